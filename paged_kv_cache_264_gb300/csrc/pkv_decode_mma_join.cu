// pkv_decode_mma_join.cu -- tensor-core decode kernels whose items join a prefix pass's partial states with
// their own (shared-prefix decode's pass over the sequences' own tokens), in each type's default ring shape.
#include "pkv_decode_mma.cuh"

namespace pkv {

template <KvType KV, int D>
static cudaError_t launch_join(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int cols, bool gen,
                               cudaStream_t stream) {
  constexpr RingShape kShape = KV != KvType::kBf16 ? (D == 64 ? kShapesQuantD64[0] : kShapesQuant[0])
                                                   : (D == 64 ? kShapesBf16D64[0] : kShapesBf16D128[0]);
  return gen ? launch_mma_cols<KV, D, kShape.stages, kShape.bps, true, true>(p, tk, tv, cols, stream)
             : launch_mma_cols<KV, D, kShape.stages, kShape.bps, false, true>(p, tk, tv, cols, stream);
}

cudaError_t launch_decode_mma_join(const DecodeParams& p, const CUtensorMap* tk, const CUtensorMap* tv, KvType kv, int cols,
                                   cudaStream_t stream) {
  if (!mma_supported(kv, p.head_dim, cols)) return cudaErrorInvalidValue;
  const bool gen = mma_needs_general(p.num_queries, p.window, cols);
  const bool wide = p.head_dim == 128;
  switch (kv) {
    case KvType::kBf16:
      return wide ? launch_join<KvType::kBf16, 128>(p, *tk, *tv, cols, gen, stream)
                  : launch_join<KvType::kBf16, 64>(p, *tk, *tv, cols, gen, stream);
    case KvType::kInt8:
      return wide ? launch_join<KvType::kInt8, 128>(p, *tk, *tv, cols, gen, stream)
                  : launch_join<KvType::kInt8, 64>(p, *tk, *tv, cols, gen, stream);
    case KvType::kFp8:
      return wide ? launch_join<KvType::kFp8, 128>(p, *tk, *tv, cols, gen, stream)
                  : launch_join<KvType::kFp8, 64>(p, *tk, *tv, cols, gen, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pkv
