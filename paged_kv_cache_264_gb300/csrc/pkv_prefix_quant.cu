// pkv_prefix_quant.cu -- the prefix pass of shared-prefix decode over INT8 and FP8 pools.
#include "pkv_prefix_tc.cuh"

namespace pkv {

cudaError_t launch_prefix_quant(const PrefixParams& p, const CUtensorMap& tk, const CUtensorMap& tv, KvType kv,
                                cudaStream_t stream) {
  if (kv == KvType::kInt8)
    return p.head_dim == 128 ? launch_prefix_tc<KvType::kInt8, 128>(p, tk, tv, stream)
                             : launch_prefix_tc<KvType::kInt8, 64>(p, tk, tv, stream);
  return p.head_dim == 128 ? launch_prefix_tc<KvType::kFp8, 128>(p, tk, tv, stream)
                           : launch_prefix_tc<KvType::kFp8, 64>(p, tk, tv, stream);
}

}  // namespace pkv
