// pkv_prefix_bf16.cu -- the prefix pass of shared-prefix decode over bf16 pools.
#include "pkv_prefix_tc.cuh"

namespace pkv {

cudaError_t launch_prefix_bf16(const PrefixParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_prefix_tc<KvType::kBf16, 128>(p, tk, tv, stream)
                           : launch_prefix_tc<KvType::kBf16, 64>(p, tk, tv, stream);
}

}  // namespace pkv
