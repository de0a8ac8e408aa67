// pkv_prompt_bf16.cu -- prompt attention's pass over bf16 keys and values: packed rows, and bf16 pools.
#include "pkv_prompt_tc.cuh"

namespace pkv {

cudaError_t launch_prompt_bf16(const PromptParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t stream) {
  if (p.head_dim == 128)
    return p.paged ? launch_prompt_tc<KvType::kBf16, 128, true>(p, tq, tk, tv, stream) : launch_prompt_tc<KvType::kBf16, 128, false>(p, tq, tk, tv, stream);
  return p.paged ? launch_prompt_tc<KvType::kBf16, 64, true>(p, tq, tk, tv, stream) : launch_prompt_tc<KvType::kBf16, 64, false>(p, tq, tk, tv, stream);
}

}  // namespace pkv
