// pkv_prompt_quant.cu -- prompt attention's pass over INT8 and FP8 pools.
#include "pkv_prompt_tc.cuh"

namespace pkv {

cudaError_t launch_prompt_quant(const PromptParams& p, const CUtensorMap& tq, KvType kv, cudaStream_t stream) {
  // codes come by plain loads: the maps of K and V are not used
  if (kv == KvType::kInt8)
    return p.head_dim == 128 ? launch_prompt_tc<KvType::kInt8, 128, true>(p, tq, tq, tq, stream)
                             : launch_prompt_tc<KvType::kInt8, 64, true>(p, tq, tq, tq, stream);
  return p.head_dim == 128 ? launch_prompt_tc<KvType::kFp8, 128, true>(p, tq, tq, tq, stream)
                           : launch_prompt_tc<KvType::kFp8, 64, true>(p, tq, tq, tq, stream);
}

}  // namespace pkv
