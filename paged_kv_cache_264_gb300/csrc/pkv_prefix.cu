// pkv_prefix.cu -- decode attention for a batch whose groups of sequences share a prefix
// ("Efficient AI Lecture 13: LLM Deployment Techniques", section "PagedAttention": shared
// prompt prefixes reuse physical blocks): each prefix is read once for its group, not once per
// sequence.
//
//     out[b][h] = sum_{t < T_b} softmax_t(scale * q[b][h] . K_b[t]) V_b[t]
//
// is formed in three passes.  (1) The prefix pass takes all query rows of a group and kv head
// together against the prefix: a matrix product of R rows, not a batch of products of G rows.
// (2) The suffix pass is the paged decode over each sequence's own tokens (pkv_decode_mma.cuh)
// on the tail of its block table.  Both leave partial softmax states (running max m in log2
// units, sum l, accumulator) per row, which (3) the merge pass joins:
//     M = max_i m_i,  out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i.
// Where each sequence's own tokens are one item and all items run at once, the items join the states
// themselves (pkv_decode_mma_join.cu) and there is no third pass.
#include <math.h>

#include "pkv_decode.cuh"
#include "pkv_prefix.cuh"

namespace pkv {
namespace {

// Join a row's partials: one warp per (sequence, query token, query head), a lane to D / 32
// consecutive values.  Bound by its chain of loads (description, states, accumulators): measured on GB300,
// 2048 rows of 20 partials of 128 7 us, 8192 rows of up to 6 11 us.
template <int D>
__global__ void __launch_bounds__(128) prefix_merge_kernel(const PrefixParams p) {
  constexpr int kDPV = D / 32;
  constexpr int kAhead = 8;
  constexpr uint32_t kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t gw = int64_t(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int per_seq = p.num_queries * p.num_q_heads;
  if (gw >= int64_t(p.num_seqs) * per_seq) return;
  const int b = int(gw / per_seq), rem = int(gw - int64_t(b) * per_seq);
  const int qi = rem / p.num_q_heads, h = rem - qi * p.num_q_heads;
  const int kvh = h / p.group;
  auto* out = static_cast<__nv_bfloat16*>(p.out) + gw * D + lane * kDPV;
  const PrefixSeq d = p.seqs[b];
  if (d.suffix_len < 0) {
    for (int i = 0; i < kDPV; ++i) out[i] = __float2bfloat16_rn(0.0f);
    return;
  }
  const int nsuf = partition_count((d.suffix_len + kBlockSize - 1) / kBlockSize, p.suffix_partition);
  const float2* sml = p.suffix_ml + gw * p.suffix_parts;
  const float* sacc = p.suffix_acc + gw * p.suffix_parts * D + lane * kDPV;
  PrefixParts pre;
  if (d.tiles > 0) pre = PrefixParts(d, kvh, d.first_row + qi * p.group + (h - kvh * p.group), p.grid);
  const int n = nsuf + pre.count;
  auto state = [&](int i) { return i < nsuf ? sml[i] : p.ml[pre.row(i - nsuf)]; };
  // lane i holds partials i, i + 32, ...; the first 32 stay in registers
  const float2 mine = lane < n ? state(lane) : make_float2(-INFINITY, 0.0f);
  float M = mine.x;
  for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, state(i).x);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  float L = 0.0f, a[kDPV] = {};
  for (int i0 = 0; i0 < n; i0 += 32) {
    // A state with a sum of 0 weighs nothing and may have no accumulator (a stream without tiles): -1 stands
    // for its weight.  A NaN sum, and a NaN accumulator under a weight of 0, go into the result.
    float f = -1.0f;
    if (i0 + lane < n) {
      const float2 s = i0 == 0 ? mine : state(i0 + lane);
      if (s.y != 0.0f) {
        f = exp2f(s.x - M);
        L = fmaf(f, s.y, L);
      }
    }
    const int here = min(32, n - i0);
    for (int j0 = 0; j0 < here; j0 += kAhead) {  // kAhead accumulators on their way at a time
      float v[kAhead][kDPV], w[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        w[u] = __shfl_sync(kFull, f, (j0 + u) & 31);
        if (j0 + u >= here || w[u] < 0.0f) {
          w[u] = 0.0f;
#pragma unroll
          for (int e = 0; e < kDPV; ++e) v[u][e] = 0.0f;
        } else {
          const int i = i0 + j0 + u;
          const float* src = i < nsuf ? sacc + int64_t(i) * D : p.acc + pre.row(i - nsuf) * D + lane * kDPV;
          if constexpr (kDPV == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[u][0] = x.x; v[u][1] = x.y;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int e = 0; e < kDPV; ++e) a[e] = fmaf(w[u], v[u][e], a[e]);
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(kFull, L, o);
  uint32_t packed[kDPV / 2];
#pragma unroll
  for (int i = 0; i < kDPV / 2; ++i)
    packed[i] = L == 0.0f ? 0u : pack_bf16x2(a[2 * i] / L, a[2 * i + 1] / L);
  if constexpr (kDPV == 4) *reinterpret_cast<uint2*>(out) = make_uint2(packed[0], packed[1]);
  else *reinterpret_cast<uint32_t*>(out) = packed[0];
}

}  // namespace

cudaError_t launch_prefix(const PrefixParams& p, const CUtensorMap& tk, const CUtensorMap& tv, KvType kv,
                          cudaStream_t stream) {
  return kv == KvType::kBf16 ? launch_prefix_bf16(p, tk, tv, stream) : launch_prefix_quant(p, tk, tv, kv, stream);
}

cudaError_t launch_prefix_merge(const PrefixParams& p, cudaStream_t stream) {
  const int64_t rows = int64_t(p.num_seqs) * p.num_queries * p.num_q_heads;
  const unsigned grid = unsigned((rows + 3) / 4);
  if (p.head_dim == 128) return launch_pdl(prefix_merge_kernel<128>, dim3(grid), dim3(128), 0, stream, p);
  return launch_pdl(prefix_merge_kernel<64>, dim3(grid), dim3(128), 0, stream, p);
}

}  // namespace pkv
