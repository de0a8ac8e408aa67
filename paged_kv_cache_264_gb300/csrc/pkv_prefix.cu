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
#include <math.h>

#include "pkv_decode.cuh"
#include "pkv_prefix.cuh"

namespace pkv {
namespace {

constexpr int kSimpleThreads = 256;

// Value of element c of a pool row.
template <KvType KV>
__device__ __forceinline__ float pool_value(const void* cache, int64_t i) {
  if constexpr (KV == KvType::kBf16) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(cache)[i]);
  } else if constexpr (KV == KvType::kInt8) {
    return float(static_cast<const int8_t*>(cache)[i]);
  } else {
    float f[4];
    e4m3x4_to_f32(static_cast<const uint8_t*>(cache)[i], f);
    return f[0];
  }
}

// One warp per query row of the CTA's stretch: 32 tokens at a time, a lane to a token for the
// logits and a lane to D / 32 values for the accumulator.
template <KvType KV, int D>
__global__ void __launch_bounds__(kSimpleThreads) prefix_simple_kernel(const PrefixParams p) {
  constexpr uint32_t kFull = 0xffffffffu;
  constexpr int kDPV = D / 32;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float qs[kSimpleThreads / 32][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  PrefixScan sc{reinterpret_cast<longlong2*>(smem) + 32, reinterpret_cast<longlong2*>(smem)};
  const int64_t total = prefix_scan<kSimpleThreads>(p, sc);
  prefix_describe<kSimpleThreads>(p, sc, total);
  if (total <= 0) return;
  PrefixWalk k;
  for (bool more = walk_begin(p, sc, total, blockIdx.x, k); more; more = walk_next(p, blockIdx.x, k)) {
    const int prefix = __ldg(p.prefix_lens + k.g);
    const int32_t* table = p.block_tables + int64_t(k.x.first_seq) * p.max_blocks_per_seq;
    for (int r = warp; r < k.nrows; r += kSimpleThreads / 32) {
      const auto* q = static_cast<const __nv_bfloat16*>(p.q) + prefix_q_row(p, k.x, k.kvh, k.row0 + r) * D;
      __syncwarp();
      for (int c = lane; c < D; c += 32) qs[warp][c] = __bfloat162float(q[c]) * p.scale_log2;
      __syncwarp();
      float m = kMaxFloor, l = 0.0f, acc[kDPV] = {};
      for (int t0 = k.tile0 * kPrefixTile; t0 < min(prefix, k.tile1 * kPrefixTile); t0 += 32) {
        const int t = t0 + lane;
        float x = -INFINITY, sv = 1.0f;
        int64_t row = -1;
        if (t < prefix) {
          const int64_t block = __ldg(table + t / kBlockSize);
          if (block < 0 || block >= p.num_blocks) {
            set_error(p.err, kErrBlockId);
          } else {
            row = (block * p.kv_heads + k.kvh) * kBlockSize + t % kBlockSize;
            x = 0.0f;
            for (int c = 0; c < D; ++c) x = fmaf(qs[warp][c], pool_value<KV>(p.k_cache, row * D + c), x);
            if constexpr (KV != KvType::kBf16) {
              x *= p.k_scale[row];
              sv = p.v_scale[row];
            }
          }
        }
        float mx = x;
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        const float mu = fmaxf(m, mx), f = fast_exp2(m - mu);
        m = mu;
        const float pr = row >= 0 ? fast_exp2(x - m) : 0.0f;
        l = l * f + pr;
        for (int i = 0; i < kDPV; ++i) acc[i] *= f;
        for (int j = 0; j < 32; ++j) {
          const float w = __shfl_sync(kFull, pr * sv, j);
          const int64_t rj = __shfl_sync(kFull, row, j);
          if (rj >= 0)
            for (int i = 0; i < kDPV; ++i) acc[i] = fmaf(w, pool_value<KV>(p.v_cache, rj * D + lane + 32 * i), acc[i]);
        }
      }
      for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
      const int64_t to = k.partial + r;
      for (int i = 0; i < kDPV; ++i) p.acc[to * D + lane + 32 * i] = acc[i];
      if (lane == 0) p.ml[to] = make_float2(m, l);
      if (k.x.rows <= kPrefixRows / 2 && lane == 0) {
        p.ml[to + k.x.rows] = make_float2(kMaxFloor, 0.0f);
        // never weighted, but read
      }
      if (k.x.rows <= kPrefixRows / 2)
        for (int i = 0; i < kDPV; ++i) p.acc[(to + k.x.rows) * D + lane + 32 * i] = 0.0f;
    }
  }
}

template <KvType KV, int D>
cudaError_t launch_prefix_simple(const PrefixParams& p, cudaStream_t stream) {
  const size_t smem = prefix_scan_bytes(p.num_groups);
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(prefix_simple_kernel<KV, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int(prefix_scan_bytes(kMaxPrefixGroups)));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(prefix_simple_kernel<KV, D>, dim3(p.grid), dim3(kSimpleThreads), smem, stream, p);
}

// Join a row's partials: one warp per (sequence, query token, query head), a lane to D / 32
// consecutive values.
template <int D>
__global__ void __launch_bounds__(128) prefix_merge_kernel(const PrefixParams p) {
  constexpr int kDPV = D / 32;
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
  // prefix partials: rows 256 apart, one per CTA (two for a unit of up to 128 rows)
  int npre = 0, twice = 0;
  int64_t first = 0;
  if (d.tiles > 0) {
    const int r = d.first_row + qi * p.group + (h - kvh * p.group);
    const int units = (d.rows + kPrefixRows - 1) / kPrefixRows;
    const int64_t w0 = d.w_base + (int64_t(kvh) * units + r / kPrefixRows) * d.tiles;
    const int ctas = stretch_ctas(d.total, p.grid);
    const int c0 = stretch_owner(d.total, ctas, w0), c1 = stretch_owner(d.total, ctas, w0 + d.tiles - 1);
    twice = d.rows <= kPrefixRows / 2;
    npre = (c1 - c0 + 1) << twice;
    first = d.row_base + int64_t(kvh) * partial_rows(d.rows) + r + int64_t(c0) * kPrefixRows;
  }
  const int n = nsuf + npre;
  auto pre_row = [&](int i) { return first + int64_t(i >> twice) * kPrefixRows + (twice && (i & 1) ? d.rows : 0); };
  auto state = [&](int i) { return i < nsuf ? sml[i] : p.ml[pre_row(i - nsuf)]; };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, state(i).x);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  float L = 0.0f, a[kDPV] = {};
  for (int i0 = 0; i0 < n; i0 += 32) {
    float f = 0.0f;
    if (i0 + lane < n) {
      const float2 s = state(i0 + lane);
      f = exp2f(s.x - M);
      L = fmaf(f, s.y, L);
    }
#pragma unroll 4
    for (int j = 0; j < min(32, n - i0); ++j) {
      const float w = __shfl_sync(kFull, f, j);
      if (w == 0.0f) continue;  // a stream without tiles leaves no accumulator
      const int i = i0 + j;
      const float* src = i < nsuf ? sacc + int64_t(i) * D : p.acc + pre_row(i - nsuf) * D + lane * kDPV;
#pragma unroll
      for (int e = 0; e < kDPV; ++e) a[e] = fmaf(w, src[e], a[e]);
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(kFull, L, o);
#pragma unroll
  for (int i = 0; i < kDPV; ++i) out[i] = __float2bfloat16_rn(L == 0.0f ? 0.0f : a[i] / L);
}

}  // namespace

cudaError_t launch_prefix(const PrefixParams& p, const CUtensorMap& tk, const CUtensorMap& tv, KvType kv,
                          cudaStream_t stream) {
  const bool wide = p.head_dim == 128;
  switch (kv) {
    case KvType::kBf16:
      return launch_prefix_bf16(p, tk, tv, stream);
    case KvType::kInt8:
      return wide ? launch_prefix_simple<KvType::kInt8, 128>(p, stream) : launch_prefix_simple<KvType::kInt8, 64>(p, stream);
    case KvType::kFp8:
      return wide ? launch_prefix_simple<KvType::kFp8, 128>(p, stream) : launch_prefix_simple<KvType::kFp8, 64>(p, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_prefix_merge(const PrefixParams& p, cudaStream_t stream) {
  const int64_t rows = int64_t(p.num_seqs) * p.num_queries * p.num_q_heads;
  const unsigned grid = unsigned((rows + 3) / 4);
  if (p.head_dim == 128) return launch_pdl(prefix_merge_kernel<128>, dim3(grid), dim3(128), 0, stream, p);
  return launch_pdl(prefix_merge_kernel<64>, dim3(grid), dim3(128), 0, stream, p);
}

}  // namespace pkv
