// pkv_prompt.cu -- attention of packed query tokens: prompts, chunks of prompts and single tokens
// side by side, over the paged cache or over packed keys and values.
//
//     out[i][h] = sum_t softmax_t(scale * q[i][h] . K[t]) V[t]   over the tokens t that query i sees
//
// in up to three launches.  (1) The plan: lengths are on the device, so one CTA forms the list of
// items there (pkv_prompt.cuh), largest first, and cuts items that are longer than a CTA's share of
// the whole call, as a few rows behind a long context are.  (2) The pass over the items.  Pieces of a cut
// item leave partial softmax states (running max m in log2 units, sum l, accumulator) per row, which (3) joins:
//     M = max_i m_i,  out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i.
#include "pkv_decode.cuh"
#include "pkv_prompt.cuh"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;  // of item sizes, for the order
constexpr int kItemCost = 2;    // an item's start and end, in tiles

template <typename T>
__device__ __forceinline__ T warp_scan(T v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// Exclusive prefix over the CTA and the total; `part` holds a value per warp.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* part, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T in = warp_scan(v);
  if (lane == 31) part[warp] = in;
  __syncthreads();
  if (warp == 0) {
    const T x = warp_scan(part[lane]);
    part[lane] = x;
  }
  __syncthreads();
  const T r = in - v + (warp ? part[warp - 1] : T(0));
  total = part[31];
  __syncthreads();
  return r;
}

struct PromptSeq {
  int row0, n, len, key0;
};
// Sequence b; false where its starts are invalid.  len is 0 where its length is.
__device__ __forceinline__ bool prompt_seq(const PromptParams& p, int b, PromptSeq& s, bool& bad_len) {
  s.row0 = __ldg(p.query_starts + b);
  const int end = __ldg(p.query_starts + b + 1);
  s.n = end - s.row0;
  s.key0 = 0;
  bad_len = false;
  if (s.row0 < 0 || end < s.row0 || end > p.num_tokens) return false;
  if (p.paged) {
    s.len = __ldg(p.context_lens + b);
    if (s.n > 0 && (s.len < s.n || s.len > p.max_context_len)) {
      bad_len = true;
      s.len = 0;
    }
    return true;
  }
  s.key0 = __ldg(p.key_starts + b);
  const int key1 = __ldg(p.key_starts + b + 1);
  s.len = key1 - s.key0;
  return s.key0 >= 0 && key1 >= s.key0 && key1 <= p.num_keys;
}

// Item `at` of the call: its sequence, rows and tiles.
__device__ __forceinline__ PromptItem prompt_item(const PromptParams& p, int at) {
  int lo = 0, hi = p.num_seqs;
  while (hi - lo > 1) {  // the last sequence whose items start at or before this one
    const int mid = (lo + hi) >> 1;
    if (p.tile_starts[mid] <= at) lo = mid; else hi = mid;
  }
  PromptSeq s;
  bool bad;
  prompt_seq(p, lo, s, bad);
  const int per = 2 * p.stream_tokens, tok0 = (at - p.tile_starts[lo]) * per;
  PromptItem x{};
  x.seq = lo;
  x.row0 = s.row0 + tok0;
  x.ntok = min(per, s.n - tok0);
  x.pos0 = s.len - s.n + tok0;
  x.len = s.len;
  x.key0 = s.key0;
  x.shared = s.n > per;
  span_tiles(prompt_span(p, x.pos0, x.pos0 + x.ntok - 1, s.len), x.tile0, x.tiles);
  return x;
}

__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const PromptParams p) {
  __shared__ int part[32];
  __shared__ int64_t part64[32];
  __shared__ int hist[kBuckets];
  __shared__ int s_most, s_parts, s_joins;
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) s_most = s_parts = s_joins = 0;
  hist[tid] = 0;
  // items of each sequence
  int items = 0;
  bool ok = true;
  for (int b0 = 0; b0 < p.num_seqs; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < p.num_seqs) {
      PromptSeq s;
      bool bad_len;
      const bool good = prompt_seq(p, b, s, bad_len);
      ok &= good;
      if (good && bad_len) set_error(p.err, kErrContextLen);
      if (good) n = (s.n + 2 * p.stream_tokens - 1) / (2 * p.stream_tokens);
    }
    int all;
    const int before = block_scan(n, part, all);
    if (b < p.num_seqs) p.tile_starts[b] = items + before;
    items += all;
  }
  if (!__syncthreads_and(ok)) {
    if (tid == 0) {
      set_error(p.err, kErrQuery);
      *p.header = PromptHeader{};
    }
    return;
  }
  // the whole call's tiles, and the largest item's
  int64_t sum = 0;
  int most = 0;
  for (int i = tid; i < items; i += kPlanThreads) {
    const int t = prompt_item(p, i).tiles;
    sum += t + kItemCost;
    most = max(most, t);
  }
  int64_t total;
  block_scan(sum, part64, total);
  atomicMax(&s_most, most);
  __syncthreads();
  most = s_most;
  // Items longer than a CTA's share are cut into equal pieces.
  const int64_t share = (total * p.units + p.grid - 1) / p.grid;
  const int limit = p.max_pieces > 0 ? int(min(max(share - kItemCost, int64_t(kPromptMinPiece)), int64_t(INT_MAX))) : INT_MAX;
  most = min(most, limit);
  auto bucket = [&](int tiles) { return kBuckets - 1 - int(int64_t(min(tiles, most)) * (kBuckets - 1) / max(most, 1)); };
  for (int i = tid; i < items; i += kPlanThreads) {
    const PromptItem x = prompt_item(p, i);
    int2 cut = make_int2(1, -1);
    if (x.tiles > limit) {
      const int pieces = (x.tiles + limit - 1) / limit;
      const int at = atomicAdd(&s_parts, pieces);
      if (at + pieces <= p.max_pieces) {
        cut = make_int2(pieces, at);
        p.joins[atomicAdd(&s_joins, 1)] = PromptJoin{x.row0, x.ntok, at, pieces};
      }
    }
    p.cuts[i] = cut;
    atomicAdd(&hist[bucket((x.tiles + cut.x - 1) / cut.x)], cut.x);
  }
  __syncthreads();
  int all;
  const int before = block_scan(hist[tid], part, all);
  hist[tid] = before;
  __syncthreads();
  for (int i = tid; i < items; i += kPlanThreads) {
    PromptItem x = prompt_item(p, i);
    const int2 cut = p.cuts[i];
    const int tile0 = x.tile0, tiles = x.tiles;
    int at = atomicAdd(&hist[bucket((tiles + cut.x - 1) / cut.x)], cut.x);
    for (int j = 0; j < cut.x; ++j) {
      const int t0 = int(int64_t(tiles) * j / cut.x), t1 = int(int64_t(tiles) * (j + 1) / cut.x);
      x.tile0 = tile0 + t0;
      x.tiles = t1 - t0;
      x.part = cut.y < 0 ? -1 : cut.y + j;
      p.list[at++] = x;
    }
  }
  if (tid == 0) *p.header = PromptHeader{0u, all, s_joins, 0};
}

// Join the pieces' states of cut items: a warp per row, a lane to D / 32 consecutive values.
template <int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptParams p) {
  constexpr int kDPV = D / 32;
  constexpr uint32_t kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t rows = int64_t(p.header->joins) * p.units * p.part_rows;
  const int64_t warps = int64_t(gridDim.x) * (blockDim.x / 32);
  for (int64_t w = int64_t(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5); w < rows; w += warps) {
    const int64_t ju = w / p.part_rows;
    const int r = int(w - ju * p.part_rows);
    const int j = int(ju / p.units), unit = int(ju - int64_t(j) * p.units);
    const PromptJoin x = p.joins[j];
    const int tok = r / p.heads, h = r - tok * p.heads;
    const int kvh = unit / p.chunks, head = (unit - kvh * p.chunks) * p.heads + h;
    if (tok >= x.ntok || head >= p.group) continue;
    auto row = [&](int i) { return (int64_t(x.part + i) * p.units + unit) * p.part_rows + r; };
    float M = kMaxFloor;
    for (int i = lane; i < x.parts; i += 32) M = fmaxf(M, p.ml[row(i)].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
    float L = 0.0f, a[kDPV] = {};
    for (int i = 0; i < x.parts; ++i) {
      const float2 s = p.ml[row(i)];
      if (s.y == 0.0f) continue;  // weighs nothing; it may have no accumulator
      const float f = exp2f(s.x - M);
      L = fmaf(f, s.y, L);
      const float* src = p.acc + row(i) * D + lane * kDPV;
#pragma unroll
      for (int e = 0; e < kDPV; ++e) a[e] = fmaf(f, src[e], a[e]);
    }
    uint32_t packed[kDPV / 2];
#pragma unroll
    for (int e = 0; e < kDPV / 2; ++e) packed[e] = L == 0.0f ? 0u : pack_bf16x2(a[2 * e] / L, a[2 * e + 1] / L);
    auto* out = static_cast<__nv_bfloat16*>(p.out) + int64_t(x.row0 + tok) * p.out_stride +
                (int64_t(kvh) * p.group + head) * D + lane * kDPV;
    if constexpr (kDPV == 4) *reinterpret_cast<uint2*>(out) = make_uint2(packed[0], packed[1]);
    else *reinterpret_cast<uint32_t*>(out) = packed[0];
  }
}

// The pass over the items, one warp to a row: a lane to a token of 32 for the logits, to D / 32
// values for the sums.
template <KvType KV, int D, bool kPaged>
__global__ void __launch_bounds__(256) prompt_simple_kernel(const PromptParams p) {
  constexpr int kDPV = D / 32;
  constexpr uint32_t kAll = 0xffffffffu;
  __shared__ float qs[8][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const int total = p.header->items * p.units;
  auto value = [&](const void* base, const float* scale, int64_t row, int c) -> float {
    if constexpr (KV == KvType::kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[row * D + c]);
    if constexpr (KV == KvType::kInt8) return scale[row] * float(static_cast<const int8_t*>(base)[row * D + c]);
    uint32_t lo, hi;
    f16x2x2_from_e4m3x4(static_cast<const uint8_t*>(base)[row * D + c], lo, hi);
    return scale[row] * __half2float(__ushort_as_half(uint16_t(lo & 0xffffu)));
  };
  for (int w = blockIdx.x; w < total; w += gridDim.x) {
    const PromptItem x = p.list[w / p.units];
    const int unit = w % p.units, kvh = unit / p.chunks, chunk = unit - kvh * p.chunks;
    for (int r = warp; r < x.ntok * p.heads; r += 8) {
      const int tok = r / p.heads, head = chunk * p.heads + r - tok * p.heads;
      if (head >= p.group) continue;
      const auto* q = static_cast<const __nv_bfloat16*>(p.q) + int64_t(x.row0 + tok) * p.q_stride +
                      (int64_t(kvh) * p.group + head) * D;
      __syncwarp();
      for (int c = lane; c < D; c += 32) qs[warp][c] = __bfloat162float(q[c]);
      __syncwarp();
      const PromptSpan span = prompt_span(p, x.pos0 + tok, x.pos0 + tok, x.len);
      const int lo = max(span.lo, x.tile0 * kPromptTile), hi = min(span.hi, (x.tile0 + x.tiles) * kPromptTile);
      float m = kMaxFloor, l = 0.0f, acc[kDPV] = {};
      for (int t0 = lo / 32 * 32; t0 < hi; t0 += 32) {
        const int t = t0 + lane;
        // row of the token's K and V (in units of head_dim values); -1: not there
        int64_t row = -1;
        if (t >= lo && t < hi) {
          if constexpr (kPaged) {
            const int id = p.block_tables[int64_t(x.seq) * p.max_blocks_per_seq + t / kBlockSize];
            if (id < 0 || id >= p.num_blocks) set_error(p.err, kErrBlockId);
            else row = (int64_t(id) * p.kv_heads + kvh) * kBlockSize + t % kBlockSize;
          } else {
            row = t;
          }
        }
        float y = -INFINITY;
        if (row >= 0) {
          float dot = 0.0f;
          for (int c = 0; c < D; ++c) {
            float k;
            if constexpr (kPaged) k = value(p.k_cache, p.k_scale, row, c);
            else k = __bfloat162float(static_cast<const __nv_bfloat16*>(p.k)[(x.key0 + row) * p.k_stride + kvh * D + c]);
            dot = fmaf(qs[warp][c], k, dot);
          }
          y = dot * p.scale_log2;
        }
        float mx = y;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o));
        const float m2 = fmaxf(m, mx), f = exp2f(m - m2), e = row >= 0 ? exp2f(y - m2) : 0.0f;
        m = m2;
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < kDPV; ++i) acc[i] *= f;
        for (int j = 0; j < 32; ++j) {
          const int64_t rj = __shfl_sync(kAll, row, j);
          const float ej = __shfl_sync(kAll, e, j);
          if (rj < 0) continue;
#pragma unroll
          for (int i = 0; i < kDPV; ++i) {
            const int c = lane * kDPV + i;
            float v;
            if constexpr (kPaged) v = value(p.v_cache, p.v_scale, rj, c);
            else v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v)[(x.key0 + rj) * p.v_stride + kvh * D + c]);
            acc[i] = fmaf(ej, v, acc[i]);
          }
        }
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
      if (x.part >= 0) {
        const int64_t at = (int64_t(x.part) * p.units + unit) * p.part_rows + r;
        for (int i = 0; i < kDPV; ++i) p.acc[at * D + lane * kDPV + i] = acc[i];
        if (lane == 0) p.ml[at] = make_float2(m, l);
        continue;
      }
      auto* out = static_cast<__nv_bfloat16*>(p.out) + int64_t(x.row0 + tok) * p.out_stride +
                  (int64_t(kvh) * p.group + head) * D;
      for (int i = 0; i < kDPV; ++i) out[lane * kDPV + i] = __float2bfloat16_rn(l == 0.0f ? 0.0f : acc[i] / l);
    }
  }
}

template <KvType KV, bool kPaged>
cudaError_t launch_simple(const PromptParams& p, cudaStream_t stream) {
  const dim3 grid(p.grid * 4);
  if (p.head_dim == 128) return launch_pdl(prompt_simple_kernel<KV, 128, kPaged>, grid, dim3(256), 0, stream, p);
  return launch_pdl(prompt_simple_kernel<KV, 64, kPaged>, grid, dim3(256), 0, stream, p);
}

}  // namespace

cudaError_t launch_prompt_plan(const PromptParams& p, cudaStream_t stream) {
  return launch_pdl(prompt_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
}

cudaError_t launch_prompt_join(const PromptParams& p, cudaStream_t stream) {
  const dim3 grid(unsigned(p.grid) * 4);
  if (p.head_dim == 128) return launch_pdl(prompt_join_kernel<128>, grid, dim3(256), 0, stream, p);
  return launch_pdl(prompt_join_kernel<64>, grid, dim3(256), 0, stream, p);
}

cudaError_t launch_prompt_simple(const PromptParams& p, KvType kv, cudaStream_t stream) {
  if (!p.paged) return launch_simple<KvType::kBf16, false>(p, stream);
  return kv == KvType::kBf16  ? launch_simple<KvType::kBf16, true>(p, stream)
         : kv == KvType::kInt8 ? launch_simple<KvType::kInt8, true>(p, stream)
                               : launch_simple<KvType::kFp8, true>(p, stream);
}

}  // namespace pkv
