// pkv_prompt.cu -- attention of packed query tokens: prompts, chunks of prompts and single tokens
// side by side, over the paged cache or over packed keys and values.
//
//     out[i][h] = sum_t softmax_t(scale * q[i][h] . K[t]) V[t]   over the tokens t that query i sees
//
// in up to three launches.  (1) The plan: lengths are on the device, so one CTA forms the list of
// work there.  (2) The pass over it (pkv_prompt_tc.cuh).  (3) Where units of work were cut, their pieces'
// partial softmax states (running max m in log2 units, sum l, accumulator) are joined, row by row:
//     M = max_i m_i,  out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i.
//
// The list takes one of two forms.  Few units of work, or one that is large beside a CTA's share of all: a line.
// The units in order, each as long as its tiles and a fixed cost, make one line that the CTAs share out in equal
// stretches, so that they end together; a unit on a border is cut there.  Many units: whole items, which
// the CTAs take one after the other, longest sequences first, so that what is left at the end is
// small.  A sequence's items of one head unit are neighbours there, and run together on their keys and values.
#include "pkv_decode.cuh"
#include "pkv_prompt.cuh"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;  // of sequences' sizes, for the order
constexpr int kHeldSeqs = 1024; // of up to this many sequences the plan holds what it needs in shared memory
// Places on the line: of a tile, of one whose rows both streams hold (up to kRowTile of them), and ahead of a unit's
// tiles, for its start and end.  Measured on GB300, cycles of a CTA, head_dim 128, 32 query and 8 kv heads: a tile of
// 256 rows 3400 (codes 5000 to 5400), of 4 and 128 rows 2900 (codes 3100 to 3700), a unit 5000 to 7000 besides.  At
// head_dim 64 a tile takes 2400 and 1800 (codes 4400 and 2450) and a unit as long, some 8 : 6 : 17, and its line is shared
// out by the same weights: stretches with more units of few tiles than others end later.
constexpr int kTileCost = 8, kTwinCost = 7, kTwinCodesCost = 5, kUnitCost = 12;
__device__ __forceinline__ int tile_cost(const PromptParams& p, int ntok) {
  return ntok > p.stream_tokens ? kTileCost : p.k_scale ? kTwinCodesCost : kTwinCost;
}

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

// The sequences' items, in shared memory where they fit.
struct PromptItems {
  const PromptParams& p;
  const PromptSeq* held;  // NULL: read again
  const int* starts;      // [num_seqs] items before each sequence's
  int items;

  // The sequence that item `at` belongs to, its items and which of them it is.
  __device__ __forceinline__ int find(int at, int& count, int& index) const {
    int lo = 0, hi = p.num_seqs;
    while (hi - lo > 1) {  // the last sequence whose items start at or before this one
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= at) lo = mid; else hi = mid;
    }
    count = (lo + 1 < p.num_seqs ? starts[lo + 1] : items) - starts[lo];
    index = at - starts[lo];
    return lo;
  }
  // Item `index` of sequence b's `count`.
  __device__ __forceinline__ PromptItem item(int b, int count, int index) const {
    PromptSeq s;
    bool bad;
    if (held) s = held[b];
    else prompt_seq(p, b, s, bad);
    return sequence_item(p, s, b, count, index);
  }
};

// CTA c's stretch of a line of `total` places starts here; the CTA whose stretch holds place w.
// (Lines are short enough for 32 bits as a rule, and a 64-bit division is some hundred instructions.)
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) { return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b; }
__device__ __forceinline__ int64_t line_start(int64_t total, int ctas, int c) { return divide(total * c, ctas); }
__device__ __forceinline__ int line_owner(int64_t total, int ctas, int64_t w) { return int(divide((w + 1) * ctas - 1, total)); }

// A unit's pieces along the line: f(CTA, first tile, tiles) for each that has tiles, or once for a unit that has none.
template <typename F>
__device__ __forceinline__ void line_pieces(int64_t total, int ctas, int64_t at, int tiles, int per, F&& f) {
  const int64_t cost = int64_t(tiles) * per + kUnitCost;
  if (tiles <= kPromptWhole) {
    f(line_owner(total, ctas, at + cost / 2), 0, tiles);
    return;
  }
  const int c1 = line_owner(total, ctas, at + cost - 1);
  for (int c = line_owner(total, ctas, at), t = 0; c <= c1; ++c) {
    const int end = c == c1 ? tiles : int(divide(max(line_start(total, ctas, c + 1) - at - kUnitCost, int64_t(0)), per));
    if (end > t) {
      f(c, t, end - t);
      t = end;
    }
  }
}

// Forming the list.  One CTA, bound by its chain of scans and barriers: 8 us for a batch of equal prompts, 10 to 14
// for hundreds of sequences, 23 where a prompt of 16384 tokens has 2048 units of work, against 1.2 ms of its pass.
__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const PromptParams p) {
  __shared__ int part[32];
  __shared__ int64_t part64[32];
  __shared__ int hist[kBuckets];  // sequences' sizes, or the CTAs' pieces
  __shared__ PromptSeq held[kHeldSeqs];
  __shared__ int held_starts[kHeldSeqs];
  __shared__ int s_most, s_joins;
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) s_most = s_joins = 0;
  hist[tid] = 0;
  // items of each sequence
  const bool hold = p.num_seqs <= kHeldSeqs;
  int* starts = hold ? held_starts : p.item_starts;
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
      if (hold) held[b] = s;
    }
    int all;
    const int before = block_scan(n, part, all);
    if (b < p.num_seqs) starts[b] = items + before;
    items += all;
  }
  if (!__syncthreads_and(ok)) {
    if (tid == 0) {
      set_error(p.err, kErrQuery);
      *p.header = PromptHeader{};
    }
    return;
  }
  const PromptItems call{p, hold ? held : nullptr, starts, items};
  // the whole call's places, and the largest item's tiles
  int64_t sum = 0;
  int most = 0, count, index;
  for (int i = tid; i < items; i += kPlanThreads) {
    const int b = call.find(i, count, index);
    const PromptItem x = call.item(b, count, index);
    sum += int64_t(x.tiles) * tile_cost(p, x.ntok) + kUnitCost;
    most = max(most, x.tiles);
  }
  if (most > 0) atomicMax(&s_most, most);
  int64_t total;
  block_scan(sum, part64, total);
  most = s_most;
  total *= p.units;
  const int work = items * p.units;
  const bool line = work <= kPromptWaves * p.grid || int64_t(most) * kTileCost * kPromptWaves > total / p.grid;
  if (line) {
    const int ctas = int(min(total, int64_t(p.grid)));
    int64_t line0 = 0;
    int entry0 = 0, part0 = 0;
    for (int w0 = 0; w0 < work; w0 += kPlanThreads) {
      // in order: sequences, their head units, their items
      const int w = w0 + tid;
      PromptItem x{};
      int pieces = 0, per = 0;
      if (w < work) {
        const int b = call.find(w / p.units, count, index);
        const int in_seq = w - starts[b] * p.units, unit = in_seq / count;
        x = call.item(b, count, in_seq - unit * count);
        x.unit = unit;
        per = tile_cost(p, x.ntok);
      }
      int64_t all64;
      const int64_t at = line0 + block_scan(w < work ? int64_t(x.tiles) * per + kUnitCost : int64_t(0), part64, all64);
      if (w < work)
        line_pieces(total, ctas, at, x.tiles, per, [&](int c, int, int) {
          atomicAdd(&hist[c], 1);
          ++pieces;
        });
      // both counts in one scan: pieces, and those of cut units
      int64_t all_pieces;
      const int64_t before = block_scan(int64_t(pieces) | int64_t(pieces > 1 ? pieces : 0) << 32, part64, all_pieces);
      int entry = entry0 + int(before & 0xffffffff);
      const int first = part0 + int(before >> 32);
      if (w < work) {
        const int tile0 = x.tile0, tiles = x.tiles;
        int to = first;
        line_pieces(total, ctas, at, tiles, per, [&](int, int t, int n) {
          x.tile0 = tile0 + t;
          x.tiles = n;
          x.part = pieces > 1 ? to++ : -1;
          p.list[entry++] = x;
        });
        if (pieces > 1) p.joins[atomicAdd(&s_joins, 1)] = PromptJoin{x.row0, x.ntok, x.unit, first, pieces};
      }
      line0 += all64;
      entry0 += int(all_pieces & 0xffffffff);
      part0 += int(all_pieces >> 32);
    }
    __syncthreads();
    int all;
    const int before = block_scan(hist[tid], part, all);
    if (tid <= p.grid) p.cta_first[tid] = before;
  } else {
    // sequences by the tiles of their last item, largest first
    auto bucket = [&](int tiles) { return kBuckets - 1 - int(int64_t(tiles) * (kBuckets - 1) / max(most, 1)); };
    for (int pass = 0; pass < 2; ++pass) {
      for (int b = tid; b < p.num_seqs; b += kPlanThreads) {
        const int n = (b + 1 < p.num_seqs ? starts[b + 1] : items) - starts[b];
        if (n == 0) continue;
        int* at = &hist[bucket(call.item(b, n, n - 1).tiles)];
        if (pass == 0) atomicAdd(at, n);
        else p.seq_entry[b] = atomicAdd(at, n);
      }
      __syncthreads();
      if (pass == 0) {
        int all;
        const int before = block_scan(hist[tid], part, all);
        hist[tid] = before;
        __syncthreads();
      }
    }
    for (int i = tid; i < items; i += kPlanThreads) {
      const int b = call.find(i, count, index);
      PromptItem x = call.item(b, count, index);
      x.unit = p.seq_entry[b];
      p.list[x.unit + count - 1 - index] = x;
    }
  }
  if (tid == 0) *p.header = PromptHeader{0u, line, items, s_joins};
}

// Join the pieces' states of cut units: half a warp per row, a lane to D / 16 consecutive values.  Bound by its chain
// of loads: the states and accumulators of kAhead pieces are on their way at a time, before it is known what each weighs.
// 5 us where few rows are cut, 14 after a prompt of 16384 tokens (152 units of 256 rows, 40 MB: 2.9 TB/s).
template <int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptParams p) {
  constexpr int kVec = D / 64;  // float4s of a lane
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 15;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t w = int64_t(blockIdx.x) * (blockDim.x / 16) + (threadIdx.x >> 4);
  const int j = int(w / p.part_rows), r = int(w - int64_t(j) * p.part_rows);
  if (j >= p.header->joins) return;
  const PromptJoin x = p.joins[j];
  const int tok = r / p.heads, h = r - tok * p.heads;
  const int kvh = x.unit / p.chunks, head = (x.unit - kvh * p.chunks) * p.heads + h;
  if (tok >= x.ntok || head >= p.group) return;
  const int64_t row0 = int64_t(x.part) * p.part_rows + r;
  float M = kMaxFloor, L = 0.0f, a[4 * kVec] = {};
  for (int i0 = 0; i0 < x.parts; i0 += kAhead) {
    float2 s[kAhead];
    float4 v[kAhead][kVec];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t row = row0 + int64_t(min(i0 + u, x.parts - 1)) * p.part_rows;
      s[u] = p.ml[row];
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[u][e] = reinterpret_cast<const float4*>(p.acc + row * D)[lane * kVec + e];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      // a sum of 0 weighs nothing, and may have no accumulator
      if (i0 + u >= x.parts || s[u].y == 0.0f) continue;
      const float top = fmaxf(M, s[u].x), f0 = exp2f(M - top), f = exp2f(s[u].x - top);
      M = top;
      L = L * f0 + s[u].y * f;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        a[4 * e] = a[4 * e] * f0 + v[u][e].x * f;
        a[4 * e + 1] = a[4 * e + 1] * f0 + v[u][e].y * f;
        a[4 * e + 2] = a[4 * e + 2] * f0 + v[u][e].z * f;
        a[4 * e + 3] = a[4 * e + 3] * f0 + v[u][e].w * f;
      }
    }
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  auto* out = static_cast<__nv_bfloat16*>(p.out) + int64_t(x.row0 + tok) * p.out_stride +
              (int64_t(kvh) * p.group + head) * D + lane * 4 * kVec;
#pragma unroll
  for (int e = 0; e < kVec; ++e)
    reinterpret_cast<uint2*>(out)[e] = make_uint2(pack_bf16x2(a[4 * e] * inv, a[4 * e + 1] * inv), pack_bf16x2(a[4 * e + 2] * inv, a[4 * e + 3] * inv));
}

}  // namespace

cudaError_t launch_prompt_plan(const PromptParams& p, cudaStream_t stream) {
  return launch_pdl(prompt_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
}

cudaError_t launch_prompt_join(const PromptParams& p, cudaStream_t stream) {
  // at most a cut unit per CTA of the pass
  const dim3 grid(unsigned((int64_t(p.grid) * p.part_rows + 15) / 16));
  if (p.head_dim == 128) return launch_pdl(prompt_join_kernel<128>, grid, dim3(256), 0, stream, p);
  return launch_pdl(prompt_join_kernel<64>, grid, dim3(256), 0, stream, p);
}

}  // namespace pkv
