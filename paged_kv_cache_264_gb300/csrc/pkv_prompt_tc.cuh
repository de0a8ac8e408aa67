// pkv_prompt_tc.cuh -- the pass over prompt attention's work on the fifth-generation tensor core: a CTA
// per SM takes pieces of work (pkv_prompt.cuh), its own of the line or whole units off the list.
//
// Two streams of up to 128 query rows run through the CTA, one under the other.  Per stream and tile of 128 tokens:
//     S = Q K^T    128 x 128 x D, both operands in shared memory, S in tensor memory (fp32)
//     P = 2^(S * scale - m)    a thread to a row
//     O += P V     128 x D x 128, P in tensor memory (bf16, over S's columns), V as it lies in memory
//                  (token-major, the contracted index outermost: an MN-major operand)
// A warp per stream issues its products: O of a tile, then S of the next, so that the tensor pipe works on one
// stream while the other's softmax runs (one warp for both was late with either: a prompt of 16384 tokens 1558 us for
// 1332).  Products complete in order, so S may be written over P behind the product that reads it, and a softmax that
// has its S knows that O is at rest: it rescales O itself where it has to.
// That is rare, for the running maximum is lazy (kMaxSlack): it moves only when a row's logits pass it by 2^8.  The
// weights enter the product over V as bf16, which the product's other operand sets (2^-8 of each at most, as in the
// paged decode); the softmax sum is over the unrounded ones.
//
// An item of up to 128 rows has both streams hold the same rows and take every other tile; their two states are
// joined on the way out.
//
// INT8 and FP8 pools: two warpgroups load codes, one K's and one V's, and turn them into operand tiles, bf16 and
// fp16, which hold every INT8 and E4M3 code exactly.  The scales stay out of the operands.  A token's K scale multiplies
// its fp32 logit, and its V scale its weight before that is rounded: with m the running maximum of logit + log2(V scale),
// p = 2^(logit - m) goes into the softmax sum and w = p * (V scale) is near 1 where it matters, so that fp16 holds it
// (2^-11 of it; below 2^-14 of the row's largest an absolute 2^-25).
//
// Warps: a warpgroup of softmax per stream; over bf16, one that turns finished accumulators into rows of out, so that
// the next unit's softmax need not wait for that, and one warp that fills the rings of K and V tiles by TMA (over the
// cache 8 blocks to a tile, each wherever it lies in the pool), which also takes pieces off the list and loads Q; over
// codes, the softmax warps write out and the two converting warpgroups fill the rings; a warp per stream issues the products.
//
// What a row does not see is masked in its logits; only tiles that some row of the warp sees in part pay for that.
// The product over V takes the steps of 16 tokens that the item sees, and rows of V within those that no row of the
// item sees are zeroed first, since a weight of 0 would not hide a NaN there.
//
// Measured, 32 query and 8 kv heads of 128: a causal prompt of 16384 tokens 1240 us in a short burst (1.77 PFLOP/s of
// its unmasked logits), 1376 in a loop that draws 1370 of 1400 W; the tensor pipe is busy for 72 % of a prompt of 8192.
// A tile of two full streams takes 3350 cycles of 2048 that its products need: the rest is the hand-over between
// softmax and products.  Over INT8 and FP8 it takes 5000 to 5400: the streams' chain again, longer by the scales and by
// the converting warps beside it (issue slots 53 % busy, shared memory about 73 %: scales, codes and operands).  Over
// bf16 24 tokens of 32 kv heads behind 32744 read the cache at 5.9 TB/s.
//
// Every wait is bounded; after one that gave up the CTA takes no further work, lets its
// copies and products land, frees its tensor memory and ends.
#pragma once

#include <atomic>

#include "pkv_decode.cuh"
#include "pkv_prompt.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

template <int N>
__device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_fewer() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// 3-D tiled tensor copy global -> shared.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

// Loads that stay where they are written: the compiler would sink plain ones to their use.
__device__ __forceinline__ int load_now(const void* at) {
  int v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_codes(const void* at) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(at));
  return v;
}

// A piece of work as the roles of a CTA see it.
struct PromptPiece {
  int seq, row0, ntok, pos0;  // sequence, first row of q and out, tokens, position of the first
  int len, key0;
  int tile0, tiles;           // tiles < 0: there is no more work
  int lo, hi;                 // tokens that some row of the item sees
  int part, kvh, head0;       // partial (-1: none), kv head, first of its query heads
  int twin;                   // both streams hold the same rows and take every other tile
  int shared;                 // the tiles are read again by other items
  int tok0[2], toks[2];       // each stream's first token and tokens
  int first[2], count[2];     // and tiles, from tile0 + first[s] on
};

template <KvType KV, int D, bool kPaged>
struct PromptCfg {
  static constexpr bool kQuant = KvTraits<KV>::kQuant;
  static constexpr int kHalves = D / 64;                       // 128-byte spans of a row
  static constexpr int kTileBytes = kPromptTile * D * 2;       // one K, V or Q tile
  static constexpr int kHalfBytes = kPromptTile * 128;         // one span of all its rows
  static constexpr int kK = D == 128 ? 2 : 4, kV = D == 128 && !kQuant ? 3 : kK;  // stages of the rings
  // A tile's scales are read by its softmax.  K of tile n + kSlots takes its stage once S of tile n + kSlots - kK
  // has been formed, behind the products over V of all tiles two or more before that.
  static constexpr int kSlots = kQuant ? (D == 128 ? 4 : 8) : 0;
  static_assert(!kQuant || kSlots >= kK + 2, "a scale slot is free when it is written again");
  static constexpr int kThreads = kQuant ? 640 : 512;
  // first warps: of the writers of out, or of the two converting warpgroups (K's and V's); of the others
  static constexpr int kOutWarp = 8, kConvertWarp = 8, kMmaWarp = kQuant ? 16 : 12, kLoadWarp = kMmaWarp + 2,
                       kListWarp = kMmaWarp + 3;
  static constexpr int kReaders = kMmaWarp + 3;                // warps that take pieces
  // Registers a thread: the launch's, shared out anew by warpgroup.
  static constexpr int kRegs = kQuant ? 96 : 128, kSoftmaxRegs = kQuant ? 152 : 192, kSideRegs = 64,
                       kLoadRegs = kQuant ? 48 : 64;
  static_assert(2 * kSoftmaxRegs + (kQuant ? 2 : 1) * kSideRegs + kLoadRegs <= kThreads / 128 * kRegs, "registers");
  static constexpr int kRingOff = 2 * kTileBytes;              // Q tiles of both streams first
  static constexpr int kVOff = kRingOff + kK * kTileBytes;
  // float [3][128] to a slot: K's scale times the softmax's, V's, and its log2
  static constexpr int kSlotOff = kVOff + kV * kTileBytes, kSlotBytes = 3 * kPromptTile * 4;
  static constexpr int kMiscOff = kSlotOff + kSlots * kSlotBytes;
  static constexpr int kStatOff = kMiscOff + 1024;             // float2 [2][128]: running max and sum
  static constexpr int kSmemBytes = kStatOff + 2 * 128 * 8;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

constexpr int kPieceQueue = 4;   // pieces handed out
constexpr int kTileMasks = 16;   // tiles whose masks are kept: more than the rings hold

// Barriers and flags of one CTA.
struct PromptSync {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];  // ring stages
  uint64_t q_full[2], q_empty[2];  // per stream from here
  uint64_t s_ready[2], p_half[2], p_ready[2];  // P's first 64 columns, and all
  uint64_t o_free[2];
  // An accumulator and its state are complete: stream 0's; stream 1's; and stream 1's of a piece whose rows both hold,
  // which others wait for (a parity wait has to see every phase).
  uint64_t o_ready[3], stat_ready[3];
  uint64_t turn[2], drain[2];
  uint64_t piece_full[kPieceQueue], piece_empty[kPieceQueue];
  PromptPiece piece[kPieceQueue];
  uint32_t mask[kTileMasks];       // which of a tile's blocks exist, by tile in load order: two to a byte
  uint32_t tmem;
  uint32_t abort;
};
static_assert(sizeof(PromptSync) <= 1024, "barriers fit their space");

template <int N>
struct RingAt {  // a place in a ring of N stages: the stage, and the parity of the phase its current use completes
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == N) {
      st = 0;
      ph ^= 1u;
    }
  }
};

// Bits [lo, hi) of a word.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t below_lo = lo >= 32 ? ~0u : lo <= 0 ? 0u : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

// Bit j: block j of a tile, from the word that holds two to a byte.
__device__ __forceinline__ uint32_t tile_mask(uint32_t w) { return (w | w >> 6 | w >> 12 | w >> 18) & 0xffu; }

template <KvType KV, int D, bool kPaged>
__global__ void __launch_bounds__(PromptCfg<KV, D, kPaged>::kThreads, 1)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const PromptParams p) {
  using C = PromptCfg<KV, D, kPaged>;
  constexpr uint32_t kAll = 0xffffffffu;
  extern __shared__ __align__(1024) unsigned char tile_smem[];  // the swizzled tiles need its alignment
  unsigned char* smem = tile_smem;
  auto* sy = reinterpret_cast<PromptSync*>(smem + C::kMiscOff);
  auto* stats = reinterpret_cast<float2*>(smem + C::kStatOff);
  const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (smem_addr(smem) & 1023u) {  // never, since it is the kernel's only shared memory: no work, the error
    griddep_wait();
    if (threadIdx.x == 0) set_error(p.err, kErrTimeout);
    return;
  }

  if (threadIdx.x == 0) {
    constexpr int kFillers = C::kQuant ? 4 : 1;
    for (int i = 0; i < C::kK; ++i) {
      mbar_init(sy->k_full + i, kFillers);
      mbar_init(sy->k_empty + i, 2);
    }
    for (int i = 0; i < C::kV; ++i) {
      mbar_init(sy->v_full + i, kFillers);
      mbar_init(sy->v_empty + i, 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(sy->q_full + s, 1);
      mbar_init(sy->q_empty + s, 1);
      mbar_init(sy->s_ready + s, 1);
      mbar_init(sy->p_half + s, 4);
      mbar_init(sy->p_ready + s, 4);
      mbar_init(sy->o_free + s, 4);
      mbar_init(sy->drain + s, 1);
      mbar_init(sy->turn + s, 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(sy->o_ready + i, 1);
      mbar_init(sy->stat_ready + i, 4);
    }
    for (int i = 0; i < kPieceQueue; ++i) {
      mbar_init(sy->piece_full + i, 1);
      mbar_init(sy->piece_empty + i, C::kReaders);
    }
    sy->abort = 0;
    fence_barrier_init();
    prefetch_tensor_map(&tmap_q);
    if constexpr (!C::kQuant) {
      prefetch_tensor_map(&tmap_k);
      prefetch_tensor_map(&tmap_v);
    }
  }
  if (warp == C::kMmaWarp) tmem_alloc(&sy->tmem, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // inputs and the list come from earlier kernels in the stream
  const uint32_t tmem = sy->tmem;
  volatile uint32_t* abort = &sy->abort;
  bool alive = true;
  // A whole warp's wait: the same answer on every lane; false after the time limit, or once another
  // warp of the CTA gave up.
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t tries = 0; !__all_sync(kAll, mbar_try_wait_short(bar, parity)); ++tries) {
      if (tries & 63u) continue;
      const uint64_t now = global_timer_ns();
      if (tries == 0) t0 = now;
      if (__any_sync(kAll, *abort != 0 || now - t0 > kWaitTimeoutNs)) return false;
    }
    return true;
  };
  // The next piece of the queue; false after the last, or once a wait gave up.  It stays in place until
  // every role is done with it.
  RingAt<kPieceQueue> queue;
  auto take = [&]() {
    alive = alive && wait_all(sy->piece_full + queue.st, queue.ph);
    return alive && sy->piece[queue.st].tiles >= 0;
  };
  auto done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(sy->piece_empty + queue.st);
    queue.next();
  };
  // Which of o_ready and stat_ready a piece completes.
  auto piece_done = [&](const PromptPiece& x) {
    return uint32_t(x.count[0] > 0) | uint32_t(x.count[1] > 0) << (x.twin ? 2 : 1);
  };
  // Finished rows of stream s (of both streams, where they hold the same): a thread to a row of the accumulator, run by
  // the four warps of a warpgroup.  Each thread stores its own: turned through shared memory first, so that an
  // instruction's stores lie in 8 lines and not 32, was no faster.
  // done3: the parities of o_ready and stat_ready, a bit each; tok, h: this thread's row.
  [[maybe_unused]] auto write_out = [&](const PromptPiece& x, int s, int wq, int tok, int h, uint32_t done3) {
    const bool any = x.count[s] > 0, both = x.twin != 0;
    const bool live = tok < x.toks[s] && x.head0 + h < p.group;
    const uint32_t o_addr = tmem + (uint32_t(wq) << 21) + 256 + s * D;
    float m = kMaxFloor, l = 0.0f, f0 = 1.0f, f1 = 0.0f;  // the state, and the streams' shares of it
    bool on0 = false, on1 = false;                        // a state without a weight may have no accumulator
    if (any) {
      if (!wait_all(sy->stat_ready + s, done3 >> s & 1) || !wait_all(sy->o_ready + s, done3 >> s & 1)) return false;
      if (both && (!wait_all(sy->stat_ready + 2, done3 >> 2) || !wait_all(sy->o_ready + 2, done3 >> 2))) return false;
      tc_fence_after();
      const int r = wq * 32 + lane;
      const float2 a = stats[s * 128 + r];
      m = a.x;
      l = a.y;
      on0 = a.y != 0.0f;
      if (both) {
        const float2 b = stats[128 + r];
        on1 = b.y != 0.0f;
        m = fmaxf(a.x, b.x);
        f0 = fast_exp2(a.x - m);
        f1 = fast_exp2(b.x - m);
        l = (on0 ? f0 * a.y : 0.0f) + (on1 ? f1 * b.y : 0.0f);
      }
    }
    if (__any_sync(kAll, live)) {
      const bool partial = x.part >= 0;
      float* acc = p.acc;
      auto* out = static_cast<__nv_bfloat16*>(p.out);
      if (live && partial) {
        const int64_t row = int64_t(x.part) * p.part_rows + x.tok0[s] * p.heads + wq * 32 + lane;
        p.ml[row] = make_float2(m, l);
        acc += row * D;
      } else if (live) {
        out += int64_t(x.row0 + x.tok0[s] + tok) * p.out_stride + (x.kvh * p.group + x.head0 + h) * D;
        const float inv = 1.0f / l;
        f0 *= inv;
        f1 *= inv;
      }
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 16) {
        float o[16], o1[16];
        if (any) {
          tmem_ld16(o_addr + c0, o);
          if (both) tmem_ld16(o_addr + D + c0, o1);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = on0 ? o[e] * f0 : 0.0f;
        if (both) {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = on1 ? fmaf(o1[e], f1, o[e]) : o[e];
        }
        if (live && partial) {
#pragma unroll
          for (int e = 0; e < 4; ++e) reinterpret_cast<float4*>(acc + c0)[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else if (live) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            reinterpret_cast<uint4*>(out + c0)[e] = make_uint4(pack_bf16x2(o[8 * e], o[8 * e + 1]), pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                                                               pack_bf16x2(o[8 * e + 4], o[8 * e + 5]), pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
        }
        __syncwarp();
      }
    }
    tc_fence_before();
    __syncwarp();
    if (any && lane == 0) {
      mbar_arrive(sy->o_free + s);
      if (both) mbar_arrive(sy->o_free + 1);
    }
    return true;
  };

  if (warp >= C::kMmaWarp) {
    regs_fewer<C::kLoadRegs>();
    if (warp == C::kListWarp) {
      // ---------------------------------------------------------------- list -> pieces
      // an int of a list entry to a lane
      static_assert(sizeof(PromptItem) == 48, "12 ints");
      bool line = true;
      int w = 0, end = 0, entry = 0;
      if (p.direct) {  // few units, at most one per CTA: no list, a lane to a sequence
        entry = direct_entry(p, lane);
        end = __shfl_sync(kAll, entry, 12);
      } else {
        line = load_now(&p.header->line) != 0;
        end = line ? load_now(p.cta_first + blockIdx.x + 1) : load_now(&p.header->items) * p.units;
        w = line ? load_now(p.cta_first + blockIdx.x) : blockIdx.x;
      }
      uint32_t solo = 0;  // the stream of the next piece that only needs one
      for (uint32_t put = 0;;) {
        PromptPiece x;
        x.tiles = -1;
        unsigned ticket = 0;
        if (!line && w < end && lane == 0) ticket = atomicAdd(&p.header->ticket, 1u);  // the unit after this one
        if (w < end) {
          // entry w of the CTA's own, or unit of work w of the list of whole items
          if (!p.direct) entry = lane < 12 ? load_now(reinterpret_cast<const int*>(p.list + (line ? w : w / p.units)) + lane) : 0;
          int unit = __shfl_sync(kAll, entry, 10);
          if (!line) {
            // some entry of the sequence: its units of work are those of a head unit after the other
            const int first = unit, count = __shfl_sync(kAll, entry, 11), in_seq = w - first * p.units;
            unit = in_seq / count;
            const int index = first + in_seq - unit * count;
            if (index != w / p.units) entry = lane < 12 ? load_now(reinterpret_cast<const int*>(p.list + index) + lane) : 0;
          }
          x.seq = __shfl_sync(kAll, entry, 0);
          x.row0 = __shfl_sync(kAll, entry, 1);
          x.ntok = __shfl_sync(kAll, entry, 2);
          x.pos0 = __shfl_sync(kAll, entry, 3);
          x.len = __shfl_sync(kAll, entry, 4);
          x.key0 = __shfl_sync(kAll, entry, 5);
          x.tile0 = __shfl_sync(kAll, entry, 6);
          x.tiles = __shfl_sync(kAll, entry, 7);
          x.part = __shfl_sync(kAll, entry, 8);
          x.shared = __shfl_sync(kAll, entry, 9);
          x.kvh = unit / p.chunks;
          x.head0 = (unit - x.kvh * p.chunks) * p.heads;
          const PromptSpan span = prompt_span(p, x.pos0, x.pos0 + x.ntok - 1, x.len);
          x.lo = span.lo;
          x.hi = span.hi;
          // Up to one stream's rows: both streams' over several tiles; over one, those of either stream in turn, so that
          // the next piece need not wait for this one.
          const bool single = x.ntok <= p.stream_tokens;
          x.twin = single && x.tiles > 1;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            x.tok0[s] = single ? 0 : s * p.stream_tokens;
            x.toks[s] = single ? (x.twin || uint32_t(s) == solo ? x.ntok : 0) : min(p.stream_tokens, x.ntok - x.tok0[s]);
            const int pos = x.pos0 + x.tok0[s];
            int f, c;
            span_tiles(prompt_span(p, pos, pos + x.toks[s] - 1, x.len), f, c);
            const int a = max(f, x.tile0), b = min(f + c, x.tile0 + x.tiles);
            x.first[s] = x.twin ? s : a - x.tile0;
            x.count[s] = x.twin ? (x.tiles + 1 - s) >> 1 : x.toks[s] > 0 ? max(0, b - a) : 0;
          }
          if (single && !x.twin) solo ^= 1u;
        }
        if (put >= kPieceQueue && !wait_all(sy->piece_empty + queue.st, queue.ph ^ 1u)) {
          alive = false;
          break;
        }
        if (lane == 0) {
          sy->piece[queue.st] = x;
          mbar_arrive(sy->piece_full + queue.st);
        }
        __syncwarp();
        queue.next();
        ++put;
        if (x.tiles < 0) break;
        w = line ? w + 1 : int(min(__shfl_sync(kAll, ticket, 0), unsigned(INT_MAX / 2))) + int(gridDim.x);
      }
    } else if (warp == C::kLoadWarp) {
      // ---------------------------------------------------------------- Q, and over bf16 K and V tiles
      // The whole warp runs this with warp-uniform values; one elected lane issues.
      const uint64_t once = l2_evict_first_policy(), again = l2_evict_last_policy();
      [[maybe_unused]] RingAt<C::kK> kr;
      [[maybe_unused]] RingAt<C::kV> vr;
      [[maybe_unused]] uint32_t k_filled = 0, v_filled = 0, tiles = 0;
      uint32_t q_used[2] = {0, 0};
      for (; take(); done()) {
        const PromptPiece x = sy->piece[queue.st];
        const int kvh = x.kvh, head = kvh * p.group + x.head0;
        auto load_q = [&]() {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (x.count[s] == 0) continue;
            if (q_used[s] > 0 && !wait_all(sy->q_empty + s, (q_used[s] - 1) & 1)) {
              alive = false;
              return;
            }
            ++q_used[s];
            if (elect_one()) {
              mbar_arrive_expect_tx(sy->q_full + s, C::kHalves * p.heads * p.stream_tokens * 128);
#pragma unroll
              for (int span = 0; span < C::kHalves; ++span)
                tma_load_3d(smem + s * C::kTileBytes + span * C::kHalfBytes, &tmap_q, span * 64, head, x.row0 + x.tok0[s],
                            sy->q_full + s, once);
            }
            __syncwarp();
          }
        };
        if constexpr (C::kQuant) {
          load_q();
          if (!alive) break;
        } else {
          const int lead = x.twin ? 2 : 1;
          const uint64_t policy = x.shared ? again : once;
          const int32_t* table = kPaged ? p.block_tables + int64_t(x.seq) * p.max_blocks_per_seq : nullptr;
          // Blocks lane % 8 of a tile, asked for a tile ahead.  Only those that hold a token of the item's are read.
          const int blk0 = x.lo / kBlockSize, blk1 = (x.hi + kBlockSize - 1) / kBlockSize;
          auto tile_id = [&](int tile) {
            const int b = tile * (kPromptTile / kBlockSize) + (lane & 7);
            return b >= blk0 && b < blk1 ? load_now(table + b) : -1;
          };
          // Of K's tile, and (a tile or two later) of V's: this lane's block, and which of them exist.
          int next = kPaged && x.tiles > 0 ? tile_id(x.tile0) : 0, ids[3] = {0, 0, 0};
          uint32_t have[3] = {0xffu, 0xffu, 0xffu};
          auto copy = [&](const CUtensorMap* map, unsigned char* dst, uint64_t* bar, int tile, int id, uint32_t blocks) {
            if constexpr (kPaged) {
              int row[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) row[j] = (__shfl_sync(kAll, id, j) * p.kv_heads + kvh) * kBlockSize;  // pools with tensor maps have < 2^31 rows
              if (elect_one()) {
                if (blocks) mbar_arrive_expect_tx(bar, __popc(blocks) * (C::kHalves * kBlockSize * 128));
                else mbar_arrive(bar);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  if (blocks >> j & 1) {
#pragma unroll
                    for (int span = 0; span < C::kHalves; ++span)
                      tma_load_2d(dst + span * C::kHalfBytes + j * (kBlockSize * 128), map, span * 64, row[j], bar, policy);
                  }
                }
              }
            } else if (elect_one()) {
              mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
              for (int span = 0; span < C::kHalves; ++span)
                tma_load_3d(dst + span * C::kHalfBytes, map, span * 64, kvh, x.key0 + tile * kPromptTile, bar, policy);
            }
            __syncwarp();
          };
#pragma unroll 1
          for (int j = -lead; j < x.tiles; ++j) {
            if (j + lead < x.tiles) {
              const int tile = x.tile0 + j + lead;
              if constexpr (kPaged) {
                ids[2] = ids[1];
                ids[1] = ids[0];
                ids[0] = next;
                have[2] = have[1];
                have[1] = have[0];
                const int b = tile * (kPromptTile / kBlockSize) + (lane & 7);
                const bool wanted = b >= blk0 && b < blk1, ok = wanted && next >= 0 && next < p.num_blocks;
                if (wanted && !ok && lane < 8) set_error(p.err, kErrBlockId);
                have[0] = __ballot_sync(kAll, ok) & 0xffu;
                if (j + lead + 1 < x.tiles) next = tile_id(tile + 1);
              }
              if (k_filled >= C::kK && !wait_all(sy->k_empty + kr.st, kr.ph ^ 1u)) {
                alive = false;
                break;
              }
              if (lane == 0) {  // published by the copy's arrival
                const uint32_t a = have[0];
                sy->mask[(tiles + j + lead) % kTileMasks] = (a & 3u) | (a & 0xcu) << 6 | (a & 0x30u) << 12 | (a & 0xc0u) << 18;
              }
              __syncwarp();
              copy(&tmap_k, smem + C::kRingOff + kr.st * C::kTileBytes, sy->k_full + kr.st, tile, ids[0], have[0]);
              ++k_filled;
              kr.next();
            } else if constexpr (kPaged) {  // K is through
              ids[2] = ids[1];
              ids[1] = ids[0];
              have[2] = have[1];
              have[1] = have[0];
            }
            if (j == -lead) load_q();  // behind the first K: that need not wait for the last piece's products
            if (!alive) break;
            if (j >= 0) {
              if (v_filled >= C::kV && !wait_all(sy->v_empty + vr.st, vr.ph ^ 1u)) {
                alive = false;
                break;
              }
              copy(&tmap_v, smem + C::kVOff + vr.st * C::kTileBytes, sy->v_full + vr.st, x.tile0 + j, lead == 1 ? ids[1] : ids[2],
                   lead == 1 ? have[1] : have[2]);
              ++v_filled;
              vr.next();
            }
          }
          tiles += x.tiles;
          if (!alive) break;
        }
      }
      // the copies in flight land before the CTA can end (the stages filled last, and Q)
      for (uint32_t j = 0; j < min(k_filled, uint32_t(C::kK)); ++j) {
        const uint32_t n = k_filled - 1 - j;
        (void)mbar_wait_bounded(sy->k_full + n % C::kK, (n / C::kK) & 1);
      }
      for (uint32_t j = 0; j < min(v_filled, uint32_t(C::kV)); ++j) {
        const uint32_t n = v_filled - 1 - j;
        (void)mbar_wait_bounded(sy->v_full + n % C::kV, (n / C::kV) & 1);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (q_used[s] > 0) (void)mbar_wait_bounded(sy->q_full + s, (q_used[s] - 1) & 1);
    } else if (warp == C::kMmaWarp || warp == C::kMmaWarp + 1) {
      // ---------------------------------------------------------------- products of stream s
      // The whole warp runs this with warp-uniform values; one elected lane issues.  Both warps wait for and
      // release every stage, those of tiles that only the other stream takes too: a barrier's wait is for a parity.
      const int s = warp - C::kMmaWarp;
      const uint32_t negate = p.scale_log2 < 0.0f ? 1u << 13 : 0u;  // -Q: the largest product is the largest logit
      const uint32_t desc_s = mma_bf16_desc(128, kPromptTile, false) | negate;
      constexpr uint32_t kDescO = C::kQuant ? mma_f16_desc(128, D, true) : mma_bf16_desc(128, D, true);
      constexpr uint32_t kHi = smem_operand_hi(1024);
      const uint32_t q_desc = smem_operand(smem_addr(smem + s * C::kTileBytes), 16);
      const uint32_t k_desc = smem_operand(smem_addr(smem + C::kRingOff), 16);
      const uint32_t v_desc = smem_operand(smem_addr(smem + C::kVOff), C::kHalfBytes);
      const uint32_t t_s = tmem + s * 128, t_o = tmem + 256 + s * D;
      RingAt<C::kK> kr;
      RingAt<C::kV> vr;
      uint32_t tiles = 0, step = 0, used = 0;  // all tiles before the piece's; parities of the stream's tiles and pieces
      bool before = false;                     // the stream has had pieces
      uint32_t turns = 0;
      for (; take(); done()) {
        const PromptPiece& x = sy->piece[queue.st];
        const int n = x.tiles, tile0 = x.tile0, twin = x.twin != 0, lead = 1 + twin;
        // the stream's tiles are first, first + lead, ... last
        const int first = x.first[s], count = x.count[s], last = first + (count - 1) * lead;
        const int lo0 = x.lo - tile0 * kPromptTile, hi0 = x.hi - tile0 * kPromptTile;
        const bool both = count > 0 && x.count[s ^ 1] > 0;
        bool fresh = true;  // O holds nothing of this piece yet
#pragma unroll 1
        for (int j = -lead; j < n; ++j) {
          const bool turn = !twin || !((j ^ first) & 1);
          const bool has_v = j >= 0, has_k = j + lead < n;
          const bool pv = turn && j >= first && j <= last, qk = turn && j + lead >= first && j + lead <= last;
          if (has_k && !(alive = wait_all(sy->k_full + kr.st, kr.ph))) break;
          if (has_v && !(alive = wait_all(sy->v_full + vr.st, vr.ph))) break;
          const uint32_t kd = __shfl_sync(kAll, k_desc + kr.st * (C::kTileBytes >> 4), 0);
          uint32_t vd = 0, vmask = 0;
          if (pv) {
            vd = __shfl_sync(kAll, v_desc + vr.st * (C::kTileBytes >> 4), 0);
            const int lo = lo0 - j * kPromptTile, hi = hi0 - j * kPromptTile;
            vmask = tile_mask(sy->mask[(tiles + j) % kTileMasks]);
            if (lo > 0 || hi < kPromptTile) {
              vmask &= bit_range(lo / 16, (hi + 15) / 16);  // steps of 16 tokens that the item sees
              // within them, tokens that it does not: zero
              const int z0 = max(0, lo) & ~15, z1 = max(0, lo), z2 = min(kPromptTile, hi), z3 = min(kPromptTile, (hi + 15) & ~15);
              unsigned char* v = smem + C::kVOff + vr.st * C::kTileBytes;
              for (int c = lane; c < (z1 - z0 + z3 - z2) * 8; c += 32) {
                const int i = c >> 3, row = i < z1 - z0 ? z0 + i : z2 + i - (z1 - z0);
#pragma unroll
                for (int span = 0; span < C::kHalves; ++span)
                  *reinterpret_cast<uint4*>(v + span * C::kHalfBytes + row * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (j == first && before) alive = wait_all(sy->o_free + s, used ^ 1u);
            alive = alive && wait_all(sy->p_half + s, step);
            if (!alive) break;
          }
          if (qk && j + lead == first && !(alive = wait_all(sy->q_full + s, used))) break;
          // Products of the two streams side by side would both be late (a prompt of 16384 tokens 1748 us for 1558, when
          // that was tried): the warps issue in turn.
          if (both) {
            if ((s == 1 || turns > 0) && !(alive = wait_all(sy->turn + s, (s == 1 ? turns : turns - 1) & 1))) break;
            ++turns;
          }
          tc_fence_after();
          if (pv) {
            bool on = !fresh;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (half) {
                if (!(alive = wait_all(sy->p_ready + s, step))) break;
                tc_fence_after();
              }
              if (elect_one()) {
                if (vmask == 0xffu) {
#pragma unroll
                  for (int i = 4 * half; i < 4 * half + 4; ++i)
                    tc_mma_ts(t_o, t_s + i * 8, vd + i * ((16 * 128) >> 4), kHi, kDescO, i > 0 || on);
                } else {
                  bool more = on;
#pragma unroll 1
                  for (int i = 4 * half; i < 4 * half + 4; ++i)
                    if (vmask >> i & 1) {
                      tc_mma_ts(t_o, t_s + i * 8, vd + i * ((16 * 128) >> 4), kHi, kDescO, more);
                      more = true;
                    }
                }
              }
              __syncwarp();
              on = on || (vmask >> (4 * half) & 0xfu);
            }
            if (!alive) break;
            fresh = !on;
            step ^= 1u;
          }
          if (elect_one()) {
            if (pv) {
              tc_commit(sy->v_empty + vr.st);
              if (j == last) tc_commit(sy->o_ready + (s + (s & twin)));
            } else if (has_v) {
              mbar_arrive(sy->v_empty + vr.st);
            }
            if (qk) {
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const uint32_t o = ((i >> 2) * C::kHalfBytes + (i & 3) * 32) >> 4;
                tc_mma_ss(t_s, q_desc + o, kd + o, kHi, desc_s, i > 0);
              }
              if (both) mbar_arrive(sy->turn + (s ^ 1));
              tc_commit(sy->s_ready + s);
              tc_commit(sy->k_empty + kr.st);
              if (j + lead == last) tc_commit(sy->q_empty + s);
            } else {
              if (both) mbar_arrive(sy->turn + (s ^ 1));
              if (has_k) mbar_arrive(sy->k_empty + kr.st);
            }
          }
          __syncwarp();
          if (has_v) vr.next();
          if (has_k) kr.next();
        }
        tiles += n;
        if (!alive) break;
        if (count > 0) {
          used ^= 1u;
          before = true;
        }
      }
      if (!alive) {
        if (elect_one()) tc_commit(sy->drain + s);  // the products in flight end before their memory is given up
        __syncwarp();
        (void)mbar_wait_bounded(sy->drain + s, 0);
      }
    }
  } else if (warp >= C::kOutWarp) {
    regs_fewer<C::kSideRegs>();
    if constexpr (!C::kQuant) {
      // ---------------------------------------------------------------- finished accumulators -> out, or partials
      uint32_t done3 = 0;
      const int wq = warp & 3, r = wq * 32 + lane, tok = r / p.heads, h = r - tok * p.heads;
      for (; take(); done()) {
        const PromptPiece& x = sy->piece[queue.st];
#pragma unroll 1
        for (int s = 0; s < (x.twin ? 1 : 2) && alive; ++s)
          if (x.toks[s] > 0) alive = write_out(x, s, wq, tok, h, done3);
        if (!alive) break;
        done3 ^= piece_done(x);
      }
    } else {
      // ---------------------------------------------------------------- codes -> operand tiles of K, or of V
      constexpr int kChunks = D / 16;          // 16-byte chunks of a row of codes
      constexpr int kRows = 32 / kChunks;      // rows that a load of the warp's lanes covers
      constexpr int kLoads = 32 / kRows;       // for the warp's 32 rows of a tile: two blocks
      const bool is_v = warp >= C::kConvertWarp + 4;
      // Of a load's rows, this lane has chunk `chunk` of row `sub`.  Eight neighbouring lanes, whose 16-byte stores go
      // together, hold four chunks of two neighbouring rows: their places in the swizzled tile are all different.
      const int wq = warp & 3;
      const int chunk = D == 128 ? (lane & 3) | (lane >> 3 & 1) << 2 : lane & 3;
      const int sub = D == 128 ? (lane >> 2 & 1) | lane >> 4 << 1 : lane >> 2;
      const float scale = p.scale_log2 == 0.0f ? 1e-30f : fabsf(p.scale_log2);  // as the softmax takes it
      const auto* cache = static_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache);
      unsigned char* ring = smem + (is_v ? C::kVOff : C::kRingOff);
      uint64_t* full = is_v ? sy->v_full : sy->k_full;
      uint64_t* empty = is_v ? sy->v_empty : sy->k_empty;
      static_assert(C::kK == C::kV, "one ring's place for both");
      RingAt<C::kK> at;
      uint32_t filled = 0, tiles = 0;
      for (; take(); done()) {
        const PromptPiece& x = sy->piece[queue.st];
        const int n = x.tiles, tile0 = x.tile0, lo = x.lo, hi = x.hi;
        const int kvh = x.kvh;
        const int32_t* table = p.block_tables + int64_t(x.seq) * p.max_blocks_per_seq;
        const int blk0 = lo / kBlockSize, blk1 = (hi + kBlockSize - 1) / kBlockSize;
        const uint8_t* mine = cache + (kvh * kBlockSize + sub) * D + chunk * 16;
        const int block_bytes = p.kv_heads * (kBlockSize * D);
        // The warp's two blocks of a tile, asked for a tile ahead of their codes: -1 where no token of the item lies in one.
        int next0 = -1, next1 = -1;
        auto ask = [&](int tile) {
          const int b = (tile0 + tile) * (kPromptTile / kBlockSize) + 2 * wq;
          next0 = tile < n && b >= blk0 && b < blk1 ? load_now(table + b) : -1;
          next1 = tile < n && b + 1 >= blk0 && b + 1 < blk1 ? load_now(table + b + 1) : -1;
        };
        const uint8_t *from0 = nullptr, *from1 = nullptr;  // this lane's first chunk in each
        uint32_t have = 0;
        float ks = 0.0f, vs = 1.0f;
        auto place = [&](int tile) {  // of the blocks that were asked for
          const bool ok0 = next0 >= 0 && next0 < p.num_blocks, ok1 = next1 >= 0 && next1 < p.num_blocks;
          const int b = (tile0 + tile) * (kPromptTile / kBlockSize) + 2 * wq;
          if (!is_v && lane == 0 && ((b >= blk0 && b < blk1 && !ok0) || (b + 1 >= blk0 && b + 1 < blk1 && !ok1)))
            set_error(p.err, kErrBlockId);
          have = uint32_t(ok0) | uint32_t(ok1) << 1;
          from0 = mine + int64_t(next0) * block_bytes;
          from1 = mine + int64_t(next1) * block_bytes;
          if (!is_v) {  // a thread to a token; what the item does not see may hold anything, its scales are 0 and 1
            const int t = (tile0 + tile) * kPromptTile + wq * 32 + lane;
            const bool ok = (lane < 16 ? ok0 : ok1) && t >= lo && t < hi;
            const int64_t row = int64_t(lane < 16 ? next0 : next1) * (p.kv_heads * kBlockSize) + kvh * kBlockSize + (lane & 15);
            ks = ok ? __int_as_float(load_now(p.k_scale + row)) : 0.0f;
            vs = ok ? __int_as_float(load_now(p.v_scale + row)) : 1.0f;
          }
        };
        uint4 w[kLoads];
        auto load = [&](int i) {
          const bool upper = i >= kLoads / 2;
          const uint8_t* from = upper ? from1 : from0;
          w[i] = have >> upper & 1 ? load_codes(from + (i - (upper ? kLoads / 2 : 0)) * kRows * D) : make_uint4(0u, 0u, 0u, 0u);
        };
        ask(0);
        if (n > 0) {
          place(0);
#pragma unroll
          for (int i = 0; i < kLoads; ++i) load(i);
        }
        ask(1);
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
          float size = 1.0f, lv = 0.0f;
          if (!is_v) {
            // A scale of 0, whose codes are 0, counts as 2^-60: the token's logit has to bound the exponent, and its
            // weight must not hide others'.  Any other counts as at least 2^-98 (values move by less than 2^-89), so that a
            // sum of weights of up to 2^15 over it stays finite for 2^15 half-tiles.
            size = vs == 0.0f ? 0x1p-60f : vs < 0x1p-98f ? 0x1p-98f : vs;
            lv = __log2f(size);
          }
          if (filled >= C::kK && !(alive = wait_all(empty + at.st, at.ph ^ 1u))) break;
          if (!is_v) {
            auto* slot = reinterpret_cast<float*>(smem + C::kSlotOff + (tiles + t) % C::kSlots * C::kSlotBytes) + wq * 32;
            slot[lane] = ks * scale;
            slot[128 + lane] = size;
            slot[256 + lane] = lv;
            if (lane == 0) reinterpret_cast<uint8_t*>(sy->mask + (tiles + t) % kTileMasks)[wq] = uint8_t(have);
          }
          unsigned char* dst = ring + at.st * C::kTileBytes + (chunk >> 2) * C::kHalfBytes + (wq * 32 + sub) * 128;
          const int c0 = 2 * (chunk & 3);
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int row = i * kRows + sub;  // of the warp's 32
            uint4 a, b;
            if (is_v) {
              f16x4_from_codes<KV>(w[i].x, a.x, a.y);
              f16x4_from_codes<KV>(w[i].y, a.z, a.w);
              f16x4_from_codes<KV>(w[i].z, b.x, b.y);
              f16x4_from_codes<KV>(w[i].w, b.z, b.w);
            } else {
              bf16x4_from_codes<KV>(w[i].x, a.x, a.y);
              bf16x4_from_codes<KV>(w[i].y, a.z, a.w);
              bf16x4_from_codes<KV>(w[i].z, b.x, b.y);
              bf16x4_from_codes<KV>(w[i].w, b.z, b.w);
            }
            *reinterpret_cast<uint4*>(dst + i * (kRows * 128) + ((c0 ^ (row & 7)) << 4)) = a;
            *reinterpret_cast<uint4*>(dst + i * (kRows * 128) + (((c0 + 1) ^ (row & 7)) << 4)) = b;
          }
          // The next tile's codes, all behind this one's: a wait for one of these would wait for loads issued
          // before it too.
          if (t + 1 < n) {
            place(t + 1);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) load(i);
          }
          ask(t + 2);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full + at.st);
          ++filled;
          at.next();
        }
        tiles += n;
        if (!alive) break;
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax of stream s, a thread to a row
    regs_more<C::kSoftmaxRegs>();
    const int s = warp >> 2, wq = warp & 3, r = threadIdx.x & 127;
    const uint32_t lanes = uint32_t(wq) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t s_addr = tmem + lanes + s * 128, o_addr = tmem + lanes + 256 + s * D;
    // a scale of zero becomes one that makes every finite logit 0, and leaves a masked one -inf
    const float scale = p.scale_log2 == 0.0f ? 1e-30f : fabsf(p.scale_log2);
    const uint64_t scale2 = f32x2(scale, scale);
    const int tok = r / p.heads;
    uint32_t step = 0, tiles = 0, done3 = 0, used = 0;
    bool before = false;  // the stream has had pieces
    for (; take(); done()) {
      const PromptPiece& x = sy->piece[queue.st];
      const int n = x.count[s], first = x.first[s], tile0 = x.tile0, stride = x.twin ? 2 : 1;
      const uint32_t tiles0 = tiles;
      tiles += x.tiles;
      if (n > 0) {
        const bool dead = tok >= x.toks[s], idle = __all_sync(kAll, dead);
        const int pos = x.pos0 + x.tok0[s] + tok;
        PromptSpan span = prompt_span(p, pos, pos, x.len);
        if (dead) span = {0, INT_MAX};  // its values go nowhere
        float m = kMaxFloor, l = 0.0f;
#pragma unroll 1
        for (int i = 0; i < n; ++i, step ^= 1u) {
          const int tile = first + i * stride;
          alive = wait_all(sy->s_ready + s, step);
          if (!alive) break;
          if (!idle) {
            tc_fence_after();
            const uint32_t have = tile_mask(sy->mask[(tiles0 + tile) % kTileMasks]);
            const int lo = span.lo - (tile0 + tile) * kPromptTile, hi = span.hi - (tile0 + tile) * kPromptTile;
            [[maybe_unused]] const auto* ks =
                reinterpret_cast<const ulonglong2*>(smem + C::kSlotOff + (C::kQuant ? (tiles0 + tile) % (C::kSlots + !C::kQuant) : 0) * C::kSlotBytes);
            [[maybe_unused]] const auto *vs = ks + kPromptTile / 4, *lv = vs + kPromptTile / 4;
            const bool cut = __any_sync(kAll, lo > 0 || hi < kPromptTile || have != 0xffu);
            auto mask = [&](int c, float* z) {  // columns 32 c .. 32 c + 31
              const uint32_t w = bit_range(lo - 32 * c, hi - 32 * c) & ((have >> (2 * c) & 1 ? 0xffffu : 0u) | (have >> (2 * c + 1) & 1 ? 0xffff0000u : 0u));
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(w >> j & 1)) z[j] = -INFINITY;
            };
            auto largest = [&](const float* z, int n, float (&mx)[4]) {
#pragma unroll
              for (int j = 0; j < n; j += 8) {
#pragma unroll
                for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], z[j + 2 * u], z[j + 2 * u + 1]);
              }
            };
            uint64_t sum[2];
            // Logits (over codes: less the maximum) -> weights, 2 n to n registers.  A warp issues in order and is alone with its row's chain, so the
            // steps of neighbouring groups of 8 are written side by side: exponentials at a time (4 cycles each)
            // with the products and sums (2) of others.
            [[maybe_unused]] __half2 halves[2];
            auto weigh = [&](int c, int n, float* z, float* w) {
              const uint64_t neg = f32x2(-m, -m);
#pragma unroll
              for (int g = 0; g < n + 8; g += 4) {
                if (!C::kQuant && g < n) {
#pragma unroll
                  for (int j = g; j < g + 4; ++j) f32x2_parts(fma2(f32x2(z[2 * j], z[2 * j + 1]), scale2, neg), z[2 * j], z[2 * j + 1]);
                }
                if (g >= 4 && g < n + 4) {
#pragma unroll
                  for (int j = 2 * g - 8; j < 2 * g; ++j) z[j] = fast_exp2(z[j]);
                }
                if (g >= 8) {
#pragma unroll
                  for (int j = g - 8; j < g - 4; ++j) {
                    sum[j & 1] = add2(sum[j & 1], f32x2(z[2 * j], z[2 * j + 1]));
                    if constexpr (C::kQuant) {
                      const ulonglong2 f = vs[8 * c + j / 2];
                      f32x2_parts(mul2(f32x2(z[2 * j], z[2 * j + 1]), j & 1 ? f.y : f.x), z[2 * j], z[2 * j + 1]);
                      const __half2 v = __floats2half2_rn(z[2 * j], z[2 * j + 1]);
                      halves[j & 1] = __hadd2(halves[j & 1], v);
                      w[j] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&v));
                    } else {
                      w[j] = __uint_as_float(pack_bf16x2(z[2 * j], z[2 * j + 1]));
                    }
                  }
                }
              }
            };
            // The maximum moves where a row's logits pass it by kMaxSlack: what was weighed with the old one counts this
            // much of it now.
            auto move = [&](const float (&mx)[4]) {
              float bm = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
              bm = C::kQuant ? ceilf(bm) : bm * scale;
              const bool grow = bm > m + kMaxSlack;
              if (!__any_sync(kAll, grow)) return 1.0f;
              const float mu = grow ? bm : m, f = fast_exp2(m - mu);
              m = mu;
              l *= f;
              if (i > 0) {
                // every product into O is done: S was issued after the last
                tmem_wait_st();  // and so is a move's in the tile's first half
#pragma unroll 1
                for (int j = 0; j < D / 16; ++j) {
                  float o[16];
                  tmem_ld16(o_addr + 16 * j, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] *= f;
                  tmem_st16(o_addr + 16 * j, o);
                }
              }
              return f;
            };
            sum[0] = sum[1] = 0;
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if constexpr (C::kQuant) {
              // Half a tile at a time, once.  The maximum is looked for in the first half of a row's tiles, and again where
              // a half's weights do not add up within fp16's range (a row that passes it has one of at least 2^9).  It moves by
              // whole powers of two, so that weights handed over already can be rescaled exactly.  (All 128 logits and
              // the scales would not stay in registers, and spilled ones are far away with shared memory this full.  The
              // loop stays rolled: the code of all roles shares an instruction cache.)
              float z[64], w[32];
#pragma unroll 1
              for (int h = 0; h < 2; ++h) {
                // A search is a turn of its own, so that the weights of a row are the same whether or not another row of the
                // warp asked for one.
                bool look = i == 0 && h == 0, looked = false;
                for (;;) {
                  tmem_ld32(s_addr + 64 * h, z);
                  tmem_ld32(s_addr + 64 * h + 32, z + 32);
                  tmem_wait_ld();
                  const uint64_t neg = look ? 0 : f32x2(-m, -m);
#pragma unroll
                  for (int j = 0; j < 16; ++j) {
                    const ulonglong2 f = ks[16 * h + j];
                    f32x2_parts(fma2(f32x2(z[4 * j], z[4 * j + 1]), f.x, neg), z[4 * j], z[4 * j + 1]);
                    f32x2_parts(fma2(f32x2(z[4 * j + 2], z[4 * j + 3]), f.y, neg), z[4 * j + 2], z[4 * j + 3]);
                  }
                  if (cut) {
                    mask(2 * h, z);
                    mask(2 * h + 1, z + 32);
                  }
                  if (look) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) mx[u] = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                      const float4 f = reinterpret_cast<const float4*>(lv)[16 * h + j];
                      mx[2 * (j & 1)] = max3(mx[2 * (j & 1)], z[4 * j] + f.x, z[4 * j + 1] + f.y);
                      mx[2 * (j & 1) + 1] = max3(mx[2 * (j & 1) + 1], z[4 * j + 2] + f.z, z[4 * j + 3] + f.w);
                    }
                    const float f = move(mx);
                    if (h == 1) {  // the lower half's weights
                      tmem_wait_st();
                      const __half2 f2 = __float2half2_rn(f);
#pragma unroll 1
                      for (int c = 0; c < 32; c += 16) {
                        float o[16];
                        tmem_ld16(s_addr + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                          const uint32_t bits = __float_as_uint(o[e]);
                          const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&bits), f2);
                          o[e] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&r));
                        }
                        tmem_st16(s_addr + c, o);
                      }
                    }
                    look = false;
                    looked = true;
                    continue;
                  }
                  sum[0] = sum[1] = 0;
                  halves[0] = halves[1] = __float2half2_rn(0.0f);
                  weigh(2 * h, 32, z, w);
                  const float2 both = __half22float2(__hadd2(halves[0], halves[1]));
                  if (looked || !__any_sync(kAll, !dead && fmaxf(both.x, both.y) > 30000.0f)) {
                    float lo_sum, hi_sum;
                    f32x2_parts(add2(sum[0], sum[1]), lo_sum, hi_sum);
                    l += lo_sum + hi_sum;
                    break;
                  }
                  look = true;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) tmem_st16(s_addr + 32 * h + 16 * c, w + 16 * c);
              }
              sum[0] = sum[1] = 0;
            } else {
              float y[128], w[32];
#pragma unroll
              for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + 32 * c, y + 32 * c);
              tmem_wait_ld();
              if (cut) {
#pragma unroll
                for (int c = 0; c < 4; ++c) mask(c, y + 32 * c);
              }
              largest(y, 128, mx);
              move(mx);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                weigh(2 * h, 32, y + 64 * h, w);
#pragma unroll
                for (int c = 0; c < 2; ++c) tmem_st16(s_addr + 32 * h + 16 * c, w + 16 * c);
                if (h == 0) {
                  tmem_wait_st();
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(sy->p_half + s);
                }
              }
            }
            float sum_lo, sum_hi;
            f32x2_parts(add2(sum[0], sum[1]), sum_lo, sum_hi);
            l += sum_lo + sum_hi;
            tmem_wait_st();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) {
            if (C::kQuant || idle) mbar_arrive(sy->p_half + s);
            mbar_arrive(sy->p_ready + s);
          }
        }
        if (!alive) break;
        // the last piece's have been read once its accumulator has
        if (before && !(alive = wait_all(sy->o_free + s, used ^ 1u))) break;
        before = true;
        used ^= 1u;
        stats[s * 128 + r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(sy->stat_ready + (s && x.twin ? 2 : s));
      }
      if constexpr (C::kQuant) {
        if (x.toks[s] > 0 && (s == 0 || !x.twin) && !(alive = write_out(x, s, wq, tok, r - tok * p.heads, done3))) break;
      }
      done3 ^= piece_done(x);
    }
  }
  if (!alive && lane == 0) {
    *abort = 1;
    set_error(p.err, kErrTimeout);
  }
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, C::kTmemCols);
  }
}

template <KvType KV, int D, bool kPaged>
cudaError_t launch_prompt_tc(const PromptParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             cudaStream_t stream) {
  using C = PromptCfg<KV, D, kPaged>;
  auto kern = prompt_tc_kernel<KV, D, kPaged>;
  static std::atomic<bool> attr_done[64];  // per device: the shared-memory limit is raised
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_done[dev].load(std::memory_order_relaxed)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev].store(true, std::memory_order_relaxed);
  }
  return launch_pdl(kern, dim3(p.grid), dim3(C::kThreads), C::kSmemBytes, stream, tq, tk, tv, p);
}

}  // namespace pkv
