// pkv_prompt_tc.cuh -- the pass over prompt attention's items on the fifth-generation tensor core: a
// CTA per SM takes work units (an item and a head unit, pkv_prompt.cuh) off the list until it is empty.
//
// Two streams of up to 128 query rows run through the CTA, one under the other.  Per stream and tile of 128 tokens:
//     S = Q K^T    128 x 128 x D, both operands in shared memory, S in tensor memory (fp32)
//     P = 2^(S * scale - m)    a thread to a row
//     O += P V     128 x D x 128, P in tensor memory (bf16, over S's columns), V as it lies in memory
//                  (token-major, the contracted index outermost: an MN-major operand)
// One warp issues all products, stream by stream: O of a tile, then S of the next, so that the tensor pipe works
// on one stream while the other's softmax runs.  Products complete in order, so S may be written over P behind the product that
// reads it, and a softmax that has its S knows that O is at rest: it rescales O itself where it
// has to.  That is rare, for the running maximum is lazy (kMaxSlack): it moves only when a row's logits pass it by
// 2^8.  The weights enter the product over V as bf16, which the product's other operand sets (2^-8 of each at
// most, as in the paged decode); the softmax sum is over the unrounded ones.
//
// Warps: a warpgroup of softmax per stream; one that turns finished accumulators into rows of out, so that the
// next unit's softmax need not wait for that; one warp that takes units off the list and
// fills Q and the ring of K and V tiles by TMA (over the cache 8 blocks to a tile, each wherever it lies in the
// pool); one that issues the products.
//
// What a row does not see is masked in its logits; only tiles that some row of the warp sees in part pay for that.  The product
// over V takes the steps of 16 tokens that the item sees, and rows of V within those that no row of the item
// sees are zeroed first, since a weight of 0 would not hide a NaN there.
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

// A unit of work as the roles of a CTA see it.
struct PromptPiece {
  int seq, row0, ntok, pos0;  // sequence, first row of q and out, tokens, position of the first
  int len, key0;
  int tile0, tiles;           // tiles < 0: there are no more units
  int lo, hi;                 // tokens that some row of the item sees
  int part, unit;
  int first[2], count[2];     // each stream's tiles: first[s] .. first[s] + count[s] - 1 of this piece's
};

template <int D, bool kPaged>
struct PromptCfg {
  static constexpr int kHalves = D / 64;                       // 128-byte spans of a row
  static constexpr int kTileBytes = kPromptTile * D * 2;       // one K, V or Q tile
  static constexpr int kHalfBytes = kPromptTile * 128;         // one span of all its rows
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kThreads = 512;
  static constexpr int kOutWarp = 8, kMmaWarp = 12, kLoadWarp = 13;
  static constexpr int kReaders = 13;                          // warps that take pieces: softmax, out, products
  static constexpr int kRingOff = 2 * kTileBytes;              // Q tiles of both streams first
  static constexpr int kStageOff = kRingOff + kStages * kTileBytes;  // rows on their way out: 4 KB a warp
  static constexpr int kMiscOff = kStageOff + 4 * 4096;
  static constexpr int kStatOff = kMiscOff + 1024;             // float2 [2][128]: running max and sum
  static constexpr int kSmemBytes = kStatOff + 2 * 128 * 8;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

constexpr int kPieceQueue = 2;   // units handed out ahead
constexpr int kTileMasks = 16;   // tiles whose masks are kept: more than the ring holds

// Barriers and flags of one CTA.
struct PromptSync {
  uint64_t full[8], empty[8];      // ring stages
  uint64_t q_full[2], q_empty[2];  // per stream from here
  uint64_t s_ready[2], p_ready[2];
  uint64_t o_ready[2], o_free[2];
  uint64_t stat_ready[2];
  uint64_t drain;
  uint64_t piece_full[kPieceQueue], piece_empty[kPieceQueue];
  PromptPiece piece[kPieceQueue];
  uint8_t mask[kTileMasks];        // which of a tile's blocks exist, by tile in load order
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

// A load that stays where it is written: the compiler would sink a plain one to its use.
__device__ __forceinline__ int load_now(const void* at) {
  int v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
  return v;
}

// Bits [lo, hi) of a word.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t below_lo = lo >= 32 ? ~0u : lo <= 0 ? 0u : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

template <int D, bool kPaged>
__global__ void __launch_bounds__(PromptCfg<D, kPaged>::kThreads, 1)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const PromptParams p) {
  using C = PromptCfg<D, kPaged>;
  constexpr int S = C::kStages;
  constexpr uint32_t kAll = 0xffffffffu;
  extern __shared__ __align__(1024) unsigned char smem[];  // the swizzled tiles need its alignment
  auto* sy = reinterpret_cast<PromptSync*>(smem + C::kMiscOff);
  auto* stats = reinterpret_cast<float2*>(smem + C::kStatOff);
  unsigned char* ring = smem + C::kRingOff;
  const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(sy->full + i, 1);
      mbar_init(sy->empty + i, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(sy->q_full + s, 1);
      mbar_init(sy->q_empty + s, 1);
      mbar_init(sy->s_ready + s, 1);
      mbar_init(sy->p_ready + s, 4);
      mbar_init(sy->o_ready + s, 1);
      mbar_init(sy->o_free + s, 4);
      mbar_init(sy->stat_ready + s, 4);
    }
    mbar_init(&sy->drain, 1);
    for (int i = 0; i < kPieceQueue; ++i) {
      mbar_init(sy->piece_full + i, 1);
      mbar_init(sy->piece_empty + i, C::kReaders);
    }
    sy->abort = 0;
    fence_barrier_init();
    prefetch_tensor_map(&tmap_q);
    prefetch_tensor_map(&tmap_k);
    prefetch_tensor_map(&tmap_v);
  }
  if (warp == C::kMmaWarp) tmem_alloc(&sy->tmem, C::kTmemCols);
  if (threadIdx.x == 0 && (smem_addr(smem) & 1023u)) set_error(p.err, kErrTimeout);  // never: the only shared memory
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
  // Tokens of stream s in an item.
  auto stream_tokens = [&](const PromptPiece& x, int s) { return max(0, min(p.stream_tokens, x.ntok - s * p.stream_tokens)); };

  if (warp >= 12) {
    regs_fewer<56>();
    if (warp == C::kLoadWarp) {
      // ---------------------------------------------------------------- units, Q, K and V tiles
      // The whole warp runs this with warp-uniform values; one elected lane issues.
      const int64_t total = int64_t(load_now(&p.header->items)) * p.units;
      const uint64_t once = l2_evict_first_policy(), again = l2_evict_last_policy();
      RingAt<S> at;
      uint32_t filled = 0, put = 0, tiles = 0;
      uint32_t q_used[2] = {0, 0};
      int64_t w = blockIdx.x;
      unsigned ticket = 0;
      // an int of the list's entry to a lane
      static_assert(sizeof(PromptItem) == 48, "12 ints");
      auto fetch = [&](int64_t unit_of_work) {
        const int* entry = reinterpret_cast<const int*>(p.list + unit_of_work / p.units);
        return unit_of_work < total && lane < 12 ? load_now(entry + lane) : 0;
      };
      int entry = fetch(w);
      for (;;) {
        PromptPiece x;
        x.tiles = -1;
        bool shared = false;  // the tiles are read again by the sequence's other items
        if (w < total) {
          x.seq = __shfl_sync(kAll, entry, 0);
          x.row0 = __shfl_sync(kAll, entry, 1);
          x.ntok = __shfl_sync(kAll, entry, 2);
          x.pos0 = __shfl_sync(kAll, entry, 3);
          x.len = __shfl_sync(kAll, entry, 4);
          x.key0 = __shfl_sync(kAll, entry, 5);
          x.tile0 = __shfl_sync(kAll, entry, 6);
          x.tiles = __shfl_sync(kAll, entry, 7);
          x.part = __shfl_sync(kAll, entry, 8);
          shared = __shfl_sync(kAll, entry, 9) != 0;
          x.unit = int(w % p.units);
          const PromptSpan span = prompt_span(p, x.pos0, x.pos0 + x.ntok - 1, x.len);
          x.lo = span.lo;
          x.hi = span.hi;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int n = stream_tokens(x, s), pos = x.pos0 + s * p.stream_tokens;
            int f, c;
            span_tiles(prompt_span(p, pos, pos + n - 1, x.len), f, c);
            const int a = max(f, x.tile0), b = min(f + c, x.tile0 + x.tiles);
            x.first[s] = a;
            x.count[s] = n > 0 ? max(0, b - a) : 0;
          }
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
        const int kvh = x.unit / p.chunks, head = kvh * p.group + (x.unit - kvh * p.chunks) * p.heads;
        const uint64_t policy = shared ? again : once;
        const int32_t* table = kPaged ? p.block_tables + int64_t(x.seq) * p.max_blocks_per_seq : nullptr;
        // Blocks lane % 8 of a tile, asked for a tile ahead.  Only those that hold a token of the item's are read.
        const int blk0 = x.lo / kBlockSize, blk1 = (x.hi + kBlockSize - 1) / kBlockSize;
        auto tile_id = [&](int tile) {
          const int b = tile * (kPromptTile / kBlockSize) + (lane & 7);
          return b >= blk0 && b < blk1 ? load_now(table + b) : -1;
        };
        int next = 0, ids = 0;
        if (kPaged && x.tiles > 0) next = tile_id(x.tile0);
        uint32_t have = 0xffu;
        int64_t w_next = total;
#pragma unroll 1
        for (int i = 0; i < 2 * x.tiles && alive; ++i) {
          const int tile = x.tile0 + (i >> 1);
          const bool is_v = i & 1;
          // the next unit: taken late, so that it goes to a CTA that will be free for it
          if (i == max(0, 2 * x.tiles - 4) && lane == 0) ticket = atomicAdd(&p.header->ticket, 1u);
          if (kPaged && !is_v) {
            ids = next;
            const int b = tile * (kPromptTile / kBlockSize) + (lane & 7);
            const bool wanted = b >= blk0 && b < blk1, ok = wanted && ids >= 0 && ids < p.num_blocks;
            if (wanted && !ok && lane < 8) set_error(p.err, kErrBlockId);
            have = __ballot_sync(kAll, ok) & 0xffu;
            if ((i >> 1) + 1 < x.tiles) next = tile_id(tile + 1);
          }
          if (filled >= S && !wait_all(sy->empty + at.st, at.ph ^ 1u)) {
            alive = false;
            break;
          }
          const CUtensorMap* map = is_v ? &tmap_v : &tmap_k;
          unsigned char* dst = ring + at.st * C::kTileBytes;
          uint64_t* bar = sy->full + at.st;
          if constexpr (kPaged) {
            int row[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) row[j] = (__shfl_sync(kAll, ids, j) * p.kv_heads + kvh) * kBlockSize;  // pools with tensor maps have < 2^31 rows
            if (elect_one()) {
              if (!is_v) sy->mask[(tiles + (i >> 1)) % kTileMasks] = uint8_t(have);  // published by the arrival
              if (have) mbar_arrive_expect_tx(bar, __popc(have) * (C::kHalves * kBlockSize * 128));
              else mbar_arrive(bar);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                if (have >> j & 1) {
#pragma unroll
                  for (int span = 0; span < C::kHalves; ++span)
                    tma_load_2d(dst + span * C::kHalfBytes + j * (kBlockSize * 128), map, span * 64, row[j], bar, policy);
                }
              }
            }
          } else {
            if (elect_one()) {
              if (!is_v) sy->mask[(tiles + (i >> 1)) % kTileMasks] = 0xffu;
              mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
              for (int span = 0; span < C::kHalves; ++span)
                tma_load_3d(dst + span * C::kHalfBytes, map, span * 64, kvh, x.key0 + tile * kPromptTile, bar, policy);
            }
          }
          __syncwarp();
          ++filled;
          at.next();
          if (i == 0) {  // Q behind the first K: that need not wait for the last unit's products
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              if (x.count[s] == 0) continue;
              if (q_used[s] > 0 && !wait_all(sy->q_empty + s, (q_used[s] - 1) & 1)) {
                alive = false;
                break;
              }
              ++q_used[s];
              if (elect_one()) {
                mbar_arrive_expect_tx(sy->q_full + s, C::kHalves * p.heads * p.stream_tokens * 128);
#pragma unroll
                for (int span = 0; span < C::kHalves; ++span)
                  tma_load_3d(smem + s * C::kTileBytes + span * C::kHalfBytes, &tmap_q, span * 64, head,
                              x.row0 + s * p.stream_tokens, sy->q_full + s, once);
              }
              __syncwarp();
            }
          }
          if (i == 2 * x.tiles - 2) {  // its entry, while the last tile's V is on its way
            w_next = int64_t(__shfl_sync(kAll, ticket, 0)) + gridDim.x;
            entry = fetch(w_next);
          }
        }
        tiles += x.tiles;
        if (!alive) break;
        if (x.tiles == 0) {
          if (lane == 0) ticket = atomicAdd(&p.header->ticket, 1u);
          w_next = int64_t(__shfl_sync(kAll, ticket, 0)) + gridDim.x;
          entry = fetch(w_next);
        }
        w = w_next;
      }
      // the copies in flight land before the CTA can end (the stages filled last, and Q)
      for (uint32_t j = 0; j < min(filled, uint32_t(S)); ++j) {
        const uint32_t n = filled - 1 - j;
        (void)mbar_wait_bounded(sy->full + n % S, (n / S) & 1);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (q_used[s] > 0) (void)mbar_wait_bounded(sy->q_full + s, (q_used[s] - 1) & 1);
    } else if (warp == C::kMmaWarp) {
      // ---------------------------------------------------------------- products
      // The whole warp runs this with warp-uniform values; one elected lane issues.
      const uint32_t negate = p.scale_log2 < 0.0f ? 1u << 13 : 0u;  // -Q: the largest product is the largest logit
      const uint32_t desc_s = mma_bf16_desc(128, kPromptTile, false) | negate;
      constexpr uint32_t kDescO = mma_bf16_desc(128, D, true);
      constexpr uint32_t kHi = smem_operand_hi(1024);
      const uint32_t q_desc = smem_operand(smem_addr(smem), 16);
      const uint32_t k_desc = smem_operand(smem_addr(ring), 16), v_desc = smem_operand(smem_addr(ring), C::kHalfBytes);
      RingAt<S> at;
      uint32_t tiles = 0;
      uint32_t steps[2] = {0, 0}, units[2] = {0, 0};  // each stream's tiles and units with tiles before now
      for (; take(); done()) {
        const PromptPiece& x = sy->piece[queue.st];
        const int x_tiles = x.tiles, x_tile0 = x.tile0, x_lo = x.lo, x_hi = x.hi;
        const int first[2] = {x.first[0], x.first[1]}, count[2] = {x.count[0], x.count[1]};
        bool fresh[2] = {true, true};  // O holds nothing of this unit yet
#pragma unroll 1
        for (int j = -1; j < x_tiles && alive; ++j) {
          const int tile = x_tile0 + j;
          const uint32_t v_st = at.st;
          uint32_t k_st = 0, vmask = 0;
          if (j >= 0) {
            if (!(alive = wait_all(sy->full + at.st, at.ph))) break;
            at.next();
            // steps of 16 tokens that the item sees
            const int lo = x_lo - tile * kPromptTile, hi = x_hi - tile * kPromptTile;
            vmask = sy->mask[(tiles + j) % kTileMasks] & bit_range(lo / 16, (hi + 15) / 16);
            // within them, tokens that it does not: zero
            const int z0 = max(0, lo) & ~15, z1 = max(0, lo), z2 = min(kPromptTile, hi), z3 = min(kPromptTile, (hi + 15) & ~15);
            if (z1 > z0 || z3 > z2) {
              unsigned char* v = ring + v_st * C::kTileBytes;
              for (int c = lane; c < (z1 - z0 + z3 - z2) * 8; c += 32) {
                const int i = c >> 3, row = i < z1 - z0 ? z0 + i : z2 + i - (z1 - z0);
#pragma unroll
                for (int span = 0; span < C::kHalves; ++span)
                  *reinterpret_cast<uint4*>(v + span * C::kHalfBytes + row * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          if (j + 1 < x_tiles) {
            if (!(alive = wait_all(sy->full + at.st, at.ph))) break;
            k_st = at.st;
            at.next();
          }
          const uint32_t vd = __shfl_sync(kAll, v_desc + v_st * (C::kTileBytes >> 4), 0);
          const uint32_t kd = __shfl_sync(kAll, k_desc + k_st * (C::kTileBytes >> 4), 0);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t t_s = tmem + s * 128, t_o = tmem + 256 + s * D;
            const int mine = tile - first[s];  // the stream's tile whose product over V is due
            if (mine >= 0 && mine < count[s]) {
              alive = alive && wait_all(sy->p_ready + s, steps[s] & 1);
              if (mine == 0 && units[s] > 0) alive = alive && wait_all(sy->o_free + s, (units[s] - 1) & 1);
              if (!alive) break;
              ++steps[s];
              tc_fence_after();
              if (elect_one()) {
                if (vmask == 0xffu) {
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    tc_mma_ts(t_o, t_s + i * 8, vd + i * ((16 * 128) >> 4), kHi, kDescO, i > 0 || !fresh[s]);
                } else {
                  bool on = !fresh[s];
#pragma unroll 1
                  for (int i = 0; i < 8; ++i)
                    if (vmask >> i & 1) {
                      tc_mma_ts(t_o, t_s + i * 8, vd + i * ((16 * 128) >> 4), kHi, kDescO, on);
                      on = true;
                    }
                }
                if (mine == count[s] - 1) tc_commit(sy->o_ready + s);
              }
              __syncwarp();
              if (vmask != 0) fresh[s] = false;
              if (mine == count[s] - 1) ++units[s];
            }
            if (mine + 1 >= 0 && mine + 1 < count[s] && j + 1 < x_tiles) {
              if (mine + 1 == 0) {
                alive = alive && wait_all(sy->q_full + s, units[s] & 1);
                if (!alive) break;
              }
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                  const uint32_t o = ((i >> 2) * C::kHalfBytes + (i & 3) * 32) >> 4;
                  tc_mma_ss(t_s, q_desc + s * (C::kTileBytes >> 4) + o, kd + o, kHi, desc_s, i > 0);
                }
                tc_commit(sy->s_ready + s);
                if (mine + 1 == count[s] - 1) tc_commit(sy->q_empty + s);
              }
              __syncwarp();
            }
          }
          if (!alive) break;
          if (elect_one()) {
            if (j >= 0) tc_commit(sy->empty + v_st);
            if (j + 1 < x_tiles) tc_commit(sy->empty + k_st);
          }
          __syncwarp();
        }
        tiles += x_tiles;
        if (!alive) break;
      }
      if (!alive) {
        if (elect_one()) tc_commit(&sy->drain);  // the products in flight end before their memory is given up
        __syncwarp();
        (void)mbar_wait_bounded(&sy->drain, 0);
      }
    }
  } else if (warp >= C::kOutWarp) {
    // ---------------------------------------------------------------- finished accumulators -> out, or partials
    regs_fewer<88>();
    const int wq = warp & 3;
    const uint32_t lanes = uint32_t(wq) << 21;  // this warp's 32 lanes of tensor memory
    unsigned char* stage = smem + C::kStageOff + wq * 4096;
    uint32_t units[2] = {0, 0};
    for (; take(); done()) {
      const PromptPiece& x = sy->piece[queue.st];
      const int kvh = x.unit / p.chunks, head0 = (x.unit - kvh * p.chunks) * p.heads;
#pragma unroll 1
      for (int s = 0; s < 2 && alive; ++s) {
        const int rows = stream_tokens(x, s) * p.heads;
        const int r = wq * 32 + lane, tok = r / p.heads, h = head0 + r - tok * p.heads;
        const bool live = r < rows && h < p.group;
        const uint32_t o_addr = tmem + lanes + 256 + s * D;
        float2 st = make_float2(kMaxFloor, 0.0f);
        const bool any = x.count[s] > 0;
        if (any) {
          alive = wait_all(sy->stat_ready + s, units[s] & 1) && wait_all(sy->o_ready + s, units[s] & 1);
          if (!alive) break;
          ++units[s];
          tc_fence_after();
          st = stats[s * 128 + r];
        }
        if (x.part >= 0) {
          const int64_t row = (int64_t(x.part) * p.units + x.unit) * p.part_rows + s * p.stream_tokens * p.heads;
          if (live) p.ml[row + r] = st;
          if (any) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              float o[32];
              tmem_ld32(o_addr + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<float4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int k = j * 4 + (lane >> 3), e = lane & 7;
                if (wq * 32 + k < rows)
                  *reinterpret_cast<float4*>(p.acc + (row + wq * 32 + k) * D + c0 + e * 4) =
                      *reinterpret_cast<const float4*>(stage + k * 128 + ((e ^ (k & 7)) << 4));
              }
              __syncwarp();
            }
          }
        } else {
          // row of out; -1: none.  A row without a weight is zero, whatever the accumulator holds.
          const int64_t to = live ? int64_t(x.row0 + s * p.stream_tokens + tok) * p.out_stride + (int64_t(kvh) * p.group + h) * D : -1;
          const float inv = 1.0f / st.y;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 64) {
            uint32_t v[32];
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
              float o[32];
              if (any) {
                tmem_ld32(o_addr + c0 + c, o);
                tmem_wait_ld();
              }
#pragma unroll
              for (int e = 0; e < 16; ++e) v[c / 2 + e] = any && st.y != 0.0f ? pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
            }
            if (any && c0 == D - 64) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(sy->o_free + s);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                  make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int k = j * 4 + (lane >> 3), e = lane & 7;
              const int64_t row = __shfl_sync(kAll, to, k);
              if (row >= 0)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + row + c0 + e * 8) =
                    *reinterpret_cast<const uint4*>(stage + k * 128 + ((e ^ (k & 7)) << 4));
            }
            __syncwarp();
          }
          continue;
        }
        if (any) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(sy->o_free + s);
        }
      }
      if (!alive) break;
    }
  } else {
    // ---------------------------------------------------------------- softmax of stream s, a thread to a row
    regs_more<184>();
    const int s = warp >> 2, wq = warp & 3, r = threadIdx.x & 127;
    const uint32_t lanes = uint32_t(wq) << 21;
    const uint32_t s_addr = tmem + lanes + s * 128, o_addr = tmem + lanes + 256 + s * D;
    // a scale of zero becomes one that makes every finite logit 0, and leaves a masked one -inf
    const float scale = p.scale_log2 == 0.0f ? 1e-30f : fabsf(p.scale_log2);
    const uint64_t scale2 = f32x2(scale, scale);
    const int tok = r / p.heads;
    uint32_t step = 0, units = 0, tiles = 0;
    for (; take(); done()) {
      const PromptPiece& x = sy->piece[queue.st];
      const int n = x.count[s], ntok = stream_tokens(x, s), first = x.first[s];
      const uint32_t mask0 = tiles - x.tile0;
      tiles += x.tiles;
      if (n == 0) continue;
      const bool dead = tok >= ntok, idle = __all_sync(kAll, dead);
      const int pos = x.pos0 + s * p.stream_tokens + tok;
      PromptSpan span = prompt_span(p, pos, pos, x.len);
      if (dead) span = {0, INT_MAX};  // its values go nowhere
      float m = kMaxFloor, l = 0.0f;
#pragma unroll 1
      for (int i = 0; i < n; ++i, step ^= 1u) {
        const int tile = first + i;
        alive = wait_all(sy->s_ready + s, step);
        if (!alive) break;
        if (!idle) {
          tc_fence_after();
          const uint32_t have = sy->mask[(mask0 + tile) % kTileMasks];
          const int lo = span.lo - tile * kPromptTile, hi = span.hi - tile * kPromptTile;
          float y[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + 32 * c, y + 32 * c);
          tmem_wait_ld();
          if (__any_sync(kAll, lo > 0 || hi < kPromptTile || have != 0xffu)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t w = bit_range(lo - 32 * c, hi - 32 * c) & ((have >> (2 * c) & 1 ? 0xffffu : 0u) | (have >> (2 * c + 1) & 1 ? 0xffff0000u : 0u));
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(w >> j & 1)) y[32 * c + j] = -INFINITY;
            }
          }
          float mx[4] = {y[0], y[1], y[2], y[3]};
#pragma unroll
          for (int j = 4; j < 124; j += 8) {
#pragma unroll
            for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], y[j + 2 * u], y[j + 2 * u + 1]);
          }
          const float bm = max3(max3(mx[0], y[124], y[125]), max3(mx[1], y[126], y[127]), fmaxf(mx[2], mx[3])) * scale;
          const bool grow = bm > m + kMaxSlack;
          if (__any_sync(kAll, grow)) {
            const float mu = grow ? bm : m, f = fast_exp2(m - mu);
            m = mu;
            l *= f;
            if (i > 0) {
              // every product into O is done: S was issued after the last
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
          }
          const uint64_t neg = f32x2(-m, -m);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float* z = y + 32 * c;
#pragma unroll
            for (int j = 0; j < 16; ++j) f32x2_parts(fma2(f32x2(z[2 * j], z[2 * j + 1]), scale2, neg), z[2 * j], z[2 * j + 1]);
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = fast_exp2(z[j]);
            float w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              sum[j & 1] = add2(sum[j & 1], f32x2(z[2 * j], z[2 * j + 1]));
              w[j] = __uint_as_float(pack_bf16x2(z[2 * j], z[2 * j + 1]));
            }
            tmem_st16(s_addr + 16 * c, w);
          }
          float sum_lo, sum_hi;
          f32x2_parts(add2(sum[0], sum[1]), sum_lo, sum_hi);
          l += sum_lo + sum_hi;
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sy->p_ready + s);
      }
      if (!alive) break;
      // the last unit's have been read once its accumulator has
      if (units > 0 && !(alive = wait_all(sy->o_free + s, (units - 1) & 1))) break;
      stats[s * 128 + r] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(sy->stat_ready + s);
      ++units;
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

template <int D, bool kPaged>
cudaError_t launch_prompt_tc(const PromptParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             cudaStream_t stream) {
  using C = PromptCfg<D, kPaged>;
  auto kern = prompt_tc_kernel<D, kPaged>;
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
