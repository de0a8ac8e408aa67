// pkv_prefix_tc.cuh -- the prefix pass of shared-prefix decode on the fifth-generation tensor
// core: up to 256 query rows of one (group, kv head) against a stretch of its prefix, a CTA per
// SM, each with its stretch of the work line (pkv_prefix.cuh).
//
// Two streams of 128 rows run through the CTA.  With more than 128 rows in the unit they hold
// different rows and take every 128-token tile; with up to 128 rows both hold the same rows and
// take every other tile, so that either way one stream's softmax runs under the other's products.  Per stream and tile:
//     S = Q K^T    128 x 128 x D, both operands in shared memory, S in tensor memory (fp32)
//     P = 2^(S * scale - m)    two threads to a row, 64 logits each in registers: no shuffles
//     O += P V     128 x D x 128, P in tensor memory (bf16, over S's columns), V as it lies in the
//                  pool (token-major, the contracted index outermost: an MN-major operand)
// A row's two threads (of two warpgroups) exchange their halves' maxima and each hand their half of P
// over: with one thread to a row its 128 logits were a chain twice as long, and nothing else was ready
// to run.  S is formed for whole tiles: its products read both operands from
// shared memory, 8 KB for 64 cycles of arithmetic at 128 columns, which is what shared memory
// delivers; at 64 columns they took as long for half the work.
// The running maximum is lazy (kMaxSlack): O is rescaled in tensor memory only when a row's
// logits pass its maximum by 2^8.  P enters the product as bf16, which the product's other operand, V, sets
// (2^-8 of each weight at most, as in the paged decode of a bf16 pool); on a bf16 pool the softmax sum adds the same rounded
// weights, so that numerator and denominator agree.
//
// INT8 and FP8 pools: TMA brings codes and scales into a ring of their own, and a warpgroup turns
// the codes into bf16 operand tiles, which holds every INT8 and E4M3 code exactly.  The scales stay
// out of the operands: a token's K scale multiplies its fp32 logit, and its V scale goes into its
// weight before that is rounded to bf16 (so the weights are rounded once, as in a bf16 pool; the
// sum adds the unrounded ones, since the rounded ones carry the scale).
//
// Warps: four warpgroups of softmax (two per stream, which also load Q and write the partials),
// one warp that fills the ring of K and V tiles by TMA (8 blocks to a tile, each wherever it lies
// in the pool), one warp per stream that issues its products (one for both let a stream's waits
// hold up the other's products), one that walks the CTA's stretch and hands its pieces to the others
// through a queue, and the converting warpgroup for INT8 and FP8.  The roles run at the same time
// and share one instruction cache, so each is kept short: loops stay rolled, and what all roles
// would compute alike (the walk) one of them does.
//
// A barrier's wait is for a parity, which tells a phase from the one before it only if the waiter
// has seen that one complete.  So one warp fills the ring, and each issuing warp waits for and
// releases every stage in ring order, those of the other stream's tiles too (a warp that filled
// only K stages, or skipped stages, could run into one still in use).
//
// What bounds it: each stream's chain of S, softmax and product over V.  At head_dim 128 S and O of two streams
// fill tensor memory, so the next S cannot lie beside this one's P; at 64 a quarter of it is free and not
// used.  Measured on GB300 with 256 rows a kv head (8), from passes of 16 and 32 steps a CTA: 3800 cycles a step
// at head_dim 128 (INT8 6050, FP8 6130) and 3200 at 64 (INT8 5240, FP8 5030), and 26 to 40 thousand around them
// (launch, the roles' code that is not in the instruction cache, Q, the partials of two or three pieces); the
// tensor pipe is busy for 45% of the cycles at 32 steps (quantised 31%, head_dim 64 29%, quantised 18%).  This
// pass alone: 256 rows over 32768 tokens 43 us, tensor pipe 37%; 16 groups of 1 to 13 rows, 32 kv heads, 284 MB,
// 66 us, 4.3 TB/s; INT8, 1024 rows over 16384 tokens 101 us, 30%; FP8 at head_dim 64, 96 rows over 4000 and 672
// over 8192 tokens 45 us, 15%.
//
// Every wait is bounded; after one that gave up the CTA takes no further work, lets its
// copies and products land, frees its tensor memory and ends.
//
// A prefix ends at a block (16 tokens), not at a tile: the product over V takes only the steps of
// 16 tokens that exist, so nothing has to be zeroed, and the logits behind them are masked.
#pragma once

#include "pkv_decode_mma.cuh"
#include "pkv_prefix.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

constexpr int kExchangeOff = 1024;             // the rows' exchange, after the barriers and flags
constexpr int kExchangeBytes = 2 * 2 * 128 * 4;  // float [stream][half][row]

template <KvType KV, int D>
struct PrefixCfg {
  static constexpr bool kQuant = KvTraits<KV>::kQuant;
  static constexpr int kHalves = D / 64;                         // 128-byte spans of a 16-bit row
  static constexpr int kTileBytes = kPrefixTile * D * 2;         // one K, V or Q tile, 16-bit
  static constexpr int kHalfBytes = kPrefixTile * 128;           // one span of all its rows
  static constexpr int kStages = kQuant ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);
  // codes as they come from the pool
  static constexpr int kRawBytes = kPrefixTile * D;
  static constexpr int kScaleBytes = 2 * kPrefixTile * 4;
  static constexpr int kRawStages = kQuant ? (D == 128 ? 3 : 8) : 1;
  // Scales of a tile wait in a slot until its softmax has used them.  The slot of tile n (in load
  // order) is written again for tile n + kSlots, when K of that tile takes a ring stage; V of tile
  // n lies at least 2 kSlots - 3 stages before it, so it has been released, and its product came
  // after its softmax.
  static constexpr int kSlots = kQuant ? (D == 128 ? 4 : 8) : 1;
  static_assert(!kQuant || 2 * kSlots - 3 >= kStages, "a scale slot is free when it is written again");
  static constexpr int kThreads = kQuant ? 768 : 640;
  static constexpr int kLoadWarp = 16, kMmaWarp = 17, kWalkWarp = 19, kConvertWarp = 20;  // 17 and 18: one per stream
  static constexpr int kReaders = kThreads / 32 - 1;             // warps that take pieces from the queue
  static constexpr int kRingOff = 2 * kTileBytes;                // Q tiles of both streams first
  static constexpr int kRawOff = kRingOff + kStages * kTileBytes;
  static constexpr int kSlotOff = kRawOff + (kQuant ? kRawStages * kRawBytes : 0);
  static constexpr int kMiscOff = kSlotOff + (kQuant ? kSlots * kScaleBytes : 0);
  static constexpr int kSmemBytes = kMiscOff + kExchangeOff + kExchangeBytes;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(size_t(kStages) * kTileBytes >= prefix_scan_bytes(kMaxPrefixGroups), "the scan fits the ring");
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

constexpr int kQueue = 4;    // pieces handed out ahead
constexpr int kMasks = 16;   // tiles whose masks are kept: more than the rings hold

// Barriers and flags of one CTA, at the start of its shared memory.
struct PrefixSync {
  uint64_t full[16], empty[16];                 // operand ring stages
  uint64_t raw_full[8], raw_empty[8];           // code ring stages
  uint64_t scales[8];                           // scale slots
  uint64_t q_ready[2], s_ready[2], p_ready[2], pv_done[2], o_free[2];  // per stream
  uint64_t pair[2][4];                          // per stream and 32 rows: both halves' values are there
  uint64_t turn[2];                             // a stream's softmax of a tile is half over
  uint64_t drain[2];
  uint64_t piece_full[kQueue], piece_empty[kQueue];
  PrefixPiece piece[kQueue];
  uint8_t mask[kMasks];                         // which of a tile's blocks exist, by tile in load order
  uint32_t tmem;
  uint32_t abort;
};
static_assert(sizeof(PrefixSync) <= kExchangeOff, "barriers fit their space");

template <int N>
struct RingPos {  // a place in a ring of N stages: the stage, and the parity of the phase its current use completes
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == N) {
      st = 0;
      ph ^= 1u;
    }
  }
};

// The i-th load of a piece of n tiles: K and V of a tile in turn where every stream takes every
// tile; K, K, V, V of a pair of tiles where the streams share them out.
struct TileLoad {
  int tile, which;
  bool is_v;
};
__device__ __forceinline__ TileLoad tile_load(bool two, int n, int i) {
  if (two) return {i >> 1, 0, bool(i & 1)};
  const int pair = i >> 2, have = min(2, n - 2 * pair), j = i & 3;
  const bool is_v = j >= have;
  const int which = is_v ? j - have : j;
  return {2 * pair + which, which, is_v};
}
// Tiles of a piece that stream s takes: all of them where the streams hold different rows.
__device__ __forceinline__ int stream_steps(const PrefixPiece& x, int s) {
  return x.nrows > 128 ? x.tiles : (x.tiles + 1 - s) / 2;
}

// Two codes in the low bytes of each half of `v` (bits 0-7 and 16-23) -> two bf16, exactly: with
// x = (low seven bits) - 128 (sign), 0x4300 | low bits is 128 + low bits, 0x4300 | sign bit is 128 or
// 256, and their difference is x.
__device__ __forceinline__ uint32_t bf16x2_from_i8(uint32_t v) {
  const uint32_t a = (v & 0x007f007fu) | 0x43004300u, b = (v & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Four codes of a word -> four bf16 in two words.
template <KvType KV>
__device__ __forceinline__ void bf16x4_from_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KV == KvType::kFp8) {
    uint32_t a, b;
    f16x2x2_from_e4m3x4(w, a, b);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
    lo = pack_bf16x2(x.x, x.y);
    hi = pack_bf16x2(y.x, y.y);
  } else {
    lo = bf16x2_from_i8(__byte_perm(w, 0u, 0x4140u));
    hi = bf16x2_from_i8(__byte_perm(w, 0u, 0x4342u));
  }
}

// A load that stays where it is written: the compiler would sink a plain one to its use, behind the
// waits that are there to cover its latency.
__device__ __forceinline__ int load_ahead(const void* at) {
  int v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(at));
  return v;
}

// Block id of lane % 8 of a tile (of the prefix's last block, past its end: tile_blocks tells).
// Asked for a step ahead of its use: a table entry is a global-memory round trip away, and any use
// of the loaded value here would wait for it.
__device__ __forceinline__ int tile_id(const int32_t* table, int nblk, int tile, int lane) {
  return load_ahead(table + min(tile * (kPrefixTile / kBlockSize) + (lane & 7), nblk - 1));
}
// Which of the tile's 8 blocks exist, bit j for block j (the same on every lane of the warp).
__device__ __forceinline__ uint32_t tile_blocks(const PrefixParams& p, int id, int nblk, int tile, int lane) {
  const bool inside = tile * (kPrefixTile / kBlockSize) + (lane & 7) < nblk;
  return __ballot_sync(0xffffffffu, inside && id >= 0 && id < p.num_blocks) & 0xffu;
}

template <KvType KV, int D>
__global__ void __launch_bounds__(PrefixCfg<KV, D>::kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                     const PrefixParams p) {
  using C = PrefixCfg<KV, D>;
  constexpr int S = C::kStages;
  constexpr uint32_t kFull = 0xffffffffu;
  extern __shared__ __align__(1024) unsigned char smem[];  // the swizzled tiles need its alignment
  auto* sy = reinterpret_cast<PrefixSync*>(smem + C::kMiscOff);
  unsigned char* ring = smem + C::kRingOff;
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(sy->full + i, C::kQuant ? 128 : 1);
      mbar_init(sy->empty + i, 2);
    }
    for (int i = 0; i < C::kRawStages; ++i) {
      mbar_init(sy->raw_full + i, 1);
      mbar_init(sy->raw_empty + i, 128);
    }
    for (int i = 0; i < C::kSlots; ++i) mbar_init(sy->scales + i, 128);
    for (int s = 0; s < 2; ++s) {
      mbar_init(sy->q_ready + s, 8);
      for (int i = 0; i < 4; ++i) mbar_init(&sy->pair[s][i], 2);
      mbar_init(sy->s_ready + s, 1);
      mbar_init(sy->p_ready + s, 8);
      mbar_init(sy->pv_done + s, 1);
      mbar_init(sy->turn + s, 8);
      mbar_init(sy->o_free + s, 8);
      mbar_init(sy->drain + s, 1);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(sy->piece_full + i, 1);
      mbar_init(sy->piece_empty + i, C::kReaders);
    }
    sy->abort = 0;
    fence_barrier_init();
    prefetch_tensor_map(&tmap_k);
    prefetch_tensor_map(&tmap_v);
  }
  if (warp == C::kMmaWarp) tmem_alloc(&sy->tmem, C::kTmemCols);
  if (threadIdx.x == 0 && (smem_addr(smem) & 1023u)) set_error(p.err, kErrTimeout);  // never: the only shared memory
  griddep_wait();  // inputs may come from the previous kernel in the stream
  // The scan of up to 32 groups is the walking warp's own; that of many lies where the ring will be,
  // and all warps describe the sequences from it first.
  const bool few = p.num_groups <= kFewGroups;
  const PrefixScan sc{reinterpret_cast<longlong2*>(ring) + 32, reinterpret_cast<longlong2*>(ring)};
  PrefixWalk k;
  int64_t total = 0;
  bool more = false;
  if (!few) {
    total = prefix_scan<C::kThreads>(p, sc);
    prefix_describe_many(p, sc, total, warp, C::kThreads / 32);
    more = walk_begin(p, sc, total, blockIdx.x, k);
  }
  tc_fence_before();
  __syncthreads();  // the ring's memory is free again; the barriers and the tensor memory are there
  tc_fence_after();
  const uint32_t tmem = sy->tmem;
  volatile uint32_t* abort = &sy->abort;
  bool alive = true;
  // A whole warp's wait: the same answer on every lane; false after the time limit, or once another
  // warp of the CTA gave up.
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t tries = 0; !__all_sync(kFull, mbar_try_wait_short(bar, parity)); ++tries) {
      if (tries & 63u) continue;
      const uint64_t now = global_timer_ns();
      if (tries == 0) t0 = now;
      if (__any_sync(kFull, *abort != 0 || now - t0 > kWaitTimeoutNs)) return false;
    }
    return true;
  };
  // Take the next piece off the queue; tiles == 0 after the last, or once a wait gave up.
  RingPos<kQueue> queue;
  auto take = [&](PrefixPiece& x) {
    alive = alive && wait_all(sy->piece_full + queue.st, queue.ph);
    if (!alive) {
      x.tiles = 0;
      return;
    }
    x = sy->piece[queue.st];
    __syncwarp();
    if (lane == 0) mbar_arrive(sy->piece_empty + queue.st);
    queue.next();
  };

  if (warp == C::kWalkWarp) {
    // ---------------------------------------------------------------- the stretch -> pieces
    PrefixLanes lanes;
    if (few) {
      total = prefix_scan_few(p, lanes);
      more = walk_begin_few(p, lanes, total, blockIdx.x, k);
    }
    for (uint32_t put = 0;;) {
      PrefixPiece x{};
      while (more && !walk_piece(p, k, blockIdx.x, x)) more = walk_next(p, k);
      if (!more) x.tiles = 0;
      alive = put < kQueue || wait_all(sy->piece_empty + queue.st, queue.ph ^ 1u);
      if (!alive) break;
      if (lane == 0) {
        sy->piece[queue.st] = x;
        mbar_arrive(sy->piece_full + queue.st);
      }
      __syncwarp();
      queue.next();
      ++put;
      if (x.tiles == 0) break;
      more = walk_next(p, k);
    }
    if (few) prefix_describe_few(p, lanes, total);
  } else if (warp == C::kLoadWarp) {
    // ---------------------------------------------------------------- K and V tiles -> ring
    // The whole warp runs this with warp-uniform values; one elected lane issues (a copy per lane
    // costs about 85 cycles each, one after the other).
    constexpr int R = C::kQuant ? C::kRawStages : S;
    uint64_t* full = C::kQuant ? sy->raw_full : sy->full;
    uint64_t* empty = C::kQuant ? sy->raw_empty : sy->empty;
    constexpr int kStage = C::kQuant ? C::kRawBytes : C::kTileBytes;
    constexpr int kBoxRows = C::kQuant && D == 64 ? kBlockSize / 2 : kBlockSize;  // pool rows of 128 bytes per block and span
    constexpr int kSpans = C::kQuant ? 1 : C::kHalves;
    constexpr int kSpanBytes = kPrefixTile / kBlockSize * kBoxRows * 128;
    unsigned char* to = C::kQuant ? smem + C::kRawOff : ring;
    fence_proxy_async_smem();  // the scan's accesses to the ring come before the copies' writes
    RingPos<R> at;
    uint32_t filled = 0, tiles = 0;
    PrefixPiece x;
    for (take(x); x.tiles > 0; take(x)) {
      const bool two = x.nrows > 128;
      const int32_t* table = p.block_tables + int64_t(x.first_seq) * p.max_blocks_per_seq;
      // tiles read again by the group's other units stay in L2; others are read once
      const uint64_t policy = x.again ? l2_evict_last_policy() : l2_evict_first_policy();
      int ids0 = 0, ids1 = 0, next = tile_id(table, x.nblk, x.tile0, lane);  // of block lane % 8
      uint32_t have0 = 0, have1 = 0;
#pragma unroll 1
      for (int i = 0; i < 2 * x.tiles; ++i) {
        const TileLoad ld = tile_load(two, x.tiles, i);
        const int tile = x.tile0 + ld.tile;
        if (!ld.is_v) {
          const uint32_t have = tile_blocks(p, next, x.nblk, tile, lane);
          if (have != 0xffu && lane < 8 && tile * (kPrefixTile / kBlockSize) + lane < x.nblk && !(have >> lane & 1))
            set_error(p.err, kErrBlockId);
          if (ld.which) { ids1 = next; have1 = have; } else { ids0 = next; have0 = have; }
          if (ld.tile + 1 < x.tiles) next = tile_id(table, x.nblk, tile + 1, lane);
        }
        const uint32_t have = ld.which ? have1 : have0;
        const int pool_tile = (ld.which ? ids1 : ids0) * p.kv_heads + x.kvh;  // pools with tensor maps have < 2^27 tiles
        if (filled >= R && !wait_all(empty + at.st, at.ph ^ 1u)) {
          alive = false;
          break;
        }
        int row[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) row[j] = __shfl_sync(kFull, pool_tile, j) * kBoxRows;
        if (elect_one()) {
          const CUtensorMap* map = ld.is_v ? &tmap_v : &tmap_k;
          unsigned char* dst = to + at.st * kStage;
          uint64_t* bar = full + at.st;
          if (!ld.is_v) sy->mask[(tiles + ld.tile) % kMasks] = uint8_t(have);  // published by the arrival
          if (have) mbar_arrive_expect_tx(bar, __popc(have) * (kSpans * kBoxRows * 128));
          else mbar_arrive(bar);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (have >> j & 1) {
#pragma unroll
              for (int span = 0; span < kSpans; ++span)
                tma_load_2d(dst + span * kSpanBytes + j * (kBoxRows * 128), map, span * 64, row[j], bar, policy);
            }
          }
        }
        __syncwarp();
        ++filled;
        at.next();
      }
      tiles += x.tiles;
      if (!alive) break;
    }
    // the copies in flight land before the CTA can end (the stages filled last)
    for (uint32_t j = 0; j < min(filled, uint32_t(R)); ++j) {
      const uint32_t n = filled - 1 - j;
      (void)mbar_wait_bounded(full + n % R, (n / R) & 1);
    }
  } else if (warp == C::kMmaWarp || warp == C::kMmaWarp + 1) {
    // ---------------------------------------------------------------- products of stream s
    // The whole warp runs this with warp-uniform values; one elected lane issues.
    constexpr uint32_t kDescS = mma_bf16_desc(128, kPrefixTile, false), kDescO = mma_bf16_desc(128, D, true);
    constexpr uint32_t kHi = smem_operand_hi(1024);
    const int s = warp - C::kMmaWarp;
    const uint32_t q_desc = smem_operand(smem_addr(smem) + s * C::kTileBytes, 16);
    const uint32_t k_desc = smem_operand(smem_addr(ring), 16), v_desc = smem_operand(smem_addr(ring), C::kHalfBytes);
    const uint32_t t_s = tmem + s * 128, t_o = tmem + 256 + s * D;
    RingPos<S> at;
    uint32_t cnt = 0, seg = 0, tiles = 0;  // the stream's steps and pieces, and all tiles, before this piece
    uint32_t step = 0;                     // parity of the stream's step
    PrefixPiece x;
    for (take(x); x.tiles > 0; take(x)) {
      const bool two = x.nrows > 128;
      const int ns = stream_steps(x, s);
      bool fresh = true;  // O holds nothing of this piece yet
      if (ns > 0) alive = wait_all(sy->q_ready + s, seg & 1);
#pragma unroll 1
      for (int i = 0; i < 2 * x.tiles && alive; ++i) {
        const TileLoad ld = tile_load(two, x.tiles, i);
        if (!wait_all(sy->full + at.st, at.ph)) {
          alive = false;
          break;
        }
        if (!two && ld.which != s) {  // the other stream's alone
          if (lane == 0) mbar_arrive(sy->empty + at.st);
        } else if (!ld.is_v) {
          // S; P lies over it until the products of the step before are done
          if (cnt > 0 && !wait_all(sy->pv_done + s, step ^ 1u)) {
            alive = false;
            break;
          }
          tc_fence_after();
          const uint32_t kd = __shfl_sync(kFull, k_desc + at.st * (C::kTileBytes >> 4), 0);
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              const uint32_t o = ((j >> 2) * C::kHalfBytes + (j & 3) * 32) >> 4;
              tc_mma_ss(t_s, q_desc + o, kd + o, kHi, kDescS, j > 0);
            }
            tc_commit(sy->s_ready + s);
            tc_commit(sy->empty + at.st);
          }
          __syncwarp();
        } else {
          if (!wait_all(sy->p_ready + s, step) || (fresh && seg > 0 && !wait_all(sy->o_free + s, (seg - 1) & 1))) {
            alive = false;
            break;
          }
          const uint32_t have = sy->mask[(tiles + ld.tile) % kMasks];
          tc_fence_after();
          const uint32_t vd = __shfl_sync(kFull, v_desc + at.st * (C::kTileBytes >> 4), 0);
          // P's two halves lie over S's: columns 0 to 31 and 64 to 95
          if (elect_one()) {
            if (have == 0xffu) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                tc_mma_ts(t_o, t_s + (j >> 2) * 64 + (j & 3) * 8, vd + j * ((kBlockSize * 128) >> 4), kHi, kDescO, j > 0 || !fresh);
            } else {  // the prefix ends in this tile, or a block is missing
              bool on = !fresh;
#pragma unroll 1
              for (int j = 0; j < 8; ++j)
                if (have >> j & 1) {
                  tc_mma_ts(t_o, t_s + (j >> 2) * 64 + (j & 3) * 8, vd + j * ((kBlockSize * 128) >> 4), kHi, kDescO, on);
                  on = true;
                }
            }
            tc_commit(sy->pv_done + s);
            tc_commit(sy->empty + at.st);
          }
          __syncwarp();
          if (have != 0) fresh = false;
          ++cnt;
          step ^= 1u;
        }
        at.next();
      }
      tiles += x.tiles;
      seg += ns > 0;
      if (!alive) break;
    }
    if (!alive) {
      if (lane == 0) tc_commit(sy->drain + s);  // the products in flight end before their memory is given up
      __syncwarp();
      (void)mbar_wait_bounded(sy->drain + s, 0);
    }
  } else if (C::kQuant && warp >= C::kConvertWarp) {
    // ---------------------------------------------------------------- codes -> operand tiles, a thread to a token
    const int t = threadIdx.x & 127;
    RingPos<S> at;
    RingPos<C::kRawStages> from;
    RingPos<C::kSlots> slot;
    uint32_t filled = 0;
    PrefixPiece x;
    for (take(x); x.tiles > 0; take(x)) {
      const bool two = x.nrows > 128;
      const int32_t* table = p.block_tables + int64_t(x.first_seq) * p.max_blocks_per_seq;
      // this token's K and V scales of the tile to come, and its block of the tile after that
      // (past the end, or of a missing block: scales that nothing uses)
      float ks = 0.0f, vs = 0.0f;
      int block = 0;
      auto block_of = [&](int tile) {
        block = load_ahead(table + min((x.tile0 + tile) * (kPrefixTile / kBlockSize) + (t >> 4), x.nblk - 1));
      };
      auto fetch = [&]() {
        const int id = max(0, min(block, int(p.num_blocks) - 1));
        const int64_t row = (int64_t(id) * p.kv_heads + x.kvh) * kBlockSize + (t & 15);
        ks = __int_as_float(load_ahead(p.k_scale + row));
        vs = __int_as_float(load_ahead(p.v_scale + row));
      };
      block_of(0);
      fetch();
      block_of(1);
#pragma unroll 1
      for (int i = 0; i < 2 * x.tiles; ++i) {
        const TileLoad ld = tile_load(two, x.tiles, i);
        if (!wait_all(sy->raw_full + from.st, from.ph) || (filled >= S && !wait_all(sy->empty + at.st, at.ph ^ 1u))) {
          alive = false;
          break;
        }
        if (!ld.is_v) {
          float* to = reinterpret_cast<float*>(smem + C::kSlotOff + slot.st * C::kScaleBytes);
          to[t] = ks;
          to[kPrefixTile + t] = vs;
          mbar_arrive(sy->scales + slot.st);
          slot.next();
          fetch();
          block_of(ld.tile + 2);
        }
        const unsigned char* raw = smem + C::kRawOff + from.st * C::kRawBytes;
        unsigned char* dst = ring + at.st * C::kTileBytes + t * 128;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {  // 16 codes -> 32 bytes
          const int off = D == 128 ? t * 128 + ((c ^ (t & 7)) << 4) : swz_off_pair(t, c);
          const uint4 w = *reinterpret_cast<const uint4*>(raw + off);
          uint4 a, b;
          bf16x4_from_codes<KV>(w.x, a.x, a.y);
          bf16x4_from_codes<KV>(w.y, a.z, a.w);
          bf16x4_from_codes<KV>(w.z, b.x, b.y);
          bf16x4_from_codes<KV>(w.w, b.z, b.w);
          unsigned char* half = dst + (c >> 2) * C::kHalfBytes;
          *reinterpret_cast<uint4*>(half + ((((2 * c) & 7) ^ (t & 7)) << 4)) = a;
          *reinterpret_cast<uint4*>(half + ((((2 * c + 1) & 7) ^ (t & 7)) << 4)) = b;
        }
        mbar_arrive(sy->raw_empty + from.st);
        fence_proxy_async_smem();
        mbar_arrive(sy->full + at.st);
        ++filled;
        at.next();
        from.next();
      }
      if (!alive) break;
    }
  } else if (warp < C::kLoadWarp) {
    // ---------------------------------------------------------------- softmax: rows of stream s, half h of each tile
    const int s = warp >> 3, h = warp >> 2 & 1, wq = warp & 3;
    const int r = threadIdx.x & 127;
    const uint32_t lanes = uint32_t(wq) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t s_addr = tmem + lanes + s * 128 + h * 64, o_addr = tmem + lanes + 256 + s * D + h * (D / 2);
    unsigned char* qt = smem + s * C::kTileBytes;
    // a negative scale goes into the sign of q, so that the largest product is the largest logit;
    // a scale of zero into a zero q, so that a masked logit stays -inf
    const float scale = p.scale_log2 == 0.0f ? 1.0f : fabsf(p.scale_log2);
    const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u, keep = p.scale_log2 == 0.0f ? 0u : ~0u;
    const uint64_t scale2 = f32x2(scale, scale);
    // The two warps of 32 rows meet; and exchange a value per row.  What was written last has to be
    // read before the next is: a maximum is, as both halves' P go into the product that the next S
    // waits for.
    float* mine_at = reinterpret_cast<float*>(smem + C::kMiscOff + kExchangeOff) + (s * 2 + h) * 128 + r;
    const float* other_at = mine_at + (h ? -128 : 128);
    uint32_t pair = 0;
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sy->pair[s][wq]);
      alive = wait_all(&sy->pair[s][wq], pair);
      pair ^= 1u;
    };
    auto exchange = [&](float v) {
      *mine_at = v;
      meet();
      return *other_at;
    };
    // At head_dim 128 the softmaxes of streams that take the same tiles take turns: left alone the
    // streams fall into step, both in their softmax and then both waiting for their products.
    // Measured on GB300, whole calls: 64 sequences over 32768 tokens 60.7 us against 62.6, 256 over 16384
    // (INT8) 148.4 against 160.1; at head_dim 64, where the products are half as long, 59.9 against 56.7.
    uint32_t turns = 0;  // before this piece
    auto turn_done = [&]() {
      if (lane == 0) mbar_arrive(sy->turn + s);
    };
    uint32_t step = 0, tiles = 0;  // parity of the stream's step; all tiles before the next piece
    // The piece done last, whose partial is written while the next one's Q is on its way, and the
    // next one's rows of this stream.
    bool pending = false, any = false;
    int nrows = 0, next_rows = 0;
    int64_t to = 0;
    float m = kMaxFloor, l = 0.0f;
    PrefixPiece x;
    for (;;) {
      take(x);
      const bool two = x.nrows > 128;
      const int ns = x.tiles > 0 ? stream_steps(x, s) : 0;
      const int row0 = two ? s * 128 : 0;                           // the stream's first row within the unit
      next_rows = x.tiles > 0 ? max(0, min(128, x.nrows - row0)) : 0;  // its rows
      constexpr int kChunksQ = D / 16;                              // this thread's half of its row of Q
      uint4 w[kChunksQ];
      if (ns > 0) {
#pragma unroll
        for (int c = 0; c < kChunksQ; ++c) w[c] = make_uint4(0u, 0u, 0u, 0u);
        if (r < next_rows) {
          const auto* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                         prefix_q_row(p, x.first_seq, x.kvh, x.row0 + row0 + r) * D) + h * kChunksQ;
#pragma unroll
          for (int c = 0; c < kChunksQ; ++c) w[c] = __ldg(q + c);
        }
      }
      // Two things to do: Q -> shared memory, and the last piece's partial, which is turned through the
      // Q tile.  Where both pieces have up to 64 rows the partial uses the tile's other half, and Q
      // goes first, so that the next S runs meanwhile.  (Every S that read the tile is done.)
      const bool q_first = nrows <= 64 && next_rows <= 64;
#pragma unroll 1
      for (int job = 0; job < 2 && alive; ++job) {
        if ((job == 0) == q_first) {
          if (ns == 0) continue;
          if (!q_first) {  // the other warp of these rows has turned its half of them
            meet();
            if (!alive) break;
          }
          if (!q_first || r < 64) {
#pragma unroll
            for (int c = 0; c < kChunksQ; ++c) {
              const int at = h * kChunksQ + c;
              w[c] = make_uint4((w[c].x ^ flip) & keep, (w[c].y ^ flip) & keep, (w[c].z ^ flip) & keep, (w[c].w ^ flip) & keep);
              *reinterpret_cast<uint4*>(qt + (at >> 3) * C::kHalfBytes + r * 128 + (((at & 7) ^ (r & 7)) << 4)) = w[c];
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(sy->q_ready + s);
          continue;
        }
        if (!pending) continue;
        // A thread holds half a row, so its stores would touch 32 lines at a time; the warp turns its 32
        // rows through shared memory, 32 values of each row at a time (16 at head_dim 64), and stores whole
        // lines (half lines).
        alive = wait_all(sy->pv_done + s, step ^ 1u);
        if (!alive) break;
        const float l_other = exchange(l);
        if (alive) meet();  // both have read
        if (!alive) break;
        const int live = min(32, nrows - wq * 32);
        if (live > 0) {
          tc_fence_after();
          constexpr int kCols = C::kTileBytes / 8 / 32 / 4;  // columns per round
          constexpr int kChunks = kCols / 4;                 // 16-byte chunks of a row in a round
          // The warp's space in the Q tile: rows 32 wq + 16 h .. + 15 of each span where Q comes after, so
          // that only its pair's Q rows lie there; a quarter of rows 64 to 127 where Q is there already
          // (two quadrants have rows then).
          float* dst = p.acc + (to + wq * 32) * D + h * (D / 2);
          const int first = q_first ? 64 + (wq * 2 + h) * 16 : wq * 32 + h * 16;
          // byte b of the warp's space: span b / 2048, 16 rows of 128 bytes in each
          auto place = [&](int b) { return qt + (b >> 11) * C::kHalfBytes + first * 128 + (b & 2047); };
#pragma unroll 1
          for (int c0 = 0; c0 < D / 2; c0 += kCols) {
            float o[kCols];
            if constexpr (kCols == 32) tmem_ld32(o_addr + c0, o);
            else tmem_ld16(o_addr + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < kChunks; ++e)
              *reinterpret_cast<float4*>(place(lane * (kCols * 4) + ((e ^ (lane % kChunks)) << 4))) =
                  any ? make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            __syncwarp();
#pragma unroll 4
            for (int j = 0; j * (32 / kChunks) < live; ++j) {
              const int row = j * (32 / kChunks) + lane / kChunks, chunk = lane % kChunks;
              if (row < live)
                *reinterpret_cast<float4*>(dst + row * D + c0 + chunk * 4) =
                    *reinterpret_cast<const float4*>(place(row * (kCols * 4) + ((chunk ^ (row % kChunks)) << 4)));
            }
            __syncwarp();
          }
          if (h == 0 && lane < live) p.ml[to + wq * 32 + lane] = make_float2(m, l + l_other);
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sy->o_free + s);
      }
      if (x.tiles == 0 || !alive) break;
      nrows = next_rows;
      to = x.partial + (two ? s * 128 : s * x.nrows);
      const uint32_t tiles0 = tiles;
      tiles += x.tiles;
      pending = ns > 0;
      if (ns == 0) {
        if (h == 0 && r < nrows) p.ml[to + r] = make_float2(kMaxFloor, 0.0f);  // no tile of its own: weighs nothing
        continue;
      }
      const bool idle = wq * 32 >= nrows;  // none of the warp's rows exists
      const int32_t* table = p.block_tables + int64_t(x.first_seq) * p.max_blocks_per_seq;
      int next = tile_id(table, x.nblk, x.tile0 + (two ? 0 : s), lane);
      m = kMaxFloor;
      l = 0.0f;
      any = false;
      const bool turning = D == 128 && two;
#pragma unroll 1
      for (int i = 0; i < ns; ++i, step ^= 1u) {
        const int tile = two ? i : 2 * i + s;
        const uint32_t have = tile_blocks(p, next, x.nblk, x.tile0 + tile, lane);
        any |= have != 0;
        if (i + 1 < ns) next = tile_id(table, x.nblk, x.tile0 + tile + (two ? 1 : 2), lane);
        const uint32_t slot = C::kQuant ? (tiles0 + tile) % C::kSlots : 0;
        alive = wait_all(sy->s_ready + s, step);
        // after S, so that the slot's barrier is at this tile's phase: the stream does not see all
        if constexpr (C::kQuant) alive = alive && wait_all(sy->scales + slot, ((tiles0 + tile) / C::kSlots) & 1);
        const uint32_t turn = turns + i;
        if (alive && turning && (s == 1 || turn > 0)) alive = wait_all(sy->turn + (s ^ 1), (s == 1 ? turn : turn - 1) & 1);
        if (!alive) break;
        if (!idle) {
          tc_fence_after();
          [[maybe_unused]] const auto* ks =
              reinterpret_cast<const ulonglong2*>(smem + C::kSlotOff + slot * C::kScaleBytes) + h * 16;
          [[maybe_unused]] const auto* vs = ks + kPrefixTile / 4;
          const uint32_t mine = have >> (4 * h) & 0xfu;
          // 32 columns at a time: the upper ones for their maximum alone, then the lower ones, whose
          // weights go over their own columns; the upper ones are read again
          float y[32];
          auto fetch = [&](int c) {
            tmem_ld32(s_addr + 32 * c, y);
            tmem_wait_ld();
            if constexpr (C::kQuant) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const ulonglong2 f = ks[8 * c + j];
                f32x2_parts(mul2(f32x2(y[4 * j], y[4 * j + 1]), f.x), y[4 * j], y[4 * j + 1]);
                f32x2_parts(mul2(f32x2(y[4 * j + 2], y[4 * j + 3]), f.y), y[4 * j + 2], y[4 * j + 3]);
              }
            }
            if (mine != 0xfu) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(mine >> (2 * c + j / 16) & 1)) y[j] = -INFINITY;
            }
          };
          auto largest = [&]() {
            float mx[4] = {y[0], y[1], y[2], y[3]};
#pragma unroll
            for (int j = 4; j < 28; j += 8) {
#pragma unroll
              for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], y[j + 2 * u], y[j + 2 * u + 1]);
            }
            return max3(max3(mx[0], y[28], y[29]), max3(mx[1], y[30], y[31]), fmaxf(mx[2], mx[3]));
          };
          fetch(1);
          float bm = largest();
          fetch(0);
          bm = fmaxf(bm, largest()) * scale;
          bm = fmaxf(bm, exchange(bm));
          if (!alive) break;
          const bool grow = bm > m + kMaxSlack;
          if (__any_sync(kFull, grow)) {
            const float mu = grow ? bm : m, f = fast_exp2(m - mu);
            m = mu;
            l *= f;
            if (i > 0) {
              // every product into O is done: S was issued after the last
#pragma unroll 1
              for (int j = 0; j < D / 32; ++j) {
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
          auto weights = [&](int c) {
            // step by step over all 32: one value's chain of operations is long
#pragma unroll
            for (int j = 0; j < 16; ++j) f32x2_parts(fma2(f32x2(y[2 * j], y[2 * j + 1]), scale2, neg), y[2 * j], y[2 * j + 1]);
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = fast_exp2(y[j]);
            if constexpr (C::kQuant) {
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[j & 1] = add2(sum[j & 1], f32x2(y[2 * j], y[2 * j + 1]));
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const ulonglong2 f = vs[8 * c + j];
                f32x2_parts(mul2(f32x2(y[4 * j], y[4 * j + 1]), f.x), y[4 * j], y[4 * j + 1]);
                f32x2_parts(mul2(f32x2(y[4 * j + 2], y[4 * j + 3]), f.y), y[4 * j + 2], y[4 * j + 3]);
              }
            }
            float pw[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t v = pack_bf16x2(y[2 * j], y[2 * j + 1]);
              pw[j] = __uint_as_float(v);
              if constexpr (!C::kQuant) sum[j & 1] = add2(sum[j & 1], f32x2(bf16lo(v), bf16hi(v)));
            }
            tmem_st16(s_addr + 16 * c, pw);
          };
          weights(0);
          if (turning) turn_done();  // the other's loads and maximum take as long as the rest
          fetch(1);
          weights(1);
          float sum_lo, sum_hi;
          f32x2_parts(add2(sum[0], sum[1]), sum_lo, sum_hi);
          l += sum_lo + sum_hi;
          tmem_wait_st();
          tc_fence_before();
        } else if (turning) {
          turn_done();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sy->p_ready + s);
      }
      if (!alive) break;
      if (turning) turns += ns;
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

template <KvType KV, int D>
cudaError_t launch_prefix_tc(const PrefixParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
  using C = PrefixCfg<KV, D>;
  auto kern = prefix_tc_kernel<KV, D>;
  static std::atomic<bool> attr_done[64];  // per device: the shared-memory limit is raised
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_done[dev].load(std::memory_order_relaxed)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev].store(true, std::memory_order_relaxed);
  }
  return launch_pdl(kern, dim3(p.grid), dim3(C::kThreads), C::kSmemBytes, stream, tk, tv, p);
}

}  // namespace pkv
