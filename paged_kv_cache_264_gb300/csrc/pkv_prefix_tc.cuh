// pkv_prefix_tc.cuh -- the prefix pass of shared-prefix decode on the fifth-generation tensor
// core: up to 256 query rows of one (group, kv head) against a stretch of its prefix, a CTA per
// SM, each with its stretch of the work line (pkv_prefix.cuh).
//
// Two streams of 128 rows run through the CTA.  With more than 128 rows in the group they hold
// different rows and take every 128-token tile; with up to 128 rows both hold the same rows and
// take the even and the odd tiles, so that either way one stream's softmax runs under the other's
// products.  Per stream and tile:
//     S = Q K^T    128 x 128 x D, both operands in shared memory, S in tensor memory (fp32)
//     P = 2^(S * scale - m)    a thread to a row, its logits in registers: no shuffles
//     O += P V     128 x D x 128, P in tensor memory (bf16, over S's columns), V as it lies in the
//                  pool (token-major, the contracted index outermost: an MN-major operand)
// The softmax hands P over in halves of 64 tokens, so that the first half's product over V runs under
// the second half's softmax.  S is formed for whole tiles: its products read both operands from
// shared memory, 8 KB for 64 cycles of arithmetic at 128 columns, which is what shared memory
// delivers; at 64 columns they took as long for half the work.
// The running maximum is lazy (kMaxSlack): O is rescaled in tensor memory only when a row's
// logits pass its maximum by 2^8.  P enters the product as bf16, and the softmax sum adds the
// same rounded weights, so that numerator and denominator agree.
//
// INT8 and FP8 pools: TMA brings codes and scales into a ring of their own, and a warpgroup turns
// the codes into bf16 operand tiles, which holds every INT8 and E4M3 code exactly.  The scales stay
// out of the operands: a token's K scale multiplies its fp32 logit, and its V scale goes into its
// weight before that is rounded to bf16 (so the weights are rounded once, as in a bf16 pool; the
// sum adds the unrounded ones, since the rounded ones carry the scale).
//
// Warps: two warpgroups of softmax (one per stream, which also load Q and write the partials),
// one warp that fills the ring of K and V tiles by TMA (8 blocks to a tile, each wherever it lies
// in the pool), one warp per stream that issues its products (one for both let a stream's waits
// hold up the other's products), and the converting warpgroup for INT8 and FP8.
//
// A barrier's wait is for a parity, which tells a phase from the one before it only if the waiter
// has seen that one complete.  So one warp fills the ring, and each issuing warp waits for and
// releases every stage in ring order, those of the other stream's tiles too (a warp that filled
// only K stages, or skipped stages, could run into one still in use).
//
// Every wait is bounded; after one that gave up the
// CTA takes no further work, lets its copies and products land, frees its tensor memory and ends.
//
// A prefix ends at a block (16 tokens), not at a tile: the product over V takes only the steps of
// 16 tokens that exist, so nothing has to be zeroed, and the logits behind them are masked.
#pragma once

#include "pkv_decode_mma.cuh"
#include "pkv_prefix.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

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
  static constexpr int kRawStages = kQuant ? (D == 128 ? 3 : 8) : 0;
  // Scales of a tile wait in a slot until its softmax has used them.  The slot of tile n (in load
  // order) is written again for tile n + kSlots, when K of that tile takes a ring stage; V of tile
  // n lies at least 2 kSlots - 3 stages before it, so it has been released, and its product came
  // after its softmax.
  static constexpr int kSlots = kQuant ? (D == 128 ? 4 : 8) : 0;
  static_assert(!kQuant || 2 * kSlots - 3 >= kStages, "a scale slot is free when it is written again");
  static constexpr int kThreads = kQuant ? 512 : 384;
  static constexpr int kLoadWarp = 8, kMmaWarp = 9, kDescribeWarp = 11, kConvertWarp = 12;  // 9 and 10: one per stream
  // Registers: the softmax threads hold a row of 128 logits; what the other warpgroups give up
  // goes to them.  The shares' sum is checked against the kernel's own count before a launch.
  static constexpr int kSoftmaxRegs = kQuant ? 184 : 200;
  static constexpr int kIssueRegs = kQuant ? 64 : 96, kConvertRegs = 80;
  static constexpr int kRegSum = 128 * (2 * kSoftmaxRegs + kIssueRegs + (kQuant ? kConvertRegs : 0));
  static constexpr int kMiscBytes = 1024;
  static constexpr int kRingOff = 2 * kTileBytes;                // Q tiles of both streams first
  static constexpr int kRawOff = kRingOff + kStages * kTileBytes;
  static constexpr int kSlotOff = kRawOff + kRawStages * kRawBytes;
  static constexpr int kSmemBytes = kMiscBytes + 1024 + kSlotOff + kSlots * kScaleBytes;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(size_t(kStages) * kTileBytes >= prefix_scan_bytes(kMaxPrefixGroups), "the scan fits the ring");
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

// Barriers and flags of one CTA, at the start of its shared memory.
struct PrefixSync {
  uint64_t full[16], empty[16];          // operand ring stages
  uint64_t raw_full[8], raw_empty[8];    // code ring stages
  uint64_t scales[8];                    // scale slots
  uint64_t q_ready[2], s_ready[2], o_free[2];   // per stream
  uint64_t p_ready[2][2], pv_done[2][2];        // per stream and half of a tile
  uint64_t drain[2];
  uint32_t tmem;
  uint32_t abort;
};
static_assert(sizeof(PrefixSync) <= 1008, "barriers fit their space");

// A place in a ring of N stages: the stage, and the parity of the phase that its current use
// completes.
template <int N>
struct RingPos {
  uint32_t st, ph;
  __device__ __forceinline__ void advance(uint32_t by) {
    st += by;
    while (st >= N) {
      st -= N;
      ph ^= 1u;
    }
  }
  static __device__ __forceinline__ RingPos at(uint32_t index) { return {index % N, (index / N) & 1u}; }
};

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

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
// Roles ask for a tile's ids one step ahead of their use: a table entry is a global-memory round trip
// away, and any use of the loaded value here would wait for it.
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
  constexpr int kRaw = C::kQuant ? C::kRawStages : 1, kSlots = C::kQuant ? C::kSlots : 1;
  constexpr uint32_t kFull = 0xffffffffu;
  extern __shared__ unsigned char smem_raw[];
  auto* sy = reinterpret_cast<PrefixSync*>((reinterpret_cast<uintptr_t>(smem_raw) + 15) & ~uintptr_t(15));
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + C::kMiscBytes + 1023) & ~uintptr_t(1023));
  unsigned char* ring = smem + C::kRingOff;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
      mbar_init(sy->q_ready + s, 128);
      mbar_init(sy->s_ready + s, 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sy->p_ready[s][h], 128);
        mbar_init(&sy->pv_done[s][h], 1);
      }
      mbar_init(sy->o_free + s, 128);
      mbar_init(sy->drain + s, 1);
    }
    sy->abort = 0;
    fence_barrier_init();
    prefetch_tensor_map(&tmap_k);
    prefetch_tensor_map(&tmap_v);
  }
  if (warp == C::kMmaWarp) tmem_alloc(&sy->tmem, C::kTmemCols);
  griddep_wait();  // inputs may come from the previous kernel in the stream
  // The scan of up to 32 groups is each warp's own, and one describes the sequences beside the work;
  // that of many lies where the ring will be, and is used up first.
  const bool few = p.num_groups <= kFewGroups;
  PrefixLanes lanes;
  PrefixWalk k;
  int64_t total;
  bool more;
  if (few) {
    total = prefix_scan_few(p, lanes);
    more = walk_begin_few(p, lanes, total, blockIdx.x, k);
  } else {
    PrefixScan sc{reinterpret_cast<longlong2*>(ring) + 32, reinterpret_cast<longlong2*>(ring)};
    total = prefix_scan<C::kThreads>(p, sc);
    prefix_describe_many(p, sc, total, warp, C::kThreads / 32);
    more = walk_begin(p, sc, total, blockIdx.x, k);
  }
  tc_fence_before();
  __syncthreads();  // the ring's memory is free again; the barriers and the tensor memory are there
  tc_fence_after();
  const uint32_t tmem = sy->tmem;
  volatile uint32_t* abort = &sy->abort;
  // A whole warp's wait: the same answer on every lane; false after the time limit, or once another
  // warp of the CTA gave up.  A barrier that is already there costs one test and a vote.
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    bool ok = false;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t tries = 0; tries < (1u << 26); ++tries) {
      if (__all_sync(kFull, mbar_try_wait(bar, parity))) {
        ok = true;
        break;
      }
      if ((tries & 63u) == 63u && __any_sync(kFull, *abort != 0 || global_timer_ns() - t0 > kWaitTimeoutNs)) break;
    }
    return ok;
  };

  // Steps of stream s over n tiles: which of the unit's tiles it takes, and how many.
  // two: the streams hold different rows; else they share the tiles out between them.
  auto steps_of = [&](bool two, int nrows, int n, int s) { return two ? (s == 0 || nrows > 128 ? n : 0) : (n + 1 - s) / 2; };

  if (warp >= C::kLoadWarp && warp < C::kLoadWarp + 4) regs_down<C::kIssueRegs>();
  if (warp == C::kLoadWarp) {
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
    uint32_t it = 0;           // stages filled so far
    bool alive = true;
    for (; more && alive; more = walk_next(p, blockIdx.x, k)) {
      const bool two = k.x.rows > 128;
      const int nblk = __ldg(p.prefix_lens + k.g) / kBlockSize;
      const int32_t* table = p.block_tables + int64_t(k.x.first_seq) * p.max_blocks_per_seq;
      // tiles read again by the group's other units stay in L2; others are read once
      const uint64_t policy = k.x.units > 1 ? l2_evict_last_policy() : l2_evict_first_policy();
      const int n = k.tile1 - k.tile0;
      int ids[2] = {}, next = tile_id(table, nblk, k.tile0, lane);  // of block lane % 8
      uint32_t blocks[2] = {};
      for (int i = 0; i < 2 * n; ++i, ++it) {
        const TileLoad ld = tile_load(two, n, i);
        if (!ld.is_v) {
          const uint32_t have = tile_blocks(p, next, nblk, k.tile0 + ld.tile, lane);
          if (have != 0xffu) {
            const int j = (k.tile0 + ld.tile) * (kPrefixTile / kBlockSize) + lane;
            if (lane < 8 && j < nblk && !(have >> lane & 1)) set_error(p.err, kErrBlockId);
          }
          if (ld.which) { ids[1] = next; blocks[1] = have; } else { ids[0] = next; blocks[0] = have; }
          if (ld.tile + 1 < n) next = tile_id(table, nblk, k.tile0 + ld.tile + 1, lane);
        }
        const int tile = (ld.which ? ids[1] : ids[0]) * p.kv_heads + k.kvh;  // pools with tensor maps have < 2^27 tiles
        const uint32_t have = ld.which ? blocks[1] : blocks[0];
        const CUtensorMap* map = ld.is_v ? &tmap_v : &tmap_k;
        const uint32_t st = it % R;
        if (it >= R && !wait_all(empty + st, ((it / R) & 1) ^ 1)) {
          alive = false;
          break;
        }
        int row[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) row[j] = __shfl_sync(kFull, tile, j) * kBoxRows;
        if (elect_one()) {
          if (have) mbar_arrive_expect_tx(full + st, __popc(have) * (kSpans * kBoxRows * 128));
          else mbar_arrive(full + st);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (have >> j & 1) {
#pragma unroll
              for (int x = 0; x < kSpans; ++x)
                tma_load_2d(to + st * kStage + x * kSpanBytes + j * (kBoxRows * 128), map, x * 64, row[j], full + st, policy);
            }
          }
        }
        __syncwarp();
      }
    }
    if (!alive && lane == 0) {
      *abort = 1;
      set_error(p.err, kErrTimeout);
    }
    // the copies in flight land before the CTA can end (the stages filled last)
    for (uint32_t j = it > R ? it - R : 0; j < it; ++j) (void)mbar_wait_bounded(full + j % R, (j / R) & 1);
  } else if (warp == C::kMmaWarp || warp == C::kMmaWarp + 1) {
    // ---------------------------------------------------------------- products of stream s
    // The whole warp runs this with warp-uniform values; one elected lane issues.
    constexpr uint32_t kDescS = mma_bf16_desc(128, kPrefixTile, false), kDescO = mma_bf16_desc(128, D, true);
    constexpr uint32_t kHi = smem_operand_hi(1024);
    auto uniform = [](uint32_t x) { return __shfl_sync(kFull, x, 0); };  // tells the compiler that it is
    const int s = uniform(warp - C::kMmaWarp);
    const uint32_t q_desc = uniform(smem_operand(smem_addr(smem) + s * C::kTileBytes, 16));
    const uint32_t k_desc = smem_operand(smem_addr(ring), 16), v_desc = smem_operand(smem_addr(ring), C::kHalfBytes);
    const uint32_t t_s = uniform(tmem + s * 128), t_o = uniform(tmem + 256 + s * D);
    RingPos<S> at{0, 0};  // the next stage in ring order
    uint32_t cnt = 0;     // steps of the stream before this piece
    uint32_t seg = 0;     // pieces that had work for it
    bool alive = true;
    // Wait for the stage at `at`; pass over one that the other stream alone uses.
    auto ready = [&]() { return wait_all(sy->full + at.st, at.ph); };
    auto pass = [&](int stages) {
      for (int j = 0; j < stages; ++j) {
        if (!ready()) return false;
        if (lane == 0) mbar_arrive(sy->empty + at.st);
        at.advance(1);
      }
      return true;
    };
    for (; more && alive; more = walk_next(p, blockIdx.x, k)) {
      const bool two = k.x.rows > 128;
      const int n = k.tile1 - k.tile0, ns = steps_of(two, k.nrows, n, s);
      if (ns == 0) {
        alive = pass(2 * n);
        continue;
      }
      const int nblk = __ldg(p.prefix_lens + k.g) / kBlockSize;
      const int32_t* table = p.block_tables + int64_t(k.x.first_seq) * p.max_blocks_per_seq;
      int next = tile_id(table, nblk, k.tile0 + (two ? 0 : s), lane);
      // stages of the other stream around this one's K and V of a step: of two tiles' K, K, V, V this
      // stream takes one each (the last tile may be alone)
      auto others = [&](int i) { return two ? 0 : min(2, n - 2 * i) - 1; };
      // S of step i
      auto issue_s = [&](int i) {
        if (s == 1 && !pass(others(i))) return false;
        // P lies over S until its products are done
        if (!ready() || (cnt + i > 0 && !wait_all(&sy->pv_done[s][1], (cnt + i - 1) & 1))) return false;
        tc_fence_after();
        const uint32_t kd = uniform(k_desc + at.st * (C::kTileBytes >> 4));
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const uint32_t o = ((j >> 2) * C::kHalfBytes + (j & 3) * 32) >> 4;
            tc_mma_ss(t_s, q_desc + o, kd + o, kHi, kDescS, j > 0);
          }
          tc_commit(sy->s_ready + s);
          tc_commit(sy->empty + at.st);  // K of the tile, once S is done
        }
        __syncwarp();
        at.advance(1);
        return s == 1 || pass(others(i));
      };
      bool fresh = true;  // O holds nothing of this piece yet
      alive = wait_all(sy->q_ready + s, seg & 1) && issue_s(0);
      if (alive && seg > 0) alive = wait_all(sy->o_free + s, (seg - 1) & 1);
      uint32_t have = 0;
      // one half of a tile at a time (rolled: the CTA's roles share one instruction cache)
#pragma unroll 1
      for (int g = 0; g < 2 * ns && alive; ++g) {
        const int i = g >> 1, h = g & 1;
        if (h == 0) {
          const int tile = two ? i : 2 * i + s;
          have = tile_blocks(p, next, nblk, k.tile0 + tile, lane);
          if (i + 1 < ns) next = tile_id(table, nblk, k.tile0 + tile + (two ? 1 : 2), lane);
          alive = (s == 0 || pass(others(i))) && ready();
        }
        alive = alive && wait_all(&sy->p_ready[s][h], (cnt + i) & 1);
        if (!alive) break;
        tc_fence_after();
        const uint32_t vd = uniform(v_desc + at.st * (C::kTileBytes >> 4) + h * ((64 * 128) >> 4)), t_p = uniform(t_s + h * 64);
        const uint32_t mine = have >> (4 * h) & 0xfu;
        if (elect_one()) {
          if (mine == 0xfu) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tc_mma_ts(t_o, t_p + j * 8, vd + j * ((kBlockSize * 128) >> 4), kHi, kDescO, j > 0 || !fresh);
          } else {  // the prefix ends in this half, or a block is missing
            bool acc = !fresh;
#pragma unroll 1
            for (int j = 0; j < 4; ++j)
              if (mine >> j & 1) {
                tc_mma_ts(t_o, t_p + j * 8, vd + j * ((kBlockSize * 128) >> 4), kHi, kDescO, acc);
                acc = true;
              }
          }
          tc_commit(&sy->pv_done[s][h]);
          if (h == 1) tc_commit(sy->empty + at.st);
        }
        if (mine) fresh = false;
        __syncwarp();
        if (h == 1) {
          at.advance(1);
          alive = (s == 1 || pass(others(i))) && (i + 1 == ns || issue_s(i + 1));
        }
      }
      // streams that share the tiles out: the last tile is alone where n is odd, and stream 1 passes it
      if (alive && !two && s == 1 && (n & 1)) alive = pass(2);
      cnt += ns;
      ++seg;
    }
    if (!alive) {
      if (lane == 0) {
        *abort = 1;
        set_error(p.err, kErrTimeout);
        tc_commit(sy->drain + s);  // the products in flight end before their memory is given up
      }
      __syncwarp();
      (void)mbar_wait_bounded(sy->drain + s, 0);
    }
  } else if (warp == C::kDescribeWarp) {
    if (few) prefix_describe_few(p, lanes, total);
  } else if (C::kQuant && warp >= C::kConvertWarp) {
    // ---------------------------------------------------------------- codes -> operand tiles, a thread to a token
    regs_down<C::kConvertRegs>();
    const int t = threadIdx.x & 127;
    uint32_t it = 0, tiles = 0;  // stages and tiles converted so far
    bool alive = true;
    for (; more && alive; more = walk_next(p, blockIdx.x, k)) {
      const bool two = k.x.rows > 128;
      const int n = k.tile1 - k.tile0;
      const int nblk = __ldg(p.prefix_lens + k.g) / kBlockSize;
      const int32_t* table = p.block_tables + int64_t(k.x.first_seq) * p.max_blocks_per_seq;
      // this token's K and V scales of the tile to come, and its block of the tile after that
      float ks = 0.0f, vs = 0.0f;
      auto block_of = [&](int tile) {
        const int j = (k.tile0 + tile) * (kPrefixTile / kBlockSize) + (t >> 4);
        return load_ahead(table + min(j, nblk - 1));  // past the end: scales that nothing uses
      };
      auto fetch = [&](int id) {
        id = max(0, min(id, int(p.num_blocks) - 1));  // a missing block's scales are not used either
        const int64_t row = (int64_t(id) * p.kv_heads + k.kvh) * kBlockSize + (t & 15);
        ks = __int_as_float(load_ahead(p.k_scale + row));
        vs = __int_as_float(load_ahead(p.v_scale + row));
      };
      fetch(block_of(0));
      int block = block_of(1);
      for (int i = 0; i < 2 * n; ++i, ++it) {
        const TileLoad ld = tile_load(two, n, i);
        const uint32_t st = it % S, rs = it % kRaw;
        if (!wait_all(sy->raw_full + rs, (it / kRaw) & 1) || (it >= S && !wait_all(sy->empty + st, ((it / S) & 1) ^ 1))) {
          alive = false;
          break;
        }
        const unsigned char* raw = smem + C::kRawOff + rs * C::kRawBytes;
        unsigned char* dst = ring + st * C::kTileBytes + t * 128;
        if (!ld.is_v) {
          const uint32_t slot = (tiles + ld.tile) % kSlots;
          float* to = reinterpret_cast<float*>(smem + C::kSlotOff + slot * C::kScaleBytes);
          to[t] = ks;
          to[kPrefixTile + t] = vs;
          mbar_arrive(sy->scales + slot);
          fetch(block);
          block = block_of(ld.tile + 2);
        }
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
        mbar_arrive(sy->raw_empty + rs);
        fence_proxy_async_smem();
        mbar_arrive(sy->full + st);
      }
      tiles += n;
    }
    if (!alive && lane == 0) {
      *abort = 1;
      set_error(p.err, kErrTimeout);
    }
  } else if (warp < C::kLoadWarp) {
    // ---------------------------------------------------------------- softmax, one thread per row
    regs_up<C::kSoftmaxRegs>();
    const int s = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t s_addr = tmem + lanes + s * 128, o_addr = tmem + lanes + 256 + s * D;
    unsigned char* qt = smem + s * C::kTileBytes;
    // a negative scale goes into the sign of q, so that the largest product is the largest logit;
    // a scale of zero into a zero q, so that a masked logit stays -inf
    const float scale = p.scale_log2 == 0.0f ? 1.0f : fabsf(p.scale_log2);
    const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u, keep = p.scale_log2 == 0.0f ? 0u : ~0u;
    const uint64_t scale2 = f32x2(scale, scale);
    uint32_t cnt = 0, tiles = 0;  // this stream's steps and all tiles before this piece
    bool alive = true;
    // The piece done last, whose partial is written while the next one's Q is on its way.
    bool pending = false, any = false, idle = false;
    int nrows = 0;
    int64_t to = 0;
    float m = kMaxFloor, l = 0.0f;
    for (;;) {
      uint4 w[D / 8];  // this thread's row of Q of the piece at k
      if (more) {
        const int row = (k.x.rows > 128 ? s * 128 : 0) + r;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) w[c] = make_uint4(0u, 0u, 0u, 0u);
        if (row < k.nrows) {
          const auto* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                         prefix_q_row(p, k.x, k.kvh, k.row0 + row) * D);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) w[c] = __ldg(q + c);
        }
      }
      if (pending) {
        // ---- its partial.  A thread holds a row, so its stores would touch 32 lines at a time; the
        // warp turns its 32 rows through its part of the Q tile (free: every S is done), 64 values
        // of each row at a time (32 at head_dim 64), and stores whole lines.
        if (!wait_all(&sy->pv_done[s][1], (cnt - 1) & 1)) {
          alive = false;
          break;
        }
        if (!idle) {
          tc_fence_after();
          unsigned char* turn = qt + (warp & 3) * (C::kTileBytes / 4);
          constexpr int kCols = C::kTileBytes / 4 / 32 / 4;  // columns per round
          constexpr int kChunks = kCols / 4;                 // 16-byte chunks of a row in a round
          const int wrow = (warp & 3) * 32, live = min(32, nrows - wrow);
          float* dst = p.acc + (to + wrow) * D;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += kCols) {
#pragma unroll
            for (int h = 0; h < kCols; h += 32) {
              float o[32];
              tmem_ld32(o_addr + c0 + h, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<float4*>(turn + lane * (kCols * 4) + (((h / 4 + e) ^ (lane % kChunks)) << 4)) =
                    any ? make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            __syncwarp();
#pragma unroll 4
            for (int j = 0; j < kChunks; ++j) {
              const int row = j * (32 / kChunks) + lane / kChunks, chunk = lane % kChunks;
              if (row < live)
                *reinterpret_cast<float4*>(dst + row * D + c0 + chunk * 4) =
                    *reinterpret_cast<const float4*>(turn + row * (kCols * 4) + ((chunk ^ (row % kChunks)) << 4));
            }
            __syncwarp();
          }
          if (r < nrows) p.ml[to + r] = make_float2(m, l);
          tc_fence_before();
        }
        mbar_arrive(sy->o_free + s);
        pending = false;
      }
      if (!more) break;
      const bool two = k.x.rows > 128;
      const int n = k.tile1 - k.tile0;
      const int ns = steps_of(two, k.nrows, n, s);
      const uint32_t tiles0 = tiles;
      tiles += n;
      const int row0 = two ? s * 128 : 0;         // the stream's first row within the unit
      nrows = min(128, k.nrows - row0);           // its rows
      to = k.partial + (two ? s * 128 : s * k.x.rows);
      if (ns == 0) {
        if (r < nrows) p.ml[to + r] = make_float2(kMaxFloor, 0.0f);  // no tile of its own: weighs nothing
        more = walk_next(p, blockIdx.x, k);
        continue;
      }
      const int tile0 = k.tile0, nblk = __ldg(p.prefix_lens + k.g) / kBlockSize;
      const int32_t* table = p.block_tables + int64_t(k.x.first_seq) * p.max_blocks_per_seq;
      int next = tile_id(table, nblk, tile0 + (two ? 0 : s), lane);
      {  // Q -> shared memory, swizzled; its last reader was the last step's S, which this thread saw
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          w[c] = make_uint4((w[c].x ^ flip) & keep, (w[c].y ^ flip) & keep, (w[c].z ^ flip) & keep, (w[c].w ^ flip) & keep);
          *reinterpret_cast<uint4*>(qt + (c >> 3) * C::kHalfBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = w[c];
        }
        fence_proxy_async_smem();
        mbar_arrive(sy->q_ready + s);
      }
      idle = (warp & 3) * 32 >= nrows;  // none of the warp's rows exists
      m = kMaxFloor;
      l = 0.0f;
      any = false;
      uint32_t have = 0, slot = 0;
#pragma unroll 1
      for (int g = 0; g < 2 * ns; ++g) {
        const int i = g >> 1, h = g & 1;
        if (h == 0) {
          const int tile = two ? i : 2 * i + s;
          have = tile_blocks(p, next, nblk, tile0 + tile, lane);
          any |= have != 0;
          if (i + 1 < ns) next = tile_id(table, nblk, tile0 + (two ? i + 1 : 2 * i + 2 + s), lane);
          if constexpr (C::kQuant) {
            slot = (tiles0 + tile) % kSlots;
            // after S, so that the slot's barrier is at this tile's phase: the stream does not see all
            alive = wait_all(sy->s_ready + s, (cnt + i) & 1) && wait_all(sy->scales + slot, ((tiles0 + tile) / kSlots) & 1);
          } else {
            alive = wait_all(sy->s_ready + s, (cnt + i) & 1);
          }
          if (!alive) break;
        }
        {
          if (!idle) {
            const auto* ks = reinterpret_cast<const ulonglong2*>(smem + C::kSlotOff + slot * C::kScaleBytes) + h * 16;
            [[maybe_unused]] const auto* vs = ks + kPrefixTile / 4;
            const uint32_t mine = have >> (4 * h) & 0xfu;
            tc_fence_after();
            float x[64];
            tmem_ld32(s_addr + h * 64, x);
            tmem_ld32(s_addr + h * 64 + 32, x + 32);
            tmem_wait_ld();
            if constexpr (C::kQuant) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const ulonglong2 f = ks[j];
                f32x2_parts(mul2(f32x2(x[4 * j], x[4 * j + 1]), f.x), x[4 * j], x[4 * j + 1]);
                f32x2_parts(mul2(f32x2(x[4 * j + 2], x[4 * j + 3]), f.y), x[4 * j + 2], x[4 * j + 3]);
              }
            }
            if (mine != 0xfu) {
#pragma unroll
              for (int j = 0; j < 64; ++j)
                if (!(mine >> (j / 16) & 1)) x[j] = -INFINITY;
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int j = 4; j < 64; ++j) mx[j & 3] = fmaxf(mx[j & 3], x[j]);
            const float bm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
            const bool grow = bm > m + kMaxSlack;
            if (__any_sync(kFull, grow)) {
              const float mu = grow ? bm : m, f = fast_exp2(m - mu);
              m = mu;
              l *= f;
              if (g > 0) {
                // every product into O so far has to be done: the half's before this one is the last
                alive = wait_all(&sy->pv_done[s][h ^ 1], (cnt + i - (h ^ 1)) & 1);
                tc_fence_after();
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
            uint32_t pw[32];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {  // four tokens at a time: one read of their V scales
              float e[4];
              f32x2_parts(fma2(f32x2(x[2 * j], x[2 * j + 1]), scale2, neg), e[0], e[1]);
              f32x2_parts(fma2(f32x2(x[2 * j + 2], x[2 * j + 3]), scale2, neg), e[2], e[3]);
#pragma unroll
              for (int u = 0; u < 4; ++u) e[u] = fast_exp2(e[u]);
              if constexpr (C::kQuant) {
                const uint64_t p0 = f32x2(e[0], e[1]), p1 = f32x2(e[2], e[3]);
                sum[0] = add2(sum[0], p0);
                sum[1] = add2(sum[1], p1);
                const ulonglong2 f = vs[j / 2];
                f32x2_parts(mul2(p0, f.x), e[0], e[1]);
                f32x2_parts(mul2(p1, f.y), e[2], e[3]);
              }
              pw[j] = pack_bf16x2(e[0], e[1]);
              pw[j + 1] = pack_bf16x2(e[2], e[3]);
              if constexpr (!C::kQuant) {
                sum[0] = add2(sum[0], f32x2(bf16lo(pw[j]), bf16hi(pw[j])));
                sum[1] = add2(sum[1], f32x2(bf16lo(pw[j + 1]), bf16hi(pw[j + 1])));
              }
            }
            tmem_st32(s_addr + h * 64, pw);
            float a, b;
            f32x2_parts(add2(sum[0], sum[1]), a, b);
            l += a + b;
            tmem_wait_st();
            tc_fence_before();
          }
          mbar_arrive(&sy->p_ready[s][h]);
        }
      }
      if (!alive) break;
      cnt += ns;
      pending = true;
      more = walk_next(p, blockIdx.x, k);
    }
    if (!alive && lane == 0) {
      *abort = 1;
      set_error(p.err, kErrTimeout);
    }
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
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    cudaFuncAttributes a;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, kern);
    if (e != cudaSuccess) return e;
    // the warpgroups' register shares come out of what the CTA is launched with
    if (a.numRegs * C::kThreads < C::kRegSum) return cudaErrorInvalidConfiguration;
    if (dev >= 0 && dev < 64) attr_done[dev].store(true, std::memory_order_relaxed);
  }
  return launch_pdl(kern, dim3(p.grid), dim3(C::kThreads), C::kSmemBytes, stream, tk, tv, p);
}

}  // namespace pkv
