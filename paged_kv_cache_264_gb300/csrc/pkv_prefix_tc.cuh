// pkv_prefix_tc.cuh -- the prefix pass of shared-prefix decode on the fifth-generation tensor
// core: up to 256 query rows of one (group, kv head) against a stretch of its prefix, a CTA per
// SM, each with its stretch of the work line (pkv_prefix.cuh).
//
// Two streams of 128 rows run through the CTA.  With more than 128 rows in the group they hold
// different rows and take every 128-token tile; with up to 128 rows both hold the same rows and
// take the even and the odd tiles, so that either way one stream's softmax runs under the other's
// products.  Per stream and tile:
//     S = Q K^T    128 x 128 x D, both operands in shared memory, S in tensor memory (fp32)
//     P = 2^(S * scale - m)    a thread to a row, all 128 logits in registers: no shuffles
//     O += P V     128 x D x 128, P in tensor memory (bf16, over S's columns), V as it lies in the
//                  pool (token-major, the contracted index outermost: an MN-major operand)
// The running maximum is lazy (kMaxSlack): O is rescaled in tensor memory only when a row's
// logits pass its maximum by 2^8.  P enters the product as bf16, and the softmax sum adds the
// same rounded weights, so that numerator and denominator agree.
//
// Warps: two warpgroups of softmax (one per stream, which also load Q and write the partials),
// one warp that fills the ring of K and V tiles by TMA (8 blocks to a tile, each wherever it lies
// in the pool), one that issues the products.  Every wait is bounded; after one that gave up the
// CTA takes no further work, lets its copies and products land, frees its tensor memory and ends.
//
// A prefix ends at a block (16 tokens), not at a tile: the product over V takes only the steps of
// 16 tokens that exist, so nothing has to be zeroed, and the logits behind them are masked.
#pragma once

#include "pkv_decode.cuh"
#include "pkv_prefix.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

template <KvType KV, int D>
struct PrefixCfg {
  static constexpr int kHalves = D / 64;                         // 128-byte spans of a 16-bit row
  static constexpr int kTileBytes = kPrefixTile * D * 2;         // one K, V or Q tile, 16-bit
  static constexpr int kHalfBytes = kPrefixTile * 128;           // one span of all its rows
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kThreads = 320;
  static constexpr int kTmaWarp = 8, kMmaWarp = 9;
  static constexpr int kMiscBytes = 1024;
  static constexpr int kRingOff = 2 * kTileBytes;                // Q tiles of both streams first
  static constexpr int kSmemBytes = kMiscBytes + 1024 + kRingOff + kStages * kTileBytes;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(size_t(kStages) * kTileBytes >= prefix_scan_bytes(kMaxPrefixGroups), "the scan fits the ring");
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

// Barriers and flags of one CTA, at the start of its shared memory.
struct PrefixSync {
  uint64_t full[16], empty[16];        // ring stages
  uint64_t q_ready[2], s_ready[2], p_ready[2], pv_done[2], o_free[2];  // per stream
  uint64_t drain;
  uint32_t tmem;
  uint32_t abort;
};

// Which of the 8 blocks of a tile exist, bit j for block j (the same on every lane of the warp);
// lane j's id in `id`.  The blocks past the prefix are absent without being an error.
__device__ __forceinline__ uint32_t tile_blocks(const PrefixParams& p, const int32_t* table, int nblk, int tile, int lane,
                                                int& id, bool flag) {
  id = -1;
  const int j = tile * (kPrefixTile / kBlockSize) + (lane & 7);
  const bool inside = j < nblk;
  if (inside) id = __ldg(table + j);
  const bool ok = inside && id >= 0 && id < p.num_blocks;
  if (flag && inside && !ok && lane < 8) set_error(p.err, kErrBlockId);
  return __ballot_sync(0xffffffffu, ok) & 0xffu;
}

template <KvType KV, int D>
__global__ void __launch_bounds__(PrefixCfg<KV, D>::kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                     const PrefixParams p) {
  using C = PrefixCfg<KV, D>;
  constexpr int S = C::kStages;
  constexpr uint32_t kFull = 0xffffffffu;
  extern __shared__ unsigned char smem_raw[];
  auto* sy = reinterpret_cast<PrefixSync*>((reinterpret_cast<uintptr_t>(smem_raw) + 15) & ~uintptr_t(15));
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + C::kMiscBytes + 1023) & ~uintptr_t(1023));
  unsigned char* ring = smem + C::kRingOff;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(sy->full + i, 1);
      mbar_init(sy->empty + i, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(sy->q_ready + s, 128);
      mbar_init(sy->s_ready + s, 1);
      mbar_init(sy->p_ready + s, 128);
      mbar_init(sy->pv_done + s, 1);
      mbar_init(sy->o_free + s, 128);
    }
    mbar_init(&sy->drain, 1);
    sy->abort = 0;
    fence_barrier_init();
    prefetch_tensor_map(&tmap_k);
    prefetch_tensor_map(&tmap_v);
  }
  if (warp == C::kMmaWarp) tmem_alloc(&sy->tmem, C::kTmemCols);
  griddep_wait();  // inputs may come from the previous kernel in the stream
  PrefixScan sc{reinterpret_cast<longlong2*>(ring) + 32, reinterpret_cast<longlong2*>(ring)};
  const int64_t total = prefix_scan<C::kThreads>(p, sc);
  prefix_describe<C::kThreads>(p, sc, total);
  PrefixWalk k;
  bool more = total > 0 && walk_begin(p, sc, total, blockIdx.x, k);
  tc_fence_before();
  __syncthreads();  // the ring's memory is free again; the barriers and the tensor memory are there
  tc_fence_after();
  const uint32_t tmem = sy->tmem;
  volatile uint32_t* abort = &sy->abort;
  // A whole warp's wait: the same answer on every lane, false once any part of the CTA gave up.
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_wait_bounded(bar, parity);
    return bool(__all_sync(kFull, ok && *abort == 0));
  };

  // Steps of stream s over n tiles: which of the unit's tiles it takes, and how many.
  // two: the streams hold different rows; else they share the tiles out between them.
  auto steps_of = [&](bool two, int nrows, int n, int s) { return two ? (s == 0 || nrows > 128 ? n : 0) : (n + 1 - s) / 2; };

  if (warp == C::kTmaWarp) {
    // ---------------------------------------------------------------- K and V tiles -> ring
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
      int ids[2];
      uint32_t blocks[2];
      for (int i = 0; i < 2 * n; ++i, ++it) {
        // order of the loads: K, V of a tile; with shared-out tiles K, K, V, V of a pair
        int tile, which;
        bool is_v;
        if (two) {
          tile = i >> 1;
          is_v = i & 1;
          which = 0;
        } else {
          const int pair = i >> 2, have = min(2, n - 2 * pair), j = i & 3;
          is_v = j >= have;
          which = is_v ? j - have : j;
          tile = 2 * pair + which;
        }
        if (!is_v) blocks[which] = tile_blocks(p, table, nblk, k.tile0 + tile, lane, ids[which], true);
        const uint32_t st = it % S;
        if (it >= S) {
          if (!wait_all(sy->empty + st, ((it / S) & 1) ^ 1)) {
            alive = false;
            break;
          }
        }
        const uint32_t have = blocks[which];
        if (lane == 0) {
          if (have) mbar_arrive_expect_tx(sy->full + st, __popc(have) * (kBlockSize * D * 2));
          else mbar_arrive(sy->full + st);
        }
        __syncwarp();
        // lane = (span, block): one copy of 16 rows x 128 bytes each
        const int block = lane & 7, half = lane >> 3;
        const int id = __shfl_sync(kFull, ids[which], block);
        if (half < C::kHalves && (have >> block & 1))
          tma_load_2d(ring + st * C::kTileBytes + half * C::kHalfBytes + block * (kBlockSize * 128), is_v ? &tmap_v : &tmap_k,
                      half * 64, (id * p.kv_heads + k.kvh) * kBlockSize, sy->full + st, policy);
      }
    }
    if (!alive) {
      if (lane == 0) {
        *abort = 1;
        set_error(p.err, kErrTimeout);
      }
    }
    // the copies in flight land before the CTA can end (the stages filled last)
    for (uint32_t j = it > S ? it - S : 0; j < it; ++j) (void)mbar_wait_bounded(sy->full + j % S, (j / S) & 1);
  } else if (warp == C::kMmaWarp) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t kDescS = mma_bf16_desc(128, kPrefixTile, false), kDescO = mma_bf16_desc(128, D, true);
    const uint32_t q_addr = smem_addr(smem), ring_addr = smem_addr(ring);
    uint32_t it = 0;                  // ring stages before this piece
    uint32_t cnt[2] = {0, 0};         // steps of each stream before this piece
    uint32_t seg[2] = {0, 0};         // pieces that had work for the stream
    bool alive = true;
    for (; more && alive; more = walk_next(p, blockIdx.x, k)) {
      const bool two = k.x.rows > 128;
      const int nblk = __ldg(p.prefix_lens + k.g) / kBlockSize;
      const int32_t* table = p.block_tables + int64_t(k.x.first_seq) * p.max_blocks_per_seq;
      const int n = k.tile1 - k.tile0;
      const int ns[2] = {steps_of(two, k.nrows, n, 0), steps_of(two, k.nrows, n, 1)};
      const int last = ns[1] > 0 ? 1 : 0;  // the stream that uses a shared tile last
      bool fresh[2] = {true, true};        // O holds nothing of this piece yet
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!alive) return;
        alive = wait_all(bar, parity);
      };
      auto k_index = [&](int i, int s) { return two ? 2 * i : 4 * i + s; };
      auto v_index = [&](int i, int s) { return two ? 2 * i + 1 : 4 * i + min(2, n - 2 * i) + s; };
      // S of stream s, step i
      auto issue_s = [&](int i, int s) {
        const uint32_t c = cnt[s] + i, idx = it + k_index(i, s);
        wait(sy->full + idx % S, (idx / S) & 1);
        if (i == 0) wait(sy->q_ready + s, seg[s] & 1);
        if (c > 0) wait(sy->pv_done + s, (c - 1) & 1);  // P lies over S until its product is done
        if (!alive) return;
        if (lane == 0) {
          tc_fence_after();
          const uint64_t qd = smem_operand(q_addr + s * C::kTileBytes, 16, 1024);
          const uint64_t kd = smem_operand(ring_addr + (idx % S) * C::kTileBytes, 16, 1024);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const uint32_t o = ((j >> 2) * C::kHalfBytes + (j & 3) * 32) >> 4;
            tc_mma_ss(tmem + s * 128, qd + o, kd + o, kDescS, j > 0);
          }
          tc_commit(sy->s_ready + s);
          if (!two || s == last) tc_commit(sy->empty + idx % S);
        }
        __syncwarp();
      };
      for (int s = 0; s < 2; ++s)
        if (ns[s] > 0) issue_s(0, s);
      for (int i = 0; i < ns[0] && alive; ++i) {
        for (int s = 0; s < 2 && alive; ++s) {
          if (i >= ns[s]) continue;
          int id;
          const uint32_t have = tile_blocks(p, table, nblk, k.tile0 + (two ? i : 2 * i + s), lane, id, false);
          const uint32_t c = cnt[s] + i, idx = it + v_index(i, s);
          wait(sy->p_ready + s, c & 1);
          wait(sy->full + idx % S, (idx / S) & 1);
          if (i == 0 && seg[s] > 0) wait(sy->o_free + s, (seg[s] - 1) & 1);
          if (!alive) break;
          if (lane == 0) {
            tc_fence_after();
            const uint64_t vd = smem_operand(ring_addr + (idx % S) * C::kTileBytes, C::kHalfBytes, 1024);
            bool acc = !fresh[s];
#pragma unroll
            for (int j = 0; j < kPrefixTile / 16; ++j)
              if (have >> j & 1) {
                tc_mma_ts(tmem + 256 + s * D, tmem + s * 128 + j * 8, vd + j * ((kBlockSize * 128) >> 4), kDescO, acc);
                acc = true;
              }
            tc_commit(sy->pv_done + s);
            if (!two || s == last) tc_commit(sy->empty + idx % S);
          }
          if (have) fresh[s] = false;
          __syncwarp();
          if (i + 1 < ns[s]) issue_s(i + 1, s);
        }
      }
      it += 2 * n;
      for (int s = 0; s < 2; ++s)
        if (ns[s] > 0) {
          cnt[s] += ns[s];
          ++seg[s];
        }
    }
    if (!alive) {
      if (lane == 0) {
        *abort = 1;
        set_error(p.err, kErrTimeout);
        tc_commit(&sy->drain);  // the products in flight end before their memory is given up
      }
      __syncwarp();
      (void)mbar_wait_bounded(&sy->drain, 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax, one thread per row
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
    uint32_t cnt = 0;
    bool alive = true;
    for (; more && alive; more = walk_next(p, blockIdx.x, k)) {
      const bool two = k.x.rows > 128;
      const int n = k.tile1 - k.tile0;
      const int ns = steps_of(two, k.nrows, n, s);
      const int row0 = two ? s * 128 : 0;              // the stream's first row within the unit
      const int nrows = min(128, k.nrows - row0);      // its rows
      const int64_t to = k.partial + (two ? s * 128 : s * k.x.rows) + r;
      if (ns == 0) {
        if (r < nrows) p.ml[to] = make_float2(kMaxFloor, 0.0f);  // no tile of its own: weighs nothing
        continue;
      }
      const int prefix = __ldg(p.prefix_lens + k.g), nblk = prefix / kBlockSize;
      const int32_t* table = p.block_tables + int64_t(k.x.first_seq) * p.max_blocks_per_seq;
      {  // Q -> shared memory, swizzled; its last reader was the last step's S, which this thread saw
        uint4 w[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) w[c] = make_uint4(0u, 0u, 0u, 0u);
        if (r < nrows) {
          const auto* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                         prefix_q_row(p, k.x, k.kvh, k.row0 + row0 + r) * D);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) w[c] = __ldg(q + c);
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          w[c] = make_uint4((w[c].x ^ flip) & keep, (w[c].y ^ flip) & keep, (w[c].z ^ flip) & keep, (w[c].w ^ flip) & keep);
          *reinterpret_cast<uint4*>(qt + (c >> 3) * C::kHalfBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = w[c];
        }
        fence_proxy_async_smem();
        mbar_arrive(sy->q_ready + s);
      }
      const bool idle = (warp & 3) * 32 >= nrows;  // none of the warp's rows exists
      float m = kMaxFloor, l = 0.0f;
      bool any = false;
      for (int i = 0; i < ns; ++i) {
        int id;
        const uint32_t have = tile_blocks(p, table, nblk, k.tile0 + (two ? i : 2 * i + s), lane, id, false);
        const uint32_t c = cnt + i;
        if (!wait_all(sy->s_ready + s, c & 1)) {
          alive = false;
          break;
        }
        any |= have != 0;
        if (!idle) {
          tc_fence_after();
          float x[128];
#pragma unroll
          for (int j = 0; j < 4; ++j) tmem_ld32(s_addr + 32 * j, x + 32 * j);
          tmem_wait_ld();
          if (have != 0xffu) {
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (!(have >> (j / 16) & 1)) x[j] = -INFINITY;
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int j = 4; j < 128; ++j) mx[j & 3] = fmaxf(mx[j & 3], x[j]);
          const float bm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
          const bool grow = bm > m + kMaxSlack;
          if (__any_sync(kFull, grow)) {
            const float mu = grow ? bm : m, f = fast_exp2(m - mu);
            m = mu;
            l *= f;
            if (i > 0) {
              // the last product into O is done: S was issued after it
#pragma unroll 1
              for (int j = 0; j < D / 32; ++j) {
                float o[32];
                tmem_ld32(o_addr + 32 * j, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f;
                tmem_st32(o_addr + 32 * j, reinterpret_cast<const uint32_t*>(o));
              }
            }
          }
          const uint64_t neg = f32x2(-m, -m);
          uint64_t sum[2] = {0, 0};
          uint32_t w[64];
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            float a, b;
            f32x2_parts(fma2(f32x2(x[2 * j], x[2 * j + 1]), scale2, neg), a, b);
            w[j] = pack_bf16x2(fast_exp2(a), fast_exp2(b));
            sum[j & 1] = add2(sum[j & 1], f32x2(bf16lo(w[j]), bf16hi(w[j])));
          }
          float a, b;
          f32x2_parts(add2(sum[0], sum[1]), a, b);
          l += a + b;
          tmem_st32(s_addr, w);
          tmem_st32(s_addr + 32, w + 32);
          tmem_wait_st();
          tc_fence_before();
        }
        mbar_arrive(sy->p_ready + s);
      }
      if (!alive) break;
      cnt += ns;
      // ---- the piece's partial
      if (!wait_all(sy->pv_done + s, (cnt - 1) & 1)) {
        alive = false;
        break;
      }
      if (!idle) {
        tc_fence_after();
        float* dst = p.acc + to * D;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          float o[32];
          tmem_ld32(o_addr + 32 * j, o);
          tmem_wait_ld();
          if (r < nrows) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(dst + 32 * j + e) =
                  any ? make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          }
        }
        if (r < nrows) p.ml[to] = make_float2(m, l);
        tc_fence_before();
      }
      mbar_arrive(sy->o_free + s);
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
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev].store(true, std::memory_order_relaxed);
  }
  return launch_pdl(kern, dim3(p.grid), dim3(C::kThreads), C::kSmemBytes, stream, tk, tv, p);
}

}  // namespace pkv
