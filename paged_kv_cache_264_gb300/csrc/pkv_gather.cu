// pkv_gather.cu -- reading a cache back: tokens of sequences, wherever their blocks lie, as packed
// bf16 rows.
//
//     k[token_starts[b] + i][h] = K_b[first_b + i][h]   (and the same for V)
//
// INT8 and FP8 pools: scale * value(code), formed in fp32 and rounded to bf16 once.
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kGatherThreads = 256;

// A CTA takes 32 tokens at a time (of a long sequence: whole blocks, which lie in one piece in the pool) and finds
// the next ones' places meanwhile.  A thread moves 16 bytes of K and of V at a time, kAhead of each on their way.
// Bound by memory: 2.2 GB read and written in 317 us from bf16 (6.8 TB/s, the copy rate), 3.3 GB in 539 us from INT8
// (6.1 TB/s, the codes' conversion beside it); a few hundred tokens take 8 us, a launch and three dependent trips to memory.
template <KvType KV, int D>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherParams p) {
  constexpr bool kQuant = KV != KvType::kBf16;
  constexpr int kValues = kQuant ? 16 : 8;   // of a 16-byte load
  constexpr int kChunks = D / kValues;       // per (token, head) row
  constexpr int kTile = 32;                  // tokens
  constexpr int kAhead = kQuant ? 2 : 4;
  __shared__ int64_t places[2][kTile];       // block * 16 + offset; -1: rows of zeros, -2: no token
  griddep_wait();
  griddep_launch_dependents();
  // The starts are checked by every CTA: one that writes must know that all are valid.
  bool ok = true;
  for (int b = threadIdx.x; b < p.num_seqs; b += kGatherThreads) {
    const int s0 = __ldg(p.token_starts + b), s1 = __ldg(p.token_starts + b + 1);
    ok &= s0 >= 0 && s1 >= s0 && s1 <= p.num_tokens;
  }
  if (!__syncthreads_and(ok)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_error(p.err, kErrQuery);
    return;
  }
  const int first = __ldg(p.token_starts), last = __ldg(p.token_starts + p.num_seqs);
  auto find = [&](int64_t t) -> int64_t {
    if (t >= last) return -2;
    int lo = 0, hi = p.num_seqs;
    while (hi - lo > 1) {  // the last sequence that starts at or before t
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.token_starts + mid) <= t) lo = mid; else hi = mid;
    }
    const int from = p.first_positions ? __ldg(p.first_positions + lo) : 0;
    const int64_t pos = int64_t(from) + (t - __ldg(p.token_starts + lo));
    if (from < 0 || pos >= int64_t(p.max_blocks_per_seq) * kBlockSize) {
      set_error(p.err, kErrContextLen);
      return -1;
    }
    const int id = __ldg(p.block_tables + int64_t(lo) * p.max_blocks_per_seq + pos / kBlockSize);
    if (id < 0 || id >= p.num_blocks) {
      set_error(p.err, kErrBlockId);
      return -1;
    }
    return int64_t(id) * kBlockSize + pos % kBlockSize;
  };
  // this thread's chunks: (token, rest) of chunk i = threadIdx.x + j * kGatherThreads, rest = head * kChunks + chunk
  const int per_token = p.kv_heads * kChunks, all = kTile * per_token;
  const int step_tok = kGatherThreads / per_token, step_rest = kGatherThreads - step_tok * per_token;
  const int tok0 = int(threadIdx.x) / per_token, rest0 = int(threadIdx.x) - tok0 * per_token;
  int64_t t0 = first + int64_t(blockIdx.x) * kTile;
  if (threadIdx.x < kTile) places[0][threadIdx.x] = find(t0 + threadIdx.x);
  for (int buf = 0; t0 < last; t0 += int64_t(gridDim.x) * kTile, buf ^= 1) {
    __syncthreads();  // places are there, and the last tile's have been read
    const int64_t t1 = t0 + int64_t(gridDim.x) * kTile;
    if (threadIdx.x < kTile && t1 < last) places[buf ^ 1][threadIdx.x] = find(t1 + threadIdx.x);
    int tok = tok0, rest = rest0;
    for (int i = threadIdx.x; i < all; i += kAhead * kGatherThreads) {
      uint4 kw[kAhead], vw[kAhead];
      float ks[kAhead], vs[kAhead];
      int64_t to[kAhead];  // row of the output; -1: none
      int off[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t at = i + u * kGatherThreads < all ? places[buf][tok] : -2;
        const int h = rest / kChunks, c = rest - h * kChunks;
        to[u] = at == -2 ? -1 : t0 + tok;
        off[u] = h * D + c * kValues;
        kw[u] = vw[u] = make_uint4(0u, 0u, 0u, 0u);
        ks[u] = vs[u] = 0.0f;
        if (at >= 0) {
          const int64_t block = at / kBlockSize, row = (block * p.kv_heads + h) * kBlockSize + (at - block * kBlockSize);
          kw[u] = __ldcs(static_cast<const uint4*>(p.k_cache) + row * kChunks + c);
          vw[u] = __ldcs(static_cast<const uint4*>(p.v_cache) + row * kChunks + c);
          if constexpr (kQuant) {
            ks[u] = __ldg(p.k_scale + row);
            vs[u] = __ldg(p.v_scale + row);
          }
        }
        tok += step_tok;
        rest += step_rest;
        if (rest >= per_token) {
          rest -= per_token;
          ++tok;
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (to[u] < 0) continue;
        auto put = [&](void* base, int64_t stride, const uint4& w, float s) {
          auto* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + to[u] * stride + off[u]);
          if constexpr (!kQuant) {
            __stcs(dst, w);
          } else {
            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
            uint32_t out[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float f[4];
              if constexpr (KV == KvType::kFp8) {
                e4m3x4_to_f32(words[q], f);
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = i8_from_flipped(words[q] ^ 0x80808080u, e);
              }
              out[2 * q] = pack_bf16x2(f[0] * s, f[1] * s);
              out[2 * q + 1] = pack_bf16x2(f[2] * s, f[3] * s);
            }
            __stcs(dst, make_uint4(out[0], out[1], out[2], out[3]));
            __stcs(dst + 1, make_uint4(out[4], out[5], out[6], out[7]));
          }
        };
        put(p.k, p.k_stride, kw[u], ks[u]);
        put(p.v, p.v_stride, vw[u], vs[u]);
      }
    }
  }
}

template <KvType KV>
cudaError_t launch(const GatherParams& p, int sms, cudaStream_t stream) {
  const int64_t tiles = (int64_t(p.num_tokens) + 31) / 32;
  const unsigned grid = unsigned(tiles < sms * 8 ? tiles : sms * 8);
  if (p.head_dim == 128) return launch_pdl(gather_kernel<KV, 128>, dim3(grid), dim3(kGatherThreads), 0, stream, p);
  return launch_pdl(gather_kernel<KV, 64>, dim3(grid), dim3(kGatherThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_gather(const GatherParams& p, KvType kv, int sms, cudaStream_t stream) {
  return kv == KvType::kBf16  ? launch<KvType::kBf16>(p, sms, stream)
         : kv == KvType::kInt8 ? launch<KvType::kInt8>(p, sms, stream)
                               : launch<KvType::kFp8>(p, sms, stream);
}

}  // namespace pkv
