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

// A CTA takes a tile of tokens at a time, finds each one's place in the pool, and then a thread moves
// 8 values at a time.
template <KvType KV, int D>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherParams p) {
  constexpr int kChunks = D / 8;  // per (token, head) row
  constexpr int kTile = 32;       // tokens
  __shared__ int64_t place[kTile];   // block * 16 + offset; -1: rows of zeros, -2: no token
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
  for (int64_t t0 = first + int64_t(blockIdx.x) * kTile; t0 < last; t0 += int64_t(gridDim.x) * kTile) {
    __syncthreads();
    if (threadIdx.x < kTile) {
      const int64_t t = t0 + threadIdx.x;
      int64_t at = -2;
      if (t < last) {
        int lo = 0, hi = p.num_seqs;
        while (hi - lo > 1) {  // the last sequence that starts at or before t
          const int mid = (lo + hi) >> 1;
          if (__ldg(p.token_starts + mid) <= t) lo = mid; else hi = mid;
        }
        const int from = p.first_positions ? __ldg(p.first_positions + lo) : 0;
        const int64_t pos = int64_t(from) + (t - __ldg(p.token_starts + lo));
        at = -1;
        if (from < 0 || pos >= int64_t(p.max_blocks_per_seq) * kBlockSize) {
          set_error(p.err, kErrContextLen);
        } else {
          const int id = __ldg(p.block_tables + int64_t(lo) * p.max_blocks_per_seq + pos / kBlockSize);
          if (id < 0 || id >= p.num_blocks) set_error(p.err, kErrBlockId);
          else at = int64_t(id) * kBlockSize + pos % kBlockSize;
        }
      }
      place[threadIdx.x] = at;
    }
    __syncthreads();
    const int per_token = p.kv_heads * kChunks;
    for (int i = threadIdx.x; i < kTile * per_token; i += kGatherThreads) {
      const int tok = i / per_token, rest = i - tok * per_token, h = rest / kChunks, c = rest - h * kChunks;
      const int64_t at = place[tok];
      if (at == -2) continue;
      const int64_t block = at / kBlockSize, row = (block * p.kv_heads + h) * kBlockSize + (at - block * kBlockSize);
      auto move = [&](const void* cache, const float* scale, void* to, int64_t stride) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (at >= 0) {
          if constexpr (KV == KvType::kBf16) {
            w = __ldg(reinterpret_cast<const uint4*>(cache) + row * kChunks + c);
          } else {
            const uint2 codes = __ldg(reinterpret_cast<const uint2*>(cache) + row * kChunks + c);
            const float s = __ldg(scale + row);
            float f[8];
            if constexpr (KV == KvType::kFp8) {
              float a[4], b[4];
              e4m3x4_to_f32(codes.x, a);
              e4m3x4_to_f32(codes.y, b);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                f[e] = a[e];
                f[4 + e] = b[e];
              }
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] = i8_from_flipped((e < 4 ? codes.x : codes.y) ^ 0x80808080u, e & 3);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= s;
            w = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
          }
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(to) + (t0 + tok) * stride + h * D + c * 8) = w;
      };
      move(p.k_cache, p.k_scale, p.k, p.k_stride);
      move(p.v_cache, p.v_scale, p.v, p.v_stride);
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
