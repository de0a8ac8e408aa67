// pkv_rope.cu -- per-head norm of queries and keys, rotary positions and the cache write of
// a step's new tokens in one pass over the projection's output, and the table of cosines
// and sines that the rotation reads.
//
// For each token and each query or key head x (D values):
//     y = x / sqrt(mean(x^2) + eps) * w                     (when that weight is given)
//     (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)          (for each rotated pair (a, b))
// with (c, s) the cosine and sine of the token's position for the pair: pair i of rot_dim / 2
// is (i, i + rot_dim / 2), or (2 i, 2 i + 1) when interleaved; values past rot_dim are not
// rotated.  Queries go to q_out in bf16; keys and values go to their pool slots as
// pkv_reshape_and_cache writes them (a straight copy, or s = max|y| / 127 or 448 and codes).
// All of it is fp32 from the bf16 inputs to the one rounding at the end: a key is not
// rounded to bf16 before it is quantised.
//
// A warp takes kRows rows (head rows of one token and one kind: query, key or value),
// D / 8 lanes to a row, 16 bytes a lane; the rows' loads are issued together, ahead of the
// arithmetic.  A lane holds its 8 values' cosines and sines, which all rows of the warp share.
// The pass is bound by memory: it reads q, k and v once and writes each result once.
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 256;

// One word of two bf16 values -> fp32.
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y); x[3] = bf16hi(w.y);
  x[4] = bf16lo(w.z); x[5] = bf16hi(w.z); x[6] = bf16lo(w.w); x[7] = bf16hi(w.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Write one row's 8 values of this lane to its slot: bf16, or codes with the row's scale.
template <KvType KV, int LPR>
__device__ __forceinline__ void store_cache(const float (&x)[8], void* cache, float* scale, int64_t row, int lr,
                                            bool write) {
  constexpr int D = LPR * 8;
  if constexpr (KV == KvType::kBf16) {
    if (write) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + row * D + lr * 8) = pack8(x);
  } else {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = __fdiv_rn(amax, KV == KvType::kFp8 ? 448.0f : 127.0f);
    uint32_t code[2] = {0u, 0u};
    if (amax != 0.0f) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float a = __fdiv_rn(x[i], s), b = __fdiv_rn(x[i + 1], s);
        uint32_t two;
        if constexpr (KV == KvType::kFp8) {
          two = e4m3x2_from_f32(a, b);
        } else {
          const int ca = min(127, max(-127, __float2int_rn(a))), cb = min(127, max(-127, __float2int_rn(b)));
          two = (uint32_t(ca) & 0xffu) | ((uint32_t(cb) & 0xffu) << 8);
        }
        code[i >> 2] |= two << (8 * (i & 3));
      }
    }
    if (write) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * D + lr * 8) = make_uint2(code[0], code[1]);
      if (lr == 0) scale[row] = s;
    }
  }
}

template <KvType KV, int D, int STEPS>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeParams p) {
  constexpr int LPR = D / 8;              // lanes per row
  constexpr int RPS = 32 / LPR;           // rows per step of a warp
  constexpr int kRows = RPS * STEPS;      // rows of one unit
  constexpr uint32_t kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int lr = lane % LPR, sub = lane / LPR;
  griddep_wait();  // the projection's output comes from the previous kernel in the stream
  griddep_launch_dependents();
  const int uq = (p.num_q_heads + kRows - 1) / kRows, uk = (p.kv_heads + kRows - 1) / kRows;
  const int upt = uq + 2 * uk;  // units per token
  const int64_t units = p.num_tokens * upt;
  const int64_t stride = int64_t(gridDim.x) * (kRopeThreads / 32);
  const int half = p.rot_dim >> 1;
  const int hl = half >> 3;  // lanes that half of the rotated values take
  for (int64_t u = int64_t(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5); u < units; u += stride) {
    const int64_t t = u / upt;
    const int v = int(u - t * upt);
    const int kind = v < uq ? 0 : v < uq + uk ? 1 : 2;  // query, key, value
    const int r0 = (kind == 0 ? v : kind == 1 ? v - uq : v - uq - uk) * kRows;
    const int heads = kind == 0 ? p.num_q_heads : p.kv_heads;
    const auto* src = static_cast<const __nv_bfloat16*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                      t * (kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride);
    uint4 raw[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int h = r0 + i * RPS + sub;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (h < heads) raw[i] = *reinterpret_cast<const uint4*>(src + int64_t(h) * D + lr * 8);
    }
    int64_t slot = -1;
    if (kind != 0) {
      slot = __ldg(p.slot_mapping + t);
      if (slot >= p.num_blocks * kBlockSize) {
        if (lane == 0 && r0 == 0 && kind == 1) set_error(p.err, kErrSlot);
        slot = -1;
      }
    }
    bool ok = true;
    float c[8], s[8];
    if (p.cos_sin) {
      const int pos = __ldg(p.positions + t);
      ok = pos >= 0 && pos < p.max_position;
      if (!ok && lane == 0 && v == 0) set_error(p.err, kErrPosition);
      if (kind != 2 && ok && lr * 8 < p.rot_dim) {
        const float* row = p.cos_sin + int64_t(pos) * p.rot_dim;
        // a lane's 8 consecutive values belong to 8 pairs, or to 4 neighbouring ones
        const float* cp = row + (p.interleaved ? lr * 4 : lr < hl ? lr * 8 : lr * 8 - half);
        const float4 c0 = __ldg(reinterpret_cast<const float4*>(cp)), s0 = __ldg(reinterpret_cast<const float4*>(cp + half));
        if (p.interleaved) {
          c[0] = c[1] = c0.x; c[2] = c[3] = c0.y; c[4] = c[5] = c0.z; c[6] = c[7] = c0.w;
          s[0] = s[1] = s0.x; s[2] = s[3] = s0.y; s[4] = s[5] = s0.z; s[6] = s[7] = s0.w;
        } else {
          const float4 c1 = __ldg(reinterpret_cast<const float4*>(cp + 4)), s1 = __ldg(reinterpret_cast<const float4*>(cp + half + 4));
          c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
          s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
        }
        // the first of a pair takes -s times its partner, the second +s
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (p.interleaved ? !(e & 1) : lr < hl) s[e] = -s[e];
      }
    }
    const void* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
    float w[8];
    if (weight) unpack8(__ldg(static_cast<const uint4*>(weight) + lr), w);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      if (r0 + i * RPS >= heads) break;  // the same for the whole warp
      const int h = r0 + i * RPS + sub;
      float x[8];
      unpack8(raw[i], x);
      if (weight) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        const float inv = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv * w[e];
      }
      if (p.cos_sin && kind != 2) {
        float y[8];  // each value's partner
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
        } else {
          const int from = (lane - lr) + (lr < hl ? lr + hl : lr < 2 * hl ? lr - hl : lr);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(kFull, x[e], from);
        }
        if (ok && lr * 8 < p.rot_dim) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], c[e], y[e] * s[e]);
        }
      }
      if (kind == 0) {
        if (h < heads)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) + t * p.out_stride + int64_t(h) * D + lr * 8) =
              ok ? pack8(x) : make_uint4(0u, 0u, 0u, 0u);
      } else {
        const int64_t row = ((slot / kBlockSize) * p.kv_heads + h) * kBlockSize + slot % kBlockSize;
        const bool write = ok && slot >= 0 && h < heads;
        if (kind == 1) store_cache<KV, LPR>(x, p.k_cache, p.k_scale, row, lr, write);
        else store_cache<KV, LPR>(x, p.v_cache, p.v_scale, row, lr, write);
      }
    }
  }
}

// Angles in 64 bits: at position 10^5 an fp32 angle is off by up to 2^-8.
__global__ void __launch_bounds__(kRopeThreads)
    rope_table_kernel(float* out, int64_t max_position, int half, double base) {
  griddep_wait();  // the previous kernel in the stream may still read the buffer
  griddep_launch_dependents();
  const int64_t n = max_position * half;
  for (int64_t i = int64_t(blockIdx.x) * kRopeThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kRopeThreads) {
    const int64_t pos = i / half;
    const int j = int(i - pos * half);
    double s, c;
    sincos(double(pos) * pow(base, -double(j) / half), &s, &c);
    out[pos * 2 * half + j] = float(c);
    out[pos * 2 * half + half + j] = float(s);
  }
}

template <KvType KV, int D>
cudaError_t launch_norm_rope_variant(const RopeParams& p, cudaStream_t stream) {
  constexpr int kSteps = 4;
  constexpr int kRows = 32 / (D / 8) * kSteps;
  const int64_t units = p.num_tokens * ((p.num_q_heads + kRows - 1) / kRows + 2 * ((p.kv_heads + kRows - 1) / kRows));
  const int64_t need = (units + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const int64_t cap = int64_t(1) << 30;
  return launch_pdl(norm_rope_kernel<KV, D, kSteps>, dim3(unsigned(need < cap ? need : cap)), dim3(kRopeThreads), 0,
                    stream, p);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeParams& p, KvType kv, cudaStream_t stream) {
  const bool wide = p.head_dim == 128;
  switch (kv) {
    case KvType::kBf16:
      return wide ? launch_norm_rope_variant<KvType::kBf16, 128>(p, stream) : launch_norm_rope_variant<KvType::kBf16, 64>(p, stream);
    case KvType::kInt8:
      return wide ? launch_norm_rope_variant<KvType::kInt8, 128>(p, stream) : launch_norm_rope_variant<KvType::kInt8, 64>(p, stream);
    case KvType::kFp8:
      return wide ? launch_norm_rope_variant<KvType::kFp8, 128>(p, stream) : launch_norm_rope_variant<KvType::kFp8, 64>(p, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_rope_table(float* out, int64_t max_position, int rot_dim, double base, cudaStream_t stream) {
  const int64_t n = max_position * (rot_dim / 2);
  const int64_t need = (n + kRopeThreads - 1) / kRopeThreads;
  return launch_pdl(rope_table_kernel, dim3(unsigned(need < 65536 ? need : 65536)), dim3(kRopeThreads), 0, stream, out,
                    max_position, rot_dim / 2, base);
}

}  // namespace pkv
