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
// A warp takes rows (heads) of one token and one kind: query, key or value; D / 8 lanes to a row,
// so 2 or 4 rows at a time, kBatch such steps' loads ahead of the arithmetic.  A lane holds both values of
// its four rotated pairs (two 8-byte pieces of the row, half the rotated part apart, or adjacent ones
// when interleaved), so the rotation needs no exchange between lanes.  What is common to a
// token's rows (weight times cosine or sine) is formed once per warp.  The pass is bound by memory:
// it reads q, k and v once and writes each result once.  Measured on GB300, 16384 tokens of 32 + 8 + 8
// heads of 128 into a bf16 pool (411 MB): 83 us, 4.9 TB/s, with 4 CTAs an SM and 2 steps ahead;
// 3 CTAs and 4 steps 95 us, 2 and 8 128 us, 8 and 1 116 us.
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kBatch = 2;  // steps whose rows are on their way together

// Write this lane's 8 values (chunks c0 and c1 of 4) of a row to its slot: bf16, or codes with the
// row's scale.
template <KvType KV, int LPR>
__device__ __forceinline__ void store_cache(const float (&x)[8], void* cache, float* scale, int64_t row, int c0, int c1,
                                            bool write, bool first) {
  constexpr int D = LPR * 8;
  if constexpr (KV == KvType::kBf16) {
    if (write) {
      auto* to = static_cast<__nv_bfloat16*>(cache) + row * D;
      *reinterpret_cast<uint2*>(to + c0 * 4) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
      *reinterpret_cast<uint2*>(to + c1 * 4) = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
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
      auto* to = static_cast<uint8_t*>(cache) + row * D;
      *reinterpret_cast<uint32_t*>(to + c0 * 4) = code[0];
      *reinterpret_cast<uint32_t*>(to + c1 * 4) = code[1];
      if (first) scale[row] = s;
    }
  }
}

template <KvType KV, int D>
__global__ void __launch_bounds__(kRopeThreads, 4) norm_rope_kernel(const RopeParams p, int rows_per_unit) {
  constexpr int LPR = D / 8;              // lanes per row
  constexpr int RPS = 32 / LPR;           // rows per step of a warp
  constexpr uint32_t kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int lr = lane % LPR, sub = lane / LPR;
  griddep_wait();  // the projection's output comes from the previous kernel in the stream
  griddep_launch_dependents();
  const int uq = (p.num_q_heads + rows_per_unit - 1) / rows_per_unit, uk = (p.kv_heads + rows_per_unit - 1) / rows_per_unit;
  const int upt = uq + 2 * uk;  // units per token
  const int64_t u = int64_t(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  if (u >= p.num_tokens * upt) return;
  const int64_t t = u / upt;
  const int v = int(u - t * upt);
  const int kind = v < uq ? 0 : v < uq + uk ? 1 : 2;  // query, key, value
  const int r0 = (kind == 0 ? v : kind == 1 ? v - uq : v - uq - uk) * rows_per_unit;
  const int r1 = min(kind == 0 ? p.num_q_heads : p.kv_heads, r0 + rows_per_unit);
  const auto* src = static_cast<const __nv_bfloat16*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                    t * (kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride);
  // The lane's two chunks of 4 values: the two halves of 4 rotated pairs, or what lies past the
  // rotated part, or (values, interleaved pairs) 8 neighbours.
  const int half4 = p.rot_dim >> 3;  // chunks of half the rotated part
  const bool apart = kind != 2 && !p.interleaved && p.rot_dim > 0;
  const bool turns = kind != 2 && lr * 8 < p.rot_dim;  // half4 lanes hold pairs, whichever way they lie
  int c0 = 2 * lr, c1 = 2 * lr + 1;
  if (apart) {
    c0 = lr < half4 ? lr : lr + half4;
    c1 = lr < half4 ? lr + half4 : lr + half4 + (D / 8 - half4);
  }
  uint2 raw[kBatch][2];
  auto load = [&](int r) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = r + i * RPS + sub;
      if (h < r1) {
        raw[i][0] = *reinterpret_cast<const uint2*>(src + int64_t(h) * D + c0 * 4);
        raw[i][1] = *reinterpret_cast<const uint2*>(src + int64_t(h) * D + c1 * 4);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kBatch; ++i) raw[i][0] = raw[i][1] = make_uint2(0u, 0u);
  load(r0);
  int64_t slot = -1;
  if (kind != 0) {
    slot = __ldg(p.slot_mapping + t);
    if (slot >= p.num_blocks * kBlockSize) {
      if (lane == 0 && r0 == 0 && kind == 1) set_error(p.err, kErrSlot);
      slot = -1;
    }
  }
  bool ok = true;
  float4 c = make_float4(1.0f, 1.0f, 1.0f, 1.0f), s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (p.cos_sin) {
    const int pos = __ldg(p.positions + t);
    ok = pos >= 0 && pos < p.max_position;
    if (!ok && lane == 0 && v == 0) set_error(p.err, kErrPosition);
    if (ok && turns) {
      const float4* row = reinterpret_cast<const float4*>(p.cos_sin + int64_t(pos) * p.rot_dim);
      c = __ldg(row + lr);
      s = __ldg(row + half4 + lr);
    }
  }
  const void* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
  float4 w0 = make_float4(1.0f, 1.0f, 1.0f, 1.0f), w1 = w0;
  if (weight) {
    const uint2 a = __ldg(static_cast<const uint2*>(weight) + c0), b = __ldg(static_cast<const uint2*>(weight) + c1);
    w0 = make_float4(bf16lo(a.x), bf16hi(a.x), bf16lo(a.y), bf16hi(a.y));
    w1 = make_float4(bf16lo(b.x), bf16hi(b.x), bf16lo(b.y), bf16hi(b.y));
  }
  // pairs (a, b) -> (a A - b B, b C + a E), two pairs to a register pair: A = w_a cos, B = w_b sin,
  // C = w_b cos, E = w_a sin.  Pairs are (x0..3, x4..7), or neighbours when interleaved (x0 x1, ...).
  uint64_t A[2], B[2], Cc[2], E[2];
  if (p.interleaved && kind != 2) {  // a = x0 x2 | x4 x6
    const float wa[4] = {w0.x, w0.z, w1.x, w1.z}, wb[4] = {w0.y, w0.w, w1.y, w1.w};
    w0 = make_float4(wa[0], wa[1], wa[2], wa[3]);
    w1 = make_float4(wb[0], wb[1], wb[2], wb[3]);
  }
  A[0] = f32x2(w0.x * c.x, w0.y * c.y); A[1] = f32x2(w0.z * c.z, w0.w * c.w);
  B[0] = f32x2(-w1.x * s.x, -w1.y * s.y); B[1] = f32x2(-w1.z * s.z, -w1.w * s.w);
  Cc[0] = f32x2(w1.x * c.x, w1.y * c.y); Cc[1] = f32x2(w1.z * c.z, w1.w * c.w);
  E[0] = f32x2(w0.x * s.x, w0.y * s.y); E[1] = f32x2(w0.z * s.z, w0.w * s.w);

  for (int r = r0; r < r1; r += kBatch * RPS) {
    uint2 cur[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      cur[i][0] = raw[i][0];
      cur[i][1] = raw[i][1];
    }
    if (r + kBatch * RPS < r1) load(r + kBatch * RPS);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (r + i * RPS >= r1) break;  // the same for the whole warp
      const int h = r + i * RPS + sub;
      float x[8] = {bf16lo(cur[i][0].x), bf16hi(cur[i][0].x), bf16lo(cur[i][0].y), bf16hi(cur[i][0].y),
                    bf16lo(cur[i][1].x), bf16hi(cur[i][1].x), bf16lo(cur[i][1].y), bf16hi(cur[i][1].y)};
      if (kind != 2) {
        uint64_t a[2], b[2];
        if (p.interleaved) {
          a[0] = f32x2(x[0], x[2]); a[1] = f32x2(x[4], x[6]);
          b[0] = f32x2(x[1], x[3]); b[1] = f32x2(x[5], x[7]);
        } else {
          a[0] = f32x2(x[0], x[1]); a[1] = f32x2(x[2], x[3]);
          b[0] = f32x2(x[4], x[5]); b[1] = f32x2(x[6], x[7]);
        }
        uint64_t inv2 = f32x2(1.0f, 1.0f);
        if (weight) {
          const uint64_t q2 = fma2(a[0], a[0], fma2(a[1], a[1], fma2(b[0], b[0], mul2(b[1], b[1]))));
          float ss, hi;
          f32x2_parts(q2, ss, hi);
          ss += hi;
#pragma unroll
          for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
          const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
          inv2 = f32x2(inv, inv);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint64_t ya = mul2(a[j], A[j]), yb = mul2(b[j], Cc[j]);
          if (turns) {  // elsewhere sine is 0, but an infinity times 0 is not
            ya = fma2(b[j], B[j], ya);
            yb = fma2(a[j], E[j], yb);
          }
          a[j] = mul2(ya, inv2);
          b[j] = mul2(yb, inv2);
        }
        if (p.interleaved) {
          f32x2_parts(a[0], x[0], x[2]); f32x2_parts(a[1], x[4], x[6]);
          f32x2_parts(b[0], x[1], x[3]); f32x2_parts(b[1], x[5], x[7]);
        } else {
          f32x2_parts(a[0], x[0], x[1]); f32x2_parts(a[1], x[2], x[3]);
          f32x2_parts(b[0], x[4], x[5]); f32x2_parts(b[1], x[6], x[7]);
        }
      }
      if (kind == 0) {
        if (h < r1) {
          auto* to = static_cast<__nv_bfloat16*>(p.q_out) + t * p.out_stride + int64_t(h) * D;
          const uint2 y0 = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
          const uint2 y1 = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
          *reinterpret_cast<uint2*>(to + c0 * 4) = ok ? y0 : make_uint2(0u, 0u);
          *reinterpret_cast<uint2*>(to + c1 * 4) = ok ? y1 : make_uint2(0u, 0u);
        }
      } else {
        const int64_t row = ((slot / kBlockSize) * p.kv_heads + h) * kBlockSize + slot % kBlockSize;
        store_cache<KV, LPR>(x, kind == 1 ? p.k_cache : p.v_cache, kind == 1 ? p.k_scale : p.v_scale, row, c0, c1,
                             ok && slot >= 0 && h < r1, lr == 0);
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
  constexpr int kWarps = kRopeThreads / 32;
  constexpr int kFewRows = 32 / (D / 8) * kBatch;  // one batch of loads
  // All of a token's heads to a warp where that fills the GPU (the token's position, table row and
  // weights are then read once for all), one batch of rows otherwise.
  const int most = p.num_q_heads > p.kv_heads ? p.num_q_heads : p.kv_heads;
  const int rows = p.num_tokens * 3 >= 152 * 32 * 2 ? most : kFewRows;
  const int64_t units = p.num_tokens * ((p.num_q_heads + rows - 1) / rows + 2 * ((p.kv_heads + rows - 1) / rows));
  const int64_t grid = (units + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(norm_rope_kernel<KV, D>, dim3(unsigned(grid)), dim3(kRopeThreads), 0, stream, p, rows);
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
