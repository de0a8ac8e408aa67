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
// A warp takes rows (heads) of one token and one kind: query, key or value; D / 16 lanes to a row,
// so 4 or 8 rows at a time.  A lane holds both values of its eight rotated pairs (two 16-byte pieces of
// the row, half the rotated part apart when the pairs are), so the rotation needs no exchange between
// lanes.  What is common to a token's rows (weights, cosines, sines) is read once per warp.
// The pass is bound by memory: it reads q, k and v once and writes each result once.  What it has on
// its way at a time decides its rate, so each lane's pieces of the next kSlots - 1 steps are copied to
// shared memory of its own (no registers held, no other lane to wait for).
// All queries' warps come first, then the keys', then the values': mixed, a CTA waited for its
// queries with half its warps done.  Measured on GB300, 16384 tokens of 32 + 8 + 8 heads of 128 into a
// bf16 pool (411 MB): 71.8 us, 5.7 TB/s (mixed 80; 6 or 4 slots the same within 2%; 5 CTAs an SM 74.8, 7
// 72.8 but slower when short); with loads of 8 bytes into registers, two steps ahead, it was 83.  Into an
// INT8 pool 4096 tokens take 23.6 us and 16384 86.2 (FP8 23.5 and 85.8; 32 + 32 + 32 heads of 64, not normalised,
// 26.4 and 94.4): the arithmetic of keys' and values' codes is in the way.  With the quotients' lower bound alone,
// which is not enough for the code, these were 20.8 and 78.4 (MHA 20.0 and 74.6).
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kSlots = 3;    // steps whose rows have a place in shared memory
constexpr int kMinCtas = 6;

__device__ __forceinline__ void copy_piece(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_next_step() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but this thread's latest kSlots - 1 steps have landed.
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory"); }

__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
  x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y); x[3] = bf16hi(w.y);
  x[4] = bf16lo(w.z); x[5] = bf16hi(w.z); x[6] = bf16lo(w.w); x[7] = bf16hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Codes of 16 values with scale s: the values divided by s, rounded, and rounded to a code, as
// pkv_reshape_and_cache forms them.
template <KvType KV>
__device__ __forceinline__ void codes_by_division(const float (&x)[16], float s, uint32_t (&code)[4]) {
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float a = __fdiv_rn(x[i], s), b = __fdiv_rn(x[i + 1], s);
    uint32_t two;
    if constexpr (KV == KvType::kFp8) {
      two = e4m3x2_from_f32(a, b);
    } else {
      const int ca = min(127, max(-127, __float2int_rn(a))), cb = min(127, max(-127, __float2int_rn(b)));
      two = (uint32_t(ca) & 0xffu) | ((uint32_t(cb) & 0xffu) << 8);
    }
    code[i >> 2] = (i & 2) ? code[i >> 2] | two << 16 : two;
  }
}

// The same codes, nearly always without a division per value.  With r = 1 / s to half a step
// (2^-24), x * r (1 - 2^-21) and x * r (1 + 2^-21) lie on either side of the rounded quotient, whose
// error is 2^-24 too, or are all too small for any code but 0.  Rounding to a code is monotone, so
// where both give one code it is the quotient's; where they do not (about one lane in 2000), and for
// NaN, this returns false.
template <KvType KV>
__device__ __forceinline__ bool codes_by_bounds(const float (&x)[16], float s, uint32_t (&code)[4]) {
  if (!(s >= 0x1p-100f && s <= 0x1p100f)) return false;  // r is a normal number
  const float r = __fdiv_rn(1.0f, s), r_lo = r * (1.0f - 0x1p-21f), r_hi = r * (1.0f + 0x1p-21f);
  const uint64_t lo2 = f32x2(r_lo, r_lo), hi2 = f32x2(r_hi, r_hi);
  bool same = true;
  if constexpr (KV == KvType::kFp8) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const uint64_t v = f32x2(x[i], x[i + 1]);
      float a, b, c, d;
      f32x2_parts(mul2(v, lo2), a, b);
      f32x2_parts(mul2(v, hi2), c, d);
      const uint32_t two = e4m3x2_from_f32(a, b);
      same = same && two == e4m3x2_from_f32(c, d);
      code[i >> 2] = (i & 2) ? code[i >> 2] | two << 16 : two;
    }
  } else {
    // adding 1.5 * 2^23 rounds to a whole number, which the sum's low byte then holds
    const uint64_t magic = f32x2(12582912.0f, 12582912.0f);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      float a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const uint64_t v = f32x2(x[i + j], x[i + j + 1]);
        f32x2_parts(fma2(v, lo2, magic), a[j], a[j + 1]);
        f32x2_parts(fma2(v, hi2, magic), b[j], b[j + 1]);
        same = same && a[j] == b[j] && a[j + 1] == b[j + 1];
      }
      code[i >> 2] = __byte_perm(__byte_perm(__float_as_uint(a[0]), __float_as_uint(a[1]), 0x0040u),
                                 __byte_perm(__float_as_uint(a[2]), __float_as_uint(a[3]), 0x0040u), 0x5410u);
    }
  }
  return same;
}

// Write this lane's 16 values (pieces c0 and c1 of 8), times the row's factor, to its slot: bf16, or codes
// with the row's scale.  The factor cancels in a code's quotient and goes into the scale alone.
template <KvType KV, int LPR>
__device__ __forceinline__ void store_cache(float (&x)[16], float factor, void* cache, float* scale, int64_t row, int c0, int c1,
                                            bool write, bool first) {
  constexpr int D = LPR * 16;
  if constexpr (KV == KvType::kBf16) {
    if (write) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= factor;
      auto* to = static_cast<__nv_bfloat16*>(cache) + row * D;
      *reinterpret_cast<uint4*>(to + c0 * 8) = pack8(x);
      *reinterpret_cast<uint4*>(to + c1 * 8) = pack8(x + 8);
    }
  } else {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = __fdiv_rn(amax, KV == KvType::kFp8 ? 448.0f : 127.0f);
    uint32_t code[4];
    if (!codes_by_bounds<KV>(x, s, code)) codes_by_division<KV>(x, s, code);
    if (amax == 0.0f) code[0] = code[1] = code[2] = code[3] = 0u;
    if (write) {
      auto* to = static_cast<uint8_t*>(cache) + row * D;
      *reinterpret_cast<uint2*>(to + c0 * 8) = make_uint2(code[0], code[1]);
      *reinterpret_cast<uint2*>(to + c1 * 8) = make_uint2(code[2], code[3]);
      if (first) scale[row] = amax == 0.0f ? 0.0f : s * factor;
    }
  }
}

template <KvType KV, int D>
__global__ void __launch_bounds__(kRopeThreads, kMinCtas) norm_rope_kernel(const RopeParams p, int rows_per_unit) {
  constexpr int LPR = D / 16;             // lanes per row
  constexpr int RPS = 32 / LPR;           // rows per step of a warp
  constexpr uint32_t kFull = 0xffffffffu;
  __shared__ uint4 stage[kSlots][2][kRopeThreads];
  const int lane = threadIdx.x & 31;
  const int lr = lane % LPR, sub = lane / LPR;
  griddep_wait();  // the projection's output comes from the previous kernel in the stream
  griddep_launch_dependents();
  // All units of queries, then those of keys, then those of values: a CTA's warps end together.
  const int64_t u = int64_t(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int uq = (p.num_q_heads + rows_per_unit - 1) / rows_per_unit, uk = (p.kv_heads + rows_per_unit - 1) / rows_per_unit;
  const int64_t nq = p.num_tokens * uq, nk = p.num_tokens * uk;
  if (u >= nq + 2 * nk) return;
  const int kind = u < nq ? 0 : u < nq + nk ? 1 : 2;  // query, key, value
  const int64_t at = u - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk);
  const int per = kind == 0 ? uq : uk;  // units per token
  const int64_t t = (at >> 32) == 0 ? int64_t(uint32_t(at) / uint32_t(per)) : at / per;
  const int r0 = int(at - t * per) * rows_per_unit;
  const int r1 = min(kind == 0 ? p.num_q_heads : p.kv_heads, r0 + rows_per_unit);
  // The lane's two pieces of 8 values: the two halves of 8 rotated pairs, or what lies past the
  // rotated part, or (values, interleaved pairs) any two.
  const bool apart = kind != 2 && !p.interleaved;
  const int half8 = apart ? p.rot_dim >> 4 : 0;  // pieces of half the rotated part
  const int c0 = lr < half8 ? lr : lr + half8, c1 = lr < half8 ? lr + half8 : lr + LPR;
  const auto* src = static_cast<const __nv_bfloat16*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                    t * (kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride);
  auto load = [&](int r, int st) {
    if (r + sub < r1) {
      copy_piece(&stage[st][0][threadIdx.x], src + int64_t(r + sub) * D + c0 * 8);
      copy_piece(&stage[st][1][threadIdx.x], src + int64_t(r + sub) * D + c1 * 8);
    }
    copies_next_step();
  };
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) load(r0 + i * RPS, i);
  int64_t slot = -1;
  if (kind != 0) {
    slot = __ldg(p.slot_mapping + t);
    if (slot >= p.num_blocks * kBlockSize) {
      if (lane == 0 && r0 == 0 && kind == 1) set_error(p.err, kErrSlot);
      slot = -1;
    }
  }
  // whether pairs of the lane's first four and of its last four are rotated
  const bool turns0 = kind != 2 && p.rot_dim > 0 && (apart ? lr < half8 : c0 * 8 < p.rot_dim);
  const bool turns1 = kind != 2 && p.rot_dim > 0 && (apart ? lr < half8 : c1 * 8 < p.rot_dim);
  bool ok = true;
  float4 cs[2] = {make_float4(1.0f, 1.0f, 1.0f, 1.0f), make_float4(1.0f, 1.0f, 1.0f, 1.0f)};
  float4 sn[2] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  if (p.cos_sin) {
    const int pos = __ldg(p.positions + t);
    ok = pos >= 0 && pos < p.max_position;
    if (!ok && lane == 0 && kind == 0 && r0 == 0) set_error(p.err, kErrPosition);
    const float4* row = reinterpret_cast<const float4*>(p.cos_sin + int64_t(pos) * p.rot_dim);
    const int half4 = p.rot_dim >> 3, i0 = apart ? 2 * lr : c0, i1 = apart ? 2 * lr + 1 : c1;
    if (ok && turns0) {
      cs[0] = __ldg(row + i0);
      sn[0] = __ldg(row + half4 + i0);
    }
    if (ok && turns1) {
      cs[1] = __ldg(row + i1);
      sn[1] = __ldg(row + half4 + i1);
    }
  }
  const void* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
  // Pairs (a, b) -> (w_a a cos - w_b b sin, w_b b cos + w_a a sin), two pairs to a register pair: a weight
  // times a value is exact in fp32, so each result has two roundings.  Pairs are a value of each piece, or
  // neighbours when interleaved.
  uint64_t wa[4], wb[4], cos2[4], sin2[4];
  {
    float w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 1.0f;
    if (weight) {
      unpack8(__ldg(static_cast<const uint4*>(weight) + c0), w);
      unpack8(__ldg(static_cast<const uint4*>(weight) + c1), w + 8);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      wa[j] = apart ? f32x2(w[2 * j], w[2 * j + 1]) : f32x2(w[4 * j], w[4 * j + 2]);
      wb[j] = apart ? f32x2(w[8 + 2 * j], w[9 + 2 * j]) : f32x2(w[4 * j + 1], w[4 * j + 3]);
      cos2[j] = j & 1 ? f32x2(cs[j >> 1].z, cs[j >> 1].w) : f32x2(cs[j >> 1].x, cs[j >> 1].y);
      sin2[j] = j & 1 ? f32x2(sn[j >> 1].z, sn[j >> 1].w) : f32x2(sn[j >> 1].x, sn[j >> 1].y);
    }
  }

  int st = 0;
#pragma unroll 1
  for (int r = r0; r < r1; r += RPS) {
    const int h = r + sub;
    load(r + (kSlots - 1) * RPS, st == 0 ? kSlots - 1 : st - 1);  // over the step before, whose values have all been used
    copies_wait();
    float x[16];
    unpack8(stage[st][0][threadIdx.x], x);
    unpack8(stage[st][1][threadIdx.x], x + 8);
    if (++st == kSlots) st = 0;
    float inv = 1.0f;  // of the row's norm
    if (kind != 2) {
      uint64_t a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[j] = apart ? f32x2(x[2 * j], x[2 * j + 1]) : f32x2(x[4 * j], x[4 * j + 2]);
        b[j] = apart ? f32x2(x[8 + 2 * j], x[9 + 2 * j]) : f32x2(x[4 * j + 1], x[4 * j + 3]);
      }
      if (weight) {
        uint64_t q2 = mul2(a[0], a[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) q2 = fma2(a[j], a[j], q2);
#pragma unroll
        for (int j = 0; j < 4; ++j) q2 = fma2(b[j], b[j], q2);
        float ss, hi;
        f32x2_parts(q2, ss, hi);
        ss += hi;
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        inv = rsqrtf(ss * (1.0f / D) + p.eps);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[j] = mul2(a[j], wa[j]);
        b[j] = mul2(b[j], wb[j]);
        if (j < 2 ? turns0 : turns1) {  // elsewhere sine is 0, but an infinity times 0 is not
          const uint64_t ya = fma2(b[j] ^ 0x8000000080000000ull, sin2[j], mul2(a[j], cos2[j]));
          b[j] = fma2(a[j], sin2[j], mul2(b[j], cos2[j]));
          a[j] = ya;
        }
      }
      if (apart) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x2_parts(a[j], x[2 * j], x[2 * j + 1]);
          f32x2_parts(b[j], x[8 + 2 * j], x[9 + 2 * j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x2_parts(a[j], x[4 * j], x[4 * j + 2]);
          f32x2_parts(b[j], x[4 * j + 1], x[4 * j + 3]);
        }
      }
    }
    if (kind == 0) {
      if (h < r1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= inv;
        auto* to = static_cast<__nv_bfloat16*>(p.q_out) + t * p.out_stride + int64_t(h) * D;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(to + c0 * 8) = ok ? pack8(x) : zero;
        *reinterpret_cast<uint4*>(to + c1 * 8) = ok ? pack8(x + 8) : zero;
      }
    } else {
      const int64_t row = ((slot / kBlockSize) * p.kv_heads + h) * kBlockSize + slot % kBlockSize;
      store_cache<KV, LPR>(x, inv, kind == 1 ? p.k_cache : p.v_cache, kind == 1 ? p.k_scale : p.v_scale, row, c0, c1,
                           ok && slot >= 0 && h < r1, lr == 0);
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
  // Rows of a unit: one step's, doubled (up to all of a token's heads) while that leaves 1.5 units for
  // each warp the GPU holds at a time.  More rows share a token's position, table row and weights; fewer
  // are done sooner.  Measured on GB300, 32 + 8 + 8 heads of 128 into a bf16 pool, 4 / 8 / 16 / 32 rows: 64
  // tokens 2.3 / 2.5 / 3.1 / 4.4 us, 1024 9.9 / 7.5 / 7.3 / 11.2, 1536 14.0 / 10.1 / 9.0 / 11.1, 2048
  // 17.7 / 12.8 / 11.5 / 10.8, 16384 142 / 97 / 80 / 72.7.
  const int most = p.num_q_heads > p.kv_heads ? p.num_q_heads : p.kv_heads;
  auto count = [&](int rows) {
    return p.num_tokens * ((p.num_q_heads + int64_t(rows) - 1) / rows + 2 * ((p.kv_heads + int64_t(rows) - 1) / rows));
  };
  int rows = 32 / (D / 16);
  while (rows < most && rows < (1 << 20) && count(2 * rows) * 2 >= 3 * 152 * kMinCtas * kWarps) rows *= 2;
  const int64_t units = count(rows);
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
