// mx_run.cuh -- 16 consecutive values of a row on their way to microscaled 4
// bits: loading (bf16, fp32, or SwiGLU of two halves), the largest magnitude,
// the block's scale and the codes.  Shared by the quantisation and by the
// product that quantises a few rows itself, so that both give the same bits.
#pragma once

#include "common.cuh"
#include "mx.cuh"

namespace aaac {

namespace {

__device__ __forceinline__ float rcp_approx(float d) {  // within a step of 1 / d
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}

// x / d from r, a reciprocal of d: the quotient x r is off by steps, its
// residual is exact in an fma, and adding the residual's quotient rounds to
// the nearest (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990; always so with r rounded to nearest, and
// all but about one time in a million with r a step off).  Three instructions
// where a division per value takes about ten.
__device__ __forceinline__ float div_by(float x, float d, float r) {
  const float q = __fmul_rn(x, r);
  return __fmaf_rn(-r, __fmaf_rn(d, q, -x), q);  // these signs keep a zero's
}

// Two values in a register pair: one instruction does for both what the scalar
// one does for each, rounded alike (SwiGLU of 65536 x 2 x 2048 to E4M3, when this
// was brought in: 148 us in scalars, 134 in pairs).
struct Two {
  uint64_t p;
  __device__ __forceinline__ Two(float a, float b) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  }
  __device__ __forceinline__ explicit Two(float a) : Two(a, a) {}
  __device__ __forceinline__ explicit Two(uint64_t p_) : p(p_) {}
  __device__ __forceinline__ void get(float& a, float& b) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
  }
};
__device__ __forceinline__ Two mul2(Two a, Two b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.p), "l"(b.p));
  return Two(r);
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a.p), "l"(b.p), "l"(c.p));
  return Two(r);
}

// div_by of two values and with every sign turned, -(x / d) with nr = -r: a
// pair has no negated operands.
__device__ __forceinline__ Two neg_div_by(Two x, Two d, Two nr) {
  const Two q = mul2(x, nr);
  return fma2(nr, fma2(d, q, x), q);
}

// silu(a) b for two columns, each step in fp32; na = -a.  The quotient is taken
// with (1 + exp(-a)) / 4, whose reciprocal is a normal number for every finite
// exp(-a); the factor is exact.  An infinite exp(-a) (a < -88.72) has the
// reciprocal 0 and the quotient -0; held finite in the residual it stays one,
// and NaN comes of an infinite a alone.  Gates that far occur (an outlier
// channel), and cost nothing here: a branch for them did, 39.5 us in place of
// 36.8 for 4099 x 2 x 8192 to E4M3 (36.0 with no care for them).
__device__ __forceinline__ void silu_mul(float na0, float na1, float b0, float b1, float& y0,
                                         float& y1) {
  const Two x(na0, na1);
  const Two d = fma2(Two(0.25f), Two(expf(na0), expf(na1)), Two(0.25f));
  float d0, d1;
  d.get(d0, d1);
  const Two nr(-rcp_approx(d0), -rcp_approx(d1));
  const Two s = neg_div_by(x, Two(fminf(d0, 0x1p126f), fminf(d1, 0x1p126f)), nr);
  mul2(mul2(s, Two(0.25f)), Two(b0, b1)).get(y0, y1);
}

// 16 values of a row.  bf16 stays packed: half the registers.
template <bool F32, bool SWIGLU>
struct Run {
  float v[16];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = 0.0f;
  }
  // NEG: with the signs turned
  template <bool NEG>
  __device__ __forceinline__ static void load16(const void* X, int64_t at, float (&o)[16]) {
    if (F32) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(X) + at);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint4 q = load_4(p + i);
        o[4 * i] = __uint_as_float(q.x ^ (NEG ? 0x80000000u : 0u));
        o[4 * i + 1] = __uint_as_float(q.y ^ (NEG ? 0x80000000u : 0u));
        o[4 * i + 2] = __uint_as_float(q.z ^ (NEG ? 0x80000000u : 0u));
        o[4 * i + 3] = __uint_as_float(q.w ^ (NEG ? 0x80000000u : 0u));
      }
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(X) + at);
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const uint4 q = load_4(p + i);
        uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
          if (NEG) w[j] ^= 0x80008000u;
          o[8 * i + 2 * j] = bf16_lo(w[j]);
          o[8 * i + 2 * j + 1] = bf16_hi(w[j]);
        }
      }
    }
  }
  // row_at: the source row's first element; col: this run's first column
  __device__ __forceinline__ void load(const void* X, int64_t row_at, int col, int K) {
    load16<SWIGLU>(X, row_at + col, v);
    if (SWIGLU) {
      float u[16];
      load16<false>(X, row_at + K + col, u);
#pragma unroll
      for (int i = 0; i < 16; i += 2)
        silu_mul(v[i], v[i + 1], u[i], u[i + 1], v[i], v[i + 1]);
    }
  }
  // the largest magnitude's bits (a NaN or infinity is above every number)
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) {
      float t;
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(t) : "f"(__uint_as_float(m)), "f"(fabsf(v[i])));
      m = __float_as_uint(t);
    }
    return m;
  }
  // half h's values times a power of two
  __device__ __forceinline__ void scaled(int h, float f, float (&o)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      mul2(Two(v[8 * h + i], v[8 * h + i + 1]), Two(f)).get(o[i], o[i + 1]);
  }
};

template <>
struct Run<false, false> {
  uint32_t w[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; i++) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const void* X, int64_t row_at, int col, int) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(X) + row_at + col);
    const uint4 a = load_4(p), b = load_4(p + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    return max(m << 16, m & 0xffff0000u);
  }
  // The product is exact in bf16 too (below 2^-126, where it is not, the code
  // is 0 either way): one multiply for two values.
  __device__ __forceinline__ void scaled(int h, float f, float (&o)[8]) const {
    const uint32_t f2 = __float_as_uint(f) | __float_as_uint(f) >> 16;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      uint32_t p;
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p) : "r"(w[4 * h + i]), "r"(f2));
      o[2 * i] = bf16_lo(p);
      o[2 * i + 1] = bf16_hi(p);
    }
  }
};

// An E4M3 byte without its sign (a scale), exact in fp32.
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  float f;
  asm("{\n .reg .b16 b, l, h;\n .reg .b32 p;\n cvt.u16.u32 b, %1;\n"
      " cvt.rn.f16x2.e4m3x2 p, b;\n mov.b32 {l, h}, p;\n cvt.f32.f16 %0, l;\n}\n"
      : "=f"(f)
      : "r"(byte & 0x7fu));
  return f;
}

// Eight E2M1 codes of eight floats, the first in the lowest nibble; round to
// nearest even, magnitudes above 6 to 6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&q)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

constexpr uint32_t kInfBits = 0x7f800000u;

// E4M3, from the bits of a row's largest magnitude: the exponent p of its power
// of two (1.3125 * 2^11 = 2688 = 6 * 448), whether the row holds a NaN or an
// infinity, and the row scale.
__device__ __forceinline__ int row_exponent(uint32_t m, bool* bad, float* row_scale) {
  *bad = m >= kInfBits;
  int p = max((int)(m >> 23) - 138 + ((m & 0x7fffffu) > 0x280000u ? 1 : 0), -126);
  if (m == 0u || *bad) p = 0;
  *row_scale = __uint_as_float(*bad ? 0x7fc00000u : (uint32_t)(127 + p) << 23);
  return p;
}

// The codes of one run (eight a word) and its block's scale byte.  Every lane of
// the warp takes part: an E8M0 block is two lanes' runs.  down: E4M3 only, 2^-p.
template <int FMT, bool F32, bool SWIGLU>
__device__ __forceinline__ uint32_t encode(const Run<F32, SWIGLU>& run, float down, bool bad_row,
                                           uint32_t (&c)[2]) {
  const uint32_t own = run.amax();
  if (FMT == kMxE8m0) {
    const uint32_t m = max(own, __shfl_xor_sync(0xffffffffu, own, 1));
    const bool bad = m >= kInfBits;
    const uint32_t byte = bad ? 255u : (uint32_t)max((int)(m >> 23) - 2, 0);
    // byte <= 252 for finite values, so 2^(127 - byte) is a normal number
    const float inv = __uint_as_float((254u - byte) << 23);
#pragma unroll
    for (int h = 0; h < 2; h++) {
      float q[8];
      run.scaled(h, inv, q);
      c[h] = bad ? 0u : e2m1x8(q);
    }
    return byte;
  }
  const float top = __fmul_rn(__uint_as_float(own), down);
  const uint32_t byte = bad_row ? 0u
                                : (uint32_t)__nv_cvt_float_to_fp8(
                                      div_by(top, 6.0f, 1.0f / 6.0f), __NV_SATFINITE, __NV_E4M3);
  const float s = e4m3_value(byte);
  // The quotient x' / s, x' = x * 2^-p.
  // bf16: with r a little below 1/s and rl = fp32_RN(r (1 - s r)) > 0, the
  // rest of 1/s, fma(x', r, x' rl) is the quotient to within 2^-24 (1 +
  // 2^-19) of it, and exactly the quotient where that is a number of few
  // bits (and keeps a zero's sign).  A border between codes is such a
  // number, and a quotient of an 8-bit x' and a 4-bit s that is not on a
  // border is 2^-9 or more away from it; so every code is the one that the
  // exact quotient has.
  // fp32 values have no such gap and take the correctly rounded quotient
  // (its residual can only underflow where the code is 0 anyway).
  float r = rcp_approx(s);
  if (F32 || SWIGLU) r = __fmaf_rn(__fmaf_rn(-s, r, 1.0f), r, r);
  else r = __fmul_rn(r, 1.0f - 0x1p-22f);
  const float rl = __fmul_rn(__fmaf_rn(-s, r, 1.0f), r);
#pragma unroll
  for (int h = 0; h < 2; h++) {
    float q[8];
    run.scaled(h, F32 || SWIGLU ? -down : down, q);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const Two x(q[i], q[i + 1]);
      const Two y = F32 || SWIGLU ? neg_div_by(x, Two(s), Two(-r))
                                  : fma2(x, Two(r), mul2(x, Two(rl)));
      y.get(q[i], q[i + 1]);
    }
    c[h] = byte == 0u ? 0u : e2m1x8(q);
  }
  return byte;
}

}  // namespace

}  // namespace aaac
