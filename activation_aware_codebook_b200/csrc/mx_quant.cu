// mx_quant.cu -- rows of bf16 or fp32 to microscaled 4 bits, and back.
//
//   E8M0 (blocks of 32):  byte = max(exponent(amax) - 2, 0) with exponent()
//     the biased exponent of the block's largest magnitude (2 is E2M1's
//     largest exponent), code = E2M1_RN_sat(x * 2^(127 - byte)): the OCP
//     microscaling conversion.
//   E4M3 (blocks of 16):  g = 2^p per row, p the smallest with
//     row amax <= 2688 * 2^p (2688 = 6 * 448, the largest value under the
//     largest scale), s = E4M3_RN(fp32_RN(block amax * 2^-p / 6)),
//     code = E2M1_RN_sat(x * 2^-p / s).
// g is a power of two so that taking it out and multiplying it back are exact:
// the choice of a code is one correctly rounded quotient away from x, and a
// row's codes depend on that row alone (a token is quantised the same
// whatever batch it comes in).  Ties go to the even code.
//
// quantize_kernel: one block a row.  Each thread holds `C` runs of 16
// consecutive values (two 16-byte loads each) in registers between the row's
// maximum and its codes, so a row is read once; a run is one E4M3 block, and
// half an E8M0 one.  Bound by HBM: 2 bytes in, 0.53 to 0.56 out per value.
#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "tcgen05.cuh"

namespace aaac {

namespace {

struct QuantArgs {
  const void* X;
  const int32_t* index;  // source row of each row, or NULL
  int64_t ldx;           // elements
  int src_rows, K;
  MxRows rows;
  uint8_t* codes;
  uint8_t* scales;
  float* row_scale;
  int64_t tiles_k;
};

// The group of row r (the number of later groups that start at or before it),
// by the whole warp; -1 when r lies in no group.
__device__ __forceinline__ int group_of(const MxRows& g, int r, int lane) {
  if (!g.offsets) return min(r / (g.rows / g.groups), g.groups - 1);
  int e = 0;
  for (int i = 1; i <= g.groups; i += 32) {
    const bool before = i + lane <= g.groups && __ldg(g.offsets + min(i + lane, g.groups)) <= r;
    const unsigned b = __ballot_sync(0xffffffffu, before);
    e += __popc(b);
    if (b != 0xffffffffu) break;
  }
  return e >= g.groups || r < __ldg(g.offsets) ? -1 : e;
}

// Where row r of group e keeps its scale bytes (of the first tile along K).
__device__ __forceinline__ int64_t scale_at(const MxRows& g, int e, int r, int64_t tiles_k) {
  int first, last;
  mx_group(g, e, &first, &last);
  const int local = max(r - first, 0);
  const int64_t band = min((int64_t)first / kMxTileRows + e + local / kMxTileRows,
                           mx_bands(g.rows, g.groups) - 1);
  const int i = local % kMxTileRows;
  return band * tiles_k * kMxTileBytes + (i % 32) * 16 + (i / 32) * 4;
}

__device__ __forceinline__ float silu_mul(float a, float b) {
  return __fmul_rn(__fdiv_rn(a, __fadd_rn(1.0f, expf(-a))), b);
}

// 16 values of a row.  bf16 stays packed: half the registers.
template <bool F32, bool SWIGLU>
struct Run {
  float v[16];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = 0.0f;
  }
  __device__ __forceinline__ static void load16(const void* X, int64_t at, float (&o)[16]) {
    if (F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(X) + at);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float4 q = __ldg(p + i);
        o[4 * i] = q.x;
        o[4 * i + 1] = q.y;
        o[4 * i + 2] = q.z;
        o[4 * i + 3] = q.w;
      }
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(X) + at);
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const uint4 q = __ldg(p + i);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
          o[8 * i + 2 * j] = bf16_lo(w[j]);
          o[8 * i + 2 * j + 1] = bf16_hi(w[j]);
        }
      }
    }
  }
  // row_at: the source row's first element; col: this run's first column
  __device__ __forceinline__ void load(const void* X, int64_t row_at, int col, int K) {
    load16(X, row_at + col, v);
    if (SWIGLU) {
      float u[16];
      load16(X, row_at + K + col, u);
#pragma unroll
      for (int i = 0; i < 16; i++) v[i] = silu_mul(v[i], u[i]);
    }
  }
  // the largest magnitude's bits (a NaN or infinity is above every number)
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ float get(int i) const { return v[i]; }
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
    const uint4 a = __ldg(p), b = __ldg(p + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    return max(m << 16, m & 0xffff0000u);
  }
  __device__ __forceinline__ float get(int i) const {
    return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
  }
};

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

// Codes and scale of one run, written out.  Every lane of the warp takes part
// (the lanes of a scale word meet in shuffles); `in` says whether this lane's
// run lies inside the row.  pbits: E4M3 only, the bits of 2^-p.
template <int FMT, bool F32, bool SWIGLU>
__device__ __forceinline__ void emit(const Run<F32, SWIGLU>& run, bool in, int col, int lane,
                                     float down, bool bad_row, uint8_t* crow, uint8_t* srow) {
  const uint32_t own = run.amax();
  uint32_t word;
  uint32_t c[2];
  if (FMT == kMxE8m0) {
    const uint32_t m = max(own, __shfl_xor_sync(0xffffffffu, own, 1));
    const bool bad = m >= kInfBits;
    const uint32_t byte = bad ? 255u : (uint32_t)max((int)(m >> 23) - 2, 0);
    // byte <= 252 for finite values, so 2^(127 - byte) is a normal number
    const float inv = bad ? 0.0f : __uint_as_float((254u - byte) << 23);
#pragma unroll
    for (int h = 0; h < 2; h++) {
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; i++) q[i] = bad ? 0.0f : __fmul_rn(run.get(8 * h + i), inv);
      c[h] = e2m1x8(q);
    }
    word = in ? byte << (8 * ((lane >> 1) & 3)) : 0u;
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
  } else {
    const float top = bad_row ? 0.0f : __fmul_rn(__uint_as_float(own), down);
    const uint32_t byte =
        (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(top, 6.0f), __NV_SATFINITE, __NV_E4M3);
    const float s = e4m3_mag(byte);
    const bool none = byte == 0u || bad_row;
    // The quotient x' / s, x' = x * 2^-p.  For bf16 inputs: with r = 1/s
    // rounded towards zero and rl = fp32_RN(1/s - r) >= 0, fma(x', r, x' * rl)
    // is the quotient to within 2^-24 (1 + 2^-21) of it, and exactly the
    // quotient where that is a number of few bits (and keeps the sign of a
    // zero).  A border between codes is such a number, and a quotient of an
    // 8-bit x' and a 4-bit s that is not on a border is 2^-9 or more away
    // from it; so every code is the one that the exact quotient has, without
    // a division per value.  fp32 inputs have no such gap and take the
    // correctly rounded division.
    const float r = none ? 0.0f : __frcp_rz(s);
    const float rl = none ? 0.0f : __fmul_rn(__fmaf_rn(-s, r, 1.0f), r);
#pragma unroll
    for (int h = 0; h < 2; h++) {
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float x = none ? 0.0f : __fmul_rn(run.get(8 * h + i), down);
        q[i] = (F32 || SWIGLU) ? (none ? 0.0f : __fdiv_rn(x, s))
                               : __fmaf_rn(x, r, __fmul_rn(x, rl));
      }
      c[h] = e2m1x8(q);
    }
    word = in ? byte << (8 * (lane & 3)) : 0u;
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
  }
  if (in) {
    *reinterpret_cast<uint2*>(crow + (col >> 1)) = make_uint2(c[0], c[1]);
    constexpr int kLanes = FMT == kMxE8m0 ? 8 : 4;  // lanes of one scale word
    if (lane % kLanes == 0)
      *reinterpret_cast<uint32_t*>(srow + (int64_t)(col / (16 * kLanes)) * kMxTileBytes) = word;
  }
}

// C > 0: the row fits in C runs a thread.  C == 0: rows of any length, read
// twice (the second time mostly from L2).
template <int FMT, bool F32, bool SWIGLU, int C>
__global__ void __launch_bounds__(1024)
quantize_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ uint32_t s_max[32];
  // the product that follows may set itself up while this kernel runs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int T = blockDim.x;
  const int src = a.index ? __ldg(a.index + row) : row;
  const bool have = src >= 0 && src < a.src_rows;
  const int64_t row_at = (int64_t)(have ? src : 0) * a.ldx;
  const int runs = a.K >> 4;
  constexpr int kHeld = C ? C : 1;
  Run<F32, SWIGLU> run[kHeld];
  if (C) {
#pragma unroll
    for (int c = 0; c < kHeld; c++) {
      const int i = c * T + threadIdx.x;
      if (have && i < runs) run[c].load(a.X, row_at, i * 16, a.K);
      else run[c].zero();
    }
  }
  const int e = group_of(a.rows, row, lane);
  if (e < 0) return;  // the whole block: a row of no group stays as it was
  float down = 1.0f;
  bool bad_row = false;
  if (FMT == kMxE4m3) {
    uint32_t m = 0;
    if (C) {
#pragma unroll
      for (int c = 0; c < kHeld; c++) m = max(m, run[c].amax());
    } else if (have) {
      for (int i = threadIdx.x; i < runs; i += T) {
        run[0].load(a.X, row_at, i * 16, a.K);
        m = max(m, run[0].amax());
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (T > 32) {
      if (lane == 0) s_max[warp] = m;
      __syncthreads();
      m = __reduce_max_sync(0xffffffffu, lane < (T >> 5) ? s_max[lane] : 0u);
    }
    bad_row = m >= kInfBits;
    int p = max((int)(m >> 23) - 138 + ((m & 0x7fffffu) > 0x280000u ? 1 : 0), -126);
    if (m == 0u || bad_row) p = 0;
    down = __uint_as_float((uint32_t)(127 - p) << 23);
    if (threadIdx.x == 0)
      a.row_scale[row] = __uint_as_float(bad_row ? 0x7fc00000u : (uint32_t)(127 + p) << 23);
  }
  uint8_t* crow = a.codes + (int64_t)row * (a.K >> 1);
  uint8_t* srow = a.scales + scale_at(a.rows, e, row, a.tiles_k);
  if (C) {
#pragma unroll
    for (int c = 0; c < kHeld; c++) {
      const int i = c * T + threadIdx.x;
      if (c * T + warp * 32 < runs)
        emit<FMT, F32, SWIGLU>(run[c], i < runs, i * 16, lane, down, bad_row, crow, srow);
    }
  } else {
    for (int i0 = warp * 32; i0 < runs; i0 += T) {
      const int i = i0 + lane;
      if (have && i < runs) run[0].load(a.X, row_at, i * 16, a.K);
      else run[0].zero();
      emit<FMT, F32, SWIGLU>(run[0], i < runs, i * 16, lane, down, bad_row, crow, srow);
    }
  }
}

template <int FMT, bool F32, bool SWIGLU>
void launch_quantize_t(const QuantArgs& a, cudaStream_t st) {
  const int runs = a.K >> 4;
  auto threads = [](int n) { return n < 1024 ? (n + 31) / 32 * 32 : 1024; };
  const unsigned grid = (unsigned)a.rows.rows;
  if (runs <= 1024)
    quantize_kernel<FMT, F32, SWIGLU, 1><<<grid, threads(runs), 0, st>>>(a);
  else if (runs <= 2048)
    quantize_kernel<FMT, F32, SWIGLU, 2><<<grid, threads((runs + 1) / 2), 0, st>>>(a);
  else
    quantize_kernel<FMT, F32, SWIGLU, 0><<<grid, 1024, 0, st>>>(a);
}

// Back to bf16 or fp32: E2M1 * scale * row scale, exact in fp32 (2 + 4 bits).
// A block walks rows; consecutive lanes take consecutive 8-value pieces (4
// bytes of codes in, 16 or 32 bytes out).
template <int FMT, bool F32>
__global__ void __launch_bounds__(256)
mx_dequant_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                  const float* __restrict__ row_scale, MxRows rows, int K, int64_t tiles_k,
                  void* __restrict__ out, int64_t ldo) {
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x;
  const int e = group_of(rows, row, lane);
  if (e < 0) return;
  const uint32_t* crow = reinterpret_cast<const uint32_t*>(codes + (int64_t)row * (K >> 1));
  const uint8_t* srow = scales + scale_at(rows, e, row, tiles_k);
  const float g = FMT == kMxE4m3 ? __ldg(row_scale + row) : 1.0f;
  constexpr int kPieces = FMT == kMxE8m0 ? 4 : 2;  // 8-value pieces of a block
#pragma unroll 4
  for (int i = threadIdx.x; i < (K >> 3); i += blockDim.x) {
    const uint32_t w = __ldg(crow + i);
    const int b = i / kPieces;
    const uint32_t sb = __ldg(srow + (int64_t)(b >> 2) * kMxTileBytes + (b & 3));
    float s;
    if (FMT == kMxE8m0)  // 2^(byte - 127); 255 is NaN
      s = sb == 255u ? __uint_as_float(0x7fc00000u)
                     : __uint_as_float(sb ? sb << 23 : 0x00400000u);
    else
      s = __fmul_rn(e4m3_mag(sb & 0x7fu), g);
    float v[8];
    uint32_t h[4];
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int j = 0; j < 4; j++) {
      float lo, hi;
      asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
          : "=f"(lo), "=f"(hi)
          : "r"(h[j]));
      v[2 * j] = __fmul_rn(lo, s);
      v[2 * j + 1] = __fmul_rn(hi, s);
    }
    if (F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + row * ldo + 8 * (int64_t)i);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t p[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        p[j] = *reinterpret_cast<const uint32_t*>(&t);
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * ldo + 8 * (int64_t)i) =
          make_uint4(p[0], p[1], p[2], p[3]);
    }
  }
}

}  // namespace

size_t mx_scale_bytes(int fmt, int64_t rows, int64_t K, int groups) {
  return (size_t)mx_bands(rows, groups) * (size_t)mx_tiles_k(fmt, K) * kMxTileBytes;
}

cudaError_t launch_mx_quantize(const MxSource& x, const MxTensor& q, cudaStream_t st) {
  QuantArgs a{x.X, x.index, x.ldx, (int)x.rows, (int)q.K,
              MxRows{q.offsets, q.groups, (int)q.rows}, q.codes, q.scales, q.row_scale,
              mx_tiles_k(q.fmt, q.K)};
  if (q.fmt == kMxE8m0) {
    if (x.f32) {
      if (x.swiglu) launch_quantize_t<kMxE8m0, true, true>(a, st);
      else launch_quantize_t<kMxE8m0, true, false>(a, st);
    } else {
      if (x.swiglu) launch_quantize_t<kMxE8m0, false, true>(a, st);
      else launch_quantize_t<kMxE8m0, false, false>(a, st);
    }
  } else {
    if (x.f32) {
      if (x.swiglu) launch_quantize_t<kMxE4m3, true, true>(a, st);
      else launch_quantize_t<kMxE4m3, true, false>(a, st);
    } else {
      if (x.swiglu) launch_quantize_t<kMxE4m3, false, true>(a, st);
      else launch_quantize_t<kMxE4m3, false, false>(a, st);
    }
  }
  return cudaGetLastError();
}

cudaError_t launch_mx_dequant(const MxTensor& q, void* out, bool f32, int64_t ldo,
                              cudaStream_t st) {
  const MxRows rows{q.offsets, q.groups, (int)q.rows};
  const int pieces = (int)(q.K >> 3);
  const int threads = pieces < 256 ? (pieces + 31) / 32 * 32 : 256;
  const unsigned grid = (unsigned)q.rows;
  const int K = (int)q.K;
  const int64_t tk = mx_tiles_k(q.fmt, q.K);
  if (q.fmt == kMxE8m0) {
    if (f32) mx_dequant_kernel<kMxE8m0, true><<<grid, threads, 0, st>>>(q.codes, q.scales, q.row_scale, rows, K, tk, out, ldo);
    else mx_dequant_kernel<kMxE8m0, false><<<grid, threads, 0, st>>>(q.codes, q.scales, q.row_scale, rows, K, tk, out, ldo);
  } else {
    if (f32) mx_dequant_kernel<kMxE4m3, true><<<grid, threads, 0, st>>>(q.codes, q.scales, q.row_scale, rows, K, tk, out, ldo);
    else mx_dequant_kernel<kMxE4m3, false><<<grid, threads, 0, st>>>(q.codes, q.scales, q.row_scale, rows, K, tk, out, ldo);
  }
  return cudaGetLastError();
}

}  // namespace aaac
