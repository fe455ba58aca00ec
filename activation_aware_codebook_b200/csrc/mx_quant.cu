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
// half an E8M0 one.  2 bytes in, 0.53 (E8M0) or 0.56 (E4M3) out per value.
// Measured back to back in a graph, on inputs larger than L2, beside the time of
// the bytes at 6.55 TB/s: 8192 x 14336 bf16 to E8M0 44 us (45), to E4M3 47 us (46);
// from fp32 76 (81) and 89 (82).  SwiGLU of 4099 x 2 x 8192 bf16 to E8M0 31.5 us
// (23), to E4M3 37 us (23): 30 instructions a value, most of them expf, the
// divisions and unpacking, which keep the issue slots busy in 75% of the active
// cycles (67% of all); from fp32 45.5 and 50 (44).
// mx_dequant_kernel: 27648 x 5120 from E4M3 to bf16 56 us (55), to fp32 98 us (99);
// mx_dequant_ragged_kernel: 8192 x 14336 in 16 groups 50 us (46).
#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "mx_run.cuh"

namespace aaac {

namespace {

// Division of n < 2^31 by a fixed d: (n m) >> (31 + l) with l = ceil(log2 d)
// and m = floor(2^(31 + l) / d) + 1; m d exceeds 2^(31 + l) by at most d <= 2^l,
// so n times that excess stays below 2^(31 + l).
struct Div {
  uint32_t m, shift, d;
  explicit Div(uint32_t d_) : d(d_) {
    uint32_t l = 0;
    while (((uint64_t)1 << l) < d) l++;
    shift = 31 + l;
    m = (uint32_t)(((uint64_t)1 << shift) / d + 1);
    if (d == 1) m = 1, shift = 0;
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * m) >> shift);
  }
};

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
  Div per;  // rows of a group, where all groups are equal
};

// The ragged group of row r (the number of later groups that start at or
// before it), by the whole warp; -1 when r lies in no group.
__device__ __forceinline__ int group_of(const MxRows& g, int r, int lane) {
  int e = 0;
  for (int i = 1; i <= g.groups; i += 32) {
    const bool before = i + lane <= g.groups && load_i32(g.offsets + min(i + lane, g.groups)) <= r;
    const unsigned b = __ballot_sync(0xffffffffu, before);
    e += __popc(b);
    if (b != 0xffffffffu) break;
  }
  return e >= g.groups || r < load_i32(g.offsets) ? -1 : e;
}

// Where row r of group e, whose first row is `first`, keeps its scale bytes (of
// the first tile along K).
__device__ __forceinline__ int64_t scale_place(uint32_t e, uint32_t first, uint32_t r,
                                               int64_t tiles_k) {
  const uint32_t local = r - first, i = local % kMxTileRows;
  return (int64_t)(first / kMxTileRows + e + local / kMxTileRows) * tiles_k * kMxTileBytes +
         (i % 32) * 16 + i / 32 * 4;
}
__device__ __forceinline__ int64_t scale_equal(const Div& per, uint32_t r, int64_t tiles_k) {
  const uint32_t e = per(r);
  return scale_place(e, e * per.d, r, tiles_k);
}
// -1 for a row of no group; inside the tensor whatever the offsets say.
__device__ __forceinline__ int64_t scale_ragged(const MxRows& g, int r, int lane,
                                                int64_t tiles_k) {
  const int e = group_of(g, r, lane);
  if (e < 0) return -1;
  int first, last;
  mx_group(g, e, &first, &last);
  return scale_place((uint32_t)e, (uint32_t)min(first, r), (uint32_t)r, tiles_k);
}

// Codes and scale of one run, written out.  Every lane of the warp takes part
// (the lanes of a scale word meet in shuffles); `in` says whether this lane's
// run lies inside the row.  down: E4M3 only, 2^-p.
template <int FMT, bool F32, bool SWIGLU>
__device__ __forceinline__ void emit(const Run<F32, SWIGLU>& run, bool in, int col, int lane,
                                     float down, bool bad_row, uint8_t* crow, uint8_t* srow) {
  uint32_t c[2];
  const uint32_t byte = encode<FMT>(run, down, bad_row, c);
  constexpr int kLanes = FMT == kMxE8m0 ? 8 : 4;  // lanes of one scale word
  uint32_t word = in ? byte << (8 * (lane % kLanes * 4 / kLanes)) : 0u;
  word |= __shfl_xor_sync(0xffffffffu, word, kLanes / 4);
  word |= __shfl_xor_sync(0xffffffffu, word, kLanes / 2);
  if (in) {
    *reinterpret_cast<uint2*>(crow + (col >> 1)) = make_uint2(c[0], c[1]);
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
  after_previous();
  let_next_start();
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int T = blockDim.x;
  const int src = a.index ? load_i32(a.index + row) : row;
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
  const int64_t at = a.rows.offsets ? scale_ragged(a.rows, row, lane, a.tiles_k)
                                    : scale_equal(a.per, (uint32_t)row, a.tiles_k);
  if (at < 0) return;  // the whole block: a row of no group stays as it was
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
    float g;
    const int p = row_exponent(m, &bad_row, &g);
    down = __uint_as_float((uint32_t)(127 - p) << 23);
    if (threadIdx.x == 0) a.row_scale[row] = g;
  }
  uint8_t* crow = a.codes + (int64_t)row * (a.K >> 1);
  uint8_t* srow = a.scales + at;
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

// A launch that may start while the kernel before it runs (see mx.cuh).
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, unsigned threads, cudaStream_t st,
                   const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

// Runs a thread holds.  With many rows: enough that a block's loads cover the
// time its predecessor on the SM takes to compute and leave (8192 x 14336 to
// E8M0: 78 us at one run a thread).  With few rows: one, for the most threads.
template <int FMT, bool F32, bool SWIGLU>
cudaError_t launch_quantize_t(const QuantArgs& a, cudaStream_t st) {
  constexpr int kMany = F32 || SWIGLU ? 2 : 4;
  const int runs = a.K >> 4;
  auto threads = [](int n) { return n < 1024 ? (n + 31) / 32 * 32 : 1024; };
  const unsigned grid = (unsigned)a.rows.rows;
  if (runs > 1024 * kMany)
    return launch(quantize_kernel<FMT, F32, SWIGLU, 0>, grid, 1024, st, a);
  if (runs > 1024 || (!SWIGLU && a.rows.rows >= 4 * 148))
    return launch(quantize_kernel<FMT, F32, SWIGLU, kMany>, grid,
                  threads((runs + kMany - 1) / kMany), st, a);
  return launch(quantize_kernel<FMT, F32, SWIGLU, 1>, grid, threads(runs), st, a);
}

// 16 values from two words of codes: E2M1 * s, exact in fp32.
__device__ __forceinline__ void expand16(uint2 w, float s, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; i++) {
    uint32_t h[4];
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(i ? w.y : w.x));
#pragma unroll
    for (int j = 0; j < 4; j++) {
      float lo, hi;
      asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
          : "=f"(lo), "=f"(hi)
          : "r"(h[j]));
      v[8 * i + 2 * j] = __fmul_rn(lo, s);
      v[8 * i + 2 * j + 1] = __fmul_rn(hi, s);
    }
  }
}

// The scale a byte stands for, times the row's g.
template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t byte, float g) {
  if (FMT == kMxE4m3) return __fmul_rn(e4m3_value(byte), g);
  return byte == 255u ? __uint_as_float(0x7fc00000u)  // 2^(byte - 127); 255 is NaN
                      : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// 32 bytes of a row: one 32-byte store where rows are so aligned.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <bool F32>
__device__ __forceinline__ void store16(void* out, int64_t at, const float (&v)[16], bool wide) {
  uint32_t w[8];
  if (F32) {
    float* o = static_cast<float*>(out) + at;
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int i = 0; i < 8; i++) w[i] = __float_as_uint(v[8 * h + i]);
      store32(o + 8 * h, w, wide);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    store32(static_cast<uint16_t*>(out) + at, w, wide);
  }
}

struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* row_scale;
  MxRows rows;
  int K;
  int64_t tiles_k;
  void* out;
  int64_t ldo;
  bool wide;
};

template <int FMT>
__device__ __forceinline__ int64_t scale_step(int run) {  // a run's byte within its row
  const int b = FMT == kMxE8m0 ? run >> 1 : run;
  return (int64_t)(b >> 2) * kMxTileBytes + (b & 3);
}

// Back to bf16 or fp32.  Groups of equal size: the tensor's 16-value runs, four
// to a thread (its loads together), whatever the row length; 8 bytes of codes
// and a scale byte in, one 32-byte store (two for fp32) out.
constexpr int kDeqThreads = 256, kDeqRuns = 4;
template <int FMT, bool F32>
__global__ void __launch_bounds__(kDeqThreads)
mx_dequant_kernel(const __grid_constant__ DequantArgs a, int row0, uint32_t total, Div runs,
                  Div per) {
  after_previous();
  let_next_start();
  const uint32_t i0 = blockIdx.x * (kDeqThreads * kDeqRuns) + threadIdx.x;
  uint2 w[kDeqRuns];
  uint32_t sb[kDeqRuns];
  float g[kDeqRuns];
  int row[kDeqRuns], run[kDeqRuns];
#pragma unroll
  for (int u = 0; u < kDeqRuns; u++) {
    const uint32_t i = min(i0 + u * kDeqThreads, total - 1);
    const uint32_t r = runs(i);
    row[u] = row0 + (int)r;
    run[u] = (int)(i - r * runs.d);
    const uint8_t* srow = a.scales + scale_equal(per, (uint32_t)row[u], a.tiles_k);
    w[u] = load_2(reinterpret_cast<const uint2*>(a.codes + (int64_t)row[u] * (a.K >> 1)) + run[u]);
    sb[u] = load_u8(srow + scale_step<FMT>(run[u]));
    g[u] = FMT == kMxE4m3 ? load_f32(a.row_scale + row[u]) : 1.0f;
  }
#pragma unroll
  for (int u = 0; u < kDeqRuns; u++) {
    float v[16];
    expand16(w[u], scale_value<FMT>(sb[u], g[u]), v);
    if (i0 + u * kDeqThreads < total)
      store16<F32>(a.out, row[u] * a.ldo + 16 * (int64_t)run[u], v, a.wide);
  }
}

// Ragged groups: a block a row, its group found once.
template <int FMT, bool F32>
__global__ void __launch_bounds__(kDeqThreads)
mx_dequant_ragged_kernel(const __grid_constant__ DequantArgs a) {
  after_previous();
  let_next_start();
  const int row = blockIdx.x;
  const int64_t at = scale_ragged(a.rows, row, threadIdx.x & 31, a.tiles_k);
  if (at < 0) return;
  const uint2* crow = reinterpret_cast<const uint2*>(a.codes + (int64_t)row * (a.K >> 1));
  const uint8_t* srow = a.scales + at;
  const float g = FMT == kMxE4m3 ? load_f32(a.row_scale + row) : 1.0f;
#pragma unroll 2
  for (int i = threadIdx.x; i < (a.K >> 4); i += blockDim.x) {
    float v[16];
    expand16(load_2(crow + i), scale_value<FMT>(load_u8(srow + scale_step<FMT>(i)), g), v);
    store16<F32>(a.out, row * a.ldo + 16 * (int64_t)i, v, a.wide);
  }
}

template <int FMT, bool F32>
cudaError_t launch_dequant_t(const DequantArgs& a, cudaStream_t st) {
  const int runs = a.K >> 4;
  if (a.rows.offsets)
    return launch(mx_dequant_ragged_kernel<FMT, F32>, (unsigned)a.rows.rows,
                  runs < kDeqThreads ? (runs + 31) / 32 * 32 : kDeqThreads, st, a);
  // as many rows to a launch as 2^30 runs hold
  const int64_t step = ((int64_t)1 << 30) / runs;
  for (int64_t r0 = 0; r0 < a.rows.rows; r0 += step) {
    const int64_t n = a.rows.rows - r0 < step ? a.rows.rows - r0 : step;
    const uint32_t total = (uint32_t)(n * runs);
    const unsigned grid = (total + kDeqThreads * kDeqRuns - 1) / (kDeqThreads * kDeqRuns);
    const cudaError_t e =
        launch(mx_dequant_kernel<FMT, F32>, grid, kDeqThreads, st, a, (int)r0, total,
               Div((uint32_t)runs), Div((uint32_t)(a.rows.rows / a.rows.groups)));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t mx_scale_bytes(int fmt, int64_t rows, int64_t K, int groups) {
  return (size_t)mx_bands(rows, groups) * (size_t)mx_tiles_k(fmt, K) * kMxTileBytes;
}

cudaError_t launch_mx_quantize(const MxSource& x, const MxTensor& q, cudaStream_t st) {
  QuantArgs a{x.X, x.index, x.ldx, (int)x.rows, (int)q.K,
              MxRows{q.offsets, q.groups, (int)q.rows}, q.codes, q.scales, q.row_scale,
              mx_tiles_k(q.fmt, q.K), Div((uint32_t)(q.rows / q.groups ? q.rows / q.groups : 1))};
  if (q.fmt == kMxE8m0) {
    if (x.f32)
      return x.swiglu ? launch_quantize_t<kMxE8m0, true, true>(a, st)
                      : launch_quantize_t<kMxE8m0, true, false>(a, st);
    return x.swiglu ? launch_quantize_t<kMxE8m0, false, true>(a, st)
                    : launch_quantize_t<kMxE8m0, false, false>(a, st);
  }
  if (x.f32)
    return x.swiglu ? launch_quantize_t<kMxE4m3, true, true>(a, st)
                    : launch_quantize_t<kMxE4m3, true, false>(a, st);
  return x.swiglu ? launch_quantize_t<kMxE4m3, false, true>(a, st)
                  : launch_quantize_t<kMxE4m3, false, false>(a, st);
}

cudaError_t launch_mx_dequant(const MxTensor& q, void* out, bool f32, int64_t ldo,
                              cudaStream_t st) {
  const int size = f32 ? 4 : 2;
  const DequantArgs a{q.codes, q.scales, q.row_scale, MxRows{q.offsets, q.groups, (int)q.rows},
                      (int)q.K, mx_tiles_k(q.fmt, q.K), out, ldo,
                      reinterpret_cast<uintptr_t>(out) % 32 == 0 && ldo * size % 32 == 0};
  if (q.fmt == kMxE8m0)
    return f32 ? launch_dequant_t<kMxE8m0, true>(a, st) : launch_dequant_t<kMxE8m0, false>(a, st);
  return f32 ? launch_dequant_t<kMxE4m3, true>(a, st) : launch_dequant_t<kMxE4m3, false>(a, st);
}

}  // namespace aaac
