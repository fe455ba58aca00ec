// mx_gemm.cu -- the product of two microscaled 4-bit tensors on the
// 5th-generation tensor cores, dense or grouped by expert:
//   Y[m][n] = gx[m] gw[n] sum_k xq[m][k] wq[e(m)][n][k]
// with the block scales applied by tcgen05.mma itself (kind::mxf4nvf4,
// block_scale) and fp32 sums in tensor memory.
//
// One CTA computes 128 weight rows x up to NT tokens of Y^T: the weights are
// the M = 128 operand and the tokens the N one, so a single token costs a
// narrow MMA and not a 128-row tile of padding, and a warp's 32 lanes hold 32
// consecutive n of one token when Y is stored.  Per stage of 256 columns of K
// (one 128-byte swizzle row of packed codes per operand row):
//   warp 0      one lane issues the TMA copies of both code tiles
//               (SWIZZLE_128B) and the bulk copies of their scale tiles;
//   warp 1      one lane copies the scale tiles to tensor memory
//               (tcgen05.cp 32x128b, one per 512-byte tile) and issues four
//               MMAs of K = 64; copies and MMAs of one thread run in order;
//   warps 2..9  epilogue: tensor memory -> registers, the accumulator handed
//               back, row scales, stores.
// The tensor core's N is the tile's own row count rounded up to 16, so a
// ragged tile costs what its rows cost.
//
// SPLIT = false: persistent CTAs walk the tiles (weight-tile major inside a
// group, so that CTAs in flight share weight rows in L2).  SPLIT = true: few
// tiles; the CTAs of a cluster take a share of K each, and add their partial
// tiles in rank order through distributed shared memory: the sum's order is
// fixed, whatever the timing.
// Waits are bounded (tcgen05.cuh); a CTA that gives up writes NaN.
#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "tcgen05.cuh"

namespace aaac {

namespace {

constexpr int kWRows = 128;        // weight rows of a tile (MMA M)
constexpr int kStageK = 256;       // columns of a stage
constexpr int kRowBytes = 128;     // of packed codes per stage and row
constexpr int kSteps = 4;          // MMAs of K = 64 per stage
constexpr int kEpiWarps = 8;
constexpr int kMxThreads = (2 + kEpiWarps) * 32;
constexpr int kWTile = kWRows * kRowBytes;  // 16 KB
constexpr int kSmemLimit = 227 * 1024;
constexpr int kSms = 148;

struct MxGemmArgs {
  const uint8_t* sx;
  const uint8_t* sw;
  const float* gx;
  const float* gw;
  void* Y;
  int64_t ldy;
  MxRows rows;        // of X and Y
  int N, K;
  int n_tiles;        // 128-row weight tiles per group
  int stages;         // ceil(K / 256)
  int tiles_k;        // scale tiles along K
  int bf16_out;
};

template <int FMT, int NT>
struct Shape {
  static constexpr int kSub = (NT + 127) / 128;             // 128-row scale bands of a token tile
  static constexpr int kAtoms = FMT == kMxE8m0 ? 2 : 4;     // scale tiles of a stage along K
  static constexpr int kScale = kAtoms * kMxTileBytes;      // of one band
  static constexpr int kXTile = NT * kRowBytes;
  static constexpr int kBox = NT < 128 ? 32 : 64;           // token rows of one TMA copy
  static constexpr int kStage = kWTile + kXTile + kScale * (1 + kSub);
  static constexpr int kStages = NT == 256 ? 4 : (NT == 128 ? 6 : (NT == 64 ? 7 : 8));
  static constexpr int kSmem = 1024 + kStages * kStage + (2 * kStages + 4) * 8 + 16;
  static_assert(kSmem + 4 * (kMxMaxGroups + 1) + 64 <= kSmemLimit, "shared memory");
};

template <int NT, bool SPLIT>
struct Tmem {
  static constexpr int kBufs = SPLIT || NT == 256 ? 1 : 2;  // accumulators
  static constexpr int kScaleX = kBufs * NT;                // columns: scales of X, then of W
  static constexpr int kScaleW = kScaleX + 16 * ((NT + 127) / 128);
  static constexpr int kUsed = kScaleW + 16;
  static constexpr int kCols = kUsed <= 64 ? 64 : (kUsed <= 128 ? 128 : (kUsed <= 256 ? 256 : 512));
};

// Descriptor of one scale tile for tcgen05.cp: no swizzle, 8-row groups of 16
// bytes a row 128 bytes apart (SBO = 8 x 16 B), descriptor version 1.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3fffu) | ((uint64_t)8 << 32) | ((uint64_t)1 << 46);
}
__device__ __forceinline__ void scale_copy(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// Instruction descriptor of the block-scaled kinds: A and B E2M1 (bits 7-9 and
// 10-12 = 1), N >> 3 at bit 17, the scale type at bit 23 (1 = UE8M0, 0 =
// UE4M3), M >> 7 at bit 27; the scale words' byte offsets of B at bit 4 and of
// A at bit 29.
template <int FMT>
__device__ __forceinline__ uint32_t mx_idesc(int N, int sf_id) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((FMT == kMxE8m0 ? 1u : 0u) << 23) | (1u << 27) | ((uint32_t)sf_id << 4) |
         ((uint32_t)sf_id << 29);
}

template <int FMT>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if (FMT == kMxE8m0)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// What a kernel launched to overlap the quantisation before it must not read
// early: the quantised X and its row scales.  Returns at once otherwise.
__device__ __forceinline__ void wait_for_x() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Columns of tensor memory to registers, without waiting.
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

struct TileAt {
  int e;       // group
  int n0;      // first weight row inside the group
  int local;   // first token inside the group
  int row;     // that token's row of X and Y
  int count;   // tokens of the tile
  int first;   // the group's first row
};

// Tile `item`; *e (the search's start) only moves forward.
template <int NT>
__device__ __forceinline__ bool tile_at(const MxGemmArgs& a, const int* s_pre, int item, int* e,
                                        TileAt* t) {
  while (*e < a.rows.groups && item >= s_pre[*e + 1] * a.n_tiles) (*e)++;
  if (*e >= a.rows.groups) return false;
  const int tt = s_pre[*e + 1] - s_pre[*e];
  const int at = item - s_pre[*e] * a.n_tiles;
  int last;
  mx_group(a.rows, *e, &t->first, &last);
  t->e = *e;
  t->n0 = (at / tt) * kWRows;
  t->local = (at % tt) * NT;
  t->row = t->first + t->local;
  t->count = min(NT, last - t->row);
  return true;
}

// One step of the producer's walk over (tile, stage).
template <int NT>
struct Walk {
  const MxGemmArgs& a;
  const int* s_pre;
  int item, step, lo, hi, st, e;
  TileAt t;
  bool valid;
  __device__ Walk(const MxGemmArgs& a_, const int* p, int item_, int step_, int lo_, int hi_)
      : a(a_), s_pre(p), item(item_), step(step_), lo(lo_), hi(hi_), st(lo_), e(0) {
    valid = tile_at<NT>(a, s_pre, item, &e, &t);
  }
  __device__ void next() {
    if (++st < hi) return;
    st = lo;
    item += step;
    valid = step > 0 && tile_at<NT>(a, s_pre, item, &e, &t);
  }
};

template <int FMT, int NT, bool SPLIT>
__global__ void __launch_bounds__(kMxThreads, 1)
mx_gemm_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
               const __grid_constant__ MxGemmArgs a) {
  using S = Shape<FMT, NT>;
  using TM = Tmem<NT, SPLIT>;
  extern __shared__ __align__(1024) unsigned char gsm[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(gsm) + 1023) & ~(uintptr_t)1023);
  unsigned char* sW = base;
  unsigned char* sX = sW + S::kStages * kWTile;
  unsigned char* sSW = sX + S::kStages * S::kXTile;
  unsigned char* sSX = sSW + S::kStages * S::kScale;
  uint64_t* full = reinterpret_cast<uint64_t*>(sSX + S::kStages * S::kScale * S::kSub);
  uint64_t* empty = full + S::kStages;
  uint64_t* acc_full = empty + S::kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;       // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  __shared__ int s_pre[kMxMaxGroups + 1];  // token tiles of the groups before
  __shared__ int s_fail;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < a.rows.groups; e += kMxThreads) {
    int first, last;
    mx_group(a.rows, e, &first, &last);
    s_pre[e + 1] = (last - first + NT - 1) / NT;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; s++) {
      mbar_init(&full[s], 1);   // the producer's expect_tx
      mbar_init(&empty[s], 1);  // MMA commit
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(&acc_full[b], 1);           // MMA commit of a tile
      mbar_init(&acc_empty[b], kEpiWarps);  // one arrive per epilogue warp
    }
    s_fail = 0;
    s_pre[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(TM::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0 && a.rows.groups > 1) {  // running sums of the tile counts
    int sum = 0;
    for (int e0 = 0; e0 < a.rows.groups; e0 += 32) {
      int v = e0 + lane < a.rows.groups ? s_pre[e0 + lane + 1] : 0;
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (e0 + lane < a.rows.groups) s_pre[e0 + lane + 1] = sum + v;
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;

  // this CTA's tiles and its share of K
  uint32_t crank = 0, csize = 1;
  if (SPLIT) {
    crank = cluster_rank();
    csize = cluster_size();
  }
  const int item0 = SPLIT ? blockIdx.y : blockIdx.x;
  const int step = SPLIT ? 0 : gridDim.x;
  const int st_lo = SPLIT ? (int)((int64_t)crank * a.stages / csize) : 0;
  const int st_hi = SPLIT ? (int)((int64_t)(crank + 1) * a.stages / csize) : a.stages;

  if (warp == 0) {
    if (lane == 0) {
      auto atoms = [&](int st) { return min(S::kAtoms, a.tiles_k - st * S::kAtoms); };
      auto bands = [&](const TileAt& t) { return (t.count + 127) / 128; };
      auto boxes = [&](const TileAt& t) { return (t.count + S::kBox - 1) / S::kBox; };
      auto load_w = [&](const Walk<NT>& w, int s) {
        const uint32_t sb = (uint32_t)(atoms(w.st) * kMxTileBytes);
        mbar_arrive_expect_tx(&full[s],
                              kWTile + boxes(w.t) * S::kBox * kRowBytes + sb * (1 + bands(w.t)));
        tma_load_2d(sW + s * kWTile, &wmap, &full[s], w.st * kRowBytes, w.t.e * a.N + w.t.n0);
        const int64_t band = (int64_t)w.t.e * a.N / kMxTileRows + w.t.e + w.t.n0 / kMxTileRows;
        bulk_load(sSW + s * S::kScale,
                  a.sw + (band * a.tiles_k + w.st * S::kAtoms) * kMxTileBytes, sb, &full[s]);
      };
      auto load_x = [&](const Walk<NT>& w, int s) {
        for (int j = 0; j < boxes(w.t); j++)  // only boxes that hold rows of the tile
          tma_load_2d(sX + s * S::kXTile + j * S::kBox * kRowBytes, &xmap, &full[s],
                      w.st * kRowBytes, w.t.row + j * S::kBox);
        const uint32_t sb = (uint32_t)(atoms(w.st) * kMxTileBytes);
        const int64_t band = w.t.first / kMxTileRows + w.t.e + w.t.local / kMxTileRows;
        for (int j = 0; j < bands(w.t); j++)
          bulk_load(sSX + (s * S::kSub + j) * S::kScale,
                    a.sx + ((band + j) * a.tiles_k + w.st * S::kAtoms) * kMxTileBytes, sb,
                    &full[s]);
      };
      // the first stages' weights do not wait for X
      int ahead = 0;
      for (Walk<NT> w(a, s_pre, item0, step, st_lo, st_hi); w.valid && ahead < S::kStages; w.next())
        load_w(w, ahead++);
      wait_for_x();
      int it = 0;
      for (Walk<NT> w(a, s_pre, item0, step, st_lo, st_hi); w.valid && !s_fail; w.next(), it++) {
        const int s = it % S::kStages;
        if (it >= ahead) {
          if (!mbar_wait(&empty[s], ((it / S::kStages) - 1) & 1)) { s_fail = 1; break; }
          load_w(w, s);
        }
        load_x(w, s);
      }
      // the last copies have landed before the CTA can exit (bounded)
      for (int j = it > S::kStages ? it - S::kStages : 0; j < it; j++)
        if (!mbar_wait(&full[j % S::kStages], (j / S::kStages) & 1)) { s_fail = 1; break; }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const int steps_all = (a.K + 63) / 64;
      TileAt t;
      int e = 0, it = 0, i = 0;
      for (int item = item0; tile_at<NT>(a, s_pre, item, &e, &t) && !s_fail; item += step, i++) {
        const int b = i % TM::kBufs;
        // the accumulator's previous tile has been read out
        if (i >= TM::kBufs && !mbar_wait(&acc_empty[b], ((i / TM::kBufs) - 1) & 1)) {
          s_fail = 1;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(b * NT);
        // A 64-token tile may start in the middle of its scale band, two
        // columns on.  A scale address must be even, so 32-token tiles are
        // only used where a group has a single one (mx_plan).
        const uint32_t shift = NT == 64 ? (uint32_t)(t.local % 128) / 32 : 0u;
        const int n_mma = (t.count + 15) & ~15;
        bool ok = true;
        for (int st = st_lo; st < st_hi; st++, it++) {
          const int s = it % S::kStages;
          if (!mbar_wait(&full[s], (it / S::kStages) & 1)) { ok = false; break; }
          tc_fence_after();
          const int na = min(S::kAtoms, a.tiles_k - st * S::kAtoms);
          for (int k = 0; k < na; k++) {
            scale_copy(tmem + TM::kScaleW + 4 * k,
                       scale_desc(smem_u32(sSW + s * S::kScale + k * kMxTileBytes)));
#pragma unroll
            for (int j = 0; j < S::kSub; j++)
              scale_copy(tmem + TM::kScaleX + 4 * (k * S::kSub + j),
                         scale_desc(smem_u32(sSX + (s * S::kSub + j) * S::kScale + k * kMxTileBytes)));
          }
          const uint32_t w0 = smem_u32(sW + s * kWTile), x0 = smem_u32(sX + s * S::kXTile);
          const int steps = min(kSteps, steps_all - st * kSteps);
          for (int k = 0; k < steps; k++) {
            const int atom = FMT == kMxE8m0 ? k / 2 : k;
            const int id = FMT == kMxE8m0 ? (k & 1) * 2 : 0;
            mma_mx<FMT>(d, sw128_desc(w0 + 32 * k), sw128_desc(x0 + 32 * k),
                        mx_idesc<FMT>(n_mma, id), tmem + TM::kScaleW + 4 * atom,
                        tmem + TM::kScaleX + 4 * S::kSub * atom + shift,
                        (st > st_lo || k > 0) ? 1u : 0u);
          }
          mma_commit(&empty[s]);
        }
        if (!ok) { s_fail = 1; break; }
        mma_commit(&acc_full[b]);
        if (SPLIT) break;
      }
    }
  } else {
    wait_for_x();  // the row scales
    const int q = warp & 3;             // the TMEM lane quadrant this warp may read
    const int half = (warp - 2) >> 2;   // which half of the token columns
    constexpr int NC = NT / 2;
    TileAt t;
    int e = 0, i = 0;
    for (int item = item0; tile_at<NT>(a, s_pre, item, &e, &t); item += step, i++) {
      const int b = i % TM::kBufs;
      const bool got = __all_sync(0xffffffffu, mbar_wait(&acc_full[b], (i / TM::kBufs) & 1));
      tc_fence_after();
      const bool fail = !got || s_fail;
      uint32_t r[NC];
      if (!fail) {
#pragma unroll
        for (int c = 0; c < NC; c += 16)
          if (half * NC + c < t.count)  // warp-uniform
            tmem_ld16_nowait(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * NT + half * NC + c),
                             r + c);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (!SPLIT && lane == 0) mbar_arrive(&acc_empty[b]);
      }
      if (SPLIT) {
        // every MMA of this CTA is complete, so the stages are free
        float* P = reinterpret_cast<float*>(base);
#pragma unroll
        for (int c = 0; c < NC; c++)
          if (half * NC + c < t.count)
            P[(half * NC + c) * kWRows + q * 32 + lane] =
                fail ? __int_as_float(0x7fc00000) : __uint_as_float(r[c]);
        break;
      }
      const int n = t.n0 + q * 32 + lane;
      const bool nok = n < a.N;
      const float gw = FMT == kMxE4m3 && nok ? __ldg(a.gw + (int64_t)t.e * a.N + n) : 1.0f;
      const int r0 = t.row + half * NC;
      const int64_t y0 = (int64_t)r0 * a.ldy + n;
#pragma unroll
      for (int c = 0; c < NC; c++) {
        if (half * NC + c >= t.count) continue;  // warp-uniform
        float v = fail ? __int_as_float(0x7fc00000) : __uint_as_float(r[c]);
        if (FMT == kMxE4m3) v = __fmul_rn(__fmul_rn(v, __ldg(a.gx + r0 + c)), gw);
        if (nok) {
          if (a.bf16_out) static_cast<__nv_bfloat16*>(a.Y)[y0 + c * a.ldy] = __float2bfloat16_rn(v);
          else static_cast<float*>(a.Y)[y0 + c * a.ldy] = v;
        }
      }
      if (fail) break;  // the MMA warp stopped; nothing more to read
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(TM::kCols));
  }
  if (SPLIT) {
    TileAt t;
    int e = 0;
    const bool have = tile_at<NT>(a, s_pre, item0, &e, &t);  // the same for the whole cluster
    cluster_sync_all();  // every CTA's partial is in its shared memory
    if (have) {
      const float* P = reinterpret_cast<const float*>(base);
      const int E = t.count * kWRows;
      const int e0 = (int)((int64_t)crank * E / csize), e1 = (int)((int64_t)(crank + 1) * E / csize);
      for (int i = e0 + threadIdx.x; i < e1; i += kMxThreads) {
        const int c = i / kWRows, n = t.n0 + i % kWRows;
        if (n < a.N) {
          float v = 0.0f;
          for (uint32_t k = 0; k < csize; k++) v = __fadd_rn(v, ld_cluster_f32(P + i, k));
          if (FMT == kMxE4m3)
            v = __fmul_rn(__fmul_rn(v, __ldg(a.gx + t.row + c)), __ldg(a.gw + (int64_t)t.e * a.N + n));
          const int64_t y = (int64_t)(t.row + c) * a.ldy + n;
          if (a.bf16_out) static_cast<__nv_bfloat16*>(a.Y)[y] = __float2bfloat16_rn(v);
          else static_cast<float*>(a.Y)[y] = v;
        }
      }
    }
    cluster_sync_all();  // no CTA leaves while another may still read its partial
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
cudaError_t code_map(EncodeTiledFn enc, CUtensorMap* map, const uint8_t* codes, int64_t rows,
                     int64_t K, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
  const cuuint32_t box[2] = {(cuuint32_t)kRowBytes, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int FMT, int NT, bool SPLIT>
cudaError_t launch_t(const CUtensorMap& xmap, const CUtensorMap& wmap, const MxGemmArgs& a,
                     const MxPlan& p, bool overlap, cudaStream_t st) {
  constexpr int smem = Shape<FMT, NT>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(mx_gemm_kernel<FMT, NT, SPLIT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = SPLIT ? dim3((unsigned)p.split, (unsigned)p.tiles, 1) : dim3((unsigned)p.ctas, 1, 1);
  cfg.blockDim = dim3(kMxThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (SPLIT) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)p.split;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    n++;
  }
  if (overlap) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    n++;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<FMT, NT, SPLIT>, xmap, wmap, a);
}

template <int FMT>
cudaError_t launch_f(const CUtensorMap& xmap, const CUtensorMap& wmap, const MxGemmArgs& a,
                     const MxPlan& p, bool overlap, cudaStream_t st) {
  if (p.split > 1) {
    switch (p.nt) {
      case 32: return launch_t<FMT, 32, true>(xmap, wmap, a, p, overlap, st);
      case 64: return launch_t<FMT, 64, true>(xmap, wmap, a, p, overlap, st);
      case 128: return launch_t<FMT, 128, true>(xmap, wmap, a, p, overlap, st);
      default: return launch_t<FMT, 256, true>(xmap, wmap, a, p, overlap, st);
    }
  }
  switch (p.nt) {
    case 32: return launch_t<FMT, 32, false>(xmap, wmap, a, p, overlap, st);
    case 64: return launch_t<FMT, 64, false>(xmap, wmap, a, p, overlap, st);
    case 128: return launch_t<FMT, 128, false>(xmap, wmap, a, p, overlap, st);
    default: return launch_t<FMT, 256, false>(xmap, wmap, a, p, overlap, st);
  }
}

}  // namespace

MxPlan mx_plan(int groups, int64_t rows, int64_t N, int64_t K) {
  MxPlan p;
  const int64_t busy = groups < rows ? groups : rows;  // groups that can hold rows
  const int64_t each = (rows + busy - 1) / busy;
  p.nt = groups == 1 && rows <= 32 ? 32 : (each <= 64 ? 64 : (each <= 128 ? 128 : 256));
  const int64_t n_tiles = (N + kWRows - 1) / kWRows;
  const int64_t stages = (K + kStageK - 1) / kStageK;
  // an upper bound of the tiles: sum ceil(c / NT) <= rows / NT + one per busy group
  p.tiles = groups == 1 ? (rows + p.nt - 1) / p.nt * n_tiles : (rows / p.nt + busy) * n_tiles;
  int64_t c = kSms / p.tiles;
  if (c > 8) c = 8;
  if (c > stages) c = stages;
  p.split = c < 1 ? 1 : (int)c;
  p.ctas = (int)(p.split > 1 ? p.tiles * p.split : (p.tiles < kSms ? p.tiles : kSms));
  p.stages = (int)stages;
  return p;
}

cudaError_t launch_mx_gemm(const MxTensor& x, const MxTensor& w, void* Y, bool f32, int64_t ldy,
                           bool overlap, cudaStream_t st) {
  EncodeTiledFn enc;
  cudaError_t e = encode_fn(&enc);
  if (e != cudaSuccess) return e;
  const int64_t N = w.rows / w.groups;
  const MxPlan p = mx_plan(x.groups, x.rows, N, x.K);
  CUtensorMap xmap, wmap;
  e = code_map(enc, &xmap, x.codes, x.rows, x.K, p.nt < 128 ? 32 : 64);
  if (e == cudaSuccess) e = code_map(enc, &wmap, w.codes, w.rows, w.K, kWRows);
  if (e != cudaSuccess) return e;
  const MxGemmArgs a{x.scales, w.scales, x.row_scale, w.row_scale, Y, ldy,
                     MxRows{x.offsets, x.groups, (int)x.rows}, (int)N, (int)x.K,
                     (int)((N + kWRows - 1) / kWRows), p.stages, (int)mx_tiles_k(x.fmt, x.K),
                     f32 ? 0 : 1};
  return x.fmt == kMxE8m0 ? launch_f<kMxE8m0>(xmap, wmap, a, p, overlap, st)
                          : launch_f<kMxE4m3>(xmap, wmap, a, p, overlap, st);
}

cudaError_t mx_timeout_flag(unsigned int* out) {
  return cudaMemcpyFromSymbol(out, g_wait_timeout, sizeof(unsigned int));
}

}  // namespace aaac
