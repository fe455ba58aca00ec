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
//   warp 0      one lane issues four TMA copies: both code tiles
//               (SWIZZLE_128B) and both operands' scale tiles;
//   warps 2..5  bring the scale tiles from shared to tensor memory, one lane
//               quadrant each (the tensor core wants a copy in all four);
//   warp 1      one lane issues four MMAs of K = 64;
//   the others  epilogue: tensor memory -> registers, the accumulator handed
//               back, row scales, stores.
// The tensor core's N is the tile's own row count rounded up to 16, so a
// ragged tile costs what its rows cost.
//
// kWalk: persistent CTAs walk the tiles (weight-tile major inside a group, so
// that CTAs in flight share weight rows in L2).  kPair: two CTAs walk tiles of
// 256 weight rows together (cta_group::2); each holds its own weight rows and
// half of the token rows, and the first issues the MMAs.  kSplit: few tiles;
// the CTAs of a cluster take a share of K each, and add their partial tiles in
// rank order through distributed shared memory: the sum's order is fixed,
// whatever the timing.
//
// What bounds it (measured; times of a launch among others):
//   14336 x 4096 at 8192 tokens, E4M3, bf16 out: 200 us, 4.8 PFLOP/s, 0.72 of
//     four times the measured bf16 rate.  MMAs alone take 145 us, copies alone
//     158: together they share shared memory (38 KB written and 32 KB read a
//     CTA and stage of 512 MMA cycles, of 128 bytes a cycle) and the power
//     limit (up to 237 us in a long run, and 252 with its quantisation).
//   5120 x 27648 at 333 tokens: 41 us, 0.31 us a stage of 37 KB, the way from
//     L2 (copies alone 35).
//   4096 x 4096 at one token: 6.8 us, of which 4.9 are a launch that loads and
//     multiplies nothing.  64 experts of 2048 x 2048, two rows each: 30 us for
//     151 MB, 0.77 of the measured HBM rate; 128 rows over 45 of them 24.5 us for
//     106 MB, 0.66: the start is the same.
// What was measured on the way: scale tiles by tcgen05.cp cost 41 ns each, in
// line with the MMAs (12 a stage: 0.49 us of 0.88); as bulk copies of 2 KB they
// cost 90 ns each to fetch, as tensor copies 18; a lane on its own in place of
// a whole warp with one lane elected pays for every descriptor and coordinate
// on its way to a uniform register (821 against 743 us at 2048 x 14336 x
// 65536).  A ring of their own for the scale tiles, with a warp to fetch them,
// was 5% slower; two sets of scale warps, or asking for the next stage before
// its turn, changed nothing.
//
// A few rows that are not quantised yet (SRC: their kind; the single tokens of
// decoding): eight more warps quantise each stage's columns straight into its
// shared memory, as mx_quant.cu would, while the weights stream in: one
// launch, and no workspace.
// Waits are bounded (tcgen05.cuh); a CTA that gives up writes NaN to the rest of
// its tiles.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "mx_run.cuh"
#include "tcgen05.cuh"

namespace aaac {

namespace {

constexpr int kWRows = 128;        // weight rows of a tile (MMA M)
constexpr int kEpiWarp = 6;        // the first epilogue warp
constexpr int kStageK = 256;       // columns of a stage
constexpr int kRowBytes = 128;     // of packed codes per stage and row
constexpr int kSteps = 4;          // MMAs of K = 64 per stage
constexpr int kWTile = kWRows * kRowBytes;  // 16 KB
constexpr int kSmemLimit = 227 * 1024;
constexpr int kSms = 148;
constexpr int kMaxSplit = 8;       // CTAs that share a tile's K

struct MxGemmArgs {
  const float* gx;
  const float* gw;
  void* Y;
  int64_t ldy;
  MxRows rows;        // of X and Y
  int N, K;
  int n_tiles;        // weight tiles per group
  int stages;         // ceil(K / 256)
  int width;          // tokens of a tile: NT, or fewer
  int box;            // token rows of one TMA copy
  int bf16_out;
  int ahead;          // all but X was ready before the kernel before this one
  int most;           // token tiles of all groups, at most
};

// Rows to quantise on the way (SRC >= 0).
struct RowsArgs {
  const void* X;
  const int32_t* index;
  int64_t ldx;
  int src_rows;
  int warps;          // warps of a stage: two rows each, a power of two
};
constexpr int kSrcNone = -1, kSrcBf16 = 0, kSrcF32 = 1, kSrcBf16Glu = 2, kSrcF32Glu = 3;
constexpr int kMaxOwnRows = 8;
constexpr int kOwnWarps = 8;

// How the CTAs of a launch share the work.
constexpr int kWalk = 0;   // each walks tiles of 128 weight rows on its own
constexpr int kSplit = 1;  // a cluster's CTAs each take a part of one tile's K
constexpr int kPair = 2;   // two CTAs walk tiles of 256 weight rows (cta_group::2)

template <int FMT, int NT, int MODE, int SRC>
struct Shape {
  static constexpr bool kOwn = SRC != kSrcNone;  // quantises its rows itself
  static constexpr bool kTwo = MODE == kPair;
  static constexpr int kTileRows = kTwo ? 2 * kWRows : kWRows;  // weight rows of a tile
  static constexpr int kSub = (NT + 127) / 128;             // 128-row scale bands a token tile meets
  static constexpr int kAtoms = FMT == kMxE8m0 ? 2 : 4;     // scale tiles of a stage along K
  static constexpr int kScale = kAtoms * kMxTileBytes;      // of one band
  static constexpr int kXTile = (kTwo ? NT / 2 : NT) * kRowBytes;  // a pair's CTAs hold half each
  static constexpr int kStage = kWTile + kXTile + kScale * (1 + kSub);
  // 64 columns an epilogue thread at most: all of them leave tensor memory in
  // one go, so that the next tile's MMAs wait for no store
  static constexpr int kEpiWarps = NT == 256 ? 16 : 8;
  static constexpr int kOwnWarp = kEpiWarp + kEpiWarps;
  static constexpr int kThreads = (kOwnWarp + (kOwn ? kOwnWarps : 0)) * 32;
  static constexpr int kStages = kTwo ? 5 : (NT == 256 ? 4 : (NT == 128 ? 6 : (NT == 64 ? 7 : 8)));
  static constexpr int kSmem = 1024 + kStages * kStage + (3 * kStages + 4) * 8 + 16;
  static_assert(kSmem + 4 * (kMxMaxGroups + 1) + 16 * NT + 64 <= kSmemLimit, "shared memory");
};

template <int NT, int MODE, int STAGES>
struct Tmem {
  static constexpr int kBufs = MODE == kSplit || NT == 256 ? 1 : 2;  // accumulators
  static constexpr int kScale = kBufs * NT;                 // first scale column
  static constexpr int kScaleX = 16 * ((NT + 127) / 128);   // of a stage: X's columns, then 16 of W
  // as many sets as stages: a set is free when its stage is, with no wait of its own
  static constexpr int kUsed = kScale + STAGES * (kScaleX + 16);
  static_assert(kUsed <= 512, "tensor memory");
  static constexpr int kCols = kUsed <= 64 ? 64 : (kUsed <= 128 ? 128 : (kUsed <= 256 ? 256 : 512));
};

// sw128_desc of a code tile whose address is given in 16-byte units.
__device__ __forceinline__ uint64_t code_desc(uint32_t at) {
  return (uint64_t)(at | 1u << 16) | ((uint64_t)(64u | 1u << 14 | 2u << 29) << 32);
}

// Instruction descriptor of the block-scaled kinds: A and B E2M1 (bits 7-9 and
// 10-12 = 1), N >> 3 at bit 17, the scale type at bit 23 (1 = UE8M0, 0 =
// UE4M3), M >> 7 at bit 27; the scale words' byte offsets of B at bit 4 and of
// A at bit 29.
template <int FMT>
__device__ __forceinline__ uint32_t mx_idesc(int M, int N) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((FMT == kMxE8m0 ? 1u : 0u) << 23) | ((uint32_t)(M >> 7) << 27);
}

#define AAAC_MX_MMA(GROUP, VEC)                                                          \
  asm volatile(                                                                          \
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"                                      \
      " tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC     \
      " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),                                 \
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)              \
      : "memory")
template <int FMT, bool TWO>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if (FMT == kMxE8m0) {
    if (TWO) AAAC_MX_MMA("2", "2X");
    else AAAC_MX_MMA("1", "2X");
  } else {
    if (TWO) AAAC_MX_MMA("2", "4X");
    else AAAC_MX_MMA("1", "4X");
  }
}
#undef AAAC_MX_MMA

// The barrier (of both CTAs of a pair) completes with the MMAs issued so far.
template <bool TWO>
__device__ __forceinline__ void commit_mx(uint64_t* bar) {
  if (TWO)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    mma_commit(bar);
}

// An arrival at the first CTA's barrier, from either CTA of a pair.  Its default
// scope is the CTA, and it need not be more, for what it orders is no plain data:
// tensor memory, by the tcgen05 fences before the arrival and after the wait, with
// the stores and loads before it complete (tcgen05.wait); and code tiles in shared
// memory, whose copies were complete (their barrier's wait) before the arrival and
// which only the tensor core reads.  Nothing that threads write may be passed to
// the other CTA under these barriers: that would take .release.cluster here and
// .acquire.cluster at the wait, measured at twice the kernel's time (1800 against
// 858 us at 2048 x 14336 x 65536).
template <bool TWO>
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  if (TWO) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(bar)));
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(at)
                 : "memory");
  } else {
    mbar_arrive(bar);
  }
}

// N consecutive columns of this warp's lane quadrant, from registers.
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t* r) {
  static_assert(N == 8 || N == 16 || N == 32, "columns");
  if (N == 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::
                     "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                 "r"(r[6]), "r"(r[7])
                 : "memory");
  else
#pragma unroll
    for (int i = 0; i < N; i += 16)
      asm volatile(
          "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
          "%11, %12, %13, %14, %15, %16};" ::"r"(taddr + i),
          "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]),
          "r"(r[i + 6]), "r"(r[i + 7]), "r"(r[i + 8]), "r"(r[i + 9]), "r"(r[i + 10]),
          "r"(r[i + 11]), "r"(r[i + 12]), "r"(r[i + 13]), "r"(r[i + 14]), "r"(r[i + 15])
          : "memory");
}


__device__ __forceinline__ float4 ld_cluster_f4(const float* local, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(rank));
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
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

// A sum times both row scales.  (sum gx) gw leaves fp32's range at gx = 2^117
// and gw = 2^-120 although Y does not; but not with 2^-100 <= gx <= 2^80, since a
// sum is 0 or between 2^-20 (the smallest product of two values under their
// block scales) and 2^24 * 2688^2 < 2^47.
__device__ __forceinline__ bool plain_scale(float gx) { return gx >= 0x1p-100f && gx <= 0x1p80f; }
// For any other gx: a factor below 1 and one above 1 are multiplied with each
// other first, others one after the other.  Row scales that the library makes
// are powers of two, so every step is exact either way.  NaN stays.
__device__ __forceinline__ float scale_sum(float sum, float gx, float gw) {
  float xl, xh, wl, wh;
  asm("min.NaN.f32 %0, %1, 0f3F800000;" : "=f"(xl) : "f"(gx));
  asm("max.NaN.f32 %0, %1, 0f3F800000;" : "=f"(xh) : "f"(gx));
  asm("min.NaN.f32 %0, %1, 0f3F800000;" : "=f"(wl) : "f"(gw));
  asm("max.NaN.f32 %0, %1, 0f3F800000;" : "=f"(wh) : "f"(gw));
  return __fmul_rn(__fmul_rn(sum, __fmul_rn(xl, wh)), __fmul_rn(xh, wl));
}

struct TileAt {
  int e;       // group
  int n0;      // first weight row inside the group
  int local;   // first token inside the group
  int row;     // that token's row of X and Y
  int count;   // tokens of the tile
  int first;   // the group's first row
};

// True in one lane of the warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(p));
  return p != 0;
}
// A wait of the whole warp, with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// A walk around the stages: the stage and the parity of its use.
template <int STAGES>
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++s == STAGES) {
      s = 0;
      phase ^= 1;
    }
  }
};

// The use before the ring's own, of the stage before, is over; at once where
// there was none (a new barrier's phase before its first is complete).
template <int STAGES>
__device__ __forceinline__ void wait_last(uint64_t* bars, const Ring<STAGES>& ring) {
  const bool back = ring.s == 0;
  warp_wait(&bars[back ? STAGES - 1 : ring.s - 1], ring.phase ^ (back ? 1u : 0u));
}

// The tensor core's N for `count` tokens; a pair's CTAs hold half of it each.
template <bool TWO>
__device__ __forceinline__ int mma_n(int count) {
  return TWO ? (count + 31) & ~31 : (count + 15) & ~15;
}

// Tile `item`, one of the s_pre[groups] * n_tiles; *e (the search's start) only
// moves forward.
template <int ROWS>
__device__ __forceinline__ void tile_at(const MxGemmArgs& a, const int* s_pre, int item, int* e,
                                        TileAt* t) {
  while (item >= s_pre[*e + 1] * a.n_tiles) (*e)++;
  const int tt = s_pre[*e + 1] - s_pre[*e];
  const int at = item - s_pre[*e] * a.n_tiles;
  int last;
  mx_group(a.rows, *e, &t->first, &last);
  t->e = *e;
  t->n0 = (at / tt) * ROWS;
  t->local = (at % tt) * a.width;
  t->row = t->first + t->local;
  t->count = min(a.width, last - t->row);
}

template <int FMT, int NT, int MODE, int SRC>
__global__ void __launch_bounds__((Shape<FMT, NT, MODE, SRC>::kThreads), 1)
mx_gemm_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
               const __grid_constant__ CUtensorMap sxmap, const __grid_constant__ CUtensorMap swmap,
               const __grid_constant__ MxGemmArgs a, const __grid_constant__ RowsArgs own) {
  using S = Shape<FMT, NT, MODE, SRC>;
  using TM = Tmem<NT, MODE, S::kStages>;
  constexpr bool SPLIT = MODE == kSplit, TWO = S::kTwo;
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
  uint64_t* scale_full = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scale_full + S::kStages);
  __shared__ int s_pre[kMxMaxGroups + 1];  // token tiles of the groups before
  __shared__ __align__(16) float s_gx[S::kEpiWarps][FMT == kMxE4m3 && !SPLIT ? NT / (S::kEpiWarps / 4) : 4];
  __shared__ uint32_t s_top[kMaxOwnRows];   // kOwn, E4M3: the rows' largest magnitudes,
  __shared__ float s_scale[kMaxOwnRows];    // and their scales
  __shared__ int s_fail;

  // The same in every lane, and known to be: the roles of warps 0 and 1 run as
  // whole warps, of which one lane issues, so that addresses and descriptors
  // are worked out in uniform registers, where TMA and MMA want them.
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  let_next_start();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; s++) {
      // the producer's expect_tx, and the warps that quantise
      mbar_init(&full[s], 1 + (S::kOwn ? own.warps : 0));
      mbar_init(&empty[s], 1);  // MMA commit
      mbar_init(&scale_full[s], TWO ? 8 : 4);  // one arrive per scale warp
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(&acc_full[b], 1);                              // MMA commit of a tile
      mbar_init(&acc_empty[b], S::kEpiWarps * (TWO ? 2 : 1));  // one arrive per epilogue warp
    }
    s_fail = 0;
    s_pre[0] = 0;
    for (int r = 0; r < kMaxOwnRows; r++) s_top[r] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if (TWO) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(TM::kCols));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(TM::kCols));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  if (!a.ahead) after_previous();
  for (int e = threadIdx.x; e < a.rows.groups; e += S::kThreads) {
    int first, last;
    mx_group(a.rows, e, &first, &last);
    s_pre[e + 1] = mx_group_tiles(last - first, a.width, a.most);
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
        if (lane >= o) v = mx_add_tiles(u, v, a.most);
      }
      v = mx_add_tiles(sum, v, a.most);
      if (e0 + lane < a.rows.groups) s_pre[e0 + lane + 1] = v;
      sum = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  if (a.rows.groups > 1) __syncthreads();
  const uint32_t tmem = *tmem_slot;

  // this CTA's tiles and its share of K
  uint32_t crank = 0, csize = 1;
  if (MODE != kWalk) {
    crank = cluster_rank();
    csize = cluster_size();
  }
  if (TWO) cluster_sync_all();  // both CTAs' barriers are set up
  const int item0 = SPLIT ? blockIdx.y : (TWO ? blockIdx.x / 2 : blockIdx.x);
  const int step = SPLIT ? 0 : (TWO ? gridDim.x / 2 : gridDim.x);
  const int wrow = TWO ? (int)crank * kWRows : 0;  // this CTA's first row of a tile
  const int st_lo = SPLIT ? (int)((int64_t)crank * a.stages / csize) : 0;
  const int st_hi = SPLIT ? (int)((int64_t)(crank + 1) * a.stages / csize) : a.stages;

  const int nst = st_hi - st_lo;
  const int items = s_pre[a.rows.groups] * a.n_tiles;

  Ring<S::kStages> mma_ring;  // warp 1's walk
  if (warp == 0) {
    const bool one = elect_one();
    // coordinates of a tile's copies: the rows of the codes and the bands of
    // the scales, of both operands
    struct At {
      int w, sw, x, sx, boxes;
    };
    auto at_of = [&](const TileAt& t) {
      At c;
      c.w = t.e * a.N + t.n0 + wrow;
      c.sw = (int)((int64_t)t.e * a.N / kMxTileRows) + t.e + (t.n0 + wrow) / kMxTileRows;
      const int half = mma_n<TWO>(t.count) / 2;
      c.x = t.row + (TWO ? (int)crank * half : 0);
      c.sx = t.first / kMxTileRows + t.e + t.local / kMxTileRows;
      // only boxes that hold rows of the tile
      c.boxes = ((TWO ? half : t.count) + a.box - 1) / a.box;
      return c;
    };
    const uint32_t box_bytes = (uint32_t)(a.box * kRowBytes);
    auto load_w = [&](const At& c, int st, int s) {
      if (one) {
        mbar_arrive_expect_tx(&full[s], S::kOwn ? kWTile + S::kScale
                                                : kWTile + c.boxes * box_bytes +
                                                      S::kScale * (1 + S::kSub));
        tma_load_2d(sW + s * kWTile, &wmap, &full[s], st * kRowBytes, c.w);
        tma_load_2d(sSW + s * S::kScale, &swmap, &full[s], st * (S::kScale / 8), c.sw);
      }
    };
    auto load_x = [&](const At& c, int st, int s) {
      if (one && !S::kOwn) {
        for (int j = 0; j < c.boxes; j++)
          tma_load_2d(sX + s * S::kXTile + j * box_bytes, &xmap, &full[s], st * kRowBytes,
                      c.x + j * a.box);
        tma_load_2d(sSX + s * S::kSub * S::kScale, &sxmap, &full[s], st * (S::kScale / 8), c.sx);
      }
    };
    TileAt t;
    int e = 0;
    // the first tile's first stages: their weights do not wait for X
    int ahead = 0;
    if (item0 < items) {
      tile_at<S::kTileRows>(a, s_pre, item0, &e, &t);
      const At c = at_of(t);
      for (; ahead < min(nst, S::kStages); ahead++) load_w(c, st_lo + ahead, ahead);
    }
    after_previous();  // X's codes and scales
    int it = 0;
    bool ok = true;
    Ring<S::kStages> ring;
    for (int item = item0; item < items && ok; item += step) {
      tile_at<S::kTileRows>(a, s_pre, item, &e, &t);
      const At c = at_of(t);
      for (int st = st_lo; st < st_hi; st++, it++, ring.next()) {
        if (it >= ahead) {
          if (it >= S::kStages) ok = warp_wait(&empty[ring.s], ring.phase ^ 1);
          if (!ok) break;
          load_w(c, st, ring.s);
        }
        load_x(c, st, ring.s);
      }
      if (SPLIT) break;
    }
    // the last copies have landed before the CTA can exit (bounded), also where
    // it gives up
    bool landed = true;
    for (int j = it > S::kStages ? it - S::kStages : 0; j < it && landed; j++)
      landed = warp_wait(&full[j % S::kStages], (j / S::kStages) & 1);
    if (!ok || !landed) s_fail = 1;
  } else if (warp == 1) {
    if (!TWO || crank == 0) {
      const bool one = elect_one();
      const int steps_all = (a.K + 63) / 64;
      // addresses in 16-byte units, as descriptors hold them
      const uint32_t w_lo = smem_u32(sW) >> 4, x_lo = smem_u32(sX) >> 4;
      TileAt t;
      int e = 0, i = 0;
      bool ok = true;
      for (int item = item0; item < items && ok; item += step, i++) {
        tile_at<S::kTileRows>(a, s_pre, item, &e, &t);
        const int b = i % TM::kBufs;
        // the accumulator's previous tile has been read out
        if (i >= TM::kBufs) ok = warp_wait(&acc_empty[b], ((i / TM::kBufs) - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(b * NT);
        // Tiles of 64 or 192 tokens may start in the middle of a scale band,
        // two columns on.  A scale address must be even, so 32-token tiles
        // are only used where there is a single one (mx_plan).
        const uint32_t shift = (uint32_t)(t.local % 128) / 32;
        const uint32_t idesc = mx_idesc<FMT>(S::kTileRows, mma_n<TWO>(t.count));
        for (int st = st_lo; st < st_hi; st++, mma_ring.next()) {
          // the scale warps arrive after the whole stage has landed
          ok = warp_wait(&scale_full[mma_ring.s], mma_ring.phase);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sc = tmem + TM::kScale + mma_ring.s * (TM::kScaleX + 16);
          const uint32_t w0 = w_lo + mma_ring.s * (kWTile >> 4);
          const uint32_t x0 = x_lo + mma_ring.s * (S::kXTile >> 4);
          const int steps = min(kSteps, steps_all - st * kSteps);
          if (one) {
#pragma unroll
            for (int k = 0; k < kSteps; k++)
              if (k < steps) {
                const int atom = FMT == kMxE8m0 ? k / 2 : k;
                const int id = FMT == kMxE8m0 ? (k & 1) * 2 : 0;
                mma_mx<FMT, TWO>(d, code_desc(w0 + 2 * k), code_desc(x0 + 2 * k),
                                 idesc | ((uint32_t)id << 4) | ((uint32_t)id << 29),
                                 sc + TM::kScaleX + 4 * atom, sc + 4 * S::kSub * atom + shift,
                                 (st > st_lo || k > 0) ? 1u : 0u);
              }
            commit_mx<TWO>(&empty[mma_ring.s]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (one) commit_mx<TWO>(&acc_full[b]);
        __syncwarp();
        if (SPLIT) break;
      }
      if (!ok) s_fail = 1;
    }
  } else if (warp < kEpiWarp) {
    // scale tiles -> tensor memory: lane l's 16 bytes of a tile are the words
    // of its rows l, l + 32, l + 64, l + 96, four consecutive columns
    const uint32_t quadrant = (uint32_t)((warp & 3) * 32) << 16;
    Ring<S::kStages> ring;
    bool ok = true;
    for (int item = item0; item < items && ok; item += step) {
      for (int st = st_lo; st < st_hi; st++, ring.next()) {
        const int s = ring.s;
        // the stage's tiles have landed, so the MMAs that read its columns the
        // last time are complete
        ok = __all_sync(0xffffffffu, mbar_wait(&full[s], ring.phase));
        if (!ok) {
          s_fail = 1;
          break;
        }
        tc_fence_after();
        uint32_t rw[4 * S::kAtoms], rx[4 * S::kAtoms * S::kSub];
        const uint4* w = reinterpret_cast<const uint4*>(sSW + s * S::kScale) + lane;
        const uint4* x = reinterpret_cast<const uint4*>(sSX + s * S::kSub * S::kScale) + lane;
#pragma unroll
        for (int k = 0; k < S::kAtoms; k++) {
          const uint4 v = w[32 * k];
          rw[4 * k] = v.x; rw[4 * k + 1] = v.y; rw[4 * k + 2] = v.z; rw[4 * k + 3] = v.w;
#pragma unroll
          for (int j = 0; j < S::kSub; j++) {
            const uint4 u = x[32 * (j * S::kAtoms + k)];
            uint32_t* o = rx + 4 * (k * S::kSub + j);
            o[0] = u.x; o[1] = u.y; o[2] = u.z; o[3] = u.w;
          }
        }
        const uint32_t sc = tmem + TM::kScale + s * (TM::kScaleX + 16) + quadrant;
        tmem_st<4 * S::kAtoms * S::kSub>(sc, rx);
        tmem_st<4 * S::kAtoms>(sc + TM::kScaleX, rw);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first<TWO>(&scale_full[s]);
      }
      if (SPLIT) break;
    }
  } else if (S::kOwn && warp >= S::kOwnWarp) {
    constexpr bool kF32 = SRC == kSrcF32 || SRC == kSrcF32Glu;
    constexpr bool kGlu = SRC == kSrcBf16Glu || SRC == kSrcF32Glu;
    const int ow = warp - S::kOwnWarp;
    int first, last;
    mx_group(a.rows, 0, &first, &last);
    const int count = min(last - first, kMaxOwnRows);
    // where the group's row r starts in X; -1: a row of zeros
    auto row_start = [&](int r) -> int64_t {
      if (r >= count) return -1;
      const int src = own.index ? load_i32(own.index + first + r) : first + r;
      return src >= 0 && src < own.src_rows ? (int64_t)src * own.ldx : -1;
    };
    if (FMT == kMxE4m3) {
      // the rows' largest magnitudes: kBatch runs a lane, their loads together
      constexpr int kBatch = kF32 || kGlu ? 2 : 4;
      const int runs = a.K >> 4, all = count * runs;
      for (int i0 = ow * 32; i0 < all; i0 += kBatch * kOwnWarps * 32) {
        Run<kF32, kGlu> run[kBatch];
        int row[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; u++) {
          const int i = i0 + u * kOwnWarps * 32 + lane;
          row[u] = min(i, all - 1) / runs;
          const int64_t at = row_start(row[u]);
          if (i < all && at >= 0) run[u].load(own.X, at, (i - row[u] * runs) * 16, a.K);
          else run[u].zero();
        }
#pragma unroll
        for (int u = 0; u < kBatch; u++) {
          if (i0 + u * kOwnWarps * 32 >= all) continue;  // warp-uniform
          uint32_t m = run[u].amax();
          const int r0 = __shfl_sync(0xffffffffu, row[u], 0);
          const int r1 = __shfl_sync(0xffffffffu, row[u], 31);
          if (r0 == r1) {
            m = __reduce_max_sync(0xffffffffu, m);
            if (lane == 0) atomicMax(&s_top[r0], m);
          } else {
            atomicMax(&s_top[row[u]], m);
          }
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kOwnWarps * 32) : "memory");
    }
    // this thread: one run of each of its set's stages
    const int set = ow / own.warps, sets = kOwnWarps / own.warps;
    const int r = (ow % own.warps) * 2 + (lane >> 4), j = lane & 15;
    const int64_t at = row_start(r);
    bool bad_row = false;
    float down = 1.0f;
    if (FMT == kMxE4m3) {
      float g;
      const int p = row_exponent(s_top[r], &bad_row, &g);
      down = __uint_as_float((uint32_t)(127 - p) << 23);
      if (j == 0) s_scale[r] = g;  // the sets write the same
    }
    // its place in a stage: the codes' 16-byte pieces in swizzled order, the
    // scale byte in the tile
    const uint32_t to = (uint32_t)(r >> 3) * 1024u + (uint32_t)(r & 7) * 128u +
                        (uint32_t)((((j >> 1) ^ (r & 7)) << 4) + (j & 1) * 8);
    const int block = FMT == kMxE8m0 ? j >> 1 : j;
    const uint32_t scale_to = (uint32_t)((block >> 2) * kMxTileBytes + r * 16 + (block & 3));
    // all its stages, over the tiles; the next one's run is fetched before this
    // one waits for its stage
    const int tiles = item0 >= items ? 0 : (SPLIT ? 1 : (items - item0 + step - 1) / step);
    const int total = tiles * nst;
    int st = st_lo + set % max(nst, 1);
    auto fetch = [&](Run<kF32, kGlu>& run) {
      const int col = st * kStageK + j * 16;
      if (at >= 0 && col < a.K) run.load(own.X, at, col, a.K);
      else run.zero();
    };
    Run<kF32, kGlu> run, next;
    if (set < total) fetch(next);
    for (int it = set; it < total; it += sets) {
      run = next;
      for (st += sets; st >= st_hi;) st -= nst;
      if (it + sets < total) fetch(next);
      const int s = it % S::kStages;
      if (it >= S::kStages && !warp_wait(&empty[s], ((it / S::kStages) - 1) & 1)) {
        s_fail = 1;
        break;
      }
      uint32_t c[2];
      const uint32_t byte = encode<FMT>(run, down, bad_row, c);
      *reinterpret_cast<uint2*>(sX + s * S::kXTile + to) = make_uint2(c[0], c[1]);
      if (FMT == kMxE4m3 || (j & 1) == 0)
        sSX[s * S::kSub * S::kScale + scale_to] = (unsigned char)byte;
      fence_proxy_async();  // generic-proxy stores -> visible to the tensor core
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
    }
  } else {
    after_previous();  // the row scales
    const int q = warp & 3;                      // the TMEM lane quadrant this warp may read
    const int part = (warp - kEpiWarp) >> 2;     // its share of the token columns
    constexpr int NC = NT / (S::kEpiWarps / 4);
    constexpr int CH = NC < 32 ? NC : 32;        // columns a thread takes at a time
    static_assert(NC == CH || NC == 2 * CH, "columns");
    float* gx = s_gx[warp - kEpiWarp];           // the row scales of its tokens
    TileAt t;
    int e = 0, i = 0;
    bool fail = false;  // a wait ran out: NaN for this tile and all that follow
    for (int item = item0; item < items; item += step, i++) {
      tile_at<S::kTileRows>(a, s_pre, item, &e, &t);
      const int b = i % TM::kBufs;
      const int n = t.n0 + wrow + q * 32 + lane;
      const bool nok = n < a.N;
      const int mine = t.count - part * NC;  // this warp's tokens
      float gw = 1.0f;
      bool plain = true;  // every row scale of this warp's tokens
      if (FMT == kMxE4m3 && !SPLIT) {  // fetched while the MMAs run
        if (nok) gw = load_f32(a.gw + (int64_t)t.e * a.N + n);
        if (!S::kOwn) {
          __syncwarp();
#pragma unroll
          for (int c = 0; c < NC; c += 32)
            if (c + lane < NC) {
              const float g = c + lane < mine ? load_f32(a.gx + t.row + part * NC + c + lane) : 1.0f;
              gx[c + lane] = g;
              plain = plain && plain_scale(g);
            }
          __syncwarp();
        }
      }
      if (!fail) fail = !epilogue_wait(&acc_full[b], (i / TM::kBufs) & 1, i);
      fail = __any_sync(0xffffffffu, fail || s_fail);
      if (fail) s_fail = 1;
      tc_fence_after();
      if (FMT == kMxE4m3 && !SPLIT && S::kOwn) {  // written before the last stage was
        __syncwarp();
        if (lane < NC) {
          gx[lane] = lane < mine ? s_scale[part * NC + lane] : 1.0f;
          plain = plain_scale(gx[lane]);
        }
        __syncwarp();
      }
      if (FMT == kMxE4m3 && !SPLIT) plain = __all_sync(0xffffffffu, plain);
      const uint32_t src = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * NT + part * NC);
      if (SPLIT) {
        // every MMA of this CTA is complete, so the stages are free
        float* P = reinterpret_cast<float*>(base) + part * NC * kWRows + q * 32 + lane;
#pragma unroll 1
        for (int c0 = 0; c0 < NC && c0 < mine; c0 += 16) {
          uint32_t r[16];
          if (!fail) tmem_ld16_nowait(src + c0, r);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; c++)
            if (c0 + c < mine)
              P[(c0 + c) * kWRows] = fail ? __int_as_float(0x7fc00000) : __uint_as_float(r[c]);
        }
        break;
      }
      const int size_y = a.bf16_out ? 2 : 4;
      const int64_t step_y = a.ldy * size_y;
      char* y = static_cast<char*>(a.Y) + (int64_t)(t.row + part * NC) * step_y + (int64_t)n * size_y;
      if (fail) {
        for (int c = 0; c < min(mine, NC) && nok; c++, y += step_y) {
          if (a.bf16_out) *reinterpret_cast<__nv_bfloat16*>(y) = __float2bfloat16_rn(__int_as_float(0x7fc00000));
          else *reinterpret_cast<float*>(y) = __int_as_float(0x7fc00000);
        }
        continue;
      }
      auto take = [&](int c0, uint32_t (&r)[CH]) {
#pragma unroll
        for (int c = 0; c < CH; c += 16) tmem_ld16_nowait(src + c0 + c, r + c);
        tmem_wait_ld();
        if (c0 + CH == NC) {  // the accumulator's last columns are in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_first<TWO>(&acc_empty[b]);
        }
        if (FMT == kMxE4m3) {
          // One answer a warp, which costs nothing: the steps of scale_sum for all
          // took 6% at 14336 x 4096 and 8192 tokens.
          if (plain) {
#pragma unroll
            for (int c = 0; c < CH; c += 4) {
              const float4 g = *reinterpret_cast<const float4*>(gx + c0 + c);
              const float gs[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
              for (int j = 0; j < 4; j++)
                r[c + j] = __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(r[c + j]), gs[j]), gw));
            }
          } else {  // a loop that stays one: little code
#pragma unroll 1
            for (int c = 0; c < CH; c++) {
              const float y = scale_sum(__uint_as_float(r[0]), gx[c0 + c], gw);
#pragma unroll
              for (int j = 0; j < CH - 1; j++) r[j] = r[j + 1];
              r[CH - 1] = __float_as_uint(y);
            }
          }
        }
      };
      auto put_f32 = [&](int c0, const uint32_t (&r)[CH]) {
#pragma unroll
        for (int c = 0; c < CH; c++) {
          if (nok && c0 + c < mine) *reinterpret_cast<uint32_t*>(y) = r[c];
          y += step_y;
        }
      };
      auto pack = [&](const uint32_t (&r)[CH], uint32_t (&h)[CH / 2]) {  // two tokens a register
#pragma unroll
        for (int c = 0; c < CH / 2; c++) {
          const __nv_bfloat162 v =
              __floats2bfloat162_rn(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1]));
          h[c] = *reinterpret_cast<const uint32_t*>(&v);
        }
      };
      auto put_bf16 = [&](int c0, const uint32_t (&h)[CH / 2]) {
#pragma unroll
        for (int c = 0; c < CH; c++) {
          if (nok && c0 + c < mine)
            *reinterpret_cast<uint16_t*>(y) = (uint16_t)(c & 1 ? h[c / 2] >> 16 : h[c / 2]);
          y += step_y;
        }
      };
      // The first columns are held as bf16 until the last ones have left
      // tensor memory: the next tile's MMAs wait for loads, not for stores.
      uint32_t r[CH], h[CH / 2];
      take(0, r);
      if (a.bf16_out) {
        pack(r, h);
        if (NC > CH) {
          take(NC - CH, r);
          put_bf16(0, h);
          pack(r, h);
        }
        put_bf16(NC - CH, h);
      } else {
        put_f32(0, r);
        if (NC > CH) {
          take(NC - CH, r);
          put_f32(NC - CH, r);
        }
      }
    }
  }
  tc_fence_before();
  // The MMAs are complete before tensor memory is given back (bounded): where
  // the epilogue gave up, it has not waited for them.
  if (TWO) {
    if (warp == 1) wait_last(empty, mma_ring);
    cluster_sync_all();  // neither CTA's memory is in use by the other
  } else {
    __syncthreads();
    if (warp == 1 && s_fail) wait_last(empty, mma_ring);
  }
  if (warp == 1) {
    tc_fence_after();
    if (TWO)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(TM::kCols));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(TM::kCols));
  }
  if (SPLIT) {
    TileAt t;
    int e = 0;
    const bool have = item0 < items;  // the same for the whole cluster
    if (have) tile_at<S::kTileRows>(a, s_pre, item0, &e, &t);
    cluster_sync_all();  // every CTA's partial is in its shared memory
    if (have) {
      // Four weight rows of a token at a time: one 16-byte read of every CTA's
      // partial, all in flight before the first sum, added in rank order.
      const float* P = reinterpret_cast<const float*>(base);
      const int E = t.count * (kWRows / 4);
      const int e0 = (int)((int64_t)crank * E / csize), e1 = (int)((int64_t)(crank + 1) * E / csize);
      const int size_y = a.bf16_out ? 2 : 4;
      const bool wide = reinterpret_cast<uintptr_t>(a.Y) % (4 * size_y) == 0 && a.ldy % 4 == 0;
      for (int i = e0 + threadIdx.x; i < e1; i += S::kThreads) {
        const int c = i / (kWRows / 4), n = t.n0 + i % (kWRows / 4) * 4;
        float4 part[kMaxSplit];
#pragma unroll
        for (int k = 0; k < kMaxSplit; k++)
          if (k < (int)csize) part[k] = ld_cluster_f4(P + 4 * i, (uint32_t)k);
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kMaxSplit; k++)
          if (k < (int)csize) {
            v[0] = __fadd_rn(v[0], part[k].x);
            v[1] = __fadd_rn(v[1], part[k].y);
            v[2] = __fadd_rn(v[2], part[k].z);
            v[3] = __fadd_rn(v[3], part[k].w);
          }
        if (FMT == kMxE4m3) {
          const float g = S::kOwn ? s_scale[c] : load_f32(a.gx + t.row + c);
          const float* gw = a.gw + (int64_t)t.e * a.N;
#pragma unroll
          for (int j = 0; j < 4; j++)
            v[j] = scale_sum(v[j], g, n + j < a.N ? load_f32(gw + n + j) : 1.0f);
        }
        const int64_t y = (int64_t)(t.row + c) * a.ldy + n;
        if (a.bf16_out) {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.Y) + y;
          if (wide && n + 3 < a.N) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(v[2], v[3]);
            *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                      *reinterpret_cast<const uint32_t*>(&hi));
          } else {
#pragma unroll
            for (int j = 0; j < 4; j++)
              if (n + j < a.N) o[j] = __float2bfloat16_rn(v[j]);
          }
        } else {
          float* o = static_cast<float*>(a.Y) + y;
          if (wide && n + 3 < a.N) {
            *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; j++)
              if (n + j < a.N) o[j] = v[j];
          }
        }
      }
    }
    cluster_sync_all();  // no CTA leaves while another may still read its partial
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
cudaError_t byte_map(EncodeTiledFn enc, CUtensorMap* map, const uint8_t* p, int64_t row_bytes,
                     int64_t rows, int unit, int box_units, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)(row_bytes / unit), (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {(cuuint32_t)box_units, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      enc(map, unit == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT64, 2,
          const_cast<uint8_t*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          unit == 1 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

struct Maps {
  CUtensorMap x, w, sx, sw;
};

// Codes as bytes, 128 of a row at a time.  Scale tiles as 8-byte units, a
// stage's tiles along K at a time (tiles past K read as zero) and as many
// bands as a token tile has.
cudaError_t make_maps(EncodeTiledFn enc, const MxTensor& t, int box_rows, int box_bands,
                      CUtensorMap* codes, CUtensorMap* scales) {
  const int units = (t.fmt == kMxE8m0 ? 2 : 4) * kMxTileBytes / 8;
  const cudaError_t e = byte_map(enc, codes, t.codes, t.K / 2, t.rows, 1, kRowBytes, box_rows);
  if (e != cudaSuccess) return e;
  return byte_map(enc, scales, t.scales, mx_tiles_k(t.fmt, t.K) * kMxTileBytes,
                  mx_bands(t.rows, t.groups), 8, units, box_bands);
}

template <int FMT, int NT, int MODE, int SRC = kSrcNone>
cudaError_t launch_t(const Maps& m, const MxGemmArgs& a, const MxPlan& p,
                     cudaStream_t st, const RowsArgs& own = RowsArgs{}) {
  using S = Shape<FMT, NT, MODE, SRC>;
  cudaError_t e = cudaFuncSetAttribute(mx_gemm_kernel<FMT, NT, MODE, SRC>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = MODE == kSplit ? dim3((unsigned)p.split, (unsigned)p.tiles, 1)
                               : dim3((unsigned)p.ctas, 1, 1);
  cfg.blockDim = dim3(S::kThreads, 1, 1);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (MODE != kWalk) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = MODE == kSplit ? (unsigned)p.split : 2u;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    n++;
  }
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  n++;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  e = cudaLaunchKernelEx(&cfg, mx_gemm_kernel<FMT, NT, MODE, SRC>, m.x, m.w, m.sx, m.sw, a, own);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <int FMT, int MODE>
cudaError_t launch_m(const Maps& m, const MxGemmArgs& a, const MxPlan& p,
                     cudaStream_t st) {
  switch (p.nt) {
    case 32: return launch_t<FMT, 32, MODE>(m, a, p, st);
    case 64: return launch_t<FMT, 64, MODE>(m, a, p, st);
    case 128: return launch_t<FMT, 128, MODE>(m, a, p, st);
    default: return launch_t<FMT, 256, MODE>(m, a, p, st);
  }
}

template <int FMT, int SRC>
cudaError_t launch_own(const Maps& m, const MxGemmArgs& a, const MxPlan& p, const RowsArgs& own,
                       cudaStream_t st) {
  return p.split > 1 ? launch_t<FMT, 32, kSplit, SRC>(m, a, p, st, own)
                     : launch_t<FMT, 32, kWalk, SRC>(m, a, p, st, own);
}

cudaError_t launch_own_s(int fmt, const Maps& m, const MxGemmArgs& a, const MxPlan& p,
                         const MxSource& x, const RowsArgs& own, cudaStream_t st) {
  if (fmt == kMxE4m3)  // no SwiGLU (mx_own_rows)
    return x.f32 ? launch_own<kMxE4m3, kSrcF32>(m, a, p, own, st)
                 : launch_own<kMxE4m3, kSrcBf16>(m, a, p, own, st);
  if (x.swiglu)
    return x.f32 ? launch_own<kMxE8m0, kSrcF32Glu>(m, a, p, own, st)
                 : launch_own<kMxE8m0, kSrcBf16Glu>(m, a, p, own, st);
  return x.f32 ? launch_own<kMxE8m0, kSrcF32>(m, a, p, own, st)
               : launch_own<kMxE8m0, kSrcBf16>(m, a, p, own, st);
}

template <int FMT>
cudaError_t launch_f(const Maps& m, const MxGemmArgs& a, const MxPlan& p,
                     cudaStream_t st) {
  if (p.pair) return launch_t<FMT, 256, kPair>(m, a, p, st);
  return p.split > 1 ? launch_m<FMT, kSplit>(m, a, p, st)
                     : launch_m<FMT, kWalk>(m, a, p, st);
}

}  // namespace

// The plan with the least estimated time, in microseconds, fitted at N = 1024 to
// 14336, K = 4096 to 27648 and 128 to 2048 tokens.  A launch's start and end, 3 to 6
// us that all plans share, are not in it (E4M3, in a graph, estimate and time: 2048
// tokens by 14336 x 4096 53 and 56, by 4096 x 4096 15 and 21, by 1024 x 4096 6 and
// 10; 333 by 5120 x 27648 35 and 41).  It does not know the format: E8M0, with half
// the scales, takes up to a tenth less.  Where it is wrong: 300 tokens by 1024 x
// 8192, 24 tiles split 6 ways, 6 and 23.  A stage of a tile takes 0.20 + 0.0011 per
// token column, of which the first part is the weight tile's way from L2 (narrow
// tiles pay it more often), and a tile's last stages and stores 0.5.  CTAs
// that split a tile run one after the other where there are too many of them,
// each with its start, and its joining of the parts, 4 for every 256 columns.
// Pairs of CTAs take tiles of twice the weight rows in the time of single
// ones and with a third less traffic, as soon as there are tiles for all: 2048
// tokens by 14336 x 16384 take 189 us with them and 202 without, hence 0.93.
MxPlan mx_plan(int groups, int64_t rows, int64_t N, int64_t K) {
  MxPlan p;
  const int64_t stages = (K + kStageK - 1) / kStageK;
  const int64_t n1 = (N + kWRows - 1) / kWRows, n2 = (N + 2 * kWRows - 1) / (2 * kWRows);
  const int64_t busy = groups < rows ? groups : rows;  // groups that can hold rows
  const double each = (double)rows / (double)busy;
  double best = 0.0;
  p.width = 0;
  // token tiles: of ragged groups, half a tile more than their rows fill
  auto token_tiles = [&](int width) {
    if (groups == 1) return (double)((rows + width - 1) / width);
    const double t = each / width + 0.5;
    return (double)busy * (t > 1.0 ? t : 1.0);
  };
  auto offer = [&](int width, int split, bool pair) {
    const double tt = token_tiles(width);
    const double columns = (double)rows / tt;
    const double tiles = tt * (double)(pair ? n2 : n1);
    const double waves = ceil(tiles * split / (pair ? kSms / 2 : kSms));
    const double stage = 0.20 + 0.0011 * columns;
    const double own = (double)((stages + split - 1) / split) * stage + 0.5;
    const double t = waves * (split > 1 ? own + 2.0 + columns / 64.0 : pair ? 0.93 * own : own);
    if (p.width == 0 || t < best) {
      best = t;
      p.width = width;
      p.split = split;
      p.pair = pair ? 1 : 0;
    }
  };
  if (groups == 1 && rows <= 32) {
    for (int s = 1; s <= kMaxSplit && s <= stages; s++) offer(32, s, false);
  } else {
    for (int w = 64; w <= 256; w += 64) {
      for (int s = 1; s <= kMaxSplit && s <= stages; s++) offer(w, s, false);
      if (w > 128 && token_tiles(w) * (double)n2 >= kSms / 2) offer(w, 1, true);
      if (w >= each) break;
    }
  }
  p.nt = p.width > 128 ? 256 : p.width;
  const int64_t n = p.pair ? n2 : n1;
  // an upper bound of the tiles: sum ceil(c / width) <= rows / width + one per busy group
  p.token_tiles = groups == 1 ? (rows + p.width - 1) / p.width : rows / p.width + busy;
  p.tiles = p.token_tiles * n;
  if (p.tiles > 65535) p.split = 1;  // a grid's y
  p.stages = (int)stages;
  p.ctas = p.pair ? kSms : (int)(p.split > 1 ? p.tiles * p.split : (p.tiles < kSms ? p.tiles : kSms));
  return p;
}

// The few rows that every CTA quantises itself, its part of K at a time; for
// E4M3 it first reads all of them for their maxima.  Measured against the
// quantisation in a launch before (us, of calls in a row in a graph):
//   E8M0  4096 x 4096, 1 row 6.6 (7.4), 8 rows 7.0 (7.6), 16 rows 7.5 (7.8);
//         5120 x 27648, 1 row 14.5 (16.9), 8 rows 15.8 (17.0), 16 rows 21.9 (17.3);
//         SwiGLU 14336 x 4096, 1 row 8.2 (8.8), 4 rows 8.7 (8.8), 8 rows 11.5 (8.8)
//   E4M3  14336 x 4096, 1 row 8.3 (9.0), 2 rows 8.9 (9.0), 4 rows 9.6 (9.0);
//         4096 x 14336, 1 row 11.5 (10.5); SwiGLU 4096 x 4096, 1 row 8.7 (7.8)
// and about 4 us less of the host's time.
bool mx_own_rows(int fmt, int groups, int64_t rows, int64_t K, bool swiglu) {
  if (groups != 1) return false;
  if (fmt == kMxE8m0) return rows <= (swiglu ? kMaxOwnRows / 2 : kMaxOwnRows);
  return !swiglu && rows <= kMaxOwnRows && rows * K <= 8192;
}

cudaError_t launch_mx_gemm(const MxTensor& x, const MxTensor& w, void* Y, bool f32, int64_t ldy,
                           const MxSource* src, bool overlap, cudaStream_t st) {
  EncodeTiledFn enc = nullptr;
  cudaError_t e = encode_fn(&enc);
  if (e != cudaSuccess) return e;
  const int64_t N = w.rows / w.groups;
  const MxPlan p = mx_plan(x.groups, x.rows, N, x.K);
  // One copy for all of a tile's token rows; ragged groups leave many tiles
  // part empty and take pieces, of which only those with rows are fetched.
  const int box = x.groups == 1 ? (p.pair ? p.width / 2 : p.width) : (p.nt < 128 ? 32 : 64);
  Maps m = {};
  e = make_maps(enc, w, kWRows, 1, &m.w, &m.sw);
  if (e == cudaSuccess && !src) e = make_maps(enc, x, box, (p.nt + 127) / 128, &m.x, &m.sx);
  if (e != cudaSuccess) return e;
  const MxGemmArgs a{x.row_scale, w.row_scale, Y, ldy,
                     MxRows{x.offsets, x.groups, (int)x.rows}, (int)N, (int)x.K,
                     (int)((N + kWRows - 1) / kWRows + p.pair) / (1 + p.pair), p.stages, p.width, box,
                     f32 ? 0 : 1, overlap ? 1 : 0, (int)p.token_tiles};
  if (src) {
    int warps = 1;
    while (2 * warps < (int)x.rows) warps *= 2;
    const RowsArgs own{src->X, src->index, src->ldx, (int)src->rows, warps};
    return launch_own_s(x.fmt, m, a, p, *src, own, st);
  }
  return x.fmt == kMxE8m0 ? launch_f<kMxE8m0>(m, a, p, st)
                          : launch_f<kMxE4m3>(m, a, p, st);
}

cudaError_t mx_timeout_flag(unsigned int* out) {
  return cudaMemcpyFromSymbol(out, g_wait_timeout, sizeof(unsigned int));
}

#ifdef AAAC_CHECKS
cudaError_t mx_set_patience(int tiles) { return cudaMemcpyToSymbol(g_patience, &tiles, sizeof(int)); }
#endif

}  // namespace aaac
