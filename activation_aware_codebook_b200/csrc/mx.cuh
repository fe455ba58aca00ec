// mx.cuh -- the microscaled 4-bit layout that mx_quant.cu writes and
// mx_gemm.cu reads.
//
// Values are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two per
// byte along K, the low nibble the even column: the order in which tcgen05
// reads packed 4-bit operands.  The block scales lie as the tensor core wants
// them in tensor memory: tiles of 128 rows x 4 blocks, 512 bytes each, row
// i's four bytes at (i % 32) * 16 + (i / 32) * 4.  Lane l's 16 bytes are then the
// words of rows l, l + 32, l + 64 and l + 96, and a warp moves a tile there with
// one load a lane and a store of four columns.  Tiles of a row band are
// consecutive along K.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace aaac {

constexpr int kMxE8m0 = 0;  // blocks of 32, power-of-two scales
constexpr int kMxE4m3 = 1;  // blocks of 16, E4M3 scales, a power of two per row
constexpr int kMxTileRows = 128;
constexpr int kMxTileBytes = 512;
constexpr int kMxMaxGroups = 1024;

__host__ __device__ constexpr int mx_block(int fmt) { return fmt == kMxE8m0 ? 32 : 16; }

// Scale tiles along K (four blocks each; the last one is padded with zeros).
__host__ __device__ inline int64_t mx_tiles_k(int fmt, int64_t K) {
  const int64_t span = 4 * mx_block(fmt);
  return (K + span - 1) / span;
}

// Rows of a tensor in groups (an expert's rows each): either `offsets`
// (device, groups + 1 values) or groups of equal size.
struct MxRows {
  const int32_t* offsets;
  int groups;
  int rows;  // of all groups
};

// Global loads of what an earlier kernel on the stream may have written while
// this one was already there (see after_previous): ordered behind the wait, and
// not through the path for data that is constant over a kernel's lifetime.
__device__ __forceinline__ int32_t load_i32(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load_u8(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float load_f32(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load_2(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 load_4(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Group e's rows [first, last), held inside the tensor whatever the offsets say.
__device__ __forceinline__ void mx_group(const MxRows& g, int e, int* first, int* last) {
  if (g.offsets) {
    const int a = min(max(load_i32(g.offsets + e), 0), g.rows);
    *first = a;
    *last = min(max(load_i32(g.offsets + e + 1), a), g.rows);
  } else {
    const int per = g.rows / g.groups;
    *first = e * per;
    *last = e * per + per;
  }
}

// Token tiles of a group of `count` rows, and sums of them over groups, each held
// at `most`: the plan's bound for sound offsets (at most 2^31 / 32 + 1024, so that
// neither a sum of two nor, by the calls' checks, its product with the weight
// tiles passes 32 bits).  Offsets that are not sound, say 0 and the last row in
// turn, can name every row in every group; the tiles beyond the bound are left out.
__host__ __device__ inline int mx_group_tiles(int count, int width, int most) {
  const int tiles = count > 0 ? (count - 1) / width + 1 : 0;
  return tiles < most ? tiles : most;
}
__host__ __device__ inline int mx_add_tiles(int a, int b, int most) {
  return a + b < most ? a + b : most;
}

// Each group's scales start a tile of their own: group e, whose first row is
// `first`, starts at band first / 128 + e.  floor(a / 128) + floor(b / 128) <=
// floor((a + b) / 128) keeps the bands of one group clear of the next one's,
// and rows / 128 + groups bands hold them all, so a band follows from the
// group's own offset with no sum over the others.
__host__ __device__ inline int64_t mx_bands(int64_t rows, int groups) {
  return rows / kMxTileRows + groups;
}

// Kernels of the microscaled calls are launched so that they may start while
// the kernel before them on the stream still runs (programmatic dependent
// launch), set themselves up, and then wait for all that came before.  A kernel
// touches no global memory before after_previous(), but for one case: the
// product behind its own quantisation reads weights and offsets earlier, which
// is sound because the quantisation lets it start only after its own wait.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace aaac
