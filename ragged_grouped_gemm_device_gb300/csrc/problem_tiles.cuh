// The problem list's 128-row tiles, for the kernels that place per-row data by tile (the scale
// atoms of the block-scaled products).
#pragma once

#include "common.cuh"

namespace moe {

// 128-row tiles of an expert's rows, which may be as many as an int holds (rows + 127 may not)
__host__ __device__ constexpr int row_tiles(int rows) { return rows / 128 + (rows % 128 > 0 ? 1 : 0); }
static_assert(row_tiles(0) == 0 && row_tiles(1) == 1 && row_tiles(128) == 1 && row_tiles(129) == 2 &&
                  row_tiles(0x7fffffff) == 1 << 24,
              "tiles of a row count");

// The problem list as the grouped GEMM derives it from the offsets: s_end[e] = inclusive end of
// expert e's rows, s_pre[e] = 128-row tiles of the experts before e (block-wide scan, 256
// threads). Offsets that decrease or end past `rows` would place rows outside the scale atoms:
// they are flagged (MOE_DEV_BAD_OFFSETS) and the function returns false in every thread.
static __device__ bool load_problem_tiles(const int32_t* __restrict__ offsets, int E, long long rows, int* s_end,
                                   int* s_pre, int32_t* status) {
  __shared__ int s_carry;
  __shared__ int wsum[8];
  if (threadIdx.x == 0) s_carry = 0;
  __syncthreads();
  for (int base = 0; base < E; base += blockDim.x) {
    const int e = base + threadIdx.x;
    int tiles = 0;
    if (e < E) {
      const int end = __ldg(offsets + e);
      const int start = e > 0 ? __ldg(offsets + e - 1) : 0;
      s_end[e] = end;
      tiles = row_tiles(end - start);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int nb = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += nb;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int before = s_carry;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (e < E) s_pre[e] = before + incl - tiles;
    __syncthreads();
    if (threadIdx.x == 0) {
      int tot = 0;
      for (int w = 0; w < 8; ++w) tot += wsum[w];
      s_carry += tot;
    }
    __syncthreads();
  }
  bool bad = false;
  for (int e = threadIdx.x; e < E; e += blockDim.x)
    bad |= (s_end[e] < (e > 0 ? s_end[e - 1] : 0)) || (e == E - 1 && s_end[e] > rows);
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) record_status(status, MOE_DEV_BAD_OFFSETS);
    return false;
  }
  return true;
}

// Tile (G) and row within the tile (r) of row p of the problem list.
__device__ __forceinline__ void row_tile(const int* s_end, const int* s_pre, int E, long long p, long long& G,
                                         int& r) {
  int lo = 0, hi = E - 1;  // first expert whose segment ends after p
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (s_end[mid] > p) hi = mid; else lo = mid + 1;
  }
  const long long start = lo > 0 ? s_end[lo - 1] : 0;
  G = s_pre[lo] + (p - start) / 128;
  r = static_cast<int>((p - start) % 128);
}

}  // namespace moe
