// Layer norm over the last dimension, forward and backward (the pre-norm of the expert block).
//
//   mean = sum x / d;  var = sum (x - mean)^2 / d;  rstd = 1 / sqrt(var + eps)
//   xhat = (x - mean) rstd;  y = xhat gamma + beta
//   dx = rstd (gamma dy - mean(gamma dy) - xhat mean(gamma dy xhat))
//   dgamma = sum_t dy xhat;  dbeta = sum_t dy
//
// Both passes are bound by memory: the forward has to read x and write y, the backward to read
// x and dy and write dx. A row is held in the registers of the TPR threads that own it, so each
// value is read once and the variance is the exact two-pass one (the sum of squared differences
// from the mean, not a difference of two large sums). All arithmetic is fp32; y and dx are rounded
// once. The forward gives a row to one warp as long as it fits (eight chunks a lane, 2048 bf16):
// no barriers, and the weights come from L1, which they stay in. The backward gives it to as many
// threads as it has 16-byte chunks, which keeps the weight, the two gradients' sums and the next
// row's loads in registers. The weight gradients are sums over all rows: each block adds the rows it owns in
// registers (a thread always owns the same columns), leaves one partial row of each gradient in
// the workspace, and a second small kernel adds the partials in block order. No atomics: the
// results do not depend on scheduling.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "trace.h"

namespace moe {
namespace {

// Blocks of the backward at most, and so rows of partial weight gradients: four for each of the
// 152 SMs. A constant, because the size of the workspace is host arithmetic.
constexpr int BWD_MAX_BLOCKS = 608;
constexpr int MAX_WIDTH = 1 << 20;

// VB consecutive elements of a row: one 16-byte access, or one element where the rows or bases
// are not 16-byte aligned.
template <typename T, int VB>
struct Chunk;
template <>
struct Chunk<bf16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  static __device__ __forceinline__ void store(bf16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Chunk<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void unpack(float (&f)[4]) const {
    f[0] = v.x;
    f[1] = v.y;
    f[2] = v.z;
    f[3] = v.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Chunk<bf16, 1> {
  bf16 v;
  __device__ __forceinline__ void load(const bf16* p) { v = *p; }
  __device__ __forceinline__ void unpack(float (&f)[1]) const { f[0] = __bfloat162float(v); }
  static __device__ __forceinline__ void store(bf16* p, const float (&f)[1]) { *p = __float2bfloat16_rn(f[0]); }
};
template <>
struct Chunk<float, 1> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = __ldg(p); }
  __device__ __forceinline__ void unpack(float (&f)[1]) const { f[0] = v; }
  static __device__ __forceinline__ void store(float* p, const float (&f)[1]) { *p = f[0]; }
};

// VB consecutive weights from column c: fp32 or bf16, `fill` where there are none.
template <int VB>
__device__ __forceinline__ void load_weight(const void* w, bool w_bf16, int c, float fill, float (&o)[VB]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < VB; ++i) o[i] = fill;
  } else if (w_bf16) {
    if constexpr (VB == 8) {
      Chunk<bf16, 8> q;
      q.load(static_cast<const bf16*>(w) + c);
      q.unpack(o);
    } else {
#pragma unroll
      for (int i = 0; i < VB; ++i) o[i] = __bfloat162float(static_cast<const bf16*>(w)[c + i]);
    }
  } else {
    if constexpr (VB % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VB; i += 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + c + i));
        o[i] = q.x;
        o[i + 1] = q.y;
        o[i + 2] = q.z;
        o[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VB; ++i) o[i] = __ldg(static_cast<const float*>(w) + c + i);
    }
  }
}

// Sum of a (and b) over the TPR threads of a row. For rows wider than a warp, `buf` is one of two
// alternating buffers: a thread that is a reduction ahead writes the other one.
template <int TPR>
__device__ __forceinline__ float2 row_sum(float a, float b, float2* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (TPR == 32) return make_float2(a, b);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) buf[warp] = make_float2(a, b);
  __syncthreads();
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < TPR / 32; ++w) {
    s.x += buf[w].x;
    s.y += buf[w].y;
  }
  return s;
}

struct NormArgs {
  const void* x;
  const void* dy;      // backward
  void* out;           // y, or dx
  long long ldx, lddy, ldo;
  const void* gamma;   // nullable
  const void* beta;    // nullable (forward)
  bool w_bf16;
  int T, d;
  float eps;
  float* mean;         // forward: nullable outputs; backward: inputs
  float* rstd;
  float* part;         // backward: [blocks][2][d] partial dgamma, dbeta (nullable: not wanted)
};

// threads of a block: a row's TPR, or four rows of one warp each
constexpr int block_threads(int tpr) { return tpr == 32 ? 128 : tpr; }

template <typename T, int VB, int NCH, int TPR>
__global__ void __launch_bounds__(block_threads(TPR)) norm_fwd_kernel(const NormArgs a) {
  constexpr int ROWS = block_threads(TPR) / TPR;
  __shared__ float2 red[2][32];
  const int t = threadIdx.x % TPR;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  for (long long row = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / TPR; row < a.T;
       row += static_cast<long long>(gridDim.x) * ROWS) {
    const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
    Chunk<T, VB> q[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (i * TPR + t) * VB;
      if (c < a.d) q[i].load(xr + c);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if ((i * TPR + t) * VB >= a.d) continue;
      float f[VB];
      q[i].unpack(f);
#pragma unroll
      for (int j = 0; j < VB; ++j) sum += f[j];
    }
    const float mean = row_sum<TPR>(sum, 0.f, red[0]).x * inv_d;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if ((i * TPR + t) * VB >= a.d) continue;
      float f[VB];
      q[i].unpack(f);
#pragma unroll
      for (int j = 0; j < VB; ++j) sq = fmaf(f[j] - mean, f[j] - mean, sq);
    }
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(sq, 0.f, red[1]).x * inv_d + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    T* yr = static_cast<T*>(a.out) + row * a.ldo;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (i * TPR + t) * VB;
      if (c >= a.d) continue;
      float f[VB], g[VB], b[VB];
      q[i].unpack(f);
      load_weight<VB>(a.gamma, a.w_bf16, c, 1.0f, g);
      load_weight<VB>(a.beta, a.w_bf16, c, 0.0f, b);
#pragma unroll
      for (int j = 0; j < VB; ++j) f[j] = fmaf((f[j] - mean) * rstd, g[j], b[j]);
      Chunk<T, VB>::store(yr + c, f);
    }
  }
}

template <typename T, int VB, int NCH, int TPR>
__global__ void __launch_bounds__(block_threads(TPR)) norm_bwd_kernel(const NormArgs a) {
  constexpr int ROWS = block_threads(TPR) / TPR;
  __shared__ float2 red[2][32];
  const int t = threadIdx.x % TPR;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float dg[NCH][VB], db[NCH][VB], g[NCH][VB];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * TPR + t) * VB;
    if (c < a.d) load_weight<VB>(a.gamma, a.w_bf16, c, 1.0f, g[i]);
#pragma unroll
    for (int j = 0; j < VB; ++j) dg[i][j] = db[i][j] = 0.f;
  }
  // the next row's loads are in flight while this one is worked on
  Chunk<T, VB> qx[NCH], qd[NCH];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](long long row) {
    const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
    const T* dr = static_cast<const T*>(a.dy) + row * a.lddy;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (i * TPR + t) * VB;
      if (c < a.d) {
        qx[i].load(xr + c);
        qd[i].load(dr + c);
      }
    }
    mean = __ldg(a.mean + row);
    rstd = __ldg(a.rstd + row);
  };
  const long long step = static_cast<long long>(gridDim.x) * ROWS;
  long long row = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / TPR;
  if (row < a.T) fetch(row);
  int par = 0;
  for (; row < a.T; row += step) {
    Chunk<T, VB> cx[NCH], cd[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      cx[i] = qx[i];
      cd[i] = qd[i];
    }
    const float mu = mean, rs = rstd;
    if (row + step < a.T) fetch(row + step);
    float s1 = 0.f, s2 = 0.f;  // sums of gamma dy and of gamma dy xhat
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if ((i * TPR + t) * VB >= a.d) continue;
      float fx[VB], fd[VB];
      cx[i].unpack(fx);
      cd[i].unpack(fd);
#pragma unroll
      for (int j = 0; j < VB; ++j) {
        const float xh = (fx[j] - mu) * rs, gd = g[i][j] * fd[j];
        s1 += gd;
        s2 = fmaf(gd, xh, s2);
        dg[i][j] = fmaf(fd[j], xh, dg[i][j]);
        db[i][j] += fd[j];
      }
    }
    const float2 s = row_sum<TPR>(s1, s2, red[par]);
    par ^= 1;
    const float m1 = s.x * inv_d, m2 = s.y * inv_d;
    T* orow = static_cast<T*>(a.out) + row * a.ldo;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (i * TPR + t) * VB;
      if (c >= a.d) continue;
      float fx[VB], fd[VB];
      cx[i].unpack(fx);
      cd[i].unpack(fd);
#pragma unroll
      for (int j = 0; j < VB; ++j) fx[j] = rs * (fmaf(g[i][j], fd[j], -m1) - (fx[j] - mu) * rs * m2);
      Chunk<T, VB>::store(orow + c, fx);
    }
  }
  if (a.part == nullptr) return;
  float* pg = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
  float* pb = pg + a.d;
  if constexpr (ROWS == 1) {
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int j = 0; j < VB; ++j) {
        const int c = (i * TPR + t) * VB + j;
        if (c < a.d) {
          pg[c] = dg[i][j];
          pb[c] = db[i][j];
        }
      }
  } else {
    // the block's warps own different rows of the same columns: add them in warp order
    __shared__ float2 acc[ROWS - 1][32];
    const int w = threadIdx.x / TPR;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int j = 0; j < VB; ++j) {
        const int c = (i * TPR + t) * VB + j;
        __syncthreads();
        if (w > 0) acc[w - 1][t] = make_float2(dg[i][j], db[i][j]);
        __syncthreads();
        if (w == 0 && c < a.d) {
          float g = dg[i][j], b = db[i][j];
#pragma unroll
          for (int r = 0; r < ROWS - 1; ++r) {
            g += acc[r][t].x;
            b += acc[r][t].y;
          }
          pg[c] = g;
          pb[c] = b;
        }
      }
  }
}

// Rows too wide for registers: three passes over the row (the later ones from L2), one block a row.
constexpr int WIDE_THREADS = 1024;

template <typename T>
__global__ void __launch_bounds__(WIDE_THREADS) norm_fwd_wide_kernel(const NormArgs a) {
  __shared__ float2 red[2][32];
  const float inv_d = 1.0f / static_cast<float>(a.d);
  for (long long row = blockIdx.x; row < a.T; row += gridDim.x) {
    const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
    T* yr = static_cast<T*>(a.out) + row * a.ldo;
    float s = 0.f, f[1], g[1], b[1];
    Chunk<T, 1> q;
    for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
      q.load(xr + c);
      q.unpack(f);
      s += f[0];
    }
    const float mean = row_sum<WIDE_THREADS>(s, 0.f, red[0]).x * inv_d;
    s = 0.f;
    for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
      q.load(xr + c);
      q.unpack(f);
      s = fmaf(f[0] - mean, f[0] - mean, s);
    }
    const float rstd = 1.0f / sqrtf(row_sum<WIDE_THREADS>(s, 0.f, red[1]).x * inv_d + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
      q.load(xr + c);
      q.unpack(f);
      load_weight<1>(a.gamma, a.w_bf16, c, 1.0f, g);
      load_weight<1>(a.beta, a.w_bf16, c, 0.0f, b);
      f[0] = fmaf((f[0] - mean) * rstd, g[0], b[0]);
      Chunk<T, 1>::store(yr + c, f);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(WIDE_THREADS) norm_bwd_wide_kernel(const NormArgs a) {
  __shared__ float2 red[2][32];
  const float inv_d = 1.0f / static_cast<float>(a.d);
  int par = 0;
  for (long long row = blockIdx.x; row < a.T; row += gridDim.x) {
    const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
    const T* dr = static_cast<const T*>(a.dy) + row * a.lddy;
    T* orow = static_cast<T*>(a.out) + row * a.ldo;
    const float mean = __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
    float s1 = 0.f, s2 = 0.f, fx[1], fd[1], g[1];
    Chunk<T, 1> qx, qd;
    for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
      qx.load(xr + c);
      qd.load(dr + c);
      qx.unpack(fx);
      qd.unpack(fd);
      load_weight<1>(a.gamma, a.w_bf16, c, 1.0f, g);
      s1 = fmaf(g[0], fd[0], s1);
      s2 = fmaf(g[0] * fd[0], (fx[0] - mean) * rstd, s2);
    }
    const float2 s = row_sum<WIDE_THREADS>(s1, s2, red[par]);
    par ^= 1;
    for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
      qx.load(xr + c);
      qd.load(dr + c);
      qx.unpack(fx);
      qd.unpack(fd);
      load_weight<1>(a.gamma, a.w_bf16, c, 1.0f, g);
      fx[0] = rstd * (fmaf(g[0], fd[0], -s.x * inv_d) - (fx[0] - mean) * rstd * (s.y * inv_d));
      Chunk<T, 1>::store(orow + c, fx);
    }
  }
}

// The weight gradients of wide rows: thread c of block (i, r) adds column c over the rows r,
// r + gridDim.y, ... and leaves the sums as partial row r.
template <typename T>
__global__ void __launch_bounds__(256) norm_wgrad_wide_kernel(const NormArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.d) return;
  float g = 0.f, b = 0.f, fx[1], fd[1];
  Chunk<T, 1> qx, qd;
  for (long long row = blockIdx.y; row < a.T; row += gridDim.y) {
    qx.load(static_cast<const T*>(a.x) + row * a.ldx + c);
    qd.load(static_cast<const T*>(a.dy) + row * a.lddy + c);
    qx.unpack(fx);
    qd.unpack(fd);
    g = fmaf(fd[0], (fx[0] - __ldg(a.mean + row)) * __ldg(a.rstd + row), g);
    b += fd[0];
  }
  float* pg = a.part + static_cast<size_t>(blockIdx.y) * 2 * a.d;
  pg[c] = g;
  pg[a.d + c] = b;
}

// out[c] = sum of the partials of column c, for both gradients: 32 columns a block, 32 threads a
// column that take every 32nd partial and are added in thread order.
__global__ void __launch_bounds__(1024) norm_partials_kernel(const float* __restrict__ part, int blocks, int d,
                                                             float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float acc[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + cx;  // of 2d: dgamma's, then dbeta's columns
  float s = 0.f;
  if (c < 2LL * d) {
#pragma unroll 10
    for (int r = ry; r < blocks; r += 32) s += __ldcs(part + static_cast<size_t>(r) * 2 * d + c);
  }
  acc[ry][cx] = s;
  __syncthreads();
  if (ry == 0 && c < 2LL * d) {
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) sum += acc[r][cx];
    float* out = c < d ? dgamma : dbeta;
    if (out != nullptr) out[c < d ? c : c - d] = sum;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

moe_status_t launched() {
  const cudaError_t err = cudaGetLastError();
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

template <typename T, int VB, int NCH, int TPR>
int launch_fwd_rows(const NormArgs& a, cudaStream_t s) {
  constexpr int ROWS = block_threads(TPR) / TPR;
  const int grid = static_cast<int>(std::min<long long>((static_cast<long long>(a.T) + ROWS - 1) / ROWS, 1 << 20));
  norm_fwd_kernel<T, VB, NCH, TPR><<<grid, block_threads(TPR), 0, s>>>(a);
  return grid;
}
template <typename T, int VB, int NCH, int TPR>
int launch_bwd_rows(const NormArgs& a, cudaStream_t s) {
  constexpr int ROWS = block_threads(TPR) / TPR;
  const int grid = static_cast<int>(std::min<long long>((static_cast<long long>(a.T) + ROWS - 1) / ROWS, BWD_MAX_BLOCKS));
  norm_bwd_kernel<T, VB, NCH, TPR><<<grid, block_threads(TPR), 0, s>>>(a);
  return grid;
}

// Threads per row and chunks (16 bytes, or one element) per thread. The functions return the blocks
// launched, 0 for a row wider than any layout.
// Forward: a warp a row up to eight chunks a lane; fewer rows than four for each SM take four
// warps a row from three chunks a lane on, for latency.
template <typename T, int VB, int U>
int fwd_by_width(const NormArgs& a, cudaStream_t s) {
  const int chunks = (a.d + VB - 1) / VB;
  const bool few = a.T <= 608;
  if (chunks <= 32 * U) return launch_fwd_rows<T, VB, U, 32>(a, s);
  if (chunks <= 64 * U) return launch_fwd_rows<T, VB, 2 * U, 32>(a, s);
  if (few && chunks <= 256 * U) return launch_fwd_rows<T, VB, 2 * U, 128>(a, s);
  if (chunks <= 128 * U) return launch_fwd_rows<T, VB, 4 * U, 32>(a, s);
  if (U == 1 && chunks <= 256) return launch_fwd_rows<T, VB, 8, 32>(a, s);
  if (chunks <= 512 * U) return launch_fwd_rows<T, VB, 4 * U, 128>(a, s);
  if (chunks <= 1024 * U) return launch_fwd_rows<T, VB, 2 * U, 512>(a, s);
  if (chunks <= 2048 * U) return launch_fwd_rows<T, VB, 4 * U, 512>(a, s);
  return 0;
}
// Backward: one chunk a thread (four elements without alignment) as long as a block has the threads.
template <typename T, int VB, int U>
int bwd_by_width(const NormArgs& a, cudaStream_t s) {
  const int chunks = (a.d + VB - 1) / VB;
  if (chunks <= 32 * U) return launch_bwd_rows<T, VB, U, 32>(a, s);
  if (chunks <= 64 * U) return launch_bwd_rows<T, VB, 2 * U, 32>(a, s);
  if (chunks <= 128 * U) return launch_bwd_rows<T, VB, U, 128>(a, s);
  if (chunks <= 256 * U) return launch_bwd_rows<T, VB, U, 256>(a, s);
  if (chunks <= 512 * U) return launch_bwd_rows<T, VB, U, 512>(a, s);
  if (chunks <= 1024 * U) return launch_bwd_rows<T, VB, U, 1024>(a, s);
  if (U == 1 && chunks <= 2048) return launch_bwd_rows<T, VB, 4, 512>(a, s);
  return 0;
}

template <typename T>
int launch_norm(const NormArgs& a, bool bwd, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int grid = bwd ? (vec ? bwd_by_width<T, V, 1>(a, s) : bwd_by_width<T, 1, 4>(a, s))
                       : (vec ? fwd_by_width<T, V, 1>(a, s) : fwd_by_width<T, 1, 4>(a, s));
  if (grid > 0) return grid;
  const int wide = static_cast<int>(std::min<long long>(a.T, 1 << 20));
  if (!bwd) {
    norm_fwd_wide_kernel<T><<<wide, WIDE_THREADS, 0, s>>>(a);
    return wide;
  }
  norm_bwd_wide_kernel<T><<<wide, WIDE_THREADS, 0, s>>>(a);
  const int parts = std::min(a.T, BWD_MAX_BLOCKS);
  if (a.part != nullptr)
    norm_wgrad_wide_kernel<T><<<dim3((a.d + 255) / 256, parts), 256, 0, s>>>(a);
  return parts;
}

bool dtype_ok(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F32; }
int dtype_bytes(int t) { return t == MOE_DTYPE_BF16 ? 2 : 4; }
bool element_aligned(const void* p, int es) { return (reinterpret_cast<uintptr_t>(p) & (es - 1)) == 0; }

}  // namespace

size_t layer_norm_bwd_workspace_bytes(int T, int d) {
  if (T < 0 || d < 1 || d > MAX_WIDTH) return 0;
  return static_cast<size_t>(std::min(T, BWD_MAX_BLOCKS)) * 2 * d * sizeof(float);
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_layer_norm_fwd(const void* x, int dtype, long long ldx, const void* gamma, const void* beta,
                                int w_dtype, int T, int d, float eps, void* y, long long ldy, float* mean,
                                float* rstd, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (T < 0 || d <= 0 || ldx < 0 || ldy < d || !dtype_ok(dtype) || !dtype_ok(w_dtype)) return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || std::isinf(eps)) return MOE_ERR_INVALID_ARG;
  if (d > MAX_WIDTH) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && (!x || !y)) return MOE_ERR_INVALID_ARG;
  const int es = dtype_bytes(dtype), ws = dtype_bytes(w_dtype);
  if (!element_aligned(x, es) || !element_aligned(y, es) || !element_aligned(gamma, ws) || !element_aligned(beta, ws) ||
      !element_aligned(mean, 4) || !element_aligned(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = check_device();
  if (st != MOE_OK || T == 0) return st;
  NormArgs a{};
  a.x = x;
  a.out = y;
  a.ldx = ldx;
  a.ldo = ldy;
  a.gamma = gamma;
  a.beta = beta;
  a.w_bf16 = w_dtype == MOE_DTYPE_BF16;
  a.T = T;
  a.d = d;
  a.eps = eps;
  a.mean = mean;
  a.rstd = rstd;
  const int v = 16 / es;
  const bool vec = d % v == 0 && ldx % v == 0 && ldy % v == 0 && aligned16(x) && aligned16(y) && aligned16(gamma) &&
                   aligned16(beta);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MOE_DTYPE_BF16) launch_norm<bf16>(a, false, vec, s);
  else launch_norm<float>(a, false, vec, s);
  return launched();
}

moe_status_t moe_layer_norm_bwd(const void* dy, long long lddy, const void* x, long long ldx, int dtype,
                                const void* gamma, int w_dtype, const float* mean, const float* rstd, int T, int d,
                                void* dx, long long lddx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                                moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (T < 0 || d <= 0 || ldx < 0 || lddy < 0 || lddx < d || !dtype_ok(dtype) || !dtype_ok(w_dtype))
    return MOE_ERR_INVALID_ARG;
  if (d > MAX_WIDTH) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && (!x || !dy || !dx || !mean || !rstd)) return MOE_ERR_INVALID_ARG;
  const int es = dtype_bytes(dtype);
  if (!element_aligned(x, es) || !element_aligned(dy, es) || !element_aligned(dx, es) ||
      !element_aligned(gamma, dtype_bytes(w_dtype)) || !element_aligned(mean, 4) || !element_aligned(rstd, 4) ||
      !element_aligned(dgamma, 4) || !element_aligned(dbeta, 4) || !element_aligned(ws, 4))
    return MOE_ERR_INVALID_ARG;
  const bool wgrad = dgamma != nullptr || dbeta != nullptr;
  if (wgrad && T > 0) {
    if (ws_bytes < layer_norm_bwd_workspace_bytes(T, d)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!ws) return MOE_ERR_INVALID_ARG;
  }
  moe_status_t st = check_device();
  if (st != MOE_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int blocks = 0;
  if (T > 0) {
    NormArgs a{};
    a.x = x;
    a.dy = dy;
    a.out = dx;
    a.ldx = ldx;
    a.lddy = lddy;
    a.ldo = lddx;
    a.gamma = gamma;
    a.w_bf16 = w_dtype == MOE_DTYPE_BF16;
    a.T = T;
    a.d = d;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.part = wgrad ? static_cast<float*>(ws) : nullptr;
    const int v = 16 / es;
    const bool vec = d % v == 0 && ldx % v == 0 && lddy % v == 0 && lddx % v == 0 && aligned16(x) && aligned16(dy) &&
                     aligned16(dx) && aligned16(gamma);
    blocks = dtype == MOE_DTYPE_BF16 ? launch_norm<bf16>(a, true, vec, s) : launch_norm<float>(a, true, vec, s);
    if ((st = launched()) != MOE_OK) return st;
  }
  if (!wgrad) return MOE_OK;
  norm_partials_kernel<<<(2 * d + 31) / 32, 1024, 0, s>>>(static_cast<const float*>(ws), blocks, d, dgamma, dbeta);
  return launched();
}

}  // extern "C"
