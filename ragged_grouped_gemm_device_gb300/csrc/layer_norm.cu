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
// once. A block works on one row after another: the weights (and the backward's gradient sums) stay
// in its registers, and the next rows are on their way into shared memory by asynchronous
// copies. Each thread copies exactly the chunks that it will read, so the ring needs no barrier;
// what it is for is bytes in flight, which registers cannot hold (with one row of prefetch in
// registers the backward took 47 us for 16384 x 2048 bf16, 34.6 now: 5.8 TB/s; the forward 20.9: 6.4).
// The weight gradients are sums over all rows: each block adds the rows it owns in registers (a
// thread always owns the same columns), leaves one partial row of each gradient in the workspace,
// and a second small kernel adds the partials in block order. No atomics: the results do not
// depend on scheduling.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "trace.h"

namespace moe {
namespace {

// Rows of partial weight gradients at most: four for each of the 152 SMs. A constant, because the
// size of the workspace is host arithmetic.
constexpr int BWD_MAX_BLOCKS = 608;
constexpr int MAX_WIDTH = 1 << 20;

// Blocks on an SM, which size the grids and bound the registers. Forward: 768 threads (16384 x 2048
// bf16: 20.8 us, the speed of a copy; 27 us with 1024, which spill). Backward: 384 threads with two
// chunks each (34.6 us, on 512 threads 35.8; at a time when it took 41.5, one chunk each on 512
// threads took 44, on 1024 threads 54: each row's reduction and addresses cost a warp as much as
// its chunks).
constexpr int fwd_blocks_per_sm(int tpr) { return tpr >= 512 ? 1 : 768 / block_threads(tpr); }
constexpr int bwd_blocks_per_sm(int tpr) { return tpr <= 128 ? 3 : tpr == 256 ? 2 : 1; }

// The chunks of one thread in the next rows of NT tensors (x; x and dy). 16-byte rows: a ring of
// asynchronous copies in shared memory; rows of single elements: one row ahead in registers. The
// row pointers advance by a constant, so that a row costs few address instructions.
template <typename T, int VB, int NCH, int TPR, int NT>
struct Feed {
  static constexpr bool ring = VB > 1;
  static constexpr int piece = block_threads(TPR) * 16;  // one chunk of every thread
  static constexpr int slot_bytes = NT * NCH * piece;
  static constexpr int depth = !ring ? 1 : slot_bytes <= 32 * 1024 ? 4 : 2;  // rows on their way
  static constexpr int smem_bytes = ring ? depth * slot_bytes : 0;
  Chunk<T, VB> q[NT][NCH];
  const T* at[NT];       // the next row to start
  long long step[NT];    // elements from one row of this block to its next
  int c0;                // this thread's first column
  uint32_t base, slot;   // shared-memory address of this thread, byte offset of the oldest row
  int left;              // rows not started yet
  bool in[NCH];

  __device__ __forceinline__ void init(uint8_t* smem, int t, int d, int rows) {
    if constexpr (ring) base = smem_u32(smem) + threadIdx.x * 16;
    slot = 0;
    left = rows;
    c0 = t * VB;
#pragma unroll
    for (int i = 0; i < NCH; ++i) in[i] = (i * TPR + t) * VB < d;
  }
  // start the copies of the next row into the slot at byte offset `to` (past the last row: none,
  // but a group of copies all the same)
  __device__ __forceinline__ void start(uint32_t to) {
    if (left > 0) {
#pragma unroll
      for (int k = 0; k < NT; ++k) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          if (!in[i]) continue;
          if constexpr (ring) copy16_async(base + to + (k * NCH + i) * piece, at[k] + c0 + i * (TPR * VB));
          else q[k][i].load(at[k] + c0 + i * (TPR * VB));
        }
        at[k] += step[k];
      }
      --left;
    }
    if constexpr (ring) copy_commit();
  }
  __device__ __forceinline__ void prime() {
#pragma unroll
    for (int s = 0; s < depth; ++s) start(s * slot_bytes);
  }
  // the oldest row's copies have landed: its chunks into q
  __device__ __forceinline__ void take() {
    if constexpr (ring) {
      copy_wait<depth - 1>();
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int i = 0; i < NCH; ++i)
          if (in[i]) q[k][i].from_shared(base + slot + (k * NCH + i) * piece);
    }
  }
  // q has been unpacked: start the row that takes its place
  __device__ __forceinline__ void next() {
    start(slot);
    slot = slot == (depth - 1) * slot_bytes ? 0 : slot + slot_bytes;
  }
};

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

template <typename T, int VB, int NCH, int TPR>
__global__ void __launch_bounds__(block_threads(TPR), fwd_blocks_per_sm(TPR)) norm_fwd_kernel(const NormArgs a) {
  grid_wait();
  constexpr int ROWS = block_threads(TPR) / TPR;
  __shared__ __align__(16) float red[2][32];
  const int t = ROWS > 1 ? threadIdx.x % TPR : threadIdx.x;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float g[NCH][VB], b[NCH][VB];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * TPR + t) * VB;
    if (c < a.d) {
      load_weight<VB>(after_wait(a.gamma), a.w_bf16, c, 1.0f, g[i]);
      load_weight<VB>(after_wait(a.beta), a.w_bf16, c, 0.0f, b[i]);
    }
  }
  extern __shared__ __align__(16) uint8_t ring[];
  Feed<T, VB, NCH, TPR, 1> feed;
  const int row0 = blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / TPR : 0), step = gridDim.x * ROWS;
  const int rows = row0 < a.T ? (a.T - 1 - row0) / step + 1 : 0;
  feed.init(ring, t, a.d, rows);
  feed.at[0] = static_cast<const T*>(after_wait(a.x)) + row0 * a.ldx;
  feed.step[0] = step * a.ldx;
  feed.prime();
  T* yr = static_cast<T*>(a.out) + row0 * a.ldo;
  const long long ystep = step * a.ldo;
  for (int k = 0; k < rows; ++k, yr += ystep) {
    float f[NCH][VB];
    float sum = 0.f;
    feed.take();
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (feed.in[i]) feed.q[0][i].unpack(f[i]);
    feed.next();
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (!feed.in[i]) continue;
#pragma unroll
      for (int j = 0; j < VB; ++j) sum += f[i][j];
    }
    const float mean = row_sum<TPR>(sum, red[0]) * inv_d;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (!feed.in[i]) continue;
#pragma unroll
      for (int j = 0; j < VB; ++j) {
        f[i][j] -= mean;
        sq = fmaf(f[i][j], f[i][j], sq);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(sq, red[1]) * inv_d + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row0 + static_cast<long long>(k) * step] = mean;
      if (a.rstd) a.rstd[row0 + static_cast<long long>(k) * step] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (!feed.in[i]) continue;
#pragma unroll
      for (int j = 0; j < VB; ++j) f[i][j] = fmaf(f[i][j] * rstd, g[i][j], b[i][j]);
      Chunk<T, VB>::store(yr + feed.c0 + i * (TPR * VB), f[i]);
    }
  }
}

template <typename T, int VB, int NCH, int TPR>
__global__ void __launch_bounds__(block_threads(TPR), bwd_blocks_per_sm(TPR)) norm_bwd_kernel(const NormArgs a) {
  grid_wait();
  constexpr int ROWS = block_threads(TPR) / TPR;
  __shared__ __align__(16) float red[2][64];
  const int t = ROWS > 1 ? threadIdx.x % TPR : threadIdx.x;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float dg[NCH][VB], db[NCH][VB], g[NCH][VB];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * TPR + t) * VB;
    if (c < a.d) load_weight<VB>(after_wait(a.gamma), a.w_bf16, c, 1.0f, g[i]);
#pragma unroll
    for (int j = 0; j < VB; ++j) dg[i][j] = db[i][j] = 0.f;
  }
  extern __shared__ __align__(16) uint8_t ring[];
  Feed<T, VB, NCH, TPR, 2> feed;
  const int row0 = blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / TPR : 0), step = gridDim.x * ROWS;
  const int rows = row0 < a.T ? (a.T - 1 - row0) / step + 1 : 0;
  feed.init(ring, t, a.d, rows);
  feed.at[0] = static_cast<const T*>(after_wait(a.x)) + row0 * a.ldx;
  feed.step[0] = step * a.ldx;
  feed.at[1] = static_cast<const T*>(after_wait(a.dy)) + row0 * a.lddy;
  feed.step[1] = step * a.lddy;
  feed.prime();
  T* orow = static_cast<T*>(a.out) + row0 * a.ldo;
  const long long ostep = step * a.ldo;
  // lane l holds the statistics of rows l, l + 32, ... of this block: one wait in 32 rows
  const int lane = threadIdx.x & 31;
  float mean32 = 0.f, rstd32 = 0.f;
  int par = 0;
  for (int k = 0; k < rows; ++k, orow += ostep) {
    float xh[NCH][VB], gd[NCH][VB];  // xhat, and dy, then gamma dy
    float s1 = 0.f, s2 = 0.f;
    if ((k & 31) == 0 && k + lane < rows) {
      mean32 = __ldg(after_wait(a.mean) + row0 + static_cast<long long>(k + lane) * step);
      rstd32 = __ldg(after_wait(a.rstd) + row0 + static_cast<long long>(k + lane) * step);
    }
    const float mu = __shfl_sync(0xffffffffu, mean32, k & 31), rs = __shfl_sync(0xffffffffu, rstd32, k & 31);
    feed.take();
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (feed.in[i]) {
        feed.q[0][i].unpack(xh[i]);
        feed.q[1][i].unpack(gd[i]);
      }
    feed.next();
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (!feed.in[i]) continue;
#pragma unroll
      for (int j = 0; j < VB; ++j) {
        xh[i][j] = (xh[i][j] - mu) * rs;
        dg[i][j] = fmaf(gd[i][j], xh[i][j], dg[i][j]);
        db[i][j] += gd[i][j];
        gd[i][j] *= g[i][j];
        s1 += gd[i][j];
        s2 = fmaf(gd[i][j], xh[i][j], s2);
      }
    }
    const float2 s = row_sum<TPR>(s1, s2, red[par]);
    par ^= 1;
    // dx = rstd (gd - m1 - xhat m2)
    const float m1 = s.x * inv_d, m2 = s.y * inv_d;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (!feed.in[i]) continue;
#pragma unroll
      for (int j = 0; j < VB; ++j) xh[i][j] = rs * (gd[i][j] - m1 - xh[i][j] * m2);
      Chunk<T, VB>::store(orow + feed.c0 + i * (TPR * VB), xh[i]);
    }
  }
  if (a.part == nullptr) return;
  float* pg = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
  float* pb = pg + a.d;
  // a block of several rows: its warps own the same columns; they are added in warp order
  __shared__ float2 acc[ROWS > 1 ? ROWS - 1 : 1][32];
  const int w = threadIdx.x / TPR;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    if constexpr (ROWS > 1) {
#pragma unroll
      for (int j = 0; j < VB; ++j) {
        __syncthreads();
        if (w > 0) acc[w - 1][t] = make_float2(dg[i][j], db[i][j]);
        __syncthreads();
        if (w == 0) {
#pragma unroll
          for (int r = 0; r < ROWS - 1; ++r) {
            dg[i][j] += acc[r][t].x;
            db[i][j] += acc[r][t].y;
          }
        }
      }
    }
    const int c = (i * TPR + t) * VB;
    if (w != 0 || c >= a.d) continue;
    if constexpr (VB > 1) {  // d is a multiple of VB: 16-byte rows of partials (one float at a time: 40 us, not 34.6)
#pragma unroll
      for (int j = 0; j < VB; j += 4) {
        *reinterpret_cast<float4*>(pg + c + j) = make_float4(dg[i][j], dg[i][j + 1], dg[i][j + 2], dg[i][j + 3]);
        *reinterpret_cast<float4*>(pb + c + j) = make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
      }
    } else {
      pg[c] = dg[i][0];
      pb[c] = db[i][0];
    }
  }
}

// Rows too wide for registers: three passes over the row (the later ones from L2), one block a row.
constexpr int WIDE_THREADS = 1024;

template <typename T>
__global__ void __launch_bounds__(WIDE_THREADS) norm_fwd_wide_kernel(const NormArgs a) {
  __shared__ __align__(16) float red[2][32];
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
    const float mean = row_sum<WIDE_THREADS>(s, red[0]) * inv_d;
    s = 0.f;
    for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
      q.load(xr + c);
      q.unpack(f);
      s = fmaf(f[0] - mean, f[0] - mean, s);
    }
    const float rstd = 1.0f / sqrtf(row_sum<WIDE_THREADS>(s, red[1]) * inv_d + a.eps);
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
  __shared__ __align__(16) float red[2][64];
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
__global__ void __launch_bounds__(1024) norm_partials_kernel(const float* part, int blocks, int d,
                                                             float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float acc[32][33];
  grid_wait();  // launched ahead of the end of the kernel that writes the partials
  part = after_wait(part);
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + cx;  // of 2d: dgamma's, then dbeta's columns
  // every load at once (a loop of a run-time length waits for each round of them)
  constexpr int ROUNDS = (BWD_MAX_BLOCKS + 31) / 32;
  float v[ROUNDS], s = 0.f;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int r = ry + 32 * i;
    v[i] = r < blocks && c < 2LL * d ? __ldcs(part + static_cast<size_t>(r) * 2 * d + c) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) s += v[i];
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

// The launches below leave the blocks launched in `grid`.
template <typename T, int VB, int NCH, int TPR>
cudaError_t launch_fwd_rows(const NormArgs& a, cudaStream_t s, int& grid) {
  constexpr int ROWS = block_threads(TPR) / TPR;
  const long long most = fwd_blocks_per_sm(TPR) * static_cast<long long>(device_sm_count());
  grid = static_cast<int>(std::min<long long>((static_cast<long long>(a.T) + ROWS - 1) / ROWS, most));
  constexpr int smem = Feed<T, VB, NCH, TPR, 1>::smem_bytes;
  if (smem > 48 * 1024) {
    const cudaError_t err = ensure_max_dynamic_smem(reinterpret_cast<const void*>(norm_fwd_kernel<T, VB, NCH, TPR>), smem);
    if (err != cudaSuccess) return err;
  }
  return launch_dependent(norm_fwd_kernel<T, VB, NCH, TPR>, grid, block_threads(TPR), smem, s, a);
}
template <typename T, int VB, int NCH, int TPR>
cudaError_t launch_bwd_rows(const NormArgs& a, cudaStream_t s, int& grid) {
  constexpr int ROWS = block_threads(TPR) / TPR;
  grid = static_cast<int>(std::min<long long>((static_cast<long long>(a.T) + ROWS - 1) / ROWS, std::min(bwd_blocks_per_sm(TPR) * device_sm_count(), BWD_MAX_BLOCKS)));
  constexpr int smem = Feed<T, VB, NCH, TPR, 2>::smem_bytes;
  if (smem > 48 * 1024) {
    const cudaError_t err = ensure_max_dynamic_smem(reinterpret_cast<const void*>(norm_bwd_kernel<T, VB, NCH, TPR>), smem);
    if (err != cudaSuccess) return err;
  }
  return launch_dependent(norm_bwd_kernel<T, VB, NCH, TPR>, grid, block_threads(TPR), smem, s, a);
}

// Threads per row and chunks (16 bytes, or one element) per thread. A row wider than any layout launches
// nothing and leaves `grid` 0.
// Forward: two chunks a thread (eight elements without alignment), so that a row takes few warps.
template <typename T, int VB, int U>
cudaError_t fwd_by_width(const NormArgs& a, cudaStream_t s, int& grid) {
  const int chunks = (a.d + VB - 1) / VB;
  if (chunks <= 32 * U) return launch_fwd_rows<T, VB, U, 32>(a, s, grid);
  if (chunks <= 64 * U) return launch_fwd_rows<T, VB, 2 * U, 32>(a, s, grid);
  if (chunks <= 128 * U) return launch_fwd_rows<T, VB, U, 128>(a, s, grid);
  if (chunks <= 256 * U) return launch_fwd_rows<T, VB, 2 * U, 128>(a, s, grid);
  if (chunks <= 512 * U) return launch_fwd_rows<T, VB, 2 * U, 256>(a, s, grid);
  if (chunks <= 1024 * U) return launch_fwd_rows<T, VB, 2 * U, 512>(a, s, grid);
  if (chunks <= 2048 * U) return launch_fwd_rows<T, VB, 2 * U, 1024>(a, s, grid);
  grid = 0;
  return cudaSuccess;
}
// Backward: the same.
template <typename T, int VB, int U>
cudaError_t bwd_by_width(const NormArgs& a, cudaStream_t s, int& grid) {
  const int chunks = (a.d + VB - 1) / VB;
  if (chunks <= 32 * U) return launch_bwd_rows<T, VB, U, 32>(a, s, grid);
  if (chunks <= 64 * U) return launch_bwd_rows<T, VB, 2 * U, 32>(a, s, grid);
  if (chunks <= 128 * U) return launch_bwd_rows<T, VB, U, 128>(a, s, grid);
  if (chunks <= 256 * U) return launch_bwd_rows<T, VB, 2 * U, 128>(a, s, grid);
  if (chunks <= 512 * U) return launch_bwd_rows<T, VB, 2 * U, 256>(a, s, grid);
  if (chunks <= 1024 * U) return launch_bwd_rows<T, VB, 2 * U, 512>(a, s, grid);
  if (chunks <= 2048 * U) return launch_bwd_rows<T, VB, 4 * U, 512>(a, s, grid);
  grid = 0;
  return cudaSuccess;
}

// `grid`: the blocks launched, or the rows of partial weight gradients that they leave
template <typename T>
cudaError_t launch_norm(const NormArgs& a, bool bwd, bool vec, cudaStream_t s, int& grid) {
  constexpr int V = 16 / sizeof(T);
  const cudaError_t err = bwd ? (vec ? bwd_by_width<T, V, 1>(a, s, grid) : bwd_by_width<T, 1, 4>(a, s, grid))
                              : (vec ? fwd_by_width<T, V, 1>(a, s, grid) : fwd_by_width<T, 1, 4>(a, s, grid));
  if (err != cudaSuccess || grid > 0) return err;
  const int wide = static_cast<int>(std::min<long long>(a.T, 1 << 20));
  if (!bwd) {
    norm_fwd_wide_kernel<T><<<wide, WIDE_THREADS, 0, s>>>(a);
    return cudaGetLastError();
  }
  // the weight gradients first: dx may lie over x or dy
  grid = std::min(a.T, BWD_MAX_BLOCKS);
  if (a.part != nullptr)
    norm_wgrad_wide_kernel<T><<<dim3((a.d + 255) / 256, grid), 256, 0, s>>>(a);
  norm_bwd_wide_kernel<T><<<wide, WIDE_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

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
  int blocks = 0;
  const cudaError_t err = dtype == MOE_DTYPE_BF16 ? launch_norm<bf16>(a, false, vec, s, blocks)
                                                  : launch_norm<float>(a, false, vec, s, blocks);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
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
    const bool vec = d % v == 0 && ldx % v == 0 && lddy % v == 0 && lddx % v == 0 && aligned16(ws) && aligned16(x) && aligned16(dy) &&
                     aligned16(dx) && aligned16(gamma);
    const cudaError_t err = dtype == MOE_DTYPE_BF16 ? launch_norm<bf16>(a, true, vec, s, blocks)
                                                    : launch_norm<float>(a, true, vec, s, blocks);
    if (err != cudaSuccess) return cuda_fail(err);
  }
  if (!wgrad) return MOE_OK;
  const cudaError_t err = launch_dependent(norm_partials_kernel, (2 * d + 31) / 32, 1024, 0, s,
                                           static_cast<const float*>(ws), blocks, d, dgamma, dbeta);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

}  // extern "C"
