// What stands between two blocks, in one pass: the norm behind a block, its gate and scale, the residual
// addition and the norm in front of the next block.
//
//   z = post(y);  r = alpha x + beta gate z;  n = pre(r),  post and pre: none, layer norm or RMS norm
//   D = dr + pre'(dn);  dx = alpha D;  dz = beta gate D;  dy = post'(dz)
//
// With yhat = (y - mean1) rstd1 and rhat = (r - mean2) rstd2 (mean 0 for RMS), every weight gradient comes
// from four sums over the rows:  S1 = sum D yhat, S0 = sum D, P1 = sum dn rhat, P0 = sum dn:
//   d_post_gamma = beta gate S1;  d_post_beta = beta gate S0;  d_gate = beta (post_gamma S1 + post_beta S0)
//   d_pre_gamma = P1;  d_pre_beta = P0
// Each block of rows leaves one partial row of each sum in the workspace; a second kernel adds them in
// block order. No atomics: the results do not depend on scheduling.
//
// Bound by memory: the forward reads x and y and writes r and n, the backward reads dn, r, dr and y and writes dx and dy, each
// once (8 and 12 bytes an element of bf16). 16384 x 2048 bf16: forward 44 us (6.05 TB/s), backward with every weight gradient 77
// us (5.25 TB/s), of which the sum of the partials 6. 16 x 2048: 3 us, a launch and a round trip to memory.
#include <algorithm>
#include <cmath>
#include <tuple>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "trace.h"

namespace moe {
namespace {

// Rows of partial weight gradients at most: four for each of the 152 SMs. A constant, because the size of
// the workspace is host arithmetic.
constexpr int BWD_MAX_BLOCKS = 608;
constexpr int MAX_WIDTH = 1 << 20;
constexpr int SUMS = 4;

struct JoinArgs {
  const void* x;   // forward
  const void* y;   // nullable: no branch
  void* r;         // forward: nullable output; backward: input
  void* n;         // forward: nullable output
  const void* dn;  // backward, nullable
  const void* dr;  // backward, nullable
  void* dx;        // backward, nullable outputs
  void* dy;
  long long ldx, ldy, ldr, ldn, lddn, lddr, lddx, lddy;
  const void* g1;    // post gamma, post beta, gate, pre gamma, pre beta: nullable
  const void* b1;
  const void* gate;
  const void* g2;
  const void* b2;
  bool w_bf16;
  int post, pre;
  int T, d;
  float eps, alpha, beta;
  float* stats;  // [4][T]: forward nullable outputs, backward inputs
  float* part;   // backward: [blocks][4][d] partial sums (nullable: not wanted)
  float* row;    // backward of wide rows: [T][2] means of the pre norm's gradient
};

// ------------------------------------------------------------------ rows of any width
// Rows wider than 8192: one block a row, single elements, one pass over the row for each reduction (the later ones from L2), bound by
// the instructions of single elements (2048 x 10000 bf16, RMS norms and gate: forward 181 us, backward with every gradient 466).
constexpr int WIDE_THREADS = 512;

template <typename T>
__device__ __forceinline__ float get(const T* p) {
  Chunk<T, 1> q;
  float f[1];
  q.load(p);
  q.unpack(f);
  return f[0];
}
template <typename T>
__device__ __forceinline__ float rounded(float v) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(__float2bfloat16_rn(v));
  else return v;
}
template <typename T>
__device__ __forceinline__ void put(T* p, float v) {
  const float f[1] = {v};
  Chunk<T, 1>::store(p, f);
}
__device__ __forceinline__ float weight(const void* w, bool w_bf16, int c, float fill) {
  float o[1];
  load_weight<1>(w, w_bf16, c, fill, o);
  return o[0];
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(WIDE_THREADS) join_fwd_wide_kernel(const JoinArgs a) {
  __shared__ __align__(16) float red[2][32];
  const float inv_d = 1.0f / static_cast<float>(a.d);
  int par = 0;
  const auto sum = [&](float v) {
    const float s = row_sum<WIDE_THREADS>(v, red[par]);
    par ^= 1;
    return s;
  };
  for (long long row = blockIdx.x; row < a.T; row += gridDim.x) {
    const TX* x = static_cast<const TX*>(a.x) + row * a.ldx;
    const TY* y = a.y ? static_cast<const TY*>(a.y) + row * a.ldy : nullptr;
    TX* r = a.r ? static_cast<TX*>(a.r) + row * a.ldr : nullptr;
    float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f, s = 0.f;
    if (a.post == MOE_NORM_LAYER) {
      for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) s += get(y + c);
      mean1 = sum(s) * inv_d;
    }
    if (a.post != MOE_NORM_NONE) {
      s = 0.f;
      for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
        const float v = get(y + c) - mean1;
        s = fmaf(v, v, s);
      }
      rstd1 = 1.0f / sqrtf(sum(s) * inv_d + a.eps);
    }
    // the row as it is stored
    const auto joined = [&](int c) {
      float v = a.alpha * get(x + c);
      if (y != nullptr) {
        const float z = fmaf((get(y + c) - mean1) * rstd1, weight(a.g1, a.w_bf16, c, 1.f), weight(a.b1, a.w_bf16, c, 0.f));
        v = fmaf(a.beta * weight(a.gate, a.w_bf16, c, 1.f), z, v);
      }
      return rounded<TX>(v);
    };
    s = 0.f;
    if (r != nullptr || a.pre == MOE_NORM_LAYER) {
      for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
        const float v = joined(c);
        if (r != nullptr) put(r + c, v);
        s += v;
      }
    }
    const auto again = [&](int c) { return r != nullptr ? get(r + c) : joined(c); };  // r may lie over x
    if (a.pre == MOE_NORM_LAYER) mean2 = sum(s) * inv_d;
    if (a.pre != MOE_NORM_NONE) {
      s = 0.f;
      for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
        const float v = again(c) - mean2;
        s = fmaf(v, v, s);
      }
      rstd2 = 1.0f / sqrtf(sum(s) * inv_d + a.eps);
      for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS)
        put(static_cast<TY*>(a.n) + row * a.ldn + c,
            fmaf((again(c) - mean2) * rstd2, weight(a.g2, a.w_bf16, c, 1.f), weight(a.b2, a.w_bf16, c, 0.f)));
    }
    if (threadIdx.x == 0 && a.stats != nullptr) {
      const size_t T = a.T;
      a.stats[row] = mean1;
      a.stats[T + row] = rstd1;
      a.stats[2 * T + row] = mean2;
      a.stats[3 * T + row] = rstd2;
    }
  }
}

// What the backward reads of one row
template <typename TX, typename TY>
struct WideRow {
  const TY *dn, *y;
  const TX *dr, *r;
  float mean1, rstd1, mean2, rstd2, m1, m2;
  __device__ __forceinline__ WideRow(const JoinArgs& a, long long row) {
    dn = a.dn ? static_cast<const TY*>(a.dn) + row * a.lddn : nullptr;
    y = a.y ? static_cast<const TY*>(a.y) + row * a.ldy : nullptr;
    dr = a.dr ? static_cast<const TX*>(a.dr) + row * a.lddr : nullptr;
    r = a.r ? static_cast<const TX*>(a.r) + row * a.ldr : nullptr;
    const size_t T = a.T;
    mean1 = a.post == MOE_NORM_LAYER ? __ldg(a.stats + row) : 0.f;
    rstd1 = a.post != MOE_NORM_NONE ? __ldg(a.stats + T + row) : 1.f;
    mean2 = a.pre == MOE_NORM_LAYER ? __ldg(a.stats + 2 * T + row) : 0.f;
    rstd2 = a.pre != MOE_NORM_NONE ? __ldg(a.stats + 3 * T + row) : 1.f;
  }
  __device__ __forceinline__ float rhat(int c) const { return (get(r + c) - mean2) * rstd2; }
  __device__ __forceinline__ float yhat(int c) const { return (get(y + c) - mean1) * rstd1; }
  // the gradient of r, with the means m1 and m2 of the pre norm's gradient
  __device__ __forceinline__ float grad(const JoinArgs& a, int c) const {
    float v = dr ? get(dr + c) : 0.f;
    if (a.pre != MOE_NORM_NONE) v += rstd2 * (weight(a.g2, a.w_bf16, c, 1.f) * get(dn + c) - m1 - rhat(c) * m2);
    return v;
  }
};

// The means of the pre norm's gradient, [T][2].
template <typename TX, typename TY>
__global__ void __launch_bounds__(WIDE_THREADS) join_bwd_means_kernel(const JoinArgs a) {
  __shared__ __align__(16) float red[2][64];
  int par = 0;
  for (long long row = blockIdx.x; row < a.T; row += gridDim.x) {
    const WideRow<TX, TY> w(a, row);
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
      const float g = weight(a.g2, a.w_bf16, c, 1.f) * get(w.dn + c);
      s1 += g;
      s2 = fmaf(g, w.rhat(c), s2);
    }
    const float2 s = row_sum<WIDE_THREADS>(s1, s2, red[par]);
    par ^= 1;
    if (threadIdx.x == 0) {
      a.row[2 * row] = a.pre == MOE_NORM_LAYER ? s.x / static_cast<float>(a.d) : 0.f;
      a.row[2 * row + 1] = s.y / static_cast<float>(a.d);
    }
  }
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(WIDE_THREADS) join_bwd_wide_kernel(const JoinArgs a) {
  __shared__ __align__(16) float red[2][64];
  const float inv_d = 1.0f / static_cast<float>(a.d);
  int par = 0;
  for (long long row = blockIdx.x; row < a.T; row += gridDim.x) {
    WideRow<TX, TY> w(a, row);
    w.m1 = a.pre != MOE_NORM_NONE ? a.row[2 * row] : 0.f;
    w.m2 = a.pre != MOE_NORM_NONE ? a.row[2 * row + 1] : 0.f;
    const auto branch = [&](int c) { return a.beta * weight(a.gate, a.w_bf16, c, 1.f) * weight(a.g1, a.w_bf16, c, 1.f); };
    float s1 = 0.f, s2 = 0.f;
    if (a.post != MOE_NORM_NONE) {
      for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
        const float g = branch(c) * w.grad(a, c);
        s1 += g;
        s2 = fmaf(g, w.yhat(c), s2);
      }
      const float2 s = row_sum<WIDE_THREADS>(s1, s2, red[par]);
      par ^= 1;
      s1 = a.post == MOE_NORM_LAYER ? s.x * inv_d : 0.f;
      s2 = s.y * inv_d;
    }
    for (int c = threadIdx.x; c < a.d; c += WIDE_THREADS) {
      const float D = w.grad(a, c);
      float g = 0.f;  // everything of this column is read before anything is written: dx and dy may lie over inputs
      if (w.y != nullptr) {
        g = branch(c) * D;
        if (a.post != MOE_NORM_NONE) g = w.rstd1 * (g - s1 - w.yhat(c) * s2);
      }
      if (a.dx != nullptr) put(static_cast<TX*>(a.dx) + row * a.lddx + c, a.alpha * D);
      if (w.y != nullptr) put(static_cast<TY*>(a.dy) + row * a.lddy + c, g);
    }
  }
}

// The four sums of wide rows: thread c of block (i, k) adds column c over the rows k, k + gridDim.y, ...
template <typename TX, typename TY>
__global__ void __launch_bounds__(256) join_wgrad_wide_kernel(const JoinArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.d) return;
  float s[SUMS] = {0.f, 0.f, 0.f, 0.f};
  for (long long row = blockIdx.y; row < a.T; row += gridDim.y) {
    WideRow<TX, TY> w(a, row);
    w.m1 = a.pre != MOE_NORM_NONE ? a.row[2 * row] : 0.f;
    w.m2 = a.pre != MOE_NORM_NONE ? a.row[2 * row + 1] : 0.f;
    if (w.y != nullptr) {
      const float D = w.grad(a, c);
      s[0] = fmaf(D, w.yhat(c), s[0]);
      s[1] += D;
    }
    if (a.pre != MOE_NORM_NONE) {
      const float g = get(w.dn + c);
      s[2] = fmaf(g, w.rhat(c), s[2]);
      s[3] += g;
    }
  }
#pragma unroll
  for (int k = 0; k < SUMS; ++k) a.part[(static_cast<size_t>(blockIdx.y) * SUMS + k) * a.d + c] = s[k];
}

// ------------------------------------------------------------------ rows in registers
// A row lies in the registers of its TPR threads, NCH chunks of eight elements each, so every value is read once and the
// variances are the exact two-pass ones. The rows to come are on their way into shared memory by asynchronous copies: a ring of
// `depth` rows that a thread (or, of fp32 tensors, a warp) fills for itself, so that it needs no barrier.
template <int NCH, int TPR, typename... Ts>
struct RowFeed {
  static constexpr int NT = sizeof...(Ts);
  static constexpr int threads = block_threads(TPR);
  __host__ __device__ static constexpr int size(int k) {
    constexpr int es[NT] = {static_cast<int>(sizeof(Ts))...};
    return es[k];
  }
  // bytes of a slot before tensor k
  __host__ __device__ static constexpr int before(int k) {
    int b = 0;
    for (int j = 0; j < k; ++j) b += NCH * threads * 8 * size(j);
    return b;
  }
  static constexpr int slot_bytes = before(NT);
  // Rows on their way: as many as leave room for the blocks of an SM. One, whose copies then start behind the row before, is left for the
  // backward of fp32 streams and branches wider than 4096 (4096 x 8192 with every gradient: 227 us, 119 for its bytes; 8192 x 4096
  // with two rows 132).
  static constexpr int depth = slot_bytes <= 16 * 1024 ? 4 : slot_bytes <= 32 * 1024 ? 3 : slot_bytes <= 96 * 1024 ? 2 : 1;
  static constexpr int smem_bytes = depth * slot_bytes;
  // A lane copies 16 bytes at a time: of bf16 rows its own chunk; of fp32 rows, whose chunks are 32 bytes, one quarter of
  // those of two lanes, so that a warp's accesses are contiguous. Its first address in the next row of each tensor:
  const uint8_t* at[NT];
  long long step[NT];     // bytes from one row of this block to its next
  bool on[NT];            // there is such a tensor
  bool in2[NCH], in4[NCH][2];  // what this lane copies lies in the row: of bf16, of fp32 rows
  uint32_t base, slot;    // shared-memory address of the ring, byte offset of the oldest row
  uint32_t own2, own4, get4;  // this lane's offsets: bf16 chunks, fp32 copies, fp32 chunks
  int c2, c4, left;       // first column that this lane copies of bf16 and of fp32 rows; rows not started yet

  __device__ __forceinline__ void init(uint8_t* smem, int t, int d, int rows) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x & ~31;
    base = smem_u32(smem);
    own2 = threadIdx.x * 16;
    own4 = warp * 32 + lane * 16;
    get4 = threadIdx.x * 32;
    c2 = t * 8;
    c4 = (t & ~31) * 8 + lane * 4;
    left = rows;
    slot = 0;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      in2[i] = c2 + i * TPR * 8 < d;
      in4[i][0] = c4 + i * TPR * 8 < d;
      in4[i][1] = c4 + i * TPR * 8 + 128 < d;
    }
  }
  __device__ __forceinline__ void tensor(int k, const void* p, long long ld, long long row0, int rows_step) {
    on[k] = p != nullptr;
    at[k] = static_cast<const uint8_t*>(p) + (row0 * ld + (size(k) == 2 ? c2 : c4)) * size(k);
    step[k] = rows_step * ld * size(k);
  }
  __device__ __forceinline__ void start(uint32_t to) {
    if (left > 0) {
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        if (!on[k]) continue;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const uint32_t chunk = base + to + before(k) + i * threads * 8 * size(k);
          const uint8_t* src = at[k] + i * TPR * 8 * size(k);
          if (size(k) == 2) {
            if (in2[i]) copy16_async(chunk + own2, src);
          } else {
            if (in4[i][0]) copy16_async(chunk + own4, src);
            if (in4[i][1]) copy16_async(chunk + own4 + 512, src + 512);
          }
        }
        at[k] += step[k];
      }
      --left;
    }
    copy_commit();
  }
  // What lies past the end of a row reads as zeros, so that the arithmetic need not ask.
  __device__ __forceinline__ void clear(uint32_t p) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(p), "r"(0) : "memory");
  }
  __device__ __forceinline__ void prime() {
    for (int s = 0; s < depth; ++s) {
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const uint32_t chunk = base + s * slot_bytes + before(k) + i * threads * 8 * size(k);
          if (size(k) == 2) {
            if (!in2[i] || !on[k]) clear(chunk + own2);
          } else {
            if (!in4[i][0] || !on[k]) clear(chunk + own4);
            if (!in4[i][1] || !on[k]) clear(chunk + own4 + 512);
          }
        }
    }
#pragma unroll
    for (int s = 0; s < depth; ++s) start(s * slot_bytes);
  }
  // the oldest row's copies have landed
  __device__ __forceinline__ void wait() {
    copy_wait<depth - 1>();
    __syncwarp();  // lanes copy for one another
  }
  template <int K>
  __device__ __forceinline__ void get(int i, float (&f)[8]) const {
    const uint32_t p = base + slot + before(K) + i * threads * 8 * size(K) + (size(K) == 2 ? own2 : get4);
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(p));
    if constexpr (size(K) == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_lo(w[j]);
        f[2 * j + 1] = bf16_hi(w[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(w[j]);
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]) : "r"(p + 16));
    }
  }
  // everything of the oldest row has been read: start the one that takes its place
  __device__ __forceinline__ void next() {
    __syncwarp();
    start(slot);
    slot = slot == (depth - 1) * slot_bytes ? 0 : slot + slot_bytes;
  }
};

// The same for rows that do not lie on the 16-byte grid: single elements from memory, neighbouring lanes neighbouring columns.
template <int NCH, int TPR, typename... Ts>
struct RowDirect {
  static constexpr int NT = sizeof...(Ts), smem_bytes = 0;
  const void* p[NT];
  long long ld[NT], row;
  int t, d, step;

  __device__ __forceinline__ void init(uint8_t*, int t_, int d_, int) {
    t = t_;
    d = d_;
  }
  __device__ __forceinline__ void tensor(int k, const void* p_, long long ld_, long long row0, int rows_step) {
    p[k] = p_;
    ld[k] = ld_;
    row = row0;
    step = rows_step;
  }
  __device__ __forceinline__ void prime() {}
  __device__ __forceinline__ void wait() {}
  __device__ __forceinline__ void next() { row += step; }
  template <int K>
  __device__ __forceinline__ void get(int i, float (&f)[8]) const {
    using T = std::tuple_element_t<K, std::tuple<Ts...>>;
    const T* at = static_cast<const T*>(p[K]) + row * ld[K];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = (i * 8 + j) * TPR + t;
      f[j] = p[K] != nullptr && c < d ? moe::get(at + c) : 0.f;
    }
  }
};
template <bool VEC, int NCH, int TPR, typename... Ts>
using Feed = std::conditional_t<VEC, RowFeed<NCH, TPR, Ts...>, RowDirect<NCH, TPR, Ts...>>;

// The column of element j of thread t's chunk i
template <bool VEC, int TPR>
__device__ __forceinline__ int column(int t, int i, int j) {
  return VEC ? (i * TPR + t) * 8 + j : (i * 8 + j) * TPR + t;
}
// Eight weights of a chunk, 0 past the row's end
template <bool VEC, int TPR>
__device__ __forceinline__ void weights8(const void* w, bool w_bf16, int t, int i, int d, float fill, float (&f)[8]) {
  if constexpr (VEC) {
    const int c = column<true, TPR>(t, i, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.f;
    if (c < d) load_weight<8>(w, w_bf16, c, fill, f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<false, TPR>(t, i, j);
      f[j] = c < d ? weight(w, w_bf16, c, fill) : 0.f;
    }
  }
}

__device__ __forceinline__ void put8(bf16* p, const float (&f)[8]) { Chunk<bf16, 8>::store(p, f); }
__device__ __forceinline__ void put8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ void pairs(const float (&f)[8], F2 (&p)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = pair(f[2 * j], f[2 * j + 1]);
}
// a chunk to its place in a row
template <bool VEC, int TPR, typename T>
__device__ __forceinline__ void put_chunk(T* row, int t, int i, int d, const float (&f)[8]) {
  if constexpr (VEC) {
    const int c = column<true, TPR>(t, i, 0);
    if (c < d) put8(row + c, f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<false, TPR>(t, i, j);
      if (c < d) put(row + c, f[j]);
    }
  }
}
template <bool VEC, int TPR, typename T>
__device__ __forceinline__ void put_chunk(T* row, int t, int i, int d, const F2 (&v)[4]) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 q = parts(v[j]);
    f[2 * j] = q.x;
    f[2 * j + 1] = q.y;
  }
  put_chunk<VEC, TPR>(row, t, i, d, f);
}

// Blocks on an SM, which size the grids and bound the registers. Forward: rows of 256 chunks go to 256 threads with one chunk each,
// three blocks, two with betas (16384 x 2048: 45.2 us, 47.5 with 128 threads of two chunks). Backward: the four sums over the rows take
// 32 registers a chunk, so such rows go to 128 threads of two chunks, three blocks (71 us without the sum of the partials; 256 threads
// of one chunk 77, four blocks 217, because they spill).
constexpr int fwd_blocks(int tpr, int nch, bool bias) { return tpr == 256 && nch == 1 ? (bias ? 2 : 3) : 512 / block_threads(tpr); }
constexpr int bwd_blocks(int tpr) { return tpr <= 128 ? 3 : 1; }

// The variances are of the rows in registers, after the mean: no cancellation. BIAS: some norm has a beta.
template <typename TX, typename TY, int NCH, int TPR, bool BIAS, bool VEC>
__global__ void __launch_bounds__(block_threads(TPR), fwd_blocks(TPR, NCH, BIAS)) join_fwd_kernel(const JoinArgs a) {
  grid_wait();
  constexpr int ROWS = block_threads(TPR) / TPR;
  __shared__ __align__(16) float red[2][32];
  extern __shared__ __align__(16) uint8_t ring[];
  const int t = ROWS > 1 ? threadIdx.x % TPR : threadIdx.x;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const int row0 = blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / TPR : 0), step = gridDim.x * ROWS;
  const int rows = row0 < a.T ? (a.T - 1 - row0) / step + 1 : 0;
  Feed<VEC, NCH, TPR, TX, TY> feed;
  feed.init(ring, t, a.d, rows);
  feed.tensor(0, after_wait(a.x), a.ldx, row0, step);
  feed.tensor(1, after_wait(a.y), a.ldy, row0, step);
  feed.prime();
  // r = alpha x + A yhat + B;  n = rhat g2 + b2
  float A[NCH][8], B[NCH][8], g2[NCH][8], b2[NCH][8];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float gate[8];
    weights8<VEC, TPR>(after_wait(a.gate), a.w_bf16, t, i, a.d, 1.f, gate);
    weights8<VEC, TPR>(after_wait(a.g1), a.w_bf16, t, i, a.d, 1.f, A[i]);
    weights8<VEC, TPR>(after_wait(a.g2), a.w_bf16, t, i, a.d, 1.f, g2[i]);
    if constexpr (BIAS) {
      weights8<VEC, TPR>(after_wait(a.b1), a.w_bf16, t, i, a.d, 0.f, B[i]);
      weights8<VEC, TPR>(after_wait(a.b2), a.w_bf16, t, i, a.d, 0.f, b2[i]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      A[i][j] *= a.beta * gate[j];
      if constexpr (BIAS) B[i][j] *= a.beta * gate[j];
    }
  }
  const auto in = [&](int i, int j) { return column<VEC, TPR>(t, i, VEC ? 0 : j) < a.d; };
  int par = 0;
  const auto sum = [&](float v) {
    const float s = row_sum<TPR>(v, red[par]);
    par ^= 1;
    return s;
  };
  for (int k = 0; k < rows; ++k) {
    const long long row = row0 + static_cast<long long>(k) * step;
    float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f, s = 0.f;
    float y[NCH][8], r[NCH][8];
    feed.wait();
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      feed.template get<0>(i, r[i]);
      feed.template get<1>(i, y[i]);
    }
    feed.next();
    const auto each = [&](auto f) {
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) f(i, j);
    };
    if (a.post == MOE_NORM_LAYER) {
      each([&](int i, int j) { s += y[i][j]; });
      mean1 = sum(s) * inv_d;
      each([&](int i, int j) { y[i][j] -= in(i, j) ? mean1 : 0.f; });
    }
    if (a.post != MOE_NORM_NONE) {
      s = 0.f;
      each([&](int i, int j) { s = fmaf(y[i][j], y[i][j], s); });
      rstd1 = 1.0f / sqrtf(sum(s) * inv_d + a.eps);
    }
    each([&](int i, int j) {
      float v = a.alpha * r[i][j];
      v = fmaf(A[i][j], y[i][j] * rstd1, BIAS ? v + B[i][j] : v);  // y reads as zeros where there is no branch
      r[i][j] = rounded<TX>(v);
    });
    if (a.r != nullptr) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) put_chunk<VEC, TPR>(static_cast<TX*>(a.r) + row * a.ldr, t, i, a.d, r[i]);
    }
    if (a.pre == MOE_NORM_LAYER) {
      s = 0.f;
      each([&](int i, int j) { s += r[i][j]; });
      mean2 = sum(s) * inv_d;
      each([&](int i, int j) { r[i][j] -= in(i, j) ? mean2 : 0.f; });
    }
    if (a.pre != MOE_NORM_NONE) {
      s = 0.f;
      each([&](int i, int j) { s = fmaf(r[i][j], r[i][j], s); });
      rstd2 = 1.0f / sqrtf(sum(s) * inv_d + a.eps);
      each([&](int i, int j) { r[i][j] = fmaf(r[i][j] * rstd2, g2[i][j], BIAS ? b2[i][j] : 0.f); });
#pragma unroll
      for (int i = 0; i < NCH; ++i) put_chunk<VEC, TPR>(static_cast<TY*>(a.n) + row * a.ldn, t, i, a.d, r[i]);
    }
    if (t == 0 && a.stats != nullptr) {
      const size_t T = a.T;
      a.stats[row] = mean1;
      a.stats[T + row] = rstd1;
      a.stats[2 * T + row] = mean2;
      a.stats[3 * T + row] = rstd2;
    }
  }
}

// Arithmetic in pairs of fp32, one instruction for two, and without branches: single values and a branch for each kind of norm took
// more instructions than memory leaves time for (16384 x 2048: 93 us, 77 so). BIAS: the sums over the rows that only the betas' gradients need (and, with a beta, the gate's) are wanted.
template <typename TX, typename TY, int NCH, int TPR, bool BIAS, bool VEC>
__global__ void __launch_bounds__(block_threads(TPR), bwd_blocks(TPR)) join_bwd_kernel(const JoinArgs a) {
  grid_wait();
  constexpr int ROWS = block_threads(TPR) / TPR;
  __shared__ __align__(16) float red[2][64];
  extern __shared__ __align__(16) uint8_t ring[];
  const int t = ROWS > 1 ? threadIdx.x % TPR : threadIdx.x, lane = threadIdx.x & 31;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const int row0 = blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / TPR : 0), step = gridDim.x * ROWS;
  const int rows = row0 < a.T ? (a.T - 1 - row0) / step + 1 : 0;
  Feed<VEC, NCH, TPR, TY, TX, TX, TY> feed;  // dn, r, dr, y
  feed.init(ring, t, a.d, rows);
  feed.tensor(0, after_wait(a.dn), a.lddn, row0, step);
  feed.tensor(1, a.pre != MOE_NORM_NONE ? after_wait(a.r) : nullptr, a.ldr, row0, step);
  feed.tensor(2, after_wait(a.dr), a.lddr, row0, step);
  feed.tensor(3, after_wait(a.y), a.ldy, row0, step);
  feed.prime();
  F2 A[NCH][4], g2[NCH][4], S1[NCH][4], S0[NCH][4], P1[NCH][4], P0[NCH][4];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float w[8], gate[8];
    weights8<VEC, TPR>(after_wait(a.gate), a.w_bf16, t, i, a.d, 1.f, gate);
    weights8<VEC, TPR>(after_wait(a.g1), a.w_bf16, t, i, a.d, 1.f, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= a.beta * gate[j];
    pairs(w, A[i]);
    weights8<VEC, TPR>(after_wait(a.g2), a.w_bf16, t, i, a.d, 1.f, w);
    pairs(w, g2[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) S1[i][j] = S0[i][j] = P1[i][j] = P0[i][j] = both(0.f);
  }
  int par = 0;
  const auto sums = [&](F2 u, F2 v) {
    const float2 p = parts(u), q = parts(v);
    const float2 s = row_sum<TPR>(p.x + p.y, q.x + q.y, red[par]);
    par ^= 1;
    return s;
  };
  const F2 alpha = both(a.alpha);
  // lane l holds the statistics of rows l, l + 32, ... of this block: one wait in 32 rows
  float st[4] = {0.f, 1.f, 0.f, 1.f};
  TX* dx = a.dx ? static_cast<TX*>(a.dx) + row0 * a.lddx : nullptr;
  TY* dy = a.dy ? static_cast<TY*>(a.dy) + row0 * a.lddy : nullptr;
  for (int k = 0; k < rows; ++k, dx += step * a.lddx, dy += step * a.lddy) {
    if ((k & 31) == 0 && k + lane < rows && a.stats != nullptr) {
      const float* p = after_wait(a.stats) + row0 + static_cast<long long>(k + lane) * step;
#pragma unroll
      for (int q = 0; q < 4; ++q) st[q] = __ldg(p + static_cast<size_t>(q) * a.T);
    }
    const float mean1 = a.post == MOE_NORM_LAYER ? __shfl_sync(0xffffffffu, st[0], k & 31) : 0.f;
    const float rstd1 = a.post != MOE_NORM_NONE ? __shfl_sync(0xffffffffu, st[1], k & 31) : 1.f;
    const float mean2 = a.pre == MOE_NORM_LAYER ? __shfl_sync(0xffffffffu, st[2], k & 31) : 0.f;
    const float rstd2 = a.pre != MOE_NORM_NONE ? __shfl_sync(0xffffffffu, st[3], k & 31) : 1.f;
    // past the end of a row everything is computed from zeros and weights of 0, and nothing stored
    const auto each = [&](auto f) {
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) f(i, j);
    };
    const auto get = [&](auto which, F2 (&v)[NCH][4]) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        float f[8];
        feed.template get<decltype(which)::value>(i, f);
        pairs(f, v[i]);
      }
    };
    F2 D[NCH][4], h[NCH][4], v[NCH][4];  // the pre norm's gamma dn, then the gradient of r; rhat, then yhat; dr
    feed.wait();
    F2 k0 = both(0.f), k1 = k0, scale = k0;  // D = scale (gamma dn) + k1 rhat + k0 + dr
    if (a.pre != MOE_NORM_NONE) {
      F2 s1 = both(0.f), s2 = s1;
      const F2 R = both(rstd2), C = both(-mean2 * rstd2);
      get(std::integral_constant<int, 0>{}, D);
      get(std::integral_constant<int, 1>{}, h);
      each([&](int i, int j) {
        h[i][j] = fma2(h[i][j], R, C);
        P1[i][j] = fma2(D[i][j], h[i][j], P1[i][j]);
        if constexpr (BIAS) P0[i][j] = add2(P0[i][j], D[i][j]);
        D[i][j] = mul2(D[i][j], g2[i][j]);
        s1 = add2(s1, D[i][j]);
        s2 = fma2(D[i][j], h[i][j], s2);
      });
      const float2 s = sums(s1, s2);
      scale = R;
      k0 = both(a.pre == MOE_NORM_LAYER ? -s.x * inv_d * rstd2 : 0.f);
      k1 = both(-s.y * inv_d * rstd2);
    } else {
      each([&](int i, int j) { D[i][j] = h[i][j] = both(0.f); });
    }
    get(std::integral_constant<int, 2>{}, v);
    each([&](int i, int j) { D[i][j] = fma2(D[i][j], scale, fma2(h[i][j], k1, add2(k0, v[i][j]))); });
    get(std::integral_constant<int, 3>{}, h);
    feed.next();
    if (a.dx != nullptr) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        F2 o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = mul2(alpha, D[i][j]);
        put_chunk<VEC, TPR>(dx, t, i, a.d, o);
      }
    }
    if (a.y != nullptr) {
      F2 s1 = both(0.f), s2 = s1;
      const F2 R = both(rstd1), C = both(-mean1 * rstd1);
      each([&](int i, int j) {
        h[i][j] = fma2(h[i][j], R, C);
        S1[i][j] = fma2(D[i][j], h[i][j], S1[i][j]);
        if constexpr (BIAS) S0[i][j] = add2(S0[i][j], D[i][j]);
        D[i][j] = mul2(D[i][j], A[i][j]);
        s1 = add2(s1, D[i][j]);
        s2 = fma2(D[i][j], h[i][j], s2);
      });
      if (a.post != MOE_NORM_NONE) {
        const float2 s = sums(s1, s2);
        const F2 m0 = both(a.post == MOE_NORM_LAYER ? -s.x * inv_d * rstd1 : 0.f), m1 = both(-s.y * inv_d * rstd1);
        each([&](int i, int j) { D[i][j] = fma2(D[i][j], R, fma2(h[i][j], m1, m0)); });
      }
#pragma unroll
      for (int i = 0; i < NCH; ++i) put_chunk<VEC, TPR>(dy, t, i, a.d, D[i]);
    }
  }
  if (a.part == nullptr) return;
  float* part = a.part + static_cast<size_t>(blockIdx.x) * SUMS * a.d;
  // a block of several rows: its warps own the same columns; they are added in warp order
  __shared__ F2 acc[ROWS > 1 ? ROWS - 1 : 1][SUMS][32];
  const int w = threadIdx.x / TPR;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    if constexpr (ROWS > 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        F2* const mine[SUMS] = {&S1[i][j], &S0[i][j], &P1[i][j], &P0[i][j]};
        __syncthreads();
        if (w > 0) {
#pragma unroll
          for (int q = 0; q < SUMS; ++q) acc[w - 1][q][t] = *mine[q];
        }
        __syncthreads();
        if (w == 0) {
#pragma unroll
          for (int r = 0; r < ROWS - 1; ++r)
#pragma unroll
            for (int q = 0; q < SUMS; ++q) *mine[q] = add2(*mine[q], acc[r][q][t]);
        }
      }
    }
    if (w != 0) continue;
    const size_t d = a.d;
    put_chunk<VEC, TPR>(part, t, i, a.d, S1[i]);
    put_chunk<VEC, TPR>(part + 2 * d, t, i, a.d, P1[i]);
    if constexpr (BIAS) {
      put_chunk<VEC, TPR>(part + d, t, i, a.d, S0[i]);
      put_chunk<VEC, TPR>(part + 3 * d, t, i, a.d, P0[i]);
    }
  }
}

struct GradOut {
  float *post_gamma, *post_beta, *gate, *pre_gamma, *pre_beta;
};

// The weight gradients from the partial sums: eight columns a block (a 32-byte piece of each partial row, so that there are
// blocks for all SMs), 32 threads for each of a column's four sums, which take every 32nd partial and are added in thread order.
constexpr int PART_COLS = 8;

__global__ void __launch_bounds__(1024) join_partials_kernel(const JoinArgs a, int blocks, bool bias, const GradOut o) {
  __shared__ float acc[SUMS][32][PART_COLS + 1];
  grid_wait();  // launched ahead of the end of the kernel that writes the partials
  const float* part = after_wait(static_cast<const float*>(a.part));
  const int cx = threadIdx.x % PART_COLS, k = threadIdx.x / PART_COLS % SUMS, ry = threadIdx.x / (PART_COLS * SUMS);
  const int c = blockIdx.x * PART_COLS + cx;
  // every load at once (a loop of a run-time length waits for each round of them)
  constexpr int ROUNDS = (BWD_MAX_BLOCKS + 31) / 32;
  float v[ROUNDS], s = 0.f;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int r = ry + 32 * i;
    v[i] = r < blocks && c < a.d && ((k & 1) == 0 || bias) ? __ldcs(part + (static_cast<size_t>(r) * SUMS + k) * a.d + c) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) s += v[i];
  acc[k][ry][cx] = s;
  __syncthreads();
  if (threadIdx.x >= PART_COLS || c >= a.d) return;
  float t[SUMS];
#pragma unroll
  for (int q = 0; q < SUMS; ++q) {
    t[q] = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t[q] += acc[q][i][cx];
  }
  const float g = a.beta * weight(a.gate, a.w_bf16, c, 1.f);
  if (o.post_gamma) o.post_gamma[c] = g * t[0];
  if (o.post_beta) o.post_beta[c] = g * t[1];
  if (o.gate) o.gate[c] = a.beta * fmaf(weight(a.g1, a.w_bf16, c, 1.f), t[0], weight(a.b1, a.w_bf16, c, 0.f) * t[1]);
  if (o.pre_gamma) o.pre_gamma[c] = t[2];
  if (o.pre_beta) o.pre_beta[c] = t[3];
}

template <bool VEC, typename TX, typename TY, int NCH, int TPR>
cudaError_t launch_fwd_rows(const JoinArgs& a, cudaStream_t s) {
  constexpr int ROWS = block_threads(TPR) / TPR, smem = Feed<VEC, NCH, TPR, TX, TY>::smem_bytes;
  const bool bias = a.b1 || a.b2;
  const int grid = static_cast<int>(std::min<long long>((static_cast<long long>(a.T) + ROWS - 1) / ROWS, fwd_blocks(TPR, NCH, bias) * static_cast<long long>(device_sm_count())));
  const auto kernel = bias ? join_fwd_kernel<TX, TY, NCH, TPR, true, VEC> : join_fwd_kernel<TX, TY, NCH, TPR, false, VEC>;
  if (smem > 40 * 1024) {  // beside the static shared memory
    const cudaError_t err = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (err != cudaSuccess) return err;
  }
  return launch_dependent(kernel, grid, block_threads(TPR), smem, s, a);
}
template <bool VEC, typename TX, typename TY, int NCH, int TPR>
cudaError_t launch_bwd_rows(const JoinArgs& a, bool bias, cudaStream_t s, int& blocks) {
  constexpr int ROWS = block_threads(TPR) / TPR, smem = Feed<VEC, NCH, TPR, TY, TX, TX, TY>::smem_bytes;
  blocks = static_cast<int>(std::min<long long>((static_cast<long long>(a.T) + ROWS - 1) / ROWS, std::min(bwd_blocks(TPR) * device_sm_count(), BWD_MAX_BLOCKS)));
  const auto kernel = bias ? join_bwd_kernel<TX, TY, NCH, TPR, true, VEC> : join_bwd_kernel<TX, TY, NCH, TPR, false, VEC>;
  if (smem > 40 * 1024) {  // beside the static shared memory
    const cudaError_t err = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (err != cudaSuccess) return err;
  }
  return launch_dependent(kernel, blocks, block_threads(TPR), smem, s, a);
}

// Rows go through registers up to a width of 8192, wider ones through the kernels of any width. Off the 16-byte grid the registers
// are filled by single elements (16384 x 2047 bf16, RMS norms and gate: forward 80 us, backward with every gradient 149; through the kernels
// of any width 414 and 677).
constexpr int REGISTER_WIDTH = 8192;

template <bool VEC, typename TX, typename TY>
cudaError_t launch_fwd_registers(const JoinArgs& a, cudaStream_t s) {
  const int chunks = (a.d + 7) / 8;
  if (chunks <= 32) return launch_fwd_rows<VEC, TX, TY, 1, 32>(a, s);
  if (chunks <= 64) return launch_fwd_rows<VEC, TX, TY, 2, 32>(a, s);
  if (chunks <= 128) return launch_fwd_rows<VEC, TX, TY, 1, 128>(a, s);
  if (chunks <= 256) return launch_fwd_rows<VEC, TX, TY, 1, 256>(a, s);
  if (chunks <= 512) return launch_fwd_rows<VEC, TX, TY, 2, 256>(a, s);
  return launch_fwd_rows<VEC, TX, TY, 2, 512>(a, s);
}
template <typename TX, typename TY>
cudaError_t launch_fwd(const JoinArgs& a, bool vec, cudaStream_t s) {
  if (a.d <= REGISTER_WIDTH) return vec ? launch_fwd_registers<true, TX, TY>(a, s) : launch_fwd_registers<false, TX, TY>(a, s);
  join_fwd_wide_kernel<TX, TY><<<std::min(a.T, 1 << 20), WIDE_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

// `blocks`: the rows of partial sums that the launch leaves; `bias`: all four sums are wanted
template <bool VEC, typename TX, typename TY>
cudaError_t launch_bwd_registers(const JoinArgs& a, bool bias, cudaStream_t s, int& blocks) {
  const int chunks = (a.d + 7) / 8;
  if (chunks <= 32) return launch_bwd_rows<VEC, TX, TY, 1, 32>(a, bias, s, blocks);
  if (chunks <= 64) return launch_bwd_rows<VEC, TX, TY, 2, 32>(a, bias, s, blocks);
  if (chunks <= 128) return launch_bwd_rows<VEC, TX, TY, 1, 128>(a, bias, s, blocks);
  if (chunks <= 256) return launch_bwd_rows<VEC, TX, TY, 2, 128>(a, bias, s, blocks);
  if (chunks <= 512) return launch_bwd_rows<VEC, TX, TY, 2, 256>(a, bias, s, blocks);
  return launch_bwd_rows<VEC, TX, TY, 2, 512>(a, bias, s, blocks);
}
template <typename TX, typename TY>
cudaError_t launch_bwd(const JoinArgs& a, bool vec, bool bias, cudaStream_t s, int& blocks) {
  if (a.d <= REGISTER_WIDTH) return vec ? launch_bwd_registers<true, TX, TY>(a, bias, s, blocks) : launch_bwd_registers<false, TX, TY>(a, bias, s, blocks);
  const int grid = std::min(a.T, 1 << 20);
  blocks = std::min(a.T, BWD_MAX_BLOCKS);
  if (a.pre != MOE_NORM_NONE) join_bwd_means_kernel<TX, TY><<<grid, WIDE_THREADS, 0, s>>>(a);
  // the weight gradients first: dx and dy may lie over inputs
  if (a.part != nullptr) join_wgrad_wide_kernel<TX, TY><<<dim3((a.d + 255) / 256, blocks), 256, 0, s>>>(a);
  join_bwd_wide_kernel<TX, TY><<<grid, WIDE_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

// 16-byte rows: base, pitch and width
bool rows16(const void* p, long long ld, int es) { return p == nullptr || (aligned16(p) && ld * es % 16 == 0); }

size_t part_floats(int T, int d) { return static_cast<size_t>(std::min(T, BWD_MAX_BLOCKS)) * SUMS * d; }

bool norm_ok(int k) { return k == MOE_NORM_NONE || k == MOE_NORM_LAYER || k == MOE_NORM_RMS; }
bool types_ok(int x, int y) { return dtype_ok(x) && dtype_ok(y) && (x == MOE_DTYPE_F32 || y == MOE_DTYPE_BF16); }

}  // namespace

size_t residual_norm_bwd_workspace_bytes(int T, int d) {
  if (T < 0 || d < 1 || d > MAX_WIDTH) return 0;
  return (part_floats(T, d) + 2 * static_cast<size_t>(T)) * sizeof(float);
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_residual_norm_fwd(const void* x, int x_dtype, long long ldx, const void* y, int y_dtype, long long ldy,
                                   int post, const void* post_gamma, const void* post_beta, const void* gate, int pre,
                                   const void* pre_gamma, const void* pre_beta, int w_dtype, int T, int d, float eps,
                                   float res_scale, float branch_scale, void* r, long long ldr, void* n, long long ldn,
                                   float* stats, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (T < 0 || d <= 0 || !types_ok(x_dtype, y_dtype) || !dtype_ok(w_dtype) || !norm_ok(post) || !norm_ok(pre))
    return MOE_ERR_INVALID_ARG;
  if (ldx < 0 || (y && ldy < 0) || (r && ldr < d) || (n && ldn < d)) return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || std::isinf(eps) || !std::isfinite(res_scale) || !std::isfinite(branch_scale)) return MOE_ERR_INVALID_ARG;
  if (d > MAX_WIDTH) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && (!x || (!r && !n) || (pre == MOE_NORM_NONE) != (n == nullptr))) return MOE_ERR_INVALID_ARG;
  if ((!y && T > 0 && (post != MOE_NORM_NONE || gate)) || (post == MOE_NORM_NONE && post_gamma) ||
      (post != MOE_NORM_LAYER && post_beta) || (pre == MOE_NORM_NONE && pre_gamma) || (pre != MOE_NORM_LAYER && pre_beta))
    return MOE_ERR_INVALID_ARG;
  const int ex = dtype_bytes(x_dtype), ey = dtype_bytes(y_dtype), ew = dtype_bytes(w_dtype);
  if (!element_aligned(x, ex) || !element_aligned(r, ex) || !element_aligned(y, ey) || !element_aligned(n, ey) ||
      !element_aligned(post_gamma, ew) || !element_aligned(post_beta, ew) || !element_aligned(gate, ew) ||
      !element_aligned(pre_gamma, ew) || !element_aligned(pre_beta, ew) || !element_aligned(stats, 4))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = check_device();
  if (st != MOE_OK || T == 0) return st;
  JoinArgs a{};
  a.x = x;
  a.y = y;
  a.r = r;
  a.n = n;
  a.ldx = ldx;
  a.ldy = ldy;
  a.ldr = ldr;
  a.ldn = ldn;
  a.g1 = post_gamma;
  a.b1 = post_beta;
  a.gate = gate;
  a.g2 = pre_gamma;
  a.b2 = pre_beta;
  a.w_bf16 = w_dtype == MOE_DTYPE_BF16;
  a.post = post;
  a.pre = pre;
  a.T = T;
  a.d = d;
  a.eps = eps;
  a.alpha = res_scale;
  a.beta = branch_scale;
  a.stats = stats;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool vec = d % 8 == 0 && rows16(x, ldx, ex) && rows16(y, ldy, ey) && rows16(r, ldr, ex) && rows16(n, ldn, ey) &&
                   aligned16(post_gamma) && aligned16(post_beta) && aligned16(gate) && aligned16(pre_gamma) && aligned16(pre_beta);
  const cudaError_t err = x_dtype == MOE_DTYPE_BF16   ? launch_fwd<bf16, bf16>(a, vec, s)
                          : y_dtype == MOE_DTYPE_BF16 ? launch_fwd<float, bf16>(a, vec, s)
                                                      : launch_fwd<float, float>(a, vec, s);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

moe_status_t moe_residual_norm_bwd(const void* dn, long long lddn, const void* dr, long long lddr, const void* r,
                                   long long ldr, int x_dtype, const void* y, long long ldy, int y_dtype, int post,
                                   const void* post_gamma, const void* post_beta, const void* gate, int pre,
                                   const void* pre_gamma, int w_dtype, const float* stats, int T, int d, float res_scale,
                                   float branch_scale, void* dx, long long lddx, void* dy, long long lddy,
                                   float* d_post_gamma, float* d_post_beta, float* d_gate, float* d_pre_gamma,
                                   float* d_pre_beta, void* ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (T < 0 || d <= 0 || !types_ok(x_dtype, y_dtype) || !dtype_ok(w_dtype) || !norm_ok(post) || !norm_ok(pre))
    return MOE_ERR_INVALID_ARG;
  if ((dn && lddn < 0) || (dr && lddr < 0) || (r && ldr < 0) || (y && ldy < 0) || (dx && lddx < d) || (dy && lddy < d))
    return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(res_scale) || !std::isfinite(branch_scale)) return MOE_ERR_INVALID_ARG;
  if (d > MAX_WIDTH) return MOE_ERR_UNSUPPORTED_SHAPE;
  const bool normed = post != MOE_NORM_NONE || pre != MOE_NORM_NONE;
  if (T > 0 && ((pre == MOE_NORM_NONE) != (dn == nullptr) || (pre != MOE_NORM_NONE && !r) || (normed && !stats) ||
                (y == nullptr) != (dy == nullptr) || (!y && (post != MOE_NORM_NONE || gate)) || (!dn && !dr) || (!dx && !dy)))
    return MOE_ERR_INVALID_ARG;
  if ((post == MOE_NORM_NONE && (post_gamma || d_post_gamma || d_post_beta)) || (post != MOE_NORM_LAYER && post_beta) ||
      (pre == MOE_NORM_NONE && (pre_gamma || d_pre_gamma || d_pre_beta)) || (T > 0 && !y && d_gate))
    return MOE_ERR_INVALID_ARG;
  const int ex = dtype_bytes(x_dtype), ey = dtype_bytes(y_dtype), ew = dtype_bytes(w_dtype);
  if (!element_aligned(dr, ex) || !element_aligned(r, ex) || !element_aligned(dx, ex) || !element_aligned(dn, ey) ||
      !element_aligned(y, ey) || !element_aligned(dy, ey) || !element_aligned(post_gamma, ew) ||
      !element_aligned(post_beta, ew) || !element_aligned(gate, ew) || !element_aligned(pre_gamma, ew) ||
      !element_aligned(stats, 4) || !element_aligned(d_post_gamma, 4) || !element_aligned(d_post_beta, 4) ||
      !element_aligned(d_gate, 4) || !element_aligned(d_pre_gamma, 4) || !element_aligned(d_pre_beta, 4) ||
      !element_aligned(ws, 4))
    return MOE_ERR_INVALID_ARG;
  if (T > 0) {
    if (ws_bytes < residual_norm_bwd_workspace_bytes(T, d)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!ws) return MOE_ERR_INVALID_ARG;
  }
  moe_status_t st = check_device();
  if (st != MOE_OK) return st;
  const GradOut o{d_post_gamma, d_post_beta, d_gate, d_pre_gamma, d_pre_beta};
  const bool wgrad = d_post_gamma || d_post_beta || d_gate || d_pre_gamma || d_pre_beta;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  JoinArgs a{};
  a.dn = dn;
  a.dr = dr;
  a.r = const_cast<void*>(r);
  a.y = y;
  a.dx = dx;
  a.dy = dy;
  a.lddn = lddn;
  a.lddr = lddr;
  a.ldr = ldr;
  a.ldy = ldy;
  a.lddx = lddx;
  a.lddy = lddy;
  a.g1 = post_gamma;
  a.b1 = post_beta;
  a.gate = gate;
  a.g2 = pre_gamma;
  a.w_bf16 = w_dtype == MOE_DTYPE_BF16;
  a.post = post;
  a.pre = pre;
  a.T = T;
  a.d = d;
  a.alpha = res_scale;
  a.beta = branch_scale;
  a.stats = const_cast<float*>(stats);
  a.part = wgrad && T > 0 ? static_cast<float*>(ws) : nullptr;
  a.row = static_cast<float*>(ws) + (T > 0 ? part_floats(T, d) : 0);
  int blocks = 0;
  const bool bias = d_post_beta || d_pre_beta || (d_gate && post_beta);
  if (T > 0) {
    const bool vec = d % 8 == 0 && rows16(dn, lddn, ey) && rows16(dr, lddr, ex) && rows16(r, ldr, ex) && rows16(y, ldy, ey) &&
                     rows16(dx, lddx, ex) && rows16(dy, lddy, ey) && aligned16(post_gamma) && aligned16(gate) && aligned16(pre_gamma) && aligned16(ws);
    const cudaError_t err = x_dtype == MOE_DTYPE_BF16   ? launch_bwd<bf16, bf16>(a, vec, bias, s, blocks)
                            : y_dtype == MOE_DTYPE_BF16 ? launch_bwd<float, bf16>(a, vec, bias, s, blocks)
                                                        : launch_bwd<float, float>(a, vec, bias, s, blocks);
    if (err != cudaSuccess) return cuda_fail(err);
  }
  if (!wgrad) return MOE_OK;
  const cudaError_t err = launch_dependent(join_partials_kernel, (d + PART_COLS - 1) / PART_COLS, 1024, 0, s, a, blocks, bias, o);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

}  // extern "C"
