// Few tokens through 4-bit integer weights with group scales: w = scale (code - zero).
//
//   matvec: y[s] = W[ids[s]] x[s / top_k];  decode: out[t] = sum_j weight[t, j] SwiGLU(x[t] W_ug,e^T) W_down,e
//
// Packed layout (include/moe_gg.h): tiles of 16 rows by chunks of 128 elements, 1024 bytes of codes each; the scales
// and zero points of a tile's rows r and r + 8 lie together.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "trace.h"

namespace moe {
namespace {

constexpr int MAX_DIM = 1 << 20;
constexpr int MAX_MATRICES = 2048;
constexpr int MAX_SLOTS = 4096;

// Where the pieces of packed matrices lie
struct Packed {
  const uint8_t* codes;
  const uint8_t* scales;
  const uint8_t* zeros;
  int tiles, chunks, per;  // 16-row tiles of a matrix, 128-element chunks of a row, groups of a chunk
};

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
int groups_of(int K, int group) { return (K + group - 1) / group; }
bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }

size_t pieces(int matrices, int N, int K) {
  return static_cast<size_t>(matrices) * ((N + 15) / 16) * ((K + 127) / 128);
}
Packed packed_at(const void* p, int matrices, int N, int K, int group) {
  Packed w;
  const size_t n = pieces(matrices, N, K);
  w.per = 128 / group;
  w.codes = static_cast<const uint8_t*>(p);
  w.scales = w.codes + n * 1024;
  w.zeros = w.scales + round256(n * 32 * w.per);
  w.tiles = (N + 15) / 16;
  w.chunks = (K + 127) / 128;
  return w;
}

// ------------------------------------------------------------------ preparing weights
// One warp a group: its smallest and largest value (and 0), the scale and the zero point between them, the codes.
__global__ void __launch_bounds__(256) w4_quantize_kernel(const bf16* w, long long rows, int K, int group, uint8_t* codes,
                                                          bf16* scales, uint8_t* zeros) {
  const int lane = threadIdx.x & 31, groups = (K + group - 1) / group;
  const long long all = rows * groups, step = static_cast<long long>(gridDim.x) * 8;
  for (long long g = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); g < all; g += step) {
    const long long row = g / groups;
    const int k0 = static_cast<int>(g % groups) * group;
    const int n = min(group, K - k0);
    const bf16* src = w + row * K + k0;
    float v[4];  // elements 2 (lane + 32 i) and the next one: a lane makes whole bytes
    float lo = 0.f, hi = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = (i >> 1) * 64 + 2 * lane + (i & 1);
      v[i] = e < n ? __bfloat162float(src[e]) : 0.f;
      lo = fminf(lo, v[i]);
      hi = fmaxf(hi, v[i]);
      bad |= !(fabsf(v[i]) <= 3.402823466e38f);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    bad = __any_sync(0xffffffffu, bad);
    // the two halves by themselves: hi - lo of the largest bf16 values is past fp32's range
    const bf16 sb = __float2bfloat16_rn(bad ? __uint_as_float(0x7FC00000u) : hi / 15.0f - lo / 15.0f);
    const float s = __bfloat162float(sb);
    const bool live = s > 0.f;
    const float z = live ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f;
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = live ? static_cast<uint32_t>(fminf(fmaxf(rintf(v[i] / s) + z, 0.f), 15.f)) : 0u;
    uint8_t* dst = codes + row * ((K + 1) / 2) + k0 / 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = i * 64 + 2 * lane;
      if (e < n) dst[e / 2] = static_cast<uint8_t>(c[2 * i] | (e + 1 < n ? c[2 * i + 1] << 4 : 0u));
    }
    if (lane == 0) {
      scales[g] = sb;
      zeros[g] = static_cast<uint8_t>(z);
    }
  }
}

// One warp a piece (16 rows, 128 elements): lane (g, t) its 16 bytes of rows g and g + 8.
__global__ void __launch_bounds__(256) w4_pack_kernel(const uint8_t* codes, const bf16* scales, const uint8_t* zeros, int N,
                                                      int K, int group, long long n, Packed p) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int groups = (K + group - 1) / group, pitch = (K + 1) / 2;
  const long long step = static_cast<long long>(gridDim.x) * 8;
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < n; i += step) {
    const int chunk = static_cast<int>(i % p.chunks);
    const long long mt = i / p.chunks;
    const int tile = static_cast<int>(mt % p.tiles);
    const long long m = mt / p.tiles;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = tile * 16 + half * 8 + g;
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k0 = chunk * 128 + q * 32 + t * 8;
        w[q] = 0;
        if (r < N && k0 < K) {
          // what lies past the row's end in its last group stands for 0
          const uint32_t z = zeros ? zeros[(m * N + r) * groups + k0 / group] & 15u : 8u;
          const uint8_t* src = codes + (m * N + r) * pitch + k0 / 2;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t c = k0 + j < K ? (src[j / 2] >> (4 * (j & 1))) & 15u : z;
            w[q] |= c << (4 * ((j >> 1) + 4 * (j & 1)));
          }
        }
      }
      *reinterpret_cast<uint4*>(const_cast<uint8_t*>(p.codes) + i * 1024 + half * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (t < p.per) {
      const int gi = chunk * p.per + t;
      uint32_t s = 0, z = 0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = tile * 16 + half * 8 + g;
        if (r >= N || gi >= groups) continue;
        const long long at = (m * N + r) * groups + gi;
        s |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(scales)[at]) << (16 * half);
        z |= (zeros ? zeros[at] & 15u : 8u) << (4 * half);
      }
      const long long at = (i * 8 + g) * p.per + t;
      reinterpret_cast<uint32_t*>(const_cast<uint8_t*>(p.scales))[at] = s;
      const_cast<uint8_t*>(p.zeros)[at] = static_cast<uint8_t>(z);
    }
  }
}

// ------------------------------------------------------------------ products
// Row `row` of matrix m times x [K], by one warp: a lane takes eight elements at a time.
__device__ __forceinline__ float dot(const Packed& p, int m, int row, const bf16* x, int K) {
  const int lane = threadIdx.x & 31, r = row & 15;
  const size_t piece0 = (static_cast<size_t>(m) * p.tiles + (row >> 4)) * p.chunks;
  float sum = 0.f;
  for (int i = lane; i < p.chunks * 16; i += 32) {
    const size_t piece = piece0 + (i >> 4);
    const int q = (i >> 2) & 3, t = i & 3, k0 = (i >> 4) * 128 + q * 32 + t * 8;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p.codes + piece * 1024 + (r >> 3) * 512 + ((r & 7) * 4 + t) * 16 + q * 4));
    const size_t at = (piece * 8 + (r & 7)) * p.per + (q * p.per >> 2);
    const uint32_t pair = __ldg(reinterpret_cast<const uint32_t*>(p.scales) + at);
    const float s = r < 8 ? bf16_lo(pair) : bf16_hi(pair);
    const int z = (p.zeros[at] >> (r < 8 ? 0 : 4)) & 15;
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = static_cast<int>((w >> (4 * ((j >> 1) + 4 * (j & 1)))) & 15u) - z;
      if (k0 + j < K) part = fmaf(static_cast<float>(c), __bfloat162float(x[k0 + j]), part);
    }
    sum = fmaf(s, part, sum);
  }
  return warp_sum(sum);
}

template <typename T>
__global__ void __launch_bounds__(256) w4_matvec_kernel(const bf16* x, long long ldx, const int32_t* ids, int top_k,
                                                        int matrices, int N, int K, const Packed w, T* y, long long ldy) {
  grid_wait();
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), s = blockIdx.y;
  if (row >= N) return;
  const int m = ids ? after_wait(ids)[s] : 0;
  float v[1] = {0.f};
  if (m >= 0 && m < matrices) v[0] = dot(w, m, row, after_wait(x) + (s / top_k) * ldx, K);
  if ((threadIdx.x & 31) == 0) Chunk<T, 1>::store(y + s * ldy + row, v);
}

__global__ void __launch_bounds__(256) w4_up_kernel(const bf16* x, long long ldx, const int32_t* ids, int top_k, int E, int d,
                                                    int h, const Packed w, bf16* a) {
  grid_wait();
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), s = blockIdx.y;
  const int e = after_wait(ids)[s];
  if (row >= h || e < 0 || e >= E) return;
  const bf16* xr = after_wait(x) + (s / top_k) * ldx;
  const float g = dot(w, 2 * e, row, xr, d), u = dot(w, 2 * e + 1, row, xr, d);
  if ((threadIdx.x & 31) == 0) a[static_cast<size_t>(s) * h + row] = __float2bfloat16_rn(g / (1.0f + expf(-g)) * u);
}

__global__ void __launch_bounds__(256) w4_down_kernel(const bf16* a, const int32_t* ids, const float* weights, int top_k, int E,
                                                      int d, int h, const Packed w, bf16* out, long long ldo) {
  grid_wait();
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), t = blockIdx.y;
  if (row >= d) return;
  float v = 0.f;
  for (int j = 0; j < top_k; ++j) {
    const int s = t * top_k + j, e = after_wait(ids)[s];
    if (e < 0 || e >= E) continue;
    const float y = dot(w, e, row, after_wait(a) + static_cast<size_t>(s) * h, h);
    v = fmaf(weights ? after_wait(weights)[s] : 1.0f, y, v);
  }
  if ((threadIdx.x & 31) == 0) out[t * ldo + row] = __float2bfloat16_rn(v);
}

bool dim_ok(int v) { return v >= 1 && v <= MAX_DIM; }

}  // namespace

size_t w4_weights_bytes(int matrices, int K, int N, int group) {
  if (matrices < 1 || matrices > MAX_MATRICES || !dim_ok(K) || !dim_ok(N) || !group_ok(group)) return 0;
  const size_t n = pieces(matrices, N, K), per = 128 / group;
  return n * 1024 + round256(n * 32 * per) + round256(n * 8 * per);
}
size_t w4_decode_workspace_bytes(long long slots, int E, int d, int h) {
  if (slots < 0 || slots > MAX_SLOTS || !dim_ok(d) || !dim_ok(h)) return 0;
  return round256(static_cast<size_t>(slots) * h * 2);
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_w4_quantize_rows(const moe_bf16* w, long long rows, int K, int group, uint8_t* codes, moe_bf16* scales,
                                  uint8_t* zeros, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (rows < 0 || K < 1) return MOE_ERR_INVALID_ARG;
  if (!group_ok(group) || K > MAX_DIM || rows >= (1LL << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows > 0 && (!w || !codes || !scales || !zeros)) return MOE_ERR_INVALID_ARG;
  if (!element_aligned(w, 2) || !element_aligned(scales, 2)) return MOE_ERR_INVALID_ARG;
  moe_status_t st = check_device();
  if (st != MOE_OK || rows == 0) return st;
  const long long blocks = (rows * groups_of(K, group) + 7) / 8;
  w4_quantize_kernel<<<static_cast<int>(std::min<long long>(blocks, 1 << 20)), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      reinterpret_cast<const bf16*>(w), rows, K, group, codes, reinterpret_cast<bf16*>(scales), zeros);
  const cudaError_t err = cudaGetLastError();
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

moe_status_t moe_w4_pack(const uint8_t* codes, const moe_bf16* scales, const uint8_t* zeros, int matrices, int N, int K,
                         int group, void* packed, size_t packed_bytes, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (matrices < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  const size_t need = w4_weights_bytes(matrices, K, N, group);
  if (need == 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (packed_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!codes || !scales || !packed || !element_aligned(scales, 2) || (reinterpret_cast<uintptr_t>(packed) & 255u) != 0)
    return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_device();
  if (st != MOE_OK) return st;
  const long long n = static_cast<long long>(pieces(matrices, N, K));
  w4_pack_kernel<<<static_cast<int>(std::min<long long>((n + 7) / 8, 1 << 20)), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      codes, reinterpret_cast<const bf16*>(scales), zeros, N, K, group, n, packed_at(packed, matrices, N, K, group));
  const cudaError_t err = cudaGetLastError();
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

moe_status_t moe_w4_matvec(const moe_bf16* x, long long ldx, const int32_t* ids, int T, int top_k, int matrices, int N,
                           int K, int group, const void* packed, void* y, int y_dtype, long long ldy,
                           moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (T < 0 || top_k < 1 || matrices < 1 || N < 1 || K < 1 || ldx < 0 || ldy < N || !dtype_ok(y_dtype)) return MOE_ERR_INVALID_ARG;
  if (top_k > 32 || matrices > MAX_MATRICES || !dim_ok(N) || !dim_ok(K) || !group_ok(group) ||
      static_cast<long long>(T) * top_k > MAX_SLOTS)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && (!x || !packed || !y)) return MOE_ERR_INVALID_ARG;
  if (!element_aligned(x, 2) || !element_aligned(ids, 4) || !element_aligned(y, dtype_bytes(y_dtype)) ||
      (reinterpret_cast<uintptr_t>(packed) & 255u) != 0)
    return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_device();
  if (st != MOE_OK || T == 0) return st;
  const Packed w = packed_at(packed, matrices, N, K, group);
  const bf16* xb = reinterpret_cast<const bf16*>(x);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((N + 7) / 8, T * top_k);
  const cudaError_t err =
      y_dtype == MOE_DTYPE_BF16
          ? launch_dependent(w4_matvec_kernel<bf16>, grid, 256, 0, s, xb, ldx, ids, top_k, matrices, N, K, w, static_cast<bf16*>(y), ldy)
          : launch_dependent(w4_matvec_kernel<float>, grid, 256, 0, s, xb, ldx, ids, top_k, matrices, N, K, w, static_cast<float*>(y), ldy);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

moe_status_t moe_w4_swiglu_decode(const moe_bf16* x, long long ldx, const int32_t* ids, const float* weights, int T,
                                  int top_k, int E, int d, int h, int group, const void* w_ug, const void* w_down,
                                  moe_bf16* out, long long ldo, void* ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (T < 0 || top_k < 1 || E < 1 || d < 1 || h < 1 || ldx < 0 || ldo < d) return MOE_ERR_INVALID_ARG;
  if (top_k > 32 || E > MAX_MATRICES / 2 || !dim_ok(d) || !dim_ok(h) || !group_ok(group) ||
      static_cast<long long>(T) * top_k > MAX_SLOTS)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && (!x || !ids || !w_ug || !w_down || !out)) return MOE_ERR_INVALID_ARG;
  if (!element_aligned(x, 2) || !element_aligned(ids, 4) || !element_aligned(weights, 4) || !element_aligned(out, 2) ||
      ((reinterpret_cast<uintptr_t>(w_ug) | reinterpret_cast<uintptr_t>(w_down) | reinterpret_cast<uintptr_t>(ws)) & 255u) != 0)
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < w4_decode_workspace_bytes(static_cast<long long>(T) * top_k, E, d, h)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (T > 0 && !ws) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_device();
  if (st != MOE_OK || T == 0) return st;
  const Packed ug = packed_at(w_ug, 2 * E, h, d, group), dn = packed_at(w_down, E, d, h, group);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  bf16* a = static_cast<bf16*>(ws);
  cudaError_t err = launch_dependent(w4_up_kernel, dim3((h + 7) / 8, T * top_k), 256, 0, s, reinterpret_cast<const bf16*>(x), ldx,
                                     ids, top_k, E, d, h, ug, a);
  if (err == cudaSuccess)
    err = launch_dependent(w4_down_kernel, dim3((d + 7) / 8, T), 256, 0, s, static_cast<const bf16*>(a), ids, weights, top_k, E, d, h,
                           dn, reinterpret_cast<bf16*>(out), ldo);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

}  // extern "C"
