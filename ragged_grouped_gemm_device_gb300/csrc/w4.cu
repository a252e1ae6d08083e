// Few tokens through 4-bit integer weights with group scales: w = scale (code - zero).
//
//   matvec: y[s] = W[ids[s]] x[s / top_k];  decode: out[t] = sum_j weight[t, j] SwiGLU(x[t] W_ug,e^T) W_down,e
//
// Packed layout (include/moe_gg.h): one piece for 16 rows by 128 elements, 1024 bytes of codes and behind them the groups'
// scales and zero points, those of rows r and r + 8 together. A lane's 16 bytes of codes are what it multiplies.
//
// 16 rows by 8 columns by 16 elements are one matrix instruction on bf16 values 16 + code, which a code becomes by one instruction
// for two; so few tokens' columns are mostly empty, but a weight is unpacked once for up to eight tokens, and unpacking is what
// bounds these products besides memory: 7 instructions of the half-rate pipe for eight codes. One token, 4096 x 4096: 3.7 us
// (2.4 TB/s; a launch and two round trips to memory, one for each segment of 2048 elements of the weights). 16 tokens, 8 of 128
// experts of 2048 x 768, groups of 32: 66.9 us (3.3 TB/s). At 63 us, before SwiGLU's output had two parts, the two products took 30 and 23
// without the arithmetic and 37 and 34 without the loads.
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
  const uint8_t* base;
  int tiles, chunks, per;  // 16-row tiles of a matrix, 128-element chunks of a row, groups of a chunk
};
__host__ __device__ constexpr int piece_bytes(int per) { return (1024 + 40 * per + 15) / 16 * 16; }

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
int groups_of(int K, int group) { return (K + group - 1) / group; }
bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }

size_t pieces(int matrices, int N, int K) {
  return static_cast<size_t>(matrices) * ((N + 15) / 16) * ((K + 127) / 128);
}
Packed packed_at(const void* p, int N, int K, int group) {
  return {static_cast<const uint8_t*>(p), (N + 15) / 16, (K + 127) / 128, 128 / group};
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
    uint8_t* piece = const_cast<uint8_t*>(p.base) + i * piece_bytes(p.per);
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
          w[q] = __funnelshift_l(w[q], w[q], 3);
        }
      }
      *reinterpret_cast<uint4*>(piece + half * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
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
      reinterpret_cast<uint32_t*>(piece + 1024)[g * p.per + t] = s;
      piece[1024 + 32 * p.per + g * p.per + t] = static_cast<uint8_t>(z);
    }
  }
}

// ------------------------------------------------------------------ products
// D[16 x 8] += A[16 x 16] B[16 x 8], bf16 operands, fp32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// This lane's part of a piece: the codes of rows g and g + 8, its groups' scales (a pair of rows in a word) and zero points.
template <typename T>
__device__ __forceinline__ T fetch_global(const uint8_t* p) {
  return __ldg(reinterpret_cast<const T*>(p));
}
template <typename T>
__device__ __forceinline__ T fetch_shared(const uint8_t* p) {
  return *reinterpret_cast<const T*>(p);
}
template <int PER>
struct Piece {
  static constexpr int bytes = piece_bytes(PER);
  uint4 lo, hi;
  uint32_t s[PER], z;
#define W4_LOAD(fetch)                                                                   \
  lo = fetch<uint4>(p + lane * 16);                                                      \
  hi = fetch<uint4>(p + 512 + lane * 16);                                                \
  const uint8_t *sc = p + 1024 + (lane >> 2) * 4 * PER, *zp = p + 1024 + 32 * PER + (lane >> 2) * PER; \
  if constexpr (PER == 4) {                                                              \
    const uint4 q = fetch<uint4>(sc);                                                    \
    s[0] = q.x, s[1] = q.y, s[2] = q.z, s[3] = q.w;                                      \
    z = fetch<uint32_t>(zp);                                                             \
  } else if constexpr (PER == 2) {                                                       \
    const uint2 q = fetch<uint2>(sc);                                                    \
    s[0] = q.x, s[1] = q.y;                                                              \
    z = fetch<uint16_t>(zp);                                                             \
  } else {                                                                               \
    s[0] = fetch<uint32_t>(sc);                                                          \
    z = fetch<uint8_t>(zp);                                                              \
  }
  __device__ __forceinline__ void load(const uint8_t* p, int lane) { W4_LOAD(fetch_global) }
  __device__ __forceinline__ void load_shared(const uint8_t* p, int lane) { W4_LOAD(fetch_shared) }
#undef W4_LOAD
};

__device__ __forceinline__ uint32_t word(const uint4& v, int q) { return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w; }

// Eight codes as four bf16 pairs of 16 + code: the code in the upper four mantissa bits of a bf16 in [16, 32). Both constants
// in registers, so that each pair takes one instruction behind its shift.
struct Unpack {
  uint32_t mask, base;
  __device__ __forceinline__ Unpack() {
    asm volatile("mov.b32 %0, 0x00780078;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x41804180;" : "=r"(base));
  }
  __device__ __forceinline__ uint32_t pick(uint32_t w) const {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "r"(base));  // (w & mask) | base
    return d;
  }
  __device__ __forceinline__ void operator()(uint32_t w, uint32_t (&p)[4]) const {
    p[0] = pick(w);
    p[1] = pick(w >> 4);
    p[2] = pick(w >> 8);
    p[3] = pick(__funnelshift_r(w, w, 12));
  }
};

// tot += factor scale (codes - zero) x of TILES pieces of the same columns. b(q, t): the 8 bf16 values of x of this lane for
// word q and column tile t, with SPLIT and `full` in tiles NT + t what is added to them; nx(q, t): minus the sums of x over the 32
// elements of word q, of this lane's two columns. A group's sum
// starts at -(16 + zero) sum x, which takes the codes' 16 and the zero point away without an instruction for each pair of
// codes: terms of up to 31 |x| instead of 15 |x| in an fp32 sum. A group of several words has two sums, so that a product need
// not wait for the one before it.
template <int PER, int NT, int TILES, bool SPLIT, typename B, typename X>
__device__ __forceinline__ void multiply(const Piece<PER> (&w)[TILES], float (&tot)[TILES][NT][4], float factor, const Unpack& unpack, const B& b, const X& nx,
                                         bool full = false) {
  constexpr int RUN = 4 / PER, SUMS = RUN > 1 ? 2 : 1;  // words of a group, sums of a group
  float acc[TILES][SUMS][NT][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int j = q / RUN;
    if (q % RUN == 0) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float2 v = nx(q, t);
#pragma unroll
        for (int r = 1; r < RUN; ++r) {
          const float2 u = nx(q + r, t);
          v.x += u.x;
          v.y += u.y;
        }
#pragma unroll
        for (int h = 0; h < TILES; ++h) {
          // 16 + zero: its four bits to bit 19 of an fp32 in [16, 32)
          const uint32_t z = w[h].z;
          const float zg = __uint_as_float(0x41800000u | ((j < 3 ? z << (j < 3 ? 19 - 8 * j : 0) : z >> 5) & 0x00780000u));
          const float zh = __uint_as_float(0x41800000u | ((j < 2 ? z << (j < 2 ? 15 - 8 * j : 0) : z >> (j < 2 ? 0 : 8 * j - 15)) & 0x00780000u));
          acc[h][0][t][0] = zg * v.x;
          acc[h][0][t][1] = zg * v.y;
          acc[h][0][t][2] = zh * v.x;
          acc[h][0][t][3] = zh * v.y;
          if constexpr (SUMS == 2) acc[h][1][t][0] = acc[h][1][t][1] = acc[h][1][t][2] = acc[h][1][t][3] = 0.f;
        }
      }
    }
    constexpr int XT = SPLIT ? 2 * NT : NT;
    uint4 v[XT];
#pragma unroll
    for (int t = 0; t < NT; ++t) v[t] = b(q, t);
    if (SPLIT && full) {
#pragma unroll
      for (int t = NT; t < XT; ++t) v[t] = b(q, t);
    }
#pragma unroll
    for (int h = 0; h < TILES; ++h) {
      uint32_t pg[4], ph[4];
      unpack(word(w[h].lo, q), pg);
      unpack(word(w[h].hi, q), ph);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma16816(acc[h][0][t], pg[0], ph[0], pg[1], ph[1], v[t].x, v[t].y);
        mma16816(acc[h][SUMS - 1][t], pg[2], ph[2], pg[3], ph[3], v[t].z, v[t].w);
      }
      if (SPLIT && full) {
#pragma unroll
        for (int t = NT; t < XT; ++t) {
          mma16816(acc[h][0][t - NT], pg[0], ph[0], pg[1], ph[1], v[t].x, v[t].y);
          mma16816(acc[h][SUMS - 1][t - NT], pg[2], ph[2], pg[3], ph[3], v[t].z, v[t].w);
        }
      }
    }
    if (q % RUN == RUN - 1) {
#pragma unroll
      for (int h = 0; h < TILES; ++h) {
        const float sg = bf16_lo(w[h].s[j]) * factor, sh = bf16_hi(w[h].s[j]) * factor;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float sum = SUMS == 2 ? acc[h][0][t][i] + acc[h][SUMS - 1][t][i] : acc[h][0][t][i];
            tot[h][t][i] = fmaf(i < 2 ? sg : sh, sum, tot[h][t][i]);
          }
        }
      }
    }
  }
}

// Eight bf16 of a row from column k: one 16-byte load, or single elements; zeros past K.
template <bool VEC>
__device__ __forceinline__ uint4 load_x(const bf16* row, int k, int K) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if constexpr (VEC) {
    if (k < K) v = *reinterpret_cast<const uint4*>(row + k);
  } else {
    const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = k + i < K ? r[k + i] : 0;
    v = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
  return v;
}

__device__ __forceinline__ float sum8(const uint4& v) {
  return ((bf16_lo(v.x) + bf16_hi(v.x)) + (bf16_lo(v.y) + bf16_hi(v.y))) + ((bf16_lo(v.z) + bf16_hi(v.z)) + (bf16_lo(v.w) + bf16_hi(v.w)));
}

// Minus the sums of x over the 32 elements of a word, of this lane's two columns: a product with -1.
__device__ __forceinline__ float2 minus_sums(const uint4& v) {
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  constexpr uint32_t one = 0xBF80BF80u;  // -1, twice
  mma16816(sum, one, one, one, one, v.x, v.y);
  mma16816(sum, one, one, one, one, v.z, v.w);
  return make_float2(sum[0], sum[1]);
}

struct W4Args {
  const bf16* x;
  long long ldx;
  const int32_t* ids;      // nullable: matrix 0 for all
  const float* weights;    // down: nullable
  int slots, top_k, xdiv;  // slot s reads row s / xdiv of x
  int E, N, K;
  Packed w;
  void* out;
  long long ldo;
  int pitch;               // SWIGLU: values of a row of the output
  bool y_bf16;
  bool early;              // ids are from before the kernel ahead, which only made x
};

constexpr int SEGMENT = 16;  // chunks of x in shared memory at a time

__device__ __forceinline__ void put_out(const W4Args& a, int slot, int row, float v) {
  if (a.y_bf16) static_cast<bf16*>(a.out)[slot * a.ldo + row] = __float2bfloat16_rn(v);
  else static_cast<float*>(a.out)[slot * a.ldo + row] = v;
}
// SwiGLU's output, as a sum of two bf16 values (off by at most 2^-16 of it; one bf16 by 2^-8, which was most of the decode step's
// error before its output is rounded): a row of the upper ones, then one of the lower. Rows past h up to the pitch: their scales are 0.
__device__ __forceinline__ void put_swiglu(const W4Args& a, int slot, int row, float gate, float up) {
  if (row >= a.pitch) return;
  const float v = gate / (1.0f + expf(-gate)) * up;
  const bf16 hi = __float2bfloat16_rn(v);
  bf16* o = static_cast<bf16*>(a.out) + slot * a.ldo + row;
  o[0] = hi;
  o[a.pitch] = __float2bfloat16_rn(v - __bfloat162float(hi));
}

// ------------------------------------------------------------------ one token
// Block (tile, slot) owns 16 rows of the slot's matrix (with SWIGLU of both halves, gate and up). Its warps share the chunks of a
// segment, U pieces (pairs of pieces) each, which are on their way at once, and add up their sums in shared memory, in warp order. SPLIT: x is a sum of two
// rows, the second behind the first, which take the first two columns of the eight.
template <int PER, int WARPS, bool SWIGLU, bool SPLIT, bool VEC>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 2 : 3) w4_slot_kernel(const W4Args a) {
  constexpr int U = SEGMENT / WARPS, TILES = SWIGLU ? 2 : 1, PARTS = SPLIT ? 2 : 1;
  __shared__ uint4 xs[SEGMENT * 4][PARTS * 4];
  __shared__ float xsum[SEGMENT * 4];  // minus the sums
  __shared__ float sums[WARPS][TILES][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tile = blockIdx.x, slot = blockIdx.y;
  if (!a.early) grid_wait();
  const int e = a.ids == nullptr ? 0 : after_wait(a.ids)[slot];
  if (e < 0 || e >= a.E) {
    if (a.early) grid_wait();
    const int row = tile * 16 + threadIdx.x;
    if (!SWIGLU && threadIdx.x < 16 && row < a.N) put_out(a, slot, row, 0.f);
    return;
  }
  const bf16* x = after_wait(a.x) + (slot / a.xdiv) * a.ldx;
  const Unpack unpack;
  float tot[TILES][1][4];
  const uint8_t* piece0[TILES];
#pragma unroll
  for (int h = 0; h < TILES; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) tot[h][0][i] = 0.f;
    piece0[h] = a.w.base + (static_cast<size_t>(e * TILES + h) * a.w.tiles + tile) * a.w.chunks * Piece<PER>::bytes;
  }
  for (int seg0 = 0; seg0 < a.w.chunks; seg0 += SEGMENT) {
    const int chunks = min(SEGMENT, a.w.chunks - seg0);
    Piece<PER> p[U][TILES];
#pragma unroll
    for (int u = 0; u < U; ++u)  // on their way while x comes
      if (warp + u * WARPS < chunks) {
#pragma unroll
        for (int h = 0; h < TILES; ++h) p[u][h].load(piece0[h] + static_cast<size_t>(seg0 + warp + u * WARPS) * Piece<PER>::bytes, lane);
      }
    if (a.early && seg0 == 0) grid_wait();
    __syncthreads();
    // Each thread eight elements, four threads the 32 of a sum; chunks * 16 is a multiple of 16, so whole groups of four
    for (int i = threadIdx.x; i < (chunks * 16 + 31 & ~31); i += WARPS * 32) {
      float sum = 0.f;
      if (i < chunks * 16) {
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
          const uint4 v = load_x<VEC>(x + part * a.K, (seg0 * 16 + i) * 8, a.K);
          xs[i >> 2][part * 4 + (i & 3)] = v;
          sum += sum8(v);
        }
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (i < chunks * 16 && (i & 3) == 0) xsum[i >> 2] = -sum;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (warp + u * WARPS >= chunks) break;
      const int s0 = (warp + u * WARPS) * 4;
      // the first columns of eight; the others' sums are not read
      multiply<PER, 1, TILES, false>(p[u], tot, 1.0f, unpack,
                                     [&](int q, int) { return lane < PARTS * 4 ? xs[s0 + q][lane] : make_uint4(0, 0, 0, 0); },
                                     [&](int q, int) { return make_float2(xsum[s0 + q], 0.f); });
    }
  }
  // columns 0 and 1: registers 0 and 2, 1 and 3 of the lanes with (lane & 3) = 0
  if ((lane & 3) == 0) {
#pragma unroll
    for (int h = 0; h < TILES; ++h) {
      sums[warp][h][lane >> 2] = SPLIT ? tot[h][0][0] + tot[h][0][1] : tot[h][0][0];
      sums[warp][h][8 + (lane >> 2)] = SPLIT ? tot[h][0][2] + tot[h][0][3] : tot[h][0][2];
    }
  }
  __syncthreads();
  if (threadIdx.x >= 16) return;
  float v[TILES];
#pragma unroll
  for (int h = 0; h < TILES; ++h) {
    v[h] = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v[h] += sums[w][h][threadIdx.x];
  }
  const int row = tile * 16 + threadIdx.x;
  if constexpr (SWIGLU) put_swiglu(a, slot, row, v[0], v[1]);
  else if (row < a.N) put_out(a, slot, row, v[0]);
}

// ------------------------------------------------------------------ several tokens
// Groups of up to 8 NT slots of one expert, each with all tiles of its weights, are one list of tasks (group, tile set) that the
// blocks share evenly, each a run of it: an expert's weights are read once for each of its groups. x of a group is fetched once or twice
// by a block while it fits shared memory, and for each task where it is longer (K above 2048, of
// moe_w4_matvec's groups of eight above 4096; 16 tokens, 8 of 64 experts of 4096 x 2048, groups of 128: 330 us for both products, 109 for their
// bytes). A warp's pieces go through a ring of its own in shared memory, filled by asynchronous copies that run ahead over tasks and
// groups, so that the copies in flight do not depend on how far the sums are, and no warp waits for another's.
struct StreamShape {
  int wk;       // warps that share K; WARPS / wk tiles (with SWIGLU pairs of tiles) are a task
  int sets;     // tasks of a group
  int xchunks;  // chunks of x in shared memory
};

template <int PER, int NT, int WARPS, bool SWIGLU, bool SPLIT>
struct StreamSmem {
  static constexpr int TILES = SWIGLU ? 2 : 1, XT = SPLIT ? 2 * NT : NT;  // XT: column tiles of x
  static constexpr int step = TILES * piece_bytes(PER);  // bytes of one ring slot
  static constexpr int depth = WARPS == 16 ? 2 : SWIGLU ? 3 : 4;  // slots of a warp's ring
  static constexpr int sum_floats = WARPS * TILES * NT * 128, buffers = WARPS == 16 ? 1 : 2;
  int ring, x, xsum, sums, list, groups, count, total;  // byte offsets
  __host__ __device__ StreamSmem(const W4Args& a, const StreamShape& sh) {
    ring = 0;
    x = ring + WARPS * depth * step;
    xsum = x + sh.xchunks * 4 * 8 * XT * 64;
    sums = xsum + sh.xchunks * 4 * 8 * NT * 4;
    list = sums + buffers * sum_floats * 4;
    groups = list + (a.slots * 4 + 15) / 16 * 16;
    count = groups + most_groups(a) * 8;
    total = count + (a.ids == nullptr ? 0 : (a.E + 1) * 4);
  }
  // groups at most: every slot alone, or as many full groups as the slots make and one that is not full of every expert
  static __host__ __device__ int most_groups(const W4Args& a) {
    if (a.ids == nullptr) return (a.slots + 8 * NT - 1) / (8 * NT);
    const int m = a.E + a.slots / (8 * NT);
    return m < a.slots ? m : a.slots;
  }
};

// SPLIT: x is a sum of two rows, the second behind the first. The second rows take the other half of the columns where a group leaves
// that free, and column tiles of their own where not, which is twice the matrix instructions (16 tokens, 8 of 128 experts: 66.9 us; 68.3
// with tiles of their own for all, 65.0 without the second rows. 128 tokens, 8 of 64, whose groups are full: 145.8 and 134.6 without).
template <int PER, int NT, int WARPS, bool SWIGLU, bool SPLIT, bool VEC>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 16 ? 1 : 2) w4_stream_kernel(const W4Args a, const StreamShape sh) {
  using Smem = StreamSmem<PER, NT, WARPS, SWIGLU, SPLIT>;
  constexpr int TILES = Smem::TILES, BYTES = Piece<PER>::bytes, COLS = 8 * NT, XT = Smem::XT, STREAM_THREADS = WARPS * 32;
  extern __shared__ __align__(16) uint8_t smem[];
  const Smem at(a, sh);
  uint4* xs = reinterpret_cast<uint4*>(smem + at.x);          // [chunks * 4][8 XT][4]
  float* xsum = reinterpret_cast<float*>(smem + at.xsum);     // [chunks * 4][COLS]: minus the sums
  int* list = reinterpret_cast<int*>(smem + at.list);         // slots, expert by expert
  int2* groups = reinterpret_cast<int2*>(smem + at.groups);   // expert, first slot in list | slots << 16
  int* count = reinterpret_cast<int*>(smem + at.count);       // slots of each expert, of none; then where the next one goes
  __shared__ int n_groups;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!a.early) grid_wait();
  const int32_t* ids = after_wait(a.ids);
  if (a.ids == nullptr) {
    for (int i = threadIdx.x; i < a.slots; i += STREAM_THREADS) {
      list[i] = i;
      if (i % COLS == 0) groups[i / COLS] = make_int2(0, i | min(COLS, a.slots - i) << 16);
    }
    if (threadIdx.x == 0) n_groups = (a.slots + COLS - 1) / COLS;
  } else {
    const auto of = [&](int i) {
      const int e = ids[i];
      return e >= 0 && e < a.E ? e : a.E;
    };
    for (int i = threadIdx.x; i <= a.E; i += STREAM_THREADS) count[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.slots; i += STREAM_THREADS) atomicAdd(count + of(i), 1);
    __syncthreads();
    if (warp == 0) {  // where each expert's slots begin, and the groups that they make
      int slots = 0, made = 0;
      for (int e0 = 0; e0 <= a.E; e0 += 32) {
        const int e = e0 + lane;
        const int c = e <= a.E ? count[e] : 0;
        const int g = e < a.E ? (c + COLS - 1) / COLS : 0;
        int sum = c | g << 16;  // both running sums in one word
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += v;
        }
        const int first = slots + (sum & 0xFFFF) - c, to = made + (sum >> 16) - g;
        if (e <= a.E) count[e] = first;
        for (int i = 0; i < g; ++i) groups[to + i] = make_int2(e, (first + COLS * i) | min(COLS, c - COLS * i) << 16);
        sum = __shfl_sync(0xffffffffu, sum, 31);
        slots += sum & 0xFFFF;
        made += sum >> 16;
      }
      if (lane == 0) n_groups = made;
      // The slots in order, by one warp: every block has to find the same slots in the same group.
      for (int i0 = 0; i0 < a.slots; i0 += 32) {
        const int i = i0 + lane, e = i < a.slots ? of(i) : a.E + 1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1)), at_e = i < a.slots ? count[e] : 0;
        __syncwarp();
        if (i < a.slots) {
          list[at_e + rank] = i;
          if (rank == 0) count[e] = at_e + __popc(same);
        }
        __syncwarp();
      }
    }
  }
  __syncthreads();
  const int wk = warp & (sh.wk - 1), wts = WARPS / sh.wk, wt = warp / sh.wk;
  const long long tasks = static_cast<long long>(n_groups) * sh.sets;
  const int t0 = static_cast<int>(tasks * blockIdx.x / gridDim.x), t1 = static_cast<int>(tasks * (blockIdx.x + 1) / gridDim.x);
  constexpr int depth = Smem::depth;
  const int chunks = a.w.chunks;

  // Where this warp's copies are: the tasks not begun yet, the next one's group and set, and in the one begun the next piece and how
  // many are left
  const int mine = wk < chunks ? (chunks - 1 - wk) / sh.wk + 1 : 0;  // pieces of a task that are this warp's
  int f_tasks = mine > 0 ? t1 - t0 : 0, f_group = t0 / sh.sets, f_set = t0 - f_group * sh.sets, f_left = 0;
  const uint8_t* f_src = nullptr;
  const size_t other = static_cast<size_t>(a.w.tiles) * chunks * BYTES;  // from a gate tile to the up tile
  const uint32_t ring = smem_u32(smem + at.ring) + warp * depth * Smem::step, ring_end = ring + depth * Smem::step;
  const uint32_t lane16 = lane * 16;
  const bool tail = lane < (BYTES - 1024) / 16;
  const int f_step = sh.wk * BYTES;
  const auto fill = [&](uint32_t to) {
    while (f_left == 0 && f_tasks > 0) {
      const int e = groups[f_group].x, tile = f_set * wts + wt;
      if (tile < a.w.tiles) {
        f_left = mine;
        f_src = a.w.base + ((static_cast<size_t>(e * TILES) * a.w.tiles + tile) * chunks + wk) * BYTES + lane16;
      }
      --f_tasks;
      if (++f_set == sh.sets) {
        f_set = 0;
        ++f_group;
      }
    }
    if (f_left > 0) {
      const uint32_t dst = to + lane16;
#pragma unroll
      for (int h = 0; h < TILES; ++h) {
        const uint8_t* src = f_src + (h == 1 ? other : 0);
        copy16_async(dst + h * BYTES, src);
        copy16_async(dst + h * BYTES + 512, src + 512);
        if (tail) copy16_async(dst + h * BYTES + 1024, src + 1024);
      }
      f_src += f_step;
      --f_left;
    }
    copy_commit();
  };
  for (uint32_t to = ring; to != ring_end; to += Smem::step) fill(to);

  if constexpr (SWIGLU) grid_release();  // the down product reads the ids and its first weights meanwhile
  if (a.early) grid_wait();
  const bf16* x = after_wait(a.x);
  if (!SWIGLU && a.ids != nullptr) {  // rows of dropped slots
    for (int i = blockIdx.x; i < a.slots; i += gridDim.x) {
      const int e = ids[i];
      if (e >= 0 && e < a.E) continue;
      for (int c = threadIdx.x; c < a.N; c += STREAM_THREADS) put_out(a, i, c, 0.f);
    }
  }
  const Unpack unpack;
  uint32_t slot = 0;  // byte offset in this warp's ring
  const uint8_t* const my_ring = smem + at.ring + warp * depth * Smem::step;
  int in_group = -1, in_seg = -1, par = 0, group = t0 / sh.sets, set = t0 - group * sh.sets;
  for (int t = t0; t < t1; ++t, ++set) {
    if (set == sh.sets) {
      set = 0;
      ++group;
    }
    const int2 info = groups[group];
    const int first = info.y & 0xFFFF, rows = info.y >> 16;
    const bool live = set * wts + wt < a.w.tiles, half = SPLIT && rows <= COLS / 2;
    float tot[TILES][NT][4];
#pragma unroll
    for (int h = 0; h < TILES; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[h][t][i] = 0.f;
    for (int seg0 = 0; seg0 < chunks; seg0 += sh.xchunks) {
      const int n = min(sh.xchunks, chunks - seg0);
      if (group != in_group || seg0 != in_seg) {
        __syncthreads();  // x there is no longer read
        // All columns, zeros where the group has fewer rows. A thread takes eight elements, four threads the 32 of a sum.
        for (int i = threadIdx.x; i < n * 16 * COLS; i += STREAM_THREADS) {
          const int col = i / (n * 16), k8 = i - col * (n * 16);
          float sum = 0.f;
#pragma unroll
          for (int part = 0; part < XT / NT; ++part) {
            if (part == 1 && half) break;
            uint4 v = make_uint4(0, 0, 0, 0);
            const int c = half ? col & (COLS / 2 - 1) : col;
            if (c < rows) v = load_x<VEC>(x + (list[first + c] / a.xdiv) * a.ldx + (part == 1 || c != col ? a.K : 0), (seg0 * 16 + k8) * 8, a.K);
            xs[((k8 >> 2) * 8 * XT + part * COLS + col) * 4 + (k8 & 3)] = v;
            sum += sum8(v);
          }
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);  // the bound is a multiple of 32: whole warps
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          if ((k8 & 3) == 0) xsum[(k8 >> 2) * COLS + col] = -sum;
        }
        __syncthreads();
        in_group = group;
        in_seg = seg0;
      }
      if (!live) continue;
      // chunks of this segment that are this warp's: those equal to wk modulo the warps that share K
      const int c0 = (wk - seg0) & (sh.wk - 1);
      const uint4* xp = xs + c0 * 128 * XT + lane;
      const float* sp = xsum + c0 * 4 * COLS + 2 * (lane & 3);
      for (int c = c0; c < n; c += sh.wk, xp += sh.wk * 128 * XT, sp += sh.wk * 4 * COLS) {
        copy_wait<depth - 1>();  // younger groups of copies may be on their way
        __syncwarp();
        Piece<PER> p[TILES];
#pragma unroll
        for (int h = 0; h < TILES; ++h) p[h].load_shared(my_ring + slot + h * BYTES, lane);
        __syncwarp();  // every lane has its part: the slot is free
        fill(ring + slot);
        slot = slot == (depth - 1) * Smem::step ? 0 : slot + Smem::step;
        const auto b = [&](int q, int t) { return xp[(q * XT + t) * 32]; };
        const auto nx = [&](int q, int t) { return *reinterpret_cast<const float2*>(sp + (q * NT + t) * 8); };
        multiply<PER, NT, TILES, SPLIT>(p, tot, 1.0f, unpack, b, nx, !half);
      }
    }
    // the sums of the warps: [warp][half][column tile][register][lane]
    float* sums = reinterpret_cast<float*>(smem + at.sums) + par * Smem::sum_floats;
    par ^= Smem::buffers - 1;
#pragma unroll
    for (int h = 0; h < TILES; ++h)
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[(((warp * TILES + h) * NT + c) * 4 + i) * 32 + lane] = tot[h][c][i];
    // only the warps that share a tile's K wait for one another
    const auto meet = [&] {
      if (sh.wk == 1) __syncwarp();
      else asm volatile("bar.sync %0, %1;" ::"r"(1 + wt), "r"(sh.wk * 32) : "memory");
    };
    meet();
    for (int i = wk * 32 + lane; i < 16 * rows; i += sh.wk * 32) {
      const int r = i & 15, col = i >> 4;  // consecutive threads: consecutive rows of the output
      // row r, column c of a tile lie in register (r / 8) 2 + c % 2 of lane (r % 8) 4 + (c % 8) / 2
      const int from = ((col >> 3) * 4 + (r >> 3) * 2 + (col & 1)) * 32 + (r & 7) * 4 + ((col & 7) >> 1);
      float v[TILES];
#pragma unroll
      for (int h = 0; h < TILES; ++h) {
        v[h] = 0.f;
        for (int w = 0; w < sh.wk; ++w) {
          const float* part = sums + ((wt * sh.wk + w) * TILES + h) * NT * 128 + from;
          v[h] += half ? part[0] + part[NT == 1 ? 2 : 128] : part[0];  // half of the columns further
        }
      }
      const int row = (set * wts + wt) * 16 + r, s = list[first + col];
      if constexpr (SWIGLU) put_swiglu(a, s, row, v[0], v[1]);
      else if (row < a.N) put_out(a, s, row, v[0]);
    }
    if (Smem::buffers == 1) meet();
  }
  copy_wait<0>();
}

// The down product and the combine of one token: block (tile, token) owns 16 columns of out[t]. The chunks of the token's top_k
// slots are one long contraction that its warps share, each slot's scales times its routing weight; no sums leave the block.
constexpr int DOWN_WARPS = 8;

template <int PER>
__global__ void __launch_bounds__(DOWN_WARPS * 32, 2) w4_down_token_kernel(const W4Args a) {
  constexpr int U = 3;
  __shared__ float sums[DOWN_WARPS][2][8];
  __shared__ int expert[32];
  __shared__ float weight[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tile = blockIdx.x, t = blockIdx.y;
  // the ids and weights are from before the kernel ahead, which only made x
  if (threadIdx.x < a.top_k) {
    const int s = t * a.top_k + threadIdx.x;
    const int e = after_wait(a.ids)[s];
    expert[threadIdx.x] = e >= 0 && e < a.E ? e : -1;
    weight[threadIdx.x] = a.weights ? after_wait(a.weights)[s] : 1.0f;
  }
  __syncthreads();
  const int items = a.top_k * a.w.chunks;
  float tot[1][1][4] = {{{0.f, 0.f, 0.f, 0.f}}};
  const Unpack unpack;
  bool waited = false;
  const bf16* x = a.x;
  for (int i0 = warp; i0 < items; i0 += DOWN_WARPS * U) {
    Piece<PER> p[U][1];
    uint4 v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * DOWN_WARPS, j = i / a.w.chunks, c = i % a.w.chunks;
      if (i >= items || expert[j] < 0) continue;
      p[u][0].load(a.w.base + ((static_cast<size_t>(expert[j]) * a.w.tiles + tile) * a.w.chunks + c) * Piece<PER>::bytes, lane);
    }
    if (!waited) {
      grid_wait();
      x = after_wait(a.x);
      waited = true;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * DOWN_WARPS, j = i / a.w.chunks, c = i % a.w.chunks;
      if (i >= items || expert[j] < 0) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q)  // SwiGLU's upper values in column 0, the lower ones in column 1
        v[u][q] = lane < 8 ? load_x<true>(x + static_cast<size_t>(t * a.top_k + j) * a.ldx + (lane >> 2) * a.K, c * 128 + q * 32 + (lane & 3) * 8, a.K)
                           : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * DOWN_WARPS, j = i / a.w.chunks;
      if (i >= items || expert[j] < 0) continue;
      // the sums of x by a product with ones: columns 0 and 1 of every row
      multiply<PER, 1, 1, false>(p[u], tot, weight[j], unpack, [&](int q, int) { return v[u][q]; }, [&](int q, int) { return minus_sums(v[u][q]); });
    }
  }
  if (!waited) grid_wait();
  // columns 0 and 1: registers 0 and 2, 1 and 3 of the lanes with (lane & 3) = 0
  if ((lane & 3) == 0) {
    sums[warp][0][lane >> 2] = tot[0][0][0] + tot[0][0][1];
    sums[warp][1][lane >> 2] = tot[0][0][2] + tot[0][0][3];
  }
  __syncthreads();
  const int row = tile * 16 + threadIdx.x;
  if (threadIdx.x < 16 && row < a.N) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < DOWN_WARPS; ++w) s += sums[w][threadIdx.x >> 3][threadIdx.x & 7];
    static_cast<bf16*>(a.out)[t * a.ldo + row] = __float2bfloat16_rn(s);
  }
}

// out[t] = sum_j weight[t, j] y[t, j] of fp32 rows, in slot order; eight rows' loads at a time
__global__ void __launch_bounds__(128) w4_combine_kernel(const float* y, long long ldy, const int32_t* ids, const float* weights,
                                                         int top_k, int E, int d, bf16* out, long long ldo) {
  __shared__ float weight[32];  // 0 of a dropped slot, whose row is not read
  __shared__ bool on[32];
  grid_wait();
  const int t = blockIdx.y;
  if (threadIdx.x < top_k) {
    const int e = after_wait(ids)[t * top_k + threadIdx.x];
    on[threadIdx.x] = e >= 0 && e < E;
    weight[threadIdx.x] = weights ? after_wait(weights)[t * top_k + threadIdx.x] : 1.0f;
  }
  __syncthreads();
  y = after_wait(y) + static_cast<long long>(t) * top_k * ldy;
  for (int c = blockIdx.x * 128 + threadIdx.x; c < d; c += gridDim.x * 128) {
    float v = 0.f;
    for (int j0 = 0; j0 < top_k; j0 += 8) {
      float r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = j0 + j < top_k && on[j0 + j] ? y[(j0 + j) * ldy + c] : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < top_k && on[j0 + j]) v = fmaf(weight[j0 + j], r[j], v);
    }
    out[t * ldo + c] = __float2bfloat16_rn(v);
  }
}

bool vec_x(const W4Args& a) { return a.K % 8 == 0 && a.ldx % 8 == 0 && aligned16(a.x); }

template <int PER, int NT, bool SWIGLU, bool SPLIT>
cudaError_t launch_stream(const W4Args& a, cudaStream_t s) {
  constexpr int WARPS = NT == 1 ? 8 : 16;
  using Smem = StreamSmem<PER, NT, WARPS, SWIGLU, SPLIT>;
  StreamShape sh;
  // Long rows are shared, three or four chunks a warp: with fewer the sums at the end of a task cost as much as its products, with more there are
  // too few tasks to share evenly. Short rows go to one warp each.
  sh.wk = a.w.chunks >= 24 ? 8 : a.w.chunks >= 12 ? 4 : 1;
  const int wts = WARPS / sh.wk;
  sh.sets = (a.w.tiles + wts - 1) / wts;
  sh.xchunks = std::min(a.w.chunks, SWIGLU || SPLIT || NT == 2 ? 16 : 32);
  const int smem = Smem(a, sh).total;
  const auto kernel = SPLIT || vec_x(a) ? w4_stream_kernel<PER, NT, WARPS, SWIGLU, SPLIT, true> : w4_stream_kernel<PER, NT, WARPS, SWIGLU, SPLIT, SPLIT>;
  const cudaError_t err = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kernel), 220 * 1024);
  if (err != cudaSuccess) return err;
  const long long most = static_cast<long long>(Smem::most_groups(a)) * sh.sets;
  const int blocks = static_cast<int>(std::min<long long>(most, (NT == 1 && smem <= 112 * 1024 ? 2 : 1) * static_cast<long long>(device_sm_count())));
  return launch_dependent(kernel, blocks, WARPS * 32, smem, s, a, sh);
}

template <int PER, bool SWIGLU, bool SPLIT>
cudaError_t launch_product(const W4Args& a, cudaStream_t s) {
  // A single token: a block for each tile, which starts sooner than a list of tasks is made. All weights of a tile's segment of 2048
  // elements are on their way at once: two pieces for each of eight warps, four pairs for each of four warps of gate and up, of which three
  // blocks fit on an SM (4096 x 4096: 5.6 us with four warps of two pieces, 3.9 so, with the second segment's weights a second
  // round trip to memory).
  if (a.slots == (a.ids == nullptr ? 1 : a.top_k)) {
    constexpr int WARPS = SWIGLU ? 4 : 8;
    const auto kernel = SPLIT || vec_x(a) ? w4_slot_kernel<PER, WARPS, SWIGLU, SPLIT, true> : w4_slot_kernel<PER, WARPS, SWIGLU, SPLIT, SPLIT>;
    return launch_dependent(kernel, dim3(a.w.tiles, a.slots), WARPS * 32, 0, s, a);
  }
  // Tokens of an expert, on average. With more than eight of them groups of 16 slots unpack its weights half as often, in one block of 16
  // warps, whose shared memory x fills (128 tokens, 8 of 64 experts of 2048 x 768: 133 us, 155 in groups of eight; with eight tokens
  // an expert both take 99 to 101, with four the larger groups 86 instead of 76; all before SwiGLU's output had two parts, with
  // which the 133 are 146).
  const int each = a.ids == nullptr ? a.slots : a.slots / a.E;
  return each <= 8 ? launch_stream<PER, 1, SWIGLU, SPLIT>(a, s) : launch_stream<PER, 2, SWIGLU, SPLIT>(a, s);
}
// SPLIT: x is a sum of two rows of K values, as put_swiglu() leaves them: 16-byte rows
template <bool SWIGLU, bool SPLIT>
cudaError_t launch_product(const W4Args& a, cudaStream_t s) {
  return a.w.per == 4   ? launch_product<4, SWIGLU, SPLIT>(a, s)
         : a.w.per == 2 ? launch_product<2, SWIGLU, SPLIT>(a, s)
                        : launch_product<1, SWIGLU, SPLIT>(a, s);
}

cudaError_t launch_down_token(const W4Args& a, int T, cudaStream_t s) {
  const dim3 grid(a.w.tiles, T);
  const auto kernel = a.w.per == 4 ? w4_down_token_kernel<4> : a.w.per == 2 ? w4_down_token_kernel<2> : w4_down_token_kernel<1>;
  return launch_dependent(kernel, grid, DOWN_WARPS * 32, 0, s, a);
}

// Whether the down product takes token by token. It then reads an expert's weights once for each slot, from the L2 but the
// first time, and saves the fp32 rows and a launch. The decode step so and by the list of tasks (us): 128 experts of 2048 x 768, 8 slots 10.5
// and 13.4, 32 slots 33.1 and 35.3, 48 slots 40.0 and 37.5, 128 slots 76.9 and 60.0; 256 of 2048 x 512, 32 slots 30.1 and 32.9, 64 slots
// 43.0 and 42.4; 8 of 2048 x 1024, 8 slots 16.8 and 21.6, 16 slots 22.4 and 23.1.
bool down_by_token(long long slots, int E) { return slots <= std::max(8, E / 4); }
int pitch_of(int h) { return (h + 7) / 8 * 8; }

bool dim_ok(int v) { return v >= 1 && v <= MAX_DIM; }

}  // namespace

size_t w4_weights_bytes(int matrices, int K, int N, int group) {
  if (matrices < 1 || matrices > MAX_MATRICES || !dim_ok(K) || !dim_ok(N) || !group_ok(group)) return 0;
  return round256(pieces(matrices, N, K) * piece_bytes(128 / group));
}
size_t w4_decode_workspace_bytes(long long slots, int E, int d, int h) {
  if (slots < 0 || slots > MAX_SLOTS || !dim_ok(d) || !dim_ok(h)) return 0;
  // SwiGLU's rows, and the fp32 rows of the down product where it does not take token by token
  return round256(static_cast<size_t>(slots) * pitch_of(h) * 4) + (down_by_token(slots, E) ? 0 : static_cast<size_t>(slots) * d * 4);
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
      codes, reinterpret_cast<const bf16*>(scales), zeros, N, K, group, n, packed_at(packed, N, K, group));
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
  W4Args a{};
  a.x = reinterpret_cast<const bf16*>(x);
  a.ldx = ldx;
  a.ids = ids;
  a.slots = T * top_k;
  a.top_k = top_k;
  a.xdiv = top_k;
  a.E = matrices;
  a.N = N;
  a.K = K;
  a.w = packed_at(packed, N, K, group);
  a.out = y;
  a.ldo = ldy;
  a.y_bf16 = y_dtype == MOE_DTYPE_BF16;
  const cudaError_t err = launch_product<false, false>(a, reinterpret_cast<cudaStream_t>(stream));
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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int slots = T * top_k, pitch = pitch_of(h);
  bf16* act = static_cast<bf16*>(ws);
  W4Args a{};
  a.x = reinterpret_cast<const bf16*>(x);
  a.ldx = ldx;
  a.ids = ids;
  a.slots = slots;
  a.top_k = top_k;
  a.xdiv = top_k;
  a.E = E;
  a.N = h;
  a.K = d;
  a.w = packed_at(w_ug, h, d, group);
  a.out = act;
  a.ldo = 2 * pitch;
  a.pitch = pitch;
  cudaError_t err = launch_product<true, false>(a, s);
  if (err != cudaSuccess) return cuda_fail(err);
  W4Args b = a;
  b.x = act;
  b.ldx = 2 * pitch;
  b.weights = weights;
  b.xdiv = 1;
  b.N = d;
  b.K = pitch;  // zeros from h on
  b.early = true;
  b.w = packed_at(w_down, d, h, group);
  if (down_by_token(slots, E)) {
    b.out = out;
    b.ldo = ldo;
    err = launch_down_token(b, T, s);
  } else {
    float* y = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + round256(static_cast<size_t>(slots) * pitch * 4));
    b.out = y;
    b.ldo = d;
    err = launch_product<false, true>(b, s);
    if (err == cudaSuccess)
      err = launch_dependent(w4_combine_kernel, dim3(std::min((d + 127) / 128, 64), T), 128, 0, s, static_cast<const float*>(y),
                             static_cast<long long>(d), ids, weights, top_k, E, d, reinterpret_cast<bf16*>(out), ldo);
  }
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

}  // extern "C"
