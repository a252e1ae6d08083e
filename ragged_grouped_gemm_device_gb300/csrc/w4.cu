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
          w[q] = __funnelshift_l(w[q], w[q], 3);
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
// D[16 x 8] += A[16 x 16] B[16 x 8], bf16 operands, fp32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// This lane's part of a piece: the codes of rows g and g + 8, its groups' scales (a pair of rows in a word) and zero points.
template <int PER>
struct Piece {
  uint4 lo, hi;
  uint32_t s[PER], z;
  __device__ __forceinline__ void load(const Packed& p, size_t piece, int lane) {
    const uint4* c = reinterpret_cast<const uint4*>(p.codes + piece * 1024) + lane;
    lo = __ldg(c);
    hi = __ldg(c + 32);
    const size_t at = (piece * 8 + (lane >> 2)) * PER;
    if constexpr (PER == 4) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p.scales + at * 4));
      s[0] = q.x, s[1] = q.y, s[2] = q.z, s[3] = q.w;
      z = __ldg(reinterpret_cast<const uint32_t*>(p.zeros + at));
    } else if constexpr (PER == 2) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p.scales + at * 4));
      s[0] = q.x, s[1] = q.y;
      z = __ldg(reinterpret_cast<const uint16_t*>(p.zeros + at));
    } else {
      s[0] = __ldg(reinterpret_cast<const uint32_t*>(p.scales + at * 4));
      z = __ldg(p.zeros + at);
    }
  }
};

__device__ __forceinline__ uint32_t word(const uint4& v, int q) { return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w; }

// Eight codes as four bf16 pairs of 16 + code: the code in the upper four mantissa bits of a bf16 in [16, 32).
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&p)[4]) {
  p[0] = (w & 0x00780078u) | 0x41804180u;
  p[1] = ((w >> 4) & 0x00780078u) | 0x41804180u;
  p[2] = ((w >> 8) & 0x00780078u) | 0x41804180u;
  p[3] = (__funnelshift_r(w, w, 12) & 0x00780078u) | 0x41804180u;
}

// tot += factor scale (codes - zero) x of one piece. b(q, t): the 8 bf16 values of x of this lane for word q and column tile t; nx(q, t):
// minus the sums of x over the 32 elements of word q, of this lane's two columns. A group's sum starts at -(16 + zero) sum x, which
// takes the codes' 16 and the zero point away without an instruction for each pair of codes: terms of up to 31 |x| instead of
// 15 |x| in an fp32 sum.
template <int PER, int NT, typename B, typename X>
__device__ __forceinline__ void multiply(const Piece<PER>& w, float (&tot)[NT][4], float factor, const B& b, const X& nx) {
  constexpr int RUN = 4 / PER;  // words of a group
  float acc[NT][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int j = q / RUN;
    if (q % RUN == 0) {
      const float zg = __uint_as_float(0x41800000u | ((j < 3 ? w.z << (19 - 8 * j > 0 ? 19 - 8 * j : 0) : w.z >> 5) & 0x00780000u));
      const float zh = __uint_as_float(0x41800000u | ((j < 2 ? w.z << (15 - 8 * j > 0 ? 15 - 8 * j : 0) : w.z >> (8 * j - 15)) & 0x00780000u));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float2 v = nx(q, t);
#pragma unroll
        for (int r = 1; r < RUN; ++r) {
          const float2 u = nx(q + r, t);
          v.x += u.x;
          v.y += u.y;
        }
        acc[t][0] = zg * v.x;
        acc[t][1] = zg * v.y;
        acc[t][2] = zh * v.x;
        acc[t][3] = zh * v.y;
      }
    }
    uint32_t pg[4], ph[4];
    unpack8(word(w.lo, q), pg);
    unpack8(word(w.hi, q), ph);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint4 v = b(q, t);
      mma16816(acc[t], pg[0], ph[0], pg[1], ph[1], v.x, v.y);
      mma16816(acc[t], pg[2], ph[2], pg[3], ph[3], v.z, v.w);
    }
    if (q % RUN == RUN - 1) {
      const float sg = bf16_lo(w.s[j]) * factor, sh = bf16_hi(w.s[j]) * factor;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        tot[t][0] = fmaf(sg, acc[t][0], tot[t][0]);
        tot[t][1] = fmaf(sg, acc[t][1], tot[t][1]);
        tot[t][2] = fmaf(sh, acc[t][2], tot[t][2]);
        tot[t][3] = fmaf(sh, acc[t][3], tot[t][3]);
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

struct W4Args {
  const bf16* x;
  long long ldx;
  const int32_t* ids;      // nullable: matrix 0 for all
  const float* weights;    // down: nullable
  int slots, top_k, xdiv;  // slot s reads row s / xdiv of x
  int E, N, K;
  int segment;             // chunks of x in shared memory at a time
  Packed w;
  void* out;
  long long ldo;
  bool y_bf16;
};

constexpr int SEGMENT = 16;  // chunks of x in shared memory at most
constexpr int WARPS = 4;

// Slots of one expert times its weights: WK warps of a block own 16 rows of the matrix (of both halves, gate and up, with
// SWIGLU) and take the slots of its expert 8 NT at a time. They share the chunks of K and add up their sums in shared
// memory, in warp order. A group is a slot that names its expert first (slots <= E), or an expert, with one more group for
// dropped slots; of a single token every slot is one.
template <int PER, int NT, int WK, bool SWIGLU, bool VEC>
__global__ void __launch_bounds__(WARPS * 32, NT == 1 ? 5 : 4) w4_group_kernel(const W4Args a) {
  constexpr int TILES = SWIGLU ? 2 : 1, COLS = 8 * NT, U = 2, WT = WARPS / WK;
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* xs = reinterpret_cast<uint4*>(smem);                                    // [chunks of a segment * 4][COLS][4]
  float* xsum = reinterpret_cast<float*>(smem + a.segment * 4 * COLS * 64);        // [chunks of a segment * 4][COLS]: minus the sums
  float* sums = xsum + a.segment * 4 * COLS;                                       // [WARPS][TILES][NT][4][32]
  int* list = reinterpret_cast<int*>(sums + WARPS * TILES * NT * 128);             // slots of this group
  __shared__ int counts[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = blockIdx.y;
  const int wk = warp % WK, tile = blockIdx.x * WT + warp / WK;  // this warp's share of K and its rows
  const bool live = tile < a.w.tiles;
  grid_wait();
  const int32_t* ids = after_wait(a.ids);
  const bool by_slot = a.slots <= a.E, single = a.ids == nullptr ? false : a.slots == a.top_k;
  int e = a.ids == nullptr ? 0 : by_slot || single ? ids[group] : group;
  const bool dropped = e < 0 || e >= a.E;
  int n = 1;
  if (single || (dropped && by_slot)) {
    if (threadIdx.x == 0) list[0] = group;
  } else if (a.ids == nullptr) {
    n = a.slots;
    for (int i = threadIdx.x; i < n; i += WARPS * 32) list[i] = i;
  } else {
    // the slots of expert e (of none of the experts: the last group) in order
    const int seg = (a.slots + WARPS * 32 - 1) / (WARPS * 32) * 32;  // slots of a warp
    const int i0 = warp * seg;
    const auto mine = [&](int i) {
      const int v = i < a.slots ? ids[i] : -1;
      return i < a.slots && (dropped ? v < 0 || v >= a.E : v == e);
    };
    int count = 0;
    for (int i = i0; i < i0 + seg; i += 32) count += __popc(__ballot_sync(0xffffffffu, mine(i + lane)));
    if (lane == 0) counts[warp] = count;
    __syncthreads();
    int at = 0;
    n = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      at += w < warp ? counts[w] : 0;
      n += counts[w];
    }
    for (int i = i0; i < i0 + seg; i += 32) {
      const bool m = mine(i + lane);
      const unsigned who = __ballot_sync(0xffffffffu, m);
      if (m) list[at + __popc(who & ((1u << lane) - 1))] = i + lane;
      at += __popc(who);
    }
  }
  __syncthreads();
  if (n == 0) return;
  if (by_slot && !single && !dropped && a.ids != nullptr && list[0] != group) return;  // an earlier slot has this expert
  if (dropped) {
    if constexpr (!SWIGLU) {
      for (int i = threadIdx.x; i < n * 16 * WT; i += WARPS * 32) {
        const int row = blockIdx.x * WT * 16 + i % (16 * WT), slot = list[i / (16 * WT)];
        if (row >= a.N) continue;
        if (a.y_bf16) static_cast<bf16*>(a.out)[slot * a.ldo + row] = __float2bfloat16_rn(0.f);
        else static_cast<float*>(a.out)[slot * a.ldo + row] = 0.f;
      }
    }
    return;
  }
  const bf16* x = after_wait(a.x);
  for (int r0 = 0; r0 < n; r0 += COLS) {
    const int rows = min(COLS, n - r0);
    float tot[TILES][NT][4];
#pragma unroll
    for (int h = 0; h < TILES; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[h][t][i] = 0.f;
    size_t piece0[TILES];
#pragma unroll
    for (int h = 0; h < TILES; ++h) piece0[h] = (static_cast<size_t>(e * TILES + h) * a.w.tiles + tile) * a.w.chunks;
    for (int seg0 = 0; seg0 < a.w.chunks; seg0 += a.segment) {
      const int chunks = min(a.segment, a.w.chunks - seg0);
      Piece<PER> p[U][TILES];
      const auto load = [&](int c) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (live && c + u * WK < chunks) {
#pragma unroll
            for (int h = 0; h < TILES; ++h) p[u][h].load(a.w, piece0[h] + seg0 + c + u * WK, lane);
          }
      };
      load(wk);  // on their way while x comes
      __syncthreads();
      // Each thread eight elements, four threads the 32 of a sum; whole warps, because of the shuffles
      const int units = rows * chunks * 16;
      for (int i = threadIdx.x; i < (units + 31 & ~31); i += WARPS * 32) {
        const int col = i / (chunks * 16), k8 = i % (chunks * 16);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (i < units) {
          v = load_x<VEC>(x + (list[r0 + col] / a.xdiv) * a.ldx, (seg0 * 16 + k8) * 8, a.K);
          xs[((k8 >> 2) * COLS + col) * 4 + (k8 & 3)] = v;
        }
        float sum = ((bf16_lo(v.x) + bf16_hi(v.x)) + (bf16_lo(v.y) + bf16_hi(v.y))) + ((bf16_lo(v.z) + bf16_hi(v.z)) + (bf16_lo(v.w) + bf16_hi(v.w)));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (i < units && (k8 & 3) == 0) xsum[(k8 >> 2) * COLS + col] = -sum;
      }
      __syncthreads();
      for (int c = wk; live && c < chunks; c += WK * U) {
        if (c != wk) load(c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (c + u * WK >= chunks) break;
          const int s0 = (c + u * WK) * 4;
          const auto b = [&](int q, int t) {
            const int col = t * 8 + (lane >> 2);
            return col < rows ? xs[((s0 + q) * COLS + col) * 4 + (lane & 3)] : make_uint4(0, 0, 0, 0);
          };
          const auto nx = [&](int q, int t) {  // columns past the last row: what lies there goes into sums that nobody reads
            return *reinterpret_cast<const float2*>(xsum + (s0 + q) * COLS + t * 8 + 2 * (lane & 3));
          };
#pragma unroll
          for (int h = 0; h < TILES; ++h) multiply<PER, NT>(p[u][h], tot[h], 1.0f, b, nx);
        }
      }
    }
    // sums of the warps: [warp][half][column tile][register][lane]
#pragma unroll
    for (int h = 0; h < TILES; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[(((warp * TILES + h) * NT + t) * 4 + i) * 32 + lane] = tot[h][t][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * WT * rows; i += WARPS * 32) {
      const int w0 = i / 16 % WT, r = i & 15, col = i / (16 * WT);  // consecutive threads: consecutive rows of the output
      // row r, column c of a tile lie in register (r / 8) 2 + c % 2 of lane (r % 8) 4 + (c % 8) / 2
      const int at = (((col >> 3) * 4) + (r >> 3) * 2 + (col & 1)) * 32 + (r & 7) * 4 + ((col & 7) >> 1);
      float v[TILES];
#pragma unroll
      for (int h = 0; h < TILES; ++h) {
        v[h] = 0.f;
#pragma unroll
        for (int w = 0; w < WK; ++w) v[h] += sums[((w0 * WK + w) * TILES + h) * NT * 128 + at];
      }
      const int row = (blockIdx.x * WT + w0) * 16 + r, slot = list[r0 + col];
      if constexpr (SWIGLU) {
        // rows past h up to the pitch: their scales are 0
        if (row < a.ldo) static_cast<bf16*>(a.out)[slot * a.ldo + row] = __float2bfloat16_rn(v[0] / (1.0f + expf(-v[0])) * v[1]);
      } else if (row < a.N) {
        if (a.y_bf16) static_cast<bf16*>(a.out)[slot * a.ldo + row] = __float2bfloat16_rn(v[0]);
        else static_cast<float*>(a.out)[slot * a.ldo + row] = v[0];
      }
    }
    __syncthreads();
  }
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
  grid_wait();
  if (threadIdx.x < a.top_k) {
    const int s = t * a.top_k + threadIdx.x;
    const int e = after_wait(a.ids)[s];
    expert[threadIdx.x] = e >= 0 && e < a.E ? e : -1;
    weight[threadIdx.x] = a.weights ? after_wait(a.weights)[s] : 1.0f;
  }
  __syncthreads();
  const int items = a.top_k * a.w.chunks;
  float tot[1][4] = {{0.f, 0.f, 0.f, 0.f}};
  const bf16* x = after_wait(a.x);
  for (int i0 = warp; i0 < items; i0 += DOWN_WARPS * U) {
    Piece<PER> p[U];
    uint4 v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * DOWN_WARPS, j = i / a.w.chunks, c = i % a.w.chunks;
      if (i >= items || expert[j] < 0) continue;
      p[u].load(a.w, (static_cast<size_t>(expert[j]) * a.w.tiles + tile) * a.w.chunks + c, lane);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[u][q] = lane < 4 ? load_x<true>(x + static_cast<size_t>(t * a.top_k + j) * a.ldx, c * 128 + q * 32 + lane * 8, a.K)
                           : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * DOWN_WARPS, j = i / a.w.chunks;
      if (i >= items || expert[j] < 0) continue;
      // the sums of x by a product with ones: column 0 of every row
      multiply<PER, 1>(p[u], tot, weight[j], [&](int q, int) { return v[u][q]; }, [&](int q, int) {
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        constexpr uint32_t one = 0xBF80BF80u;  // -1, twice
        mma16816(sum, one, one, one, one, v[u][q].x, v[u][q].y);
        mma16816(sum, one, one, one, one, v[u][q].z, v[u][q].w);
        return make_float2(sum[0], sum[1]);
      });
    }
  }
  // column 0: registers 0 and 2 of the lanes with (lane & 3) = 0
  if ((lane & 3) == 0) {
    sums[warp][0][lane >> 2] = tot[0][0];
    sums[warp][1][lane >> 2] = tot[0][2];
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

// out[t] = sum_j weight[t, j] y[t, j] of fp32 rows, in slot order
__global__ void __launch_bounds__(128) w4_combine_kernel(const float* y, long long ldy, const int32_t* ids, const float* weights,
                                                         int top_k, int E, int d, bf16* out, long long ldo) {
  grid_wait();
  const int t = blockIdx.y;
  y = after_wait(y);
  for (int c = blockIdx.x * 128 + threadIdx.x; c < d; c += gridDim.x * 128) {
    float v = 0.f;
    for (int j = 0; j < top_k; ++j) {
      const int s = t * top_k + j, e = after_wait(ids)[s];
      if (e >= 0 && e < E) v = fmaf(weights ? after_wait(weights)[s] : 1.0f, y[s * ldy + c], v);
    }
    out[t * ldo + c] = __float2bfloat16_rn(v);
  }
}

template <int PER, int NT, int WK, bool SWIGLU, bool VEC>
cudaError_t launch_group_as(const W4Args& a, int groups, cudaStream_t s) {
  const int x_bytes = 4 * 8 * NT * 68, sum_bytes = WARPS * (SWIGLU ? 2 : 1) * NT * 512;
  const auto kernel = w4_group_kernel<PER, NT, WK, SWIGLU, VEC>;
  const int smem = a.segment * x_bytes + sum_bytes + std::max(1, a.slots) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t err = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kernel), SEGMENT * x_bytes + sum_bytes + MAX_SLOTS * 4);
    if (err != cudaSuccess) return err;
  }
  return launch_dependent(kernel, dim3((a.w.tiles * WK + WARPS - 1) / WARPS, groups), WARPS * 32, smem, s, a);
}
template <int PER, int NT, bool SWIGLU>
cudaError_t launch_group_split(const W4Args& a, int groups, cudaStream_t s) {
  const bool vec = a.K % 8 == 0 && a.ldx % 8 == 0 && aligned16(a.x);
  // The warps of a block share K where that gives no more than eight blocks for each SM: few blocks leave SMs idle, many have each its
  // share of reading ids and x.
  const bool few = static_cast<long long>(a.w.tiles) * groups <= 8LL * device_sm_count();
  if (few) return vec ? launch_group_as<PER, NT, 4, SWIGLU, true>(a, groups, s) : launch_group_as<PER, NT, 4, SWIGLU, false>(a, groups, s);
  return vec ? launch_group_as<PER, NT, 1, SWIGLU, true>(a, groups, s) : launch_group_as<PER, NT, 1, SWIGLU, false>(a, groups, s);
}

template <int PER, bool SWIGLU>
cudaError_t launch_group(W4Args a, cudaStream_t s) {
  a.segment = std::min(a.w.chunks, SEGMENT);
  const int groups = a.ids == nullptr ? 1 : a.slots <= a.E ? a.slots : a.slots == a.top_k ? a.slots : a.E + (SWIGLU ? 0 : 1);
  // tokens of an expert, on average: what one pass over its weights should take
  const int each = a.ids == nullptr ? a.slots : a.slots / a.E;
  return each <= 8 ? launch_group_split<PER, 1, SWIGLU>(a, groups, s) : launch_group_split<PER, 2, SWIGLU>(a, groups, s);
}
template <bool SWIGLU>
cudaError_t launch_group(const W4Args& a, cudaStream_t s) {
  return a.w.per == 4 ? launch_group<4, SWIGLU>(a, s) : a.w.per == 2 ? launch_group<2, SWIGLU>(a, s) : launch_group<1, SWIGLU>(a, s);
}

cudaError_t launch_down_token(const W4Args& a, int T, cudaStream_t s) {
  const dim3 grid(a.w.tiles, T);
  const auto kernel = a.w.per == 4 ? w4_down_token_kernel<4> : a.w.per == 2 ? w4_down_token_kernel<2> : w4_down_token_kernel<1>;
  return launch_dependent(kernel, grid, DOWN_WARPS * 32, 0, s, a);
}

// Whether the down product takes token by token. It then reads an expert's weights once for each slot, from the L2 but the
// first time, and saves the fp32 rows and a launch.
bool down_by_token(long long slots, int E) { return slots <= std::max(8, E / 4); }
int pitch_of(int h) { return (h + 7) / 8 * 8; }

bool dim_ok(int v) { return v >= 1 && v <= MAX_DIM; }

}  // namespace

size_t w4_weights_bytes(int matrices, int K, int N, int group) {
  if (matrices < 1 || matrices > MAX_MATRICES || !dim_ok(K) || !dim_ok(N) || !group_ok(group)) return 0;
  const size_t n = pieces(matrices, N, K), per = 128 / group;
  return n * 1024 + round256(n * 32 * per) + round256(n * 8 * per);
}
size_t w4_decode_workspace_bytes(long long slots, int E, int d, int h) {
  if (slots < 0 || slots > MAX_SLOTS || !dim_ok(d) || !dim_ok(h)) return 0;
  // SwiGLU's rows, and the fp32 rows of the down product where it does not take token by token
  return round256(static_cast<size_t>(slots) * pitch_of(h) * 2) + (down_by_token(slots, E) ? 0 : static_cast<size_t>(slots) * d * 4);
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
  a.w = packed_at(packed, matrices, N, K, group);
  a.out = y;
  a.ldo = ldy;
  a.y_bf16 = y_dtype == MOE_DTYPE_BF16;
  const cudaError_t err = launch_group<false>(a, reinterpret_cast<cudaStream_t>(stream));
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
  a.w = packed_at(w_ug, 2 * E, h, d, group);
  a.out = act;
  a.ldo = pitch;
  cudaError_t err = launch_group<true>(a, s);
  if (err != cudaSuccess) return cuda_fail(err);
  W4Args b = a;
  b.x = act;
  b.ldx = pitch;
  b.weights = weights;
  b.xdiv = 1;
  b.N = d;
  b.K = pitch;  // zeros from h on
  b.w = packed_at(w_down, E, d, h, group);
  if (down_by_token(slots, E)) {
    b.out = out;
    b.ldo = ldo;
    err = launch_down_token(b, T, s);
  } else {
    float* y = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + round256(static_cast<size_t>(slots) * pitch * 2));
    b.out = y;
    b.ldo = d;
    err = launch_group<false>(b, s);
    if (err == cudaSuccess)
      err = launch_dependent(w4_combine_kernel, dim3(std::min((d + 127) / 128, 64), T), 128, 0, s, static_cast<const float*>(y),
                             static_cast<long long>(d), ids, weights, top_k, E, d, reinterpret_cast<bf16*>(out), ldo);
  }
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

}  // extern "C"
