// MXFP4 experts: quantization of rows and weights to 4-bit floating point, and the grouped SwiGLU
// forward with both operands of every product in MXFP4 (serving: weights and activations take
// an eighth of the bytes of fp32 and a quarter of those of bf16).
//
// Format (OCP Microscaling MXFP4): blocks of 32 consecutive elements along the contraction
// dimension share one power-of-two scale 2^s stored as E8M0 (s + 127); each element is E2M1, one
// of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign. s = floor(log2(max |v|)) - 2 (2: the exponent of
// E2M1's largest value), not below -127 (-127 for an all-zero block); elements are v / 2^s rounded
// to nearest, ties to the even code, saturated at 6. E2M1 has no NaN or infinity: a block
// that holds one gets the scale 0xFF (E8M0's NaN), so everything computed from it is NaN.
//
// Layouts. Codes of an operand [rows, K]: K / 2 bytes a row, element 2i in the low half of byte i.
// Scales in the 512-byte atoms of the MXFP8 operands (mx_quant.cu), one per (128-row tile,
// 128-element chunk of K), with the chunks of a row padded to an even number KC = 2 ceil(K / 256):
// a pipeline stage of the product is 256 elements of K (128 bytes of codes, one swizzle row)
// and takes two atoms a tile. The scales of blocks past K are 2^0 (their codes are TMA zero fill).
//   activations: tiles are the problem list's 128-row tiles;
//   W_ug [E, 2h, d]: the gate and the up half of an expert are cut into tiles separately, tile
//     (2e + half) NTh + n / 128 with NTh = ceil(h / 128), so h needs no alignment beyond 32;
//   W_down^T [E, d, h]: tile e NTd + n / 128 with NTd = ceil(d / 128) rounded up to even.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "problem_tiles.cuh"
#include "trace.h"

namespace moe {
namespace {

constexpr int MXB = 32;  // elements per scale block
constexpr int MAX_E = 1024;
constexpr int MAX_TOPK = 32;

__host__ __device__ constexpr int mx4_kc(int K) { return 2 * ((K + 255) / 256); }

// ------------------------------------------------------------------------------ quantization
// E8M0 code of a block from the largest magnitude's bit pattern (as an unsigned number, which
// orders magnitudes, with infinity and NaN above all others).
__device__ __forceinline__ uint32_t mx4_scale_code(uint32_t abs_bits) {
  const int eb = static_cast<int>(abs_bits >> 23);
  if (eb == 255) return 255u;
  return static_cast<uint32_t>(max(eb - 2, 0));  // floor(log2) = eb - 127; subnormals: 0
}

// 1 / 2^s of an E8M0 code in [0, 252]: a normal power of two (1 for the NaN code, whose element
// codes carry nothing)
__device__ __forceinline__ float mx4_inv_scale(uint32_t code) {
  return code == 255u ? 1.0f : __uint_as_float((254u - code) << 23);
}

// 8 values (already divided by the scale) -> 8 E2M1 codes, the first in the low four bits
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
      "mov.b32 %0, {t0, t1, t2, t3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// A warp quantizes PASSES x 256 consecutive elements, 8 a lane and pass (four lanes hold a block):
// this lane's 8 codes of each pass, and a word of the four scale codes of a 128-element chunk: in
// lane l with l % 16 < PASSES that of pass l % 16, its first chunk for l < 16, its second above.
// Lanes past the row's end (pass i: v0 + 32 i >= vec) count as blocks of scale 2^0. What holds the
// row kernels besides memory is the integer pipe, so the passes share their shuffles: the block
// maxima go two to a word, and the four lanes of a block carry one pass's scale each.
template <int PASSES>
__device__ __forceinline__ uint32_t quantize(const uint4 (&in)[PASSES], int v0, int vec, uint32_t (&codes)[PASSES]) {
  static_assert(PASSES == 1 || PASSES == 4, "one pass, or one for each lane of a block");
  const int lane = threadIdx.x & 31;
  // largest magnitudes as bf16 bit patterns, two at a time (patterns without the sign order as
  // numbers, infinity and NaN above all others)
  uint32_t m[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i)
    m[i] = __vmaxu2(__vmaxu2(in[i].x & 0x7fff7fffu, in[i].y & 0x7fff7fffu),
                    __vmaxu2(in[i].z & 0x7fff7fffu, in[i].w & 0x7fff7fffu));
  uint32_t top[PASSES];  // of this lane's block, as a bf16 bit pattern in the high half
  if constexpr (PASSES == 1) {
    m[0] = __vmaxu2(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
    m[0] = __vmaxu2(m[0], __shfl_xor_sync(0xffffffffu, m[0], 2));
    top[0] = max(m[0] & 0xffff0000u, m[0] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < PASSES; i += 2) {
      uint32_t two = __vmaxu2(__byte_perm(m[i], m[i + 1], 0x5410), __byte_perm(m[i], m[i + 1], 0x7632));
      two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, 1));
      two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, 2));
      top[i] = two << 16;
      top[i + 1] = two & 0xffff0000u;
    }
  }
  uint32_t mine = 0u;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const uint32_t code = mx4_scale_code(top[i]);
    const uint32_t s = v0 + 32 * i < vec ? code : 127u;
    if ((lane & (PASSES - 1)) == i) mine = s;
    // v / 2^s in bf16: exact, or below the smallest normal number, which rounds to code 0
    const uint32_t inv = __float_as_uint(mx4_inv_scale(code)) >> 16;
    const uint32_t inv2 = inv << 16 | inv;
    const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
    float f[8];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t v;
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(w[t]), "r"(inv2));
      f[2 * t] = bf16_lo(v);
      f[2 * t + 1] = bf16_hi(v);
    }
    codes[i] = e2m1x8(f);
  }
  mine <<= 8 * ((lane >> 2) & 3);
  mine |= __shfl_xor_sync(0xffffffffu, mine, 4);
  mine |= __shfl_xor_sync(0xffffffffu, mine, 8);
  return mine;
}

// Address of the four scale bytes of row r of tile G in chunk kc.
__device__ __forceinline__ uint32_t* chunk_word(uint8_t* sf, long long G, int KC, int kc, int r) {
  return reinterpret_cast<uint32_t*>(sf + static_cast<size_t>(G * KC + kc) * 512 + (r & 31) * 16 + (r >> 5) * 4);
}

// The row kernels below are bound by memory (they read 2 bytes an element and write about half of
// one, or the reverse). A warp takes PASSES * 256 elements of a row at a time, all of its loads in
// flight before it works on them: 4 passes when there are rows enough for every warp of the
// GPU, 1 for few rows, so that a row is spread over more warps. Measured, 131072 x 2048: quantize
// 111 us (6.1 TB/s of reads and writes; 125 with the shuffles of each pass on their own), its
// inverse 119 us (5.7 TB/s, four fifths of them writes; a table in shared memory was no slower);
// the gather with quantization of 16384 tokens to 8 rows each 40 us (5.2 TB/s, two thirds writes);
// 333 x 1024 2.4 us each, a launch and a round trip to memory.
constexpr int ROW_PASSES = 4;

// Row and piece of item `it` (32-bit division unless there are 2^32 items).
__device__ __forceinline__ long long item_row(long long it, int pieces, bool small) {
  return small ? static_cast<long long>(static_cast<uint32_t>(it) / static_cast<uint32_t>(pieces)) : it / pieces;
}

// Rows along K. With offsets: the rows p < M of a problem list; else `rows` rows of weights in
// groups of `sub` rows, ntpad tiles a group.
template <int PASSES>
__global__ void __launch_bounds__(256) mx4_quant_rows_kernel(const uint4* src, long long rows, int K,
                                                             const int32_t* offsets, int E, int sub,
                                                             int ntpad, uint32_t* __restrict__ q,
                                                             uint8_t* __restrict__ sf, long long sf_tiles,
                                                             int32_t* status) {
  __shared__ int s_end[MAX_E];
  __shared__ int s_pre[MAX_E];
  grid_wait();
  src = after_wait(src);
  offsets = after_wait(offsets);
  const bool list = offsets != nullptr;
  const int lane = threadIdx.x & 31, vec = K / 8, KC = mx4_kc(K);
  const int pieces = (vec + 32 * PASSES - 1) / (32 * PASSES);
  const bool narrow = rows * pieces <= 0xffffffffll;
  const long long step = static_cast<long long>(gridDim.x) * 8;
  long long it = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5), p = 0;
  int v0 = 0;
  uint4 w[PASSES];
  auto load = [&]() {
    p = item_row(it, pieces, narrow);
    v0 = static_cast<int>(it - p * pieces) * (32 * PASSES) + lane;
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      w[i] = v0 + 32 * i < vec ? __ldcs(src + p * vec + v0 + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
  };
  // the first loads do not wait for the problem list, and those of the next item go ahead of this
  // one's stores
  if (it < rows * pieces) load();
  if (list && !load_problem_tiles(offsets, E, rows, s_end, s_pre, status)) return;
  const long long M = list ? s_end[E - 1] : rows;
  const long long items = M * pieces;
  while (it < items) {
    long long G;
    int r;
    if (list) {
      row_tile(s_end, s_pre, E, p, G, r);
    } else {
      const long long g = p / sub, n = p - g * sub;
      G = g * ntpad + n / 128;
      r = static_cast<int>(n % 128);
    }
    const bool tile_ok = MOE_DBG_IN(DBG_MX_TILE, G, sf_tiles);
    uint32_t codes[PASSES];
    const uint32_t word = quantize(w, v0, vec, codes);
    uint32_t* out = q + p * vec + v0;
    const int left = vec - v0;                    // element groups of the row from this lane's first
    const int vs = v0 - lane + 32 * (lane & 15);  // the first element group of the pass whose scales it holds
    it += step;
    if (it < items) load();
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      if (32 * i < left) out[32 * i] = codes[i];
    if ((lane & 15) < PASSES && vs < vec && tile_ok) *chunk_word(sf, G, KC, (vs + (lane & 16)) >> 4, r) = word;
  }
}

// The permute's gather and the quantization along d in one pass, token by token: a token's row is
// read and quantized once and its codes and scales are written to the rows of its top_k slots.
template <int PASSES>
__global__ void __launch_bounds__(256) mx4_permute_kernel(const uint4* x,
                                                          const int32_t* inv_map,
                                                          const int32_t* offsets, int E, int T, int k,
                                                          int d, uint32_t* __restrict__ q, uint8_t* __restrict__ sf,
                                                          long long sf_tiles, int32_t* status) {
  __shared__ int s_end[MAX_E];
  __shared__ int s_pre[MAX_E];
  grid_wait();
  x = after_wait(x);
  inv_map = after_wait(inv_map);
  offsets = after_wait(offsets);
  const int lane = threadIdx.x & 31, vec = d / 8, KC = mx4_kc(d);
  const int pieces = (vec + 32 * PASSES - 1) / (32 * PASSES);
  const long long items = static_cast<long long>(T) * pieces;
  const long long step = static_cast<long long>(gridDim.x) * 8;
  long long it = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  int v0 = 0, slot = -1;
  uint4 w[PASSES];
  auto load = [&]() {
    const long long t = item_row(it, pieces, items <= 0xffffffffll);
    v0 = static_cast<int>(it - t * pieces) * (32 * PASSES) + lane;
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      w[i] = v0 + 32 * i < vec ? __ldg(x + t * vec + v0 + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
    slot = lane < k ? __ldg(inv_map + t * k + lane) : -1;
  };
  if (it < items) load();  // as in the kernel above
  const long long n = static_cast<long long>(T) * k;
  if (!load_problem_tiles(offsets, E, n, s_end, s_pre, status)) return;
  const int M = s_end[E - 1];
  while (it < items) {
    // lane j < k holds slot j's row, its tile and the row within the tile
    int my_p = -1, my_r = 0, my_g = 0;
    if (lane < k) {
      const int p = slot;
      if (p >= 0 && p < M) {
        long long G;
        row_tile(s_end, s_pre, E, p, G, my_r);
        if (MOE_DBG_IN(DBG_MX_TILE, G, sf_tiles)) {
          my_p = p;
          my_g = static_cast<int>(G);
        }
      }
    }
    uint32_t codes[PASSES];
    const uint32_t word = quantize(w, v0, vec, codes);
    const int at = v0, vs = v0 - lane + 32 * (lane & 15);
    const bool scales = (lane & 15) < PASSES && vs < vec;
    it += step;
    if (it < items) load();
    for (int j = 0; j < k; ++j) {
      const int p = __shfl_sync(0xffffffffu, my_p, j);
      const int g = __shfl_sync(0xffffffffu, my_g, j), r = __shfl_sync(0xffffffffu, my_r, j);
      if (p < 0) continue;  // warp-uniform
#pragma unroll
      for (int i = 0; i < PASSES; ++i)
        if (at + 32 * i < vec) q[static_cast<size_t>(p) * vec + at + 32 * i] = codes[i];
      if (scales) *chunk_word(sf, g, KC, (vs + (lane & 16)) >> 4, r) = word;
    }
  }
}

// Eight 4-bit codes times the bf16 pair scale2, in pairs of bf16. A byte permute is a table of
// eight bytes: one looks up the low bytes of four magnitudes 0 0.5 1 1.5 2 3 4 6, one the high.
__device__ __forceinline__ uint4 e2m1_scaled(uint32_t c, uint32_t scale2) {
  constexpr uint32_t LO0 = 0xc0800000u, LO1 = 0xc0804000u, HI0 = 0x3f3f3f00u, HI1 = 0x40404040u;
  const uint32_t mag = c & 0x77777777u, up = c << 4;  // byte j: code 2j + 1's sign in c, code 2j's in up
  uint32_t w[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t sel = mag >> (16 * h);  // four nibbles
    const uint32_t lo = __byte_perm(LO0, LO1, sel), hi = __byte_perm(HI0, HI1, sel);
    w[2 * h] = __byte_perm(lo, hi, 0x5140) | (__byte_perm(up, c, h ? 0x6020 : 0x4000) & 0x80008000u);
    w[2 * h + 1] = __byte_perm(lo, hi, 0x7362) | (__byte_perm(up, c, h ? 0x7030 : 0x5010) & 0x80008000u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(w[i]) : "r"(w[i]), "r"(scale2));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The bf16 values that rows p < M of codes and scales stand for (exact: an E2M1 value times a
// power of two has two significant bits); a block with a NaN scale reads as NaN.
template <int PASSES>
__global__ void __launch_bounds__(256) mx4_dequant_rows_kernel(const uint32_t* q,
                                                               const uint8_t* sf, long long rows, int K,
                                                               const int32_t* offsets, int E,
                                                               uint4* __restrict__ x, long long sf_tiles,
                                                               int32_t* status) {
  __shared__ int s_end[MAX_E];
  __shared__ int s_pre[MAX_E];
  grid_wait();
  q = after_wait(q);
  sf = after_wait(sf);
  offsets = after_wait(offsets);
  const int lane = threadIdx.x & 31, vec = K / 8, KC = mx4_kc(K);
  const int pieces = (vec + 32 * PASSES - 1) / (32 * PASSES);
  const bool narrow = rows * pieces <= 0xffffffffll;
  const long long step = static_cast<long long>(gridDim.x) * 8;
  long long it = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5), next_p = 0;
  int next_v0 = 0;
  uint32_t next[PASSES];
  auto load = [&]() {
    next_p = item_row(it, pieces, narrow);
    next_v0 = static_cast<int>(it - next_p * pieces) * (32 * PASSES) + lane;
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      next[i] = next_v0 + 32 * i < vec ? __ldcs(q + next_p * vec + next_v0 + 32 * i) : 0u;
  };
  if (it < rows * pieces) load();  // as in the quantizer
  if (!load_problem_tiles(offsets, E, rows, s_end, s_pre, status)) return;
  const int M = s_end[E - 1];
  const long long items = static_cast<long long>(M) * pieces;
  while (it < items) {
    const long long p = next_p;
    const int v0 = next_v0;
    uint32_t codes[PASSES], sc[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) codes[i] = next[i];
    it += step;
    if (it < items) load();
    long long G;
    int r;
    row_tile(s_end, s_pre, E, p, G, r);
    if (!MOE_DBG_IN(DBG_MX_TILE, G, sf_tiles)) continue;
    const uint8_t* scale = sf + atom_byte(G, KC, v0 >> 2, r);  // a pass is two chunks
#pragma unroll
    for (int i = 0; i < PASSES; ++i) sc[i] = v0 + 32 * i < vec ? __ldg(scale + 1024 * i) : 0u;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int v = v0 + 32 * i;
      if (v >= vec) break;
      // 2^(sc - 127) in bf16: 2^-127 is subnormal, 255 stands for NaN
      const uint32_t s = sc[i] == 255u ? 0x7fc0u : sc[i] == 0u ? 0x0040u : sc[i] << 7;
      __stcs(x + p * vec + v, e2m1_scaled(codes[i], s << 16 | s));
    }
  }
}

// A weight [E, R, C] quantized along R: codes [E, C, R / 2], tiles by expert and 128 columns of
// C. One thread per (expert, 32-block of R, column), columns fastest: the strided reads of a
// thread are coalesced across the warp. The blocks past R of the padded chunks get scale 2^0.
__global__ void __launch_bounds__(256) mx4_quant_cols_kernel(const bf16* __restrict__ w, int E, int R, int C, int ntpad,
                                                             uint8_t* __restrict__ q, uint8_t* __restrict__ sf) {
  const int nb = R / MXB, KC = mx4_kc(R), nbp = 4 * KC;
  const long long items = static_cast<long long>(E) * nbp * C;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < items;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int c = static_cast<int>(i % C);
    const long long rest = i / C;
    const int b = static_cast<int>(rest % nbp);
    const int e = static_cast<int>(rest / nbp);
    uint32_t code = 127u;
    if (b < nb) {
      const bf16* col = w + (static_cast<long long>(e) * R + static_cast<long long>(b) * MXB) * C + c;
      float v[MXB];
      uint32_t m = 0u;
#pragma unroll
      for (int j = 0; j < MXB; ++j) {
        v[j] = __bfloat162float(col[static_cast<long long>(j) * C]);
        m = max(m, abs_bits(v[j]));
      }
      code = mx4_scale_code(m);
      const float inv = mx4_inv_scale(code);
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) f[t] = v[8 * j + t] * inv;
        o[j] = e2m1x8(f);
      }
      *reinterpret_cast<uint4*>(q + ((static_cast<long long>(e) * C + c) * R + b * MXB) / 2) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
    sf[atom_byte(static_cast<long long>(e) * ntpad + c / 128, KC, b, c % 128)] = static_cast<uint8_t>(code);
  }
}

// ------------------------------------------------------------------------------ the product
// Persistent grouped GEMM on block-scaled 4-bit operands: the problem list, tile order, roles and
// bounded waits of the grouped GEMM (grouped_gemm.cu), one CTA per SM.
//   warp 0      TMA producer of A (the tile's rows x 256 elements of K, and their scale atoms)
//   warp 1      tensor-memory allocator and MMA issuer: per stage four block-scaled MMAs of K = 64
//               (MX4_DOWN: after copies of the scale atoms into tensor memory)
//   warp 2      TMA producer of B
//   warps 4..7  MX4_UP: scale atoms from the stage into tensor memory
//   the last 8  epilogue, two per lane quadrant
// MX4_UP:   B = BN / 2 gate and BN / 2 up rows of W_ug; the epilogue computes A = silu(gate) up in
//           fp32 and quantizes it along h from fp32 (no bf16 rounding in between).
// MX4_DOWN: B = BN rows of W_down^T; bf16 store, one rounding, staged through shared memory so
//           that a warp writes whole 128-byte lines. y is bf16 as in the BF16 and MXFP8 forwards: fp32 rows
//           would double what is written here and read by the combine, half of the time of many tokens.
//           It costs a second rounding: the combined rows are within 0.0024 of 64 bits (norm relative)
//           where one rounding gives 0.0017.
// What bounds it, at 131072 rows of 256 experts, d = 2048, h = 512 (up 153 us, 3.6 PFLOP/s; down
// 149 us): up moves 1.7 GB of tiles through the L2's output to the SMs, 51 KB for each
// 128 x 256 x 256, alone 116 us; its MMAs take 0.33 us a stage and about a microsecond a tile for
// handing the accumulator over, alone 97 us; a ring of four stages does not hide one behind the
// other entirely. Down writes 537 MB of y, 136 us at the rate of a kernel that only writes.
// Tried and slower: pairs of CTAs (35 KB instead of 51, but 181 and 152 us, and 56 us against 36 for
// 128 rows over 128 experts), 128-column tiles (57 us against 39 there: an MMA of half the columns
// takes about as long), two accumulators of 192 columns (down 213 us), prefetching the next tile
// into the L2 (up 186 us).
// Scales: tcgen05.cp by the MMA issuer runs in order with the MMAs, 0.17 us a stage. In the up
// product four warps write them with tcgen05.st while earlier MMAs run (up 162 -> 153 us; one row
// in each of 8 experts 14.1 -> 13.4). In the down product, two or three stages a tile, the extra
// hop costs more than it saves (149 against 160 us), so the issuer copies.
// A row tile that its expert does not fill loads only its own rows, 16 at a time; the other rows
// of the stage hold what was there before, and nothing reads the rows of the product that they
// give (the rows of a product are independent).
enum { MX4_UP = 0, MX4_DOWN = 1 };

constexpr int BM = 128;                        // as row_tiles() counts
constexpr int BN = 256;
constexpr int STAGE_K = 256;                 // elements of K per stage: 128 bytes of codes
constexpr int UK = 64;                       // K of one MMA
constexpr int A_BYTES = BM * STAGE_K / 2;    // 16 KB
constexpr int A_BOX = 16;                    // rows of the small box of A
constexpr int SF_BYTES = 2 * 512;            // scale atoms of a 128-row tile: two chunks
constexpr int SF_STAGE_BYTES = 3 * SF_BYTES; // A, and two tiles of B
constexpr int EPI_WARPS = 8;
constexpr int PRODUCER_B_WARP = 2;
constexpr int SCALE_WARP = 4;                // MX4_UP: warps 4..7, one per lane quadrant
// MX4_UP: registers a thread by warpgroup; the epilogue's two take over what the others leave of
// the launch's 4 x 128.
constexpr int ROLE_REGS = 72, SCALE_REGS = 56, EPI_REGS = 192;
static_assert(ROLE_REGS + SCALE_REGS + 2 * EPI_REGS <= 4 * 128, "register shares");
constexpr int TMEM_COLS = 512;
constexpr int SF_TMEM_COL = 256;             // 32 columns of scales per stage after the accumulator
constexpr int RASTER_M = 16;                 // row tiles per raster group
constexpr int MAX_STAGES = 4;
constexpr int OUT_BYTES = 32 * 128;          // MX4_DOWN: a warp's staging, 32 rows of 64 bf16
constexpr int CTL_BYTES = 256;

template <int MODE>
struct Shape {
  static constexpr int cols = MODE == MX4_UP ? BN / 2 : BN;  // output columns per tile
  static constexpr int b_bytes = BN * STAGE_K / 2;
  static constexpr int stage_bytes = A_BYTES + b_bytes;
  static constexpr int stages = MODE == MX4_UP ? 4 : 3;
  static constexpr bool scale_warps = MODE == MX4_UP;
  static constexpr int epi_warp = scale_warps ? 8 : 4;
  static constexpr int threads = 32 * (epi_warp + EPI_WARPS);
  static constexpr int out_bytes = MODE == MX4_DOWN ? EPI_WARPS * OUT_BYTES : 0;
  static constexpr int fixed = 1024 + stages * (stage_bytes + SF_STAGE_BYTES) + out_bytes + CTL_BYTES;
  static_assert(stages <= MAX_STAGES && SF_TMEM_COL + 32 * stages <= TMEM_COLS, "stages");
  static size_t smem(int E) { return fixed + 2 * sizeof(int) * static_cast<size_t>(E + 2); }
};

struct Ctl {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t scales[MAX_STAGES];
  uint64_t tfull;
  uint64_t tempty;
  uint64_t done;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Ctl) <= CTL_BYTES, "control block too large");

struct Maps {
  CUtensorMap a, a16, b;  // boxes of 128 and of 16 rows of A
};

struct Args {
  const int32_t* offsets;
  int E, cap;
  int N;               // output columns (MX4_UP: h)
  int K;
  int h;               // MX4_UP: half width of W_ug
  const uint8_t* sfa;  // scale atoms of A by the problem list's tiles
  const uint8_t* sfb;  // of B, tiles_b tiles per expert (MX4_UP: per half)
  int kc;              // chunks per row, even
  int tiles_b;
  bf16* y;             // MX4_DOWN
  uint8_t* pq;         // MX4_UP: codes [cap, h / 2] and scale atoms of A = silu(gate) up
  uint8_t* psf;
  int pkc;
  long long dbg_a_tiles, dbg_b_tiles;
  int32_t* status;
  long long timeout_ns, drain_ns;
};

struct Tile {
  int e, g, row0, rows, n0;
};

struct Sched {
  const int* offs;
  const int* pre;
  int E, nt, total;
};

// Tile t of the problem list; inside an expert, groups of up to RASTER_M row tiles are walked
// column tile by column tile (row tile fastest).
__device__ __forceinline__ Tile decode_tile(const Sched& s, int t, int cols_per_tile) {
  Tile ti;
  const int gq = t / s.nt;
  int lo = 0, hi = s.E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.pre[mid] <= gq) lo = mid; else hi = mid;
  }
  ti.e = lo;
  const int mt_e = s.pre[lo + 1] - s.pre[lo];
  const int l = t - s.pre[lo] * s.nt;
  const int grp = l / (RASTER_M * s.nt);
  const int gm = min(RASTER_M, mt_e - grp * RASTER_M);
  const int within = l - grp * RASTER_M * s.nt;
  const int m_local = grp * RASTER_M + within % gm;
  ti.g = s.pre[lo] + m_local;
  ti.row0 = s.offs[lo] + m_local * BM;
  ti.rows = min(BM, s.offs[lo + 1] - ti.row0);
  ti.n0 = (within / gm) * cols_per_tile;
  return ti;
}

__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

__device__ __forceinline__ float silu_f(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

template <int MODE>
__global__ void __launch_bounds__(Shape<MODE>::threads, 1) mx4_gemm_kernel(const __grid_constant__ Maps maps, const Args args) {
  typedef Shape<MODE> S;
  constexpr int COLS = S::cols;
  constexpr int STAGES = S::stages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sf_ring = smem + STAGES * S::stage_bytes;
  uint8_t* staging = sf_ring + STAGES * SF_STAGE_BYTES;
  Ctl* ctl = reinterpret_cast<Ctl*>(staging + S::out_bytes);
  int* offs = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(ctl) + CTL_BYTES);
  const int E = args.E;
  int* pre = offs + (E + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- barriers and tensor memory, which do not depend on the kernel before this one
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 2);  // both producers
      mbar_init(smem_u32(&ctl->empty[s]), 1);
      mbar_init(smem_u32(&ctl->scales[s]), 4);  // the scale warps
    }
    mbar_init(smem_u32(&ctl->tfull), 1);
    mbar_init(smem_u32(&ctl->tempty), EPI_WARPS);  // one arrival per epilogue warp
    mbar_init(smem_u32(&ctl->done), 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.a16);
    prefetch_tmap(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl->tmem_base), TMEM_COLS);
    tmem_relinquish();
  }
  // The up product waits here for everything before it; what the down product reads before its own
  // wait (offsets, weights) is then complete, because the up product releases it after this wait. The
  // down product itself does not release: a combine placed while it still runs lands two blocks to an
  // SM (16384 tokens 465 us instead of 430).
  if constexpr (MODE == MX4_UP) {
    grid_wait();
    grid_release();
  }

  // ---- problem list
  const int32_t* offsets = after_wait(args.offsets);
  for (int i = tid; i <= E; i += S::threads) offs[i] = i == 0 ? 0 : __ldg(offsets + i - 1);
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < E; i += S::threads) bad |= (offs[i + 1] < offs[i]) || (offs[i] < 0);
  if (tid == 0) bad |= offs[E] > args.cap;
  if (warp == 0) {
    int carry = 0;
    if (lane == 0) pre[0] = 0;
    for (int base = 0; base < E; base += 32) {
      const int e = base + lane;
      int v = (e < E) ? row_tiles(offs[e + 1] - offs[e]) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int nb = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += nb;
      }
      if (e < E) pre[e + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  tc_fence_before();
  bad = __syncthreads_or(bad);
  tc_fence_after();
  if (bad && tid == 0 && blockIdx.x == 0) record_status(args.status, MOE_DEV_BAD_OFFSETS);

  Sched sc;
  sc.offs = offs;
  sc.pre = pre;
  sc.E = E;
  sc.nt = (args.N + COLS - 1) / COLS;
  sc.total = bad ? 0 : pre[E] * sc.nt;  // bad offsets: no work, only the teardown
  const int kblocks = (args.K + STAGE_K - 1) / STAGE_K;
  const uint32_t tmem_base = ctl->tmem_base;
  volatile int* abort_flag = &ctl->abort_flag;
  const long long tmo = args.timeout_ns;
  const uint32_t stage0 = smem_u32(smem);
  const uint32_t sf0 = smem_u32(sf_ring);

  if (S::scale_warps && warp < SCALE_WARP) set_regs_down<ROLE_REGS>();
  if (warp == 0 || warp == PRODUCER_B_WARP) {
    // =========================================================== TMA producers
    if (lane == 0) {
      const bool is_a = warp == 0;
      if (MODE == MX4_DOWN && is_a) grid_wait();  // A is the up product's output
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < sc.total && ok; t += gridDim.x) {
        const Tile ti = decode_tile(sc, t, COLS);
        // first scale atoms of the tile(s): consecutive chunks of a tile are consecutive atoms
        long long s0, s1 = 0;
        if (is_a) {
          s0 = ti.g;
          if (!MOE_DBG_IN(DBG_GG_SFA, s0, args.dbg_a_tiles)) s0 = 0;
        } else {
          if constexpr (MODE == MX4_UP) {
            s0 = static_cast<long long>(2 * ti.e) * args.tiles_b + ti.n0 / 128;
            s1 = s0 + args.tiles_b;
          } else {
            s0 = static_cast<long long>(ti.e) * args.tiles_b + ti.n0 / 128;
            s1 = s0 + 1;
          }
          if (!MOE_DBG_IN(DBG_GG_SFB, s0, args.dbg_b_tiles)) s0 = 0;
          if (!MOE_DBG_IN(DBG_GG_SFB, s1, args.dbg_b_tiles)) s1 = 0;
        }
        const int boxes = ti.rows > BM - A_BOX ? 0 : (ti.rows + A_BOX - 1) / A_BOX;  // 0: the whole tile
        const uint32_t a_bytes = boxes == 0 ? A_BYTES : boxes * (A_BYTES / (BM / A_BOX));
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const int s = it % STAGES;
          // the weights of the first stages load while the up product still runs; the clock of
          // this thread's waits starts after it
          if (MODE == MX4_DOWN && !is_a && it == STAGES) grid_wait();
          if (!mbar_wait(smem_u32(&ctl->empty[s]), ((it / STAGES) & 1u) ^ 1u, abort_flag, args.status, tmo)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&ctl->full[s]);
          const uint32_t sa = stage0 + s * S::stage_bytes, sb = sa + A_BYTES;
          const uint32_t sfs = sf0 + s * SF_STAGE_BYTES;
          const int k0 = kb * (STAGE_K / 2);  // in bytes of codes
          if (is_a) {
            mbar_arrive_expect_tx(fb, a_bytes + SF_BYTES);
            if (boxes == 0) tma_load_2d(sa, &maps.a, k0, ti.row0, fb);
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(sa + i * (A_BYTES / (BM / A_BOX)), &maps.a16, k0, ti.row0 + i * A_BOX, fb);
            bulk_load(sfs, args.sfa + (s0 * args.kc + 2 * kb) * 512, SF_BYTES, fb);
          } else {
            mbar_arrive_expect_tx(fb, S::b_bytes + 2 * SF_BYTES);
            if constexpr (MODE == MX4_UP) {
              tma_load_3d(sb, &maps.b, k0, ti.n0, ti.e, fb);                            // gate rows
              tma_load_3d(sb + S::b_bytes / 2, &maps.b, k0, args.h + ti.n0, ti.e, fb);  // up rows
            } else {
              tma_load_3d(sb, &maps.b, k0, ti.n0, ti.e, fb);
            }
            bulk_load(sfs + SF_BYTES, args.sfb + (s0 * args.kc + 2 * kb) * 512, SF_BYTES, fb);
            bulk_load(sfs + 2 * SF_BYTES, args.sfb + (s1 * args.kc + 2 * kb) * 512, SF_BYTES, fb);
          }
        }
      }
      // the copies this thread issued must land before the CTA can exit (see grouped_gemm.cu)
      const uint32_t first = it > STAGES ? it - STAGES : 0u;
      for (uint32_t j = first; j < it; ++j)
        if (!mbar_wait(smem_u32(&ctl->full[j % STAGES]), (j / STAGES) & 1u, abort_flag, args.status, args.drain_ns, false))
          break;
    }
  } else if (warp == 1) {
    // =========================================================== MMA issuer
    if (MODE == MX4_DOWN) grid_wait();  // the clock of its waits starts after the up product
    uint32_t it = 0, n = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < sc.total && ok; t += gridDim.x, ++n) {
      ok = warp_all(mbar_wait(smem_u32(&ctl->tempty), (n & 1u) ^ 1u, abort_flag, args.status, tmo));
      if (!ok) break;
      tc_fence_after();
      for (int kb = 0; kb < kblocks; ++kb, ++it) {
        const int s = it % STAGES;
        ok = warp_all(mbar_wait(smem_u32(&ctl->full[s]), (it / STAGES) & 1u, abort_flag, args.status, tmo) &&
                      (!S::scale_warps ||
                       mbar_wait(smem_u32(&ctl->scales[s]), (it / STAGES) & 1u, abort_flag, args.status, tmo)));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t sa = stage0 + s * S::stage_bytes, sb = sa + A_BYTES;
          const uint32_t sft = tmem_base + SF_TMEM_COL + s * 32;
          if (!S::scale_warps) {
            const uint32_t sfs = sf0 + s * SF_STAGE_BYTES;
#pragma unroll
            for (int i = 0; i < 6; ++i)
              tmem_cp_32x128b_x4(sft + 4 * i, smem_desc_rows16(sfs + (i % 3) * SF_BYTES + (i / 3) * 512));
          }
#pragma unroll
          for (int ks = 0; ks < STAGE_K / UK; ++ks) {
            constexpr uint32_t idesc = idesc_mxf4(BM, BN);
            const uint64_t ad = smem_desc_sw128(sa + ks * (UK / 2), 16, 1024);
            const uint64_t bd = smem_desc_sw128(sb + ks * (UK / 2), 16, 1024);
            const uint32_t sfc = sft + 12 * (ks >> 1);
            mma_mxf4_ss(tmem_base, ad, bd, idesc | idesc_sf_ids(2u * (ks & 1)), sfc, sfc + 4, (kb | ks) != 0 ? 1u : 0u);
          }
          mma_commit(smem_u32(&ctl->empty[s]));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (lane == 0) mma_commit(smem_u32(&ctl->tfull));
      __syncwarp();
    }
    // every MMA this thread issued must finish before tensor memory is released
    if (lane == 0) mma_commit(smem_u32(&ctl->done));
    __syncwarp();
    mbar_wait(smem_u32(&ctl->done), 0u, abort_flag, args.status, args.drain_ns, false);
  } else if (S::scale_warps && warp >= SCALE_WARP && warp < S::epi_warp) {
    // =========================================================== scales
    // The scale atoms of a stage into its 32 columns of tensor memory, per 128-element chunk 4 columns
    // of A, then 8 of B; every lane quadrant holds all 32 rows of an atom. A stage that is full has
    // columns that no MMA reads any more: its ring slot was free before it was loaded.
    set_regs_down<SCALE_REGS>();
    const uint32_t sft = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + SF_TMEM_COL;
    const int mine = sc.total > static_cast<int>(blockIdx.x) ? (sc.total - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    const uint32_t stages = static_cast<uint32_t>(mine) * kblocks;
    for (uint32_t it = 0; it < stages; ++it) {
      const int s = it % STAGES;
      if (!warp_all(mbar_wait(smem_u32(&ctl->full[s]), (it / STAGES) & 1u, abort_flag, args.status, tmo))) break;
      tc_fence_after();
      const uint8_t* atoms = sf_ring + s * SF_STAGE_BYTES + lane * 16;
      uint4 v[6];
#pragma unroll
      for (int i = 0; i < 6; ++i) v[i] = *reinterpret_cast<const uint4*>(atoms + (i % 3) * SF_BYTES + (i / 3) * 512);
#pragma unroll
      for (int i = 0; i < 6; i += 2) tmem_st8(sft + s * 32 + 4 * i, v[i], v[i + 1]);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->scales[s]));
    }
  } else if (warp >= S::epi_warp) {
    // =========================================================== epilogue
    if (S::scale_warps) set_regs_up<EPI_REGS>();
    if (MODE == MX4_DOWN) grid_wait();  // the clock of its waits starts after the up product
    const int q = warp & 3, half = (warp - S::epi_warp) >> 2;
    const int r_in = q * 32 + lane;
    const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    auto release_acc = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty));
    };
    uint32_t n = 0;
    for (int t = blockIdx.x; t < sc.total; t += gridDim.x, ++n) {
      const Tile ti = decode_tile(sc, t, COLS);
      if (!warp_all(mbar_wait(smem_u32(&ctl->tfull), n & 1u, abort_flag, args.status, tmo))) break;
      tc_fence_after();
      if (q * 32 >= ti.rows) {  // warp-uniform: none of this quadrant's rows
        release_acc();
        continue;
      }
      const long long row = static_cast<long long>(ti.row0) + r_in;
      bool rv = r_in < ti.rows;
      if (rv && !MOE_DBG_IN(DBG_GG_ROW, row, args.cap)) rv = false;
      if constexpr (MODE == MX4_UP) {
        // this warp's gate and up columns into registers, so that the accumulator goes back to the
        // MMA issuer before they are worked on
        constexpr int BLOCKS = 2;  // blocks of 32 output columns per warp
        uint32_t g[2 * BLOCKS][16], u[2 * BLOCKS][16];
#pragma unroll
        for (int i = 0; i < 2 * BLOCKS; ++i) {
          tmem_ld16(tb + half * (32 * BLOCKS) + i * 16, g[i]);
          tmem_ld16(tb + COLS + half * (32 * BLOCKS) + i * 16, u[i]);
        }
#pragma unroll
        for (int i = 0; i < 2 * BLOCKS; ++i) tmem_ld_wait2(g[i], u[i]);
        release_acc();
        if (!rv || !MOE_DBG_IN(DBG_GG_MXSF, ti.g, args.dbg_a_tiles)) continue;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          const int col = ti.n0 + half * (32 * BLOCKS) + b * 32;  // h % 32 == 0: a block is all in or all out
          uint8_t* sfp = args.psf + atom_byte(ti.g, args.pkc, col >> 5, r_in);
          if (col >= args.h) {
            *sfp = 127;
            continue;
          }
          float p[32];
          uint32_t m = 0u;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            p[j] = silu_f(__uint_as_float(g[2 * b + (j >> 4)][j & 15])) * __uint_as_float(u[2 * b + (j >> 4)][j & 15]);
            m = max(m, abs_bits(p[j]));
          }
          const uint32_t code = mx4_scale_code(m);
          const float inv = mx4_inv_scale(code);
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = p[8 * j + i] * inv;
            o[j] = e2m1x8(f);
          }
          *reinterpret_cast<uint4*>(args.pq + row * (args.h / 2) + col / 2) = make_uint4(o[0], o[1], o[2], o[3]);
          *sfp = static_cast<uint8_t>(code);
        }
        // the last column tile also writes the scales of the blocks that no tile covers, up to
        // the end of the row's last (256-element) stage
        if (ti.n0 + COLS >= args.h)
          for (int kb = (ti.n0 + COLS) / 32 + half; kb < 4 * args.pkc; kb += 2)
            args.psf[atom_byte(ti.g, args.pkc, kb, r_in)] = 127;
      } else {
        // 64 columns at a time: packed into this warp's staging (16-byte piece j of row r at
        // piece j ^ (r & 7): no bank conflicts either way), then out in whole 128-byte lines,
        // four rows an instruction
        constexpr int CHUNKS = 2;
        uint32_t p[32 * CHUNKS];
#pragma unroll
        for (int i = 0; i < 4 * CHUNKS; i += 2) {
          uint32_t v0[16], v1[16];
          tmem_ld16(tb + half * (BN / 2) + i * 16, v0);
          tmem_ld16(tb + half * (BN / 2) + (i + 1) * 16, v1);
          tmem_ld_wait2(v0, v1);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            p[8 * i + j] = pack_bf16x2(__uint_as_float(v0[2 * j]), __uint_as_float(v0[2 * j + 1]));
            p[8 * i + 8 + j] = pack_bf16x2(__uint_as_float(v1[2 * j]), __uint_as_float(v1[2 * j + 1]));
          }
        }
        release_acc();
        uint8_t* sbuf = staging + (warp - S::epi_warp) * OUT_BYTES;
        const int rows_here = min(32, ti.rows - q * 32);
        const unsigned valid = __ballot_sync(0xffffffffu, rv);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          const int col0 = ti.n0 + half * (BN / 2) + c * 64;
          if (col0 >= args.N) break;  // warp-uniform
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(sbuf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(p[32 * c + 4 * j], p[32 * c + 4 * j + 1], p[32 * c + 4 * j + 2], p[32 * c + 4 * j + 3]);
          __syncwarp();
          const int piece = lane & 7, col = col0 + piece * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            if (i * 4 >= rows_here) break;
            if (col < args.N && ((valid >> r) & 1u))  // N % 32 == 0: a piece is all in or all out
              *reinterpret_cast<uint4*>(args.y + (static_cast<long long>(ti.row0) + q * 32 + r) * args.N + col) =
                  *reinterpret_cast<const uint4*>(sbuf + r * 128 + ((piece ^ (r & 7)) << 4));
          }
        }
      }
    }
  }

  // ---- teardown: every role has finished (or given up); release tensor memory
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------------------------ host side
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
bool width_ok(int v) { return v > 0 && v % MXB == 0 && v <= (1 << 20); }
bool shape_ok(int E, int d, int h) { return E >= 1 && E <= MAX_E && width_ok(d) && width_ok(h); }

// 128-row tiles of any problem list with at most `rows` rows
long long list_tiles(long long rows, int E) { return (rows + 127LL * E) / 128; }
int tiles128(int n) { return (n + 127) / 128; }
int down_tiles(int d) { return 2 * ((tiles128(d) + 1) / 2); }

size_t codes_bytes(long long rows, int K) { return round256(static_cast<size_t>(rows) * (K / 2)); }
size_t atoms_bytes(long long tiles, int K) { return round256(static_cast<size_t>(tiles) * mx4_kc(K) * 512); }

struct Weights {
  uint8_t *ug_q, *ug_sf, *dn_q, *dn_sf;
};
size_t ug_sf_bytes(int E, int d, int h) { return atoms_bytes(2LL * E * tiles128(h), d); }
size_t dn_sf_bytes(int E, int d, int h) { return atoms_bytes(static_cast<long long>(E) * down_tiles(d), h); }
size_t weights_bytes(int E, int d, int h) {
  return codes_bytes(2LL * E * h, d) + ug_sf_bytes(E, d, h) + codes_bytes(static_cast<long long>(E) * d, h) +
         dn_sf_bytes(E, d, h);
}
Weights carve_weights(const void* base, int E, int d, int h) {
  Weights w;
  w.ug_q = const_cast<uint8_t*>(static_cast<const uint8_t*>(base));
  w.ug_sf = w.ug_q + codes_bytes(2LL * E * h, d);
  w.dn_q = w.ug_sf + ug_sf_bytes(E, d, h);
  w.dn_sf = w.dn_q + codes_bytes(static_cast<long long>(E) * d, h);
  return w;
}
size_t fwd_ws_bytes(long long cap, int E, int h) { return codes_bytes(cap, h) + atoms_bytes(list_tiles(cap, E), h); }

moe_status_t launched() {
  const cudaError_t err = cudaGetLastError();
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

// Whether `rows` rows of K elements are at least 16 pieces of ROW_PASSES passes for each SM
bool many_rows(long long rows, int K) {
  return rows * ((K + 256 * ROW_PASSES - 1) / (256 * ROW_PASSES)) >= 16LL * device_sm_count();
}
// blocks of eight warps for the pieces of `rows` rows
int row_blocks(long long rows, int K, int passes) {
  const long long items = rows * ((K + 256 * passes - 1) / (256 * passes));
  return static_cast<int>(std::max(1LL, std::min((items + 7) / 8, 8LL * device_sm_count())));
}
template <typename Many, typename Few, typename... Given>
moe_status_t launch_rows(Many many, Few few, long long rows, int K, cudaStream_t s, Given... given) {
  const cudaError_t err = many_rows(rows, K)
                              ? launch_dependent(many, row_blocks(rows, K, ROW_PASSES), 256, 0, s, given...)
                              : launch_dependent(few, row_blocks(rows, K, 1), 256, 0, s, given...);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

template <int MODE>
moe_status_t launch_gemm(const uint8_t* a_codes, const uint8_t* b_codes, long long b_rows, Args a, cudaStream_t s) {
  typedef Shape<MODE> S;
  a.timeout_ns = wait_timeout_ns();
  a.drain_ns = std::max(a.timeout_ns, 2000000000LL);
  Maps m;
  if (!make_map_u8_rows2d(&m.a, a_codes, a.cap, a.K / 2, BM) || !make_map_u8_rows2d(&m.a16, a_codes, a.cap, a.K / 2, A_BOX) ||
      !make_map_u8_weight3d(&m.b, b_codes, a.E, b_rows, a.K / 2, MODE == MX4_UP ? BN / 2 : BN))
    return cuda_fail(cudaErrorInvalidValue);
  const cudaError_t aerr = ensure_max_dynamic_smem(reinterpret_cast<const void*>(mx4_gemm_kernel<MODE>),
                                                   static_cast<int>(S::smem(MAX_E)));
  if (aerr != cudaSuccess) return cuda_fail(aerr);
  const long long tiles = list_tiles(a.cap, a.E) * ((a.N + S::cols - 1) / S::cols);
  const unsigned grid = static_cast<unsigned>(std::max(1LL, std::min<long long>(device_sm_count(), tiles)));
  const cudaError_t err = launch_dependent(mx4_gemm_kernel<MODE>, grid, S::threads, S::smem(a.E), s, m, a);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

}  // namespace

MOE_DBG_DEFINE_COLLECTOR(dbg_collect_mx4)

size_t mx4_workspace_bytes(int op, long long n, int E, int d, int h) {
  if (!shape_ok(E, d, h)) return 0;
  switch (op) {
    case MOE_OP_MX4_WEIGHTS: return weights_bytes(E, d, h);
    case MOE_OP_MX4_FWD: return fwd_ws_bytes(n, E, h);
    case MOE_OP_MX4_ROW_SCALES: return atoms_bytes(list_tiles(n, E), d);
  }
  return 0;
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_mx4_prepare_weights(const moe_bf16* w_ug, const moe_bf16* w_down, int E, int d, int h, void* mxw,
                                     size_t mxw_bytes, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (E < 1 || d <= 0 || h <= 0) return MOE_ERR_INVALID_ARG;
  if (!shape_ok(E, d, h)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!w_ug || !w_down || !mxw || !aligned(w_ug, 16) || !aligned(w_down, 16) || !aligned(mxw, 256))
    return MOE_ERR_INVALID_ARG;
  if (mxw_bytes < weights_bytes(E, d, h)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  moe_status_t st = check_device();
  if (st != MOE_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const Weights w = carve_weights(mxw, E, d, h);
  const long long ug_rows = 2LL * E * h;
  st = launch_rows(mx4_quant_rows_kernel<ROW_PASSES>, mx4_quant_rows_kernel<1>, ug_rows, d, s,
                   reinterpret_cast<const uint4*>(w_ug), ug_rows, d, nullptr, E, h, tiles128(h),
                   reinterpret_cast<uint32_t*>(w.ug_q), w.ug_sf, 2LL * E * tiles128(h), nullptr);
  if (st != MOE_OK) return st;
  const long long items = static_cast<long long>(E) * d * 4 * mx4_kc(h);
  const int blocks = static_cast<int>(std::max(1LL, std::min((items + 255) / 256, 16LL * device_sm_count())));
  mx4_quant_cols_kernel<<<blocks, 256, 0, s>>>(reinterpret_cast<const bf16*>(w_down), E, h, d, down_tiles(d), w.dn_q,
                                               w.dn_sf);
  return launched();
}

moe_status_t moe_mx4_quantize_rows(const moe_bf16* x, const int32_t* offsets, int E, int cap, int K, uint8_t* q,
                                   uint8_t* sf, int32_t* dev_status, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (cap < 0 || K <= 0 || E < 1) return MOE_ERR_INVALID_ARG;
  if (E > MAX_E || !width_ok(K)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!offsets || (cap > 0 && (!x || !q || !sf))) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 16)) return MOE_ERR_INVALID_ARG;
  moe_status_t st = check_device();
  if (st != MOE_OK || cap == 0) return st;
  return launch_rows(mx4_quant_rows_kernel<ROW_PASSES>, mx4_quant_rows_kernel<1>, cap, K,
                     reinterpret_cast<cudaStream_t>(stream), reinterpret_cast<const uint4*>(x), cap, K, offsets, E, 0, 0,
                     reinterpret_cast<uint32_t*>(q), sf, list_tiles(cap, E), dev_status);
}

moe_status_t moe_mx4_dequantize_rows(const uint8_t* q, const uint8_t* sf, const int32_t* offsets, int E, int cap, int K,
                                     moe_bf16* x, int32_t* dev_status, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (cap < 0 || K <= 0 || E < 1) return MOE_ERR_INVALID_ARG;
  if (E > MAX_E || !width_ok(K)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!offsets || (cap > 0 && (!x || !q || !sf))) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 16)) return MOE_ERR_INVALID_ARG;
  moe_status_t st = check_device();
  if (st != MOE_OK || cap == 0) return st;
  return launch_rows(mx4_dequant_rows_kernel<ROW_PASSES>, mx4_dequant_rows_kernel<1>, cap, K,
                     reinterpret_cast<cudaStream_t>(stream), reinterpret_cast<const uint32_t*>(q), sf, cap, K, offsets, E,
                     reinterpret_cast<uint4*>(x), list_tiles(cap, E), dev_status);
}

moe_status_t moe_permute_mxfp4(const moe_bf16* x, const int32_t* inv_map, const int32_t* offsets, int T, int top_k,
                               int E, int d, uint8_t* q, uint8_t* sf, int32_t* dev_status, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (T < 0 || top_k < 1 || d <= 0 || E < 1) return MOE_ERR_INVALID_ARG;
  if (top_k > MAX_TOPK || E > MAX_E || !width_ok(d)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const long long n = static_cast<long long>(T) * top_k;
  if (n >= (1LL << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!offsets || (n > 0 && (!x || !inv_map || !q || !sf))) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 16)) return MOE_ERR_INVALID_ARG;
  moe_status_t st = check_device();
  if (st != MOE_OK || n == 0) return st;
  return launch_rows(mx4_permute_kernel<ROW_PASSES>, mx4_permute_kernel<1>, T, d, reinterpret_cast<cudaStream_t>(stream),
                     reinterpret_cast<const uint4*>(x), inv_map, offsets, E, T, top_k, d, reinterpret_cast<uint32_t*>(q),
                     sf, list_tiles(n, E), dev_status);
}

moe_status_t moe_grouped_swiglu_fwd_mxfp4(const uint8_t* xq, const uint8_t* xsf, const int32_t* offsets, int E, int cap,
                                          int d, int h, const void* mxw, moe_bf16* y, void* ws, size_t ws_bytes,
                                          int32_t* dev_status, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (cap < 0 || d <= 0 || h <= 0 || E < 1) return MOE_ERR_INVALID_ARG;
  if (!shape_ok(E, d, h)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!offsets || !mxw || !aligned(mxw, 256) || (cap > 0 && (!xq || !xsf || !y || !ws))) return MOE_ERR_INVALID_ARG;
  if (!aligned(xq, 16) || !aligned(xsf, 16) || !aligned(y, 16) || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  // tile indices are int
  if (list_tiles(cap, E) * std::max(tiles128(h), (d + BN - 1) / BN) >= (1LL << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (ws_bytes < fwd_ws_bytes(cap, E, h)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  moe_status_t st = check_device();
  if (st != MOE_OK || cap == 0) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const Weights w = carve_weights(mxw, E, d, h);
  uint8_t* pq = static_cast<uint8_t*>(ws);
  uint8_t* psf = pq + codes_bytes(cap, h);
  Args a{};
  a.offsets = offsets;
  a.E = E;
  a.cap = cap;
  a.N = h;
  a.K = d;
  a.h = h;
  a.sfa = xsf;
  a.sfb = w.ug_sf;
  a.kc = mx4_kc(d);
  a.tiles_b = tiles128(h);
  a.pq = pq;
  a.psf = psf;
  a.pkc = mx4_kc(h);
  a.dbg_a_tiles = list_tiles(cap, E);
  a.dbg_b_tiles = 2LL * E * tiles128(h);
  a.status = dev_status;
  if ((st = launch_gemm<MX4_UP>(xq, w.ug_q, 2LL * h, a, s)) != MOE_OK) return st;
  a.N = d;
  a.K = h;
  a.sfa = psf;
  a.sfb = w.dn_sf;
  a.kc = mx4_kc(h);
  a.tiles_b = down_tiles(d);
  a.dbg_b_tiles = static_cast<long long>(E) * down_tiles(d);
  a.y = reinterpret_cast<bf16*>(y);
  return launch_gemm<MX4_DOWN>(pq, w.dn_q, d, a, s);
}

}  // extern "C"
