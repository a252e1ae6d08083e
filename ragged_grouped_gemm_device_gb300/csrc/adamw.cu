// AdamW over many tensors in one launch, with states in 32 or 8 bits, and the gradients' global norm.
//
//   g' = c g;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// Bound by memory with fp32 states: p, m and v are read and written once, g is read once (28 bytes an element, 30 with a bf16 copy:
// 201 million elements 900 us, 6.7 TB/s, and the norm before, which reads g once more, 122). Bound by instructions with 8-bit states:
// 12 bytes an element, but about 80 instructions, the random roundings among them (192 million elements 499 us, 4.7 TB/s).
// Many small tensors: 72 tensors 34 us, 28 for their bytes. The tensors are cut into pieces of
// CHUNK elements, of which each block takes a run; the descriptors travel in the kernel's parameters, and a block finds its first
// tensor by bisecting the first pieces. A thread owns eight consecutive elements, moved 16 bytes at a time where the
// pointers allow it. All arithmetic is fp32; the bias corrections are -expm1(t log b), whose error is a unit in the
// last place for small t too, where 1 - b^t cancels.
//
// 8-bit states: blocks of 32 E4M3 elements share a power of two. v is kept as its square root, whose range the
// elements' 4 exponent bits hold (2^18 within a block). Both are rounded stochastically: with round-to-nearest
// an element that changes by less than half a step (3 to 6%) would never change, and v moves by 1 - b2 a step. A v that is
// not zero is not rounded to zero, because the step divides by it. v gains the variance of its root's rounding:
// about 5% at b2 = 0.999, which makes steps 2.5% shorter.
#include <algorithm>
#include <cmath>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "root.cuh"
#include "rows.cuh"
#include "trace.h"

namespace moe {
namespace {

constexpr int THREADS = 256;
constexpr int VB = 8;         // elements of a thread in one round
constexpr int CHUNK = 4096;   // elements of a piece: two rounds
constexpr int step_blocks(int bits) { return bits == 8 ? 3 : 4; }  // on an SM; four of 8-bit states would spill
// Tensors of a launch: 12 KB of parameters, or 1.5 KB for the few tensors of one block, whose launch would wait for them.
constexpr int MAX_TENSORS = 128, FEW_TENSORS = 16;
constexpr int NORM_BLOCKS = 1216;

template <int N>
struct Batch {
  int count;
  int first;                          // index of the first tensor in the call
  unsigned chunk0[N + 1];   // first piece of each tensor, and the end
  moe_adamw_tensor_t t[N];
  unsigned char wide[N];    // 1: 16-byte accesses
};

// the tensor of piece c: the last one that starts at or before it and is not empty
template <int N>
__device__ __forceinline__ int find_tensor(const Batch<N>& b, unsigned c) {
  int lo = 0, hi = b.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.chunk0[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The finalizer of MurmurHash3 (A. Appleby), a bijection of 32-bit words whose output bits all depend on all
// input bits.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x85EBCA6Bu;
  x ^= x >> 13;
  x *= 0xC2B2AE35u;
  return x ^ (x >> 16);
}

// eight elements from p, the first `k` of them (0 for the rest)
__device__ __forceinline__ void load8(const float* p, int k, bool wide, float (&f)[VB]) {
  if (wide && k == VB) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < VB; ++i) f[i] = i < k ? p[i] : 0.f;
  }
}
__device__ __forceinline__ void load8(const bf16* p, int k, bool wide, float (&f)[VB]) {
  if (wide && k == VB) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VB; ++i) f[i] = i < k ? __bfloat162float(p[i]) : 0.f;
  }
}
__device__ __forceinline__ void store8(float* p, int k, bool wide, const float (&f)[VB]) {
  if (wide && k == VB) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
  } else {
#pragma unroll
    for (int i = 0; i < VB; ++i)
      if (i < k) p[i] = f[i];
  }
}
// to nearest
__device__ __forceinline__ void store8(bf16* p, int k, bool wide, const float (&f)[VB]) {
  if (wide && k == VB) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                              pack_bf16x2(f[6], f[7]));
  } else {
#pragma unroll
    for (int i = 0; i < VB; ++i)
      if (i < k) p[i] = __float2bfloat16_rn(f[i]);
  }
}
__device__ __forceinline__ void load8(const uint8_t* p, int k, bool wide, uint32_t (&w)[2]) {
  if (wide && k == VB) {
    const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p));
    w[0] = a.x, w[1] = a.y;
  } else {
    w[0] = w[1] = 0;
#pragma unroll
    for (int i = 0; i < VB; ++i)
      if (i < k) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  }
}
__device__ __forceinline__ void store8(uint8_t* p, int k, bool wide, const uint32_t (&w)[2]) {
  if (wide && k == VB) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
  } else {
#pragma unroll
    for (int i = 0; i < VB; ++i)
      if (i < k) p[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
}

// the upper halves
__device__ __forceinline__ void store8_upper(bf16* p, int k, bool wide, const float (&f)[VB]) {
  if (wide && k == VB) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __byte_perm(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]), 0x7632);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < VB; ++i)
      if (i < k) reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(__float_as_uint(f[i]) >> 16);
  }
}

// Asynchronous 8-byte copy global -> shared
__device__ __forceinline__ void copy8_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// ------------------------------------------------------------------ 8-bit states
// An E4M3 magnitude is the top 7 bits below the sign of an fp32 value 2^120 times smaller: the exponent biases differ
// by 120, and the subnormals of both types meet.
constexpr float E4M3_DOWN = 0x1p-120f;

__device__ __forceinline__ float block_scale(uint32_t byte) {
  return byte == 0xFF ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}
// two codes of a word
__device__ __forceinline__ float2 from_e4m3x2(uint32_t w, float scale) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
  const float2 v = __half22float2(__half2(h));
  return make_float2(v.x * scale, v.y * scale);
}
// the scale byte of a block from the bits of its largest magnitude
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 0xFF;
  const int b = static_cast<int>(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
  return b > 0 ? b : 0;
}

// Eight values of this thread's quarter of a block into codes; returns the scale byte of the block. All threads of the warp call it.
// KEEP: the values are not negative, and what is not 0 does not become 0.
template <bool KEEP, int SHIFT>
__device__ __forceinline__ uint32_t to_e4m3(const float (&x)[VB], const uint32_t (&rnd)[VB], uint32_t (&w)[2]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < VB; ++i) top = max(top, KEEP ? __float_as_uint(x[i]) : __float_as_uint(x[i]) & 0x7FFFFFFFu);  // by bits: a NaN is the largest
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const uint32_t byte = scale_byte(top);
  w[0] = w[1] = 0;
  if (byte == 0xFF) return byte;
  const auto encode = [&](auto scaled) {
    uint32_t c[VB];
#pragma unroll
    for (int i = 0; i < VB; ++i) {
      c[i] = (__float_as_uint(scaled(fabsf(x[i]))) + (SHIFT == 16 ? rnd[i] >> 16 : rnd[i] & 0xFFFFu) * 16u) >> 20;
      if (KEEP) c[i] = max(c[i], min(__float_as_uint(x[i]), 1u));
    }
#pragma unroll
    for (int i = 0; i < VB; i += 4) {
      w[i >> 2] = __byte_perm(__byte_perm(c[i], c[i + 1], 0x0040), __byte_perm(c[i + 2], c[i + 3], 0x0040), 0x5410);
      // The signs: the highest bytes of four values. (Joined to a code shifted left by 4 before the bytes are packed, nvcc
      // 13.0.88 lost the code.)
      if (!KEEP) {
        const uint32_t lo = __byte_perm(__float_as_uint(x[i]), __float_as_uint(x[i + 1]), 0x0073);
        const uint32_t hi = __byte_perm(__float_as_uint(x[i + 2]), __float_as_uint(x[i + 3]), 0x0073);
        w[i >> 2] |= __byte_perm(lo, hi, 0x5410) & 0x80808080u;
      }
    }
  };
  // 2^-s 2^-120 is an fp32 (subnormal from s = 7 on) up to s = 29; blocks from s = 24 on, whose largest state is above 224 * 2^24, take
  // the two steps apart
  const float inv = __uint_as_float((254u - byte) << 23);
  if (byte <= 150) {
    const float down = inv * E4M3_DOWN;
    encode([&](float v) { return v * down; });
  } else {
    encode([&](float v) { return v * inv * E4M3_DOWN; });
  }
  return byte;
}

struct StepArgs {
  float lr, b1, omb1, b2, omb2, log_b1, log_b2, eps;
  uint32_t seed;
  int32_t* steps;
  const float* lr_scale;
  const float* grad_scale;
  unsigned blocks;  // of this launch
  bool last;        // the call's last launch counts the step
};

// to two units; 0 beyond 2^126
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// What a thread reads of one round, as it lies in memory where that takes 16-byte accesses
template <int BITS>
struct Raw {
  float g[VB], p[VB], m[VB], v[VB];
  uint32_t wm[2], wv[2], sm, sv;

  __device__ __forceinline__ void load(const moe_adamw_tensor_t& q, long long i0, int k, bool wide) {
    if (q.g_dtype == MOE_DTYPE_BF16) load8(static_cast<const bf16*>(q.g) + i0, k, wide, g);
    else load8(static_cast<const float*>(q.g) + i0, k, wide, g);
    if (q.p_dtype == MOE_DTYPE_BF16) load8(static_cast<const bf16*>(q.p) + i0, k, wide, p);
    else load8(static_cast<const float*>(q.p) + i0, k, wide, p);
    if constexpr (BITS == 8) {
      load8(static_cast<const uint8_t*>(q.m) + i0, k, wide, wm);
      load8(static_cast<const uint8_t*>(q.v) + i0, k, wide, wv);
      sm = k > 0 ? q.m_scale[i0 >> 5] : 0;
      sv = k > 0 ? q.v_scale[i0 >> 5] : 0;
    } else {
      load8(static_cast<const float*>(q.m) + i0, k, wide, m);
      load8(static_cast<const float*>(q.v) + i0, k, wide, v);
    }
  }
};

// What the next round of 8-bit states reads, on its way into shared memory during the arithmetic of this one (192 million elements:
// 520 us with four blocks on an SM that load as they go, 487 so; in registers it would spill, two rounds ahead took 512). A warp copies its 256 elements' gradients and parameters as they lie, 16 bytes a lane, and of m and v each lane its own eight
// bytes; the scales, single bytes, wait in registers.
struct Ahead {
  static constexpr int WARP = 32 * (32 + 32 + 8 + 8), BYTES = THREADS / 32 * WARP;
  const uint8_t *g, *p, *m, *v, *ms, *vs;  // of this lane's next copies
  uint32_t at, sm, sv;                     // this warp's shared memory; scales
  int eg, ep, left;                        // element bytes, rounds not begun

  __device__ __forceinline__ void start() {
    if (left > 0) {
      const uint32_t lane = threadIdx.x & 31;
      copy16_async(at + lane * 16, g);
      if (eg == 4) copy16_async(at + 512 + lane * 16, g + 512);
      copy16_async(at + 1024 + lane * 16, p);
      if (ep == 4) copy16_async(at + 1536 + lane * 16, p + 512);
      copy8_async(at + 2048 + lane * 8, m);
      copy8_async(at + 2304 + lane * 8, v);
      sm = *ms, sv = *vs;
      constexpr int n = THREADS * VB;
      g += n * eg, p += n * ep, m += n, v += n, ms += n / 32, vs += n / 32;
      --left;
    }
    copy_commit();
  }
  // this lane's first element, and the rounds
  __device__ __forceinline__ void begin(const moe_adamw_tensor_t& q, long long i0, int rounds, uint8_t* smem) {
    const int lane = threadIdx.x & 31;
    const long long w0 = i0 - lane * VB;
    eg = q.g_dtype == MOE_DTYPE_BF16 ? 2 : 4;
    ep = q.p_dtype == MOE_DTYPE_BF16 ? 2 : 4;
    g = static_cast<const uint8_t*>(q.g) + w0 * eg + lane * 16;
    p = static_cast<const uint8_t*>(q.p) + w0 * ep + lane * 16;
    m = static_cast<const uint8_t*>(q.m) + i0;
    v = static_cast<const uint8_t*>(q.v) + i0;
    ms = q.m_scale + (i0 >> 5);
    vs = q.v_scale + (i0 >> 5);
    left = rounds;
    at = smem_u32(smem) + (threadIdx.x >> 5) * WARP;
    start();
  }
  __device__ __forceinline__ void get(uint32_t from, int es, float (&f)[VB]) const {
    const uint32_t lane = threadIdx.x & 31;
    uint32_t w[4];
    if (es == 2) {
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from + lane * 16));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from + lane * 32 + j * 16));
#pragma unroll
        for (int i = 0; i < 4; ++i) f[4 * j + i] = __uint_as_float(w[i]);
      }
    }
  }
  template <typename R>
  __device__ __forceinline__ void take(R& d) {
    copy_wait<0>();
    __syncwarp();  // lanes copy for one another
    const uint32_t lane = threadIdx.x & 31;
    get(at, eg, d.g);
    get(at + 1024, ep, d.p);
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(d.wm[0]), "=r"(d.wm[1]) : "r"(at + 2048 + lane * 8));
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(d.wv[0]), "=r"(d.wv[1]) : "r"(at + 2304 + lane * 8));
    d.sm = sm, d.sv = sv;
    __syncwarp();
    start();
  }
};

struct TensorStep {
  float c, step, root, decay;
  uint32_t key;
};

// One round: eight elements from i0, k of them the tensor's (FULL: all, by 16-byte accesses). All threads of a warp call it.
template <int BITS, bool FULL>
__device__ __forceinline__ void adamw_round(const moe_adamw_tensor_t& q, const StepArgs& a, const TensorStep& u, long long i0, int k,
                                            bool wide, Raw<BITS>& d) {
  if constexpr (FULL) k = VB, wide = true;
  float r[VB];
  if constexpr (BITS == 8) {
    const float sm = block_scale(d.sm), sv = block_scale(d.sv);
#pragma unroll
    for (int i = 0; i < VB; i += 2) {
      const float2 m = from_e4m3x2(d.wm[i >> 2] >> (8 * (i & 3)), sm), v = from_e4m3x2(d.wv[i >> 2] >> (8 * (i & 3)), sv);
      d.m[i] = m.x, d.m[i + 1] = m.y;
      d.v[i] = v.x * v.x, d.v[i + 1] = v.y * v.y;
    }
  }
  // Each operation is rounded by itself: a stochastic rounding goes the other way where its argument differs in the last place, and
  // m and v are to be what the formula written out gives.
  float odd = 0.f;  // not 0 when a root is not finite
#pragma unroll
  for (int i = 0; i < VB; ++i) {
    const float gc = __fmul_rn(d.g[i], u.c);
    d.m[i] = __fadd_rn(__fmul_rn(a.b1, d.m[i]), __fmul_rn(a.omb1, gc));
    d.v[i] = __fadd_rn(__fmul_rn(a.b2, d.v[i]), __fmul_rn(__fmul_rn(a.omb2, gc), gc));
    r[i] = sqrt_normal(d.v[i]);
    odd = fmaf(r[i], 0.f, odd);
  }
  if (!(odd == 0.f)) {  // zeros, subnormals, infinities or NaNs among the v
#pragma unroll
    for (int i = 0; i < VB; ++i) r[i] = sqrtf(d.v[i]);
  }
  // What is taken from p, the quotient to two units: a small part of p. A bf16 p is rounded by its fraction, of which only whole units
  // matter there: cut off, not rounded, so that this rounding decides none (486 -> 499 us for 192 million elements with 8-bit states).
#pragma unroll
  for (int i = 0; i < VB; ++i) {
    const float less = fmaf(d.p[i], u.decay, (u.step * d.m[i]) * reciprocal(fmaf(r[i], u.root, a.eps)));
    d.p[i] = q.p_dtype == MOE_DTYPE_BF16 ? __fsub_rz(d.p[i], less) : d.p[i] - less;
  }
  uint32_t rnd[VB];
  if (BITS == 8 || q.p_dtype == MOE_DTYPE_BF16) {
    const uint32_t x0 = u.key + static_cast<uint32_t>(i0) * 0x9E3779B9u + static_cast<uint32_t>(i0 >> 32) * 0x85EBCA6Bu;
#pragma unroll
    for (int i = 0; i < VB; ++i) rnd[i] = mix(x0 + static_cast<uint32_t>(i) * 0x9E3779B9u);
  }
  if (q.p_dtype == MOE_DTYPE_BF16) {
    // To bf16, up in magnitude where the fraction and u / 2^16 reach 1: the upper half of the sum of the bits. A NaN, whose sum could
    // leave the NaNs, stays.
    float nan = 0.f;
#pragma unroll
    for (int i = 0; i < VB; ++i) nan = fmaf(d.p[i], 0.f, nan);
    if (nan == 0.f) {
#pragma unroll
      for (int i = 0; i < VB; ++i) d.p[i] = __uint_as_float(__float_as_uint(d.p[i]) + __byte_perm(rnd[i], 0, 0x4421));  // the middle 16 bits
    } else {
#pragma unroll
      for (int i = 0; i < VB; ++i)
        if (d.p[i] == d.p[i]) d.p[i] = __uint_as_float(__float_as_uint(d.p[i]) + __byte_perm(rnd[i], 0, 0x4421));
    }
    store8_upper(static_cast<bf16*>(q.p) + i0, k, wide, d.p);
  } else {
    store8(static_cast<float*>(q.p) + i0, k, wide, d.p);
    if (q.copy != nullptr) store8(static_cast<bf16*>(q.copy) + i0, k, wide, d.p);
  }
  if constexpr (BITS == 8) {
    if constexpr (!FULL) {
#pragma unroll
      for (int i = 0; i < VB; ++i) {  // what lies behind the tensor's end takes no part in its last block
        d.m[i] = i < k ? d.m[i] : 0.f;
        r[i] = i < k ? r[i] : 0.f;
      }
    }
    uint32_t w[2];
    uint32_t byte = to_e4m3<false, 0>(d.m, rnd, w);
    store8(static_cast<uint8_t*>(q.m) + i0, k, wide, w);
    if (k > 0 && (threadIdx.x & 3) == 0) q.m_scale[i0 >> 5] = static_cast<uint8_t>(byte);
    byte = to_e4m3<true, 16>(r, rnd, w);
    store8(static_cast<uint8_t*>(q.v) + i0, k, wide, w);
    if (k > 0 && (threadIdx.x & 3) == 0) q.v_scale[i0 >> 5] = static_cast<uint8_t>(byte);
  } else {
    store8(static_cast<float*>(q.m) + i0, k, wide, d.m);
    store8(static_cast<float*>(q.v) + i0, k, wide, d.v);
  }
}

template <int BITS, int N>
__global__ void __launch_bounds__(THREADS, step_blocks(BITS)) adamw_kernel(const __grid_constant__ Batch<N> batch, const StepArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];  // 8-bit states: Ahead::BYTES
  grid_wait();
  TensorStep u;
  u.c = a.grad_scale ? *after_wait(a.grad_scale) : 1.0f;
  if (u.c != u.c) return;  // the norm was not finite: the step is skipped
  const int t = *reinterpret_cast<volatile int32_t*>(a.steps) + 1;
  const unsigned long long all = batch.chunk0[batch.count];
  const unsigned c1 = static_cast<unsigned>(all * (blockIdx.x + 1) / gridDim.x);
  unsigned c = static_cast<unsigned>(all * blockIdx.x / gridDim.x);
  if (c < c1) {
    const float lr = a.lr_scale ? a.lr * *after_wait(a.lr_scale) : a.lr;
    u.step = lr / -expm1f(static_cast<float>(t) * a.log_b1);
    u.root = 1.0f / sqrtf(-expm1f(static_cast<float>(t) * a.log_b2));
    for (int j = find_tensor(batch, c); c < c1; ++j) {
      const moe_adamw_tensor_t& q = batch.t[j];
      const unsigned end = min(c1, batch.chunk0[j + 1]);
      u.decay = lr * q.weight_decay;
      u.key = mix(a.seed ^ mix(0x9E3779B9u * static_cast<uint32_t>(t) + static_cast<uint32_t>(batch.first + j)));
      const bool wide = batch.wide[j] != 0;
      long long i0 = static_cast<long long>(c - batch.chunk0[j]) * CHUNK + threadIdx.x * VB;
      const long long last = min(q.n, static_cast<long long>(end - batch.chunk0[j]) * CHUNK);  // of this block's run
      Raw<BITS> d;
      if constexpr (BITS == 8) {
        const int rounds = wide ? static_cast<int>((last - (i0 - threadIdx.x * VB)) / (THREADS * VB)) : 0;
        Ahead ahead;
        if (rounds > 0) ahead.begin(q, i0, rounds, smem);
        for (int k = 0; k < rounds; ++k, i0 += THREADS * VB) {
          ahead.take(d);
          adamw_round<BITS, true>(q, a, u, i0, VB, true, d);
        }
      } else {
        for (; i0 - threadIdx.x * VB + THREADS * VB <= last && wide; i0 += THREADS * VB) {
          d.load(q, i0, VB, true);
          adamw_round<BITS, true>(q, a, u, i0, VB, true, d);
        }
      }
      for (; i0 - threadIdx.x * VB < last; i0 += THREADS * VB) {
        const int k = static_cast<int>(max(0LL, min(static_cast<long long>(VB), last - i0)));  // elements of this thread
        d.load(q, i0, k, wide);
        adamw_round<BITS, false>(q, a, u, i0, k, wide, d);
      }
      c = end;
    }
  }
  // The last block to end counts the step: by then every thread has read the count.
  if (!a.last) return;
  __syncthreads();
  if (threadIdx.x != 0) return;
  __threadfence();
  if (atomicAdd(a.steps + 1, 1) == static_cast<int>(a.blocks) - 1) {
    a.steps[1] = 0;
    a.steps[0] = t;
  }
}

// Partial sums of g^2, one fp64 per block: the pieces blockIdx.x, blockIdx.x + gridDim.x, ... of a launch's tensors, added to
// what the launches before it left.
template <int N>
__global__ void __launch_bounds__(THREADS) grad_norm_kernel(const __grid_constant__ Batch<N> batch, double* part, bool first) {
  __shared__ __align__(16) float red[2][32];
  grid_wait();
  double sum = 0.0;
  int par = 0;
  for (unsigned c = blockIdx.x; c < batch.chunk0[batch.count]; c += gridDim.x) {
    const int j = find_tensor(batch, c);
    const moe_adamw_tensor_t& q = batch.t[j];
    const bool wide = batch.wide[j] != 0;
    float s = 0.f;
#pragma unroll
    for (int round = 0; round < CHUNK / (THREADS * VB); ++round) {
      const long long i0 = static_cast<long long>(c - batch.chunk0[j]) * CHUNK + (round * THREADS + threadIdx.x) * VB;
      const int k = static_cast<int>(max(0LL, min(static_cast<long long>(VB), q.n - i0)));
      float g[VB];
      if (q.g_dtype == MOE_DTYPE_BF16) load8(static_cast<const bf16*>(q.g) + i0, k, wide, g);
      else load8(static_cast<const float*>(q.g) + i0, k, wide, g);
#pragma unroll
      for (int i = 0; i < VB; ++i) s = fmaf(g[i], g[i], s);
    }
    sum += static_cast<double>(row_sum<THREADS>(s, red[par]));
    par ^= 1;
  }
  if (threadIdx.x == 0) part[blockIdx.x] = first ? sum : part[blockIdx.x] + sum;
}

// The norm and the coefficient from the partial sums, in index order within each thread and by a fixed tree.
__global__ void __launch_bounds__(256) grad_norm_end_kernel(const double* part, int blocks, float max_norm, float* norm) {
  __shared__ double acc[8];
  grid_wait();
  part = after_wait(part);
  constexpr int ROUNDS = (NORM_BLOCKS + 255) / 256;
  double v[ROUNDS], s = 0.0;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) v[i] = threadIdx.x + 256 * i < blocks ? part[threadIdx.x + 256 * i] : 0.0;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) s += v[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) acc[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  s = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
  const float n = static_cast<float>(sqrt(s));
  norm[0] = n;
  norm[1] = n <= 3.402823466e38f ? max_norm / fmaxf(n, max_norm) : __uint_as_float(0x7FC00000u);
}

bool aligned_to(const void* p, int b) { return (reinterpret_cast<uintptr_t>(p) & (b - 1)) == 0; }

// What a call's tensors have to be; `grads` only g, g_dtype and n
moe_status_t check_tensors(const moe_adamw_tensor_t* t, int count, bool grads, int bits) {
  if (count < 0 || (count > 0 && !t)) return MOE_ERR_INVALID_ARG;
  unsigned long long total = 0;
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor_t& q = t[i];
    if (q.n < 0 || !dtype_ok(q.g_dtype)) return MOE_ERR_INVALID_ARG;
    if (q.n >= (1LL << 43)) return MOE_ERR_UNSUPPORTED_SHAPE;
    total += (static_cast<unsigned long long>(q.n) + CHUNK - 1) / CHUNK;
    if (total >= (1ull << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!aligned_to(q.g, dtype_bytes(q.g_dtype)) || (q.n > 0 && !q.g)) return MOE_ERR_INVALID_ARG;
    if (grads) continue;
    if (!dtype_ok(q.p_dtype) || q.reserved != 0 || !std::isfinite(q.weight_decay)) return MOE_ERR_INVALID_ARG;
    if (q.copy && q.p_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(q.p, dtype_bytes(q.p_dtype)) || !aligned_to(q.copy, 2)) return MOE_ERR_INVALID_ARG;
    if (bits == 32 && (!aligned_to(q.m, 4) || !aligned_to(q.v, 4))) return MOE_ERR_INVALID_ARG;
    if (q.n > 0 && (!q.p || !q.m || !q.v || (bits == 8 && (!q.m_scale || !q.v_scale)))) return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

// the tensors i, i + 1, ... that one launch takes
template <int N>
int fill(Batch<N>& b, const moe_adamw_tensor_t* t, int i, int count, bool grads, int bits) {
  const int n = std::min(count - i, N);
  b.count = n;
  b.first = i;
  unsigned at = 0;
  for (int k = 0; k < n; ++k) {
    const moe_adamw_tensor_t& q = t[i + k];
    b.t[k] = q;
    b.chunk0[k] = at;
    at += static_cast<unsigned>((q.n + CHUNK - 1) / CHUNK);
    b.wide[k] = aligned16(q.g) && (grads || (aligned16(q.p) && aligned16(q.copy) && aligned_to(q.m, bits == 8 ? 8 : 16) &&
                                             aligned_to(q.v, bits == 8 ? 8 : 16)));
  }
  b.chunk0[n] = at;
  return n;
}

template <int N>
cudaError_t launch_norm(const moe_adamw_tensor_t* tensors, int count, int blocks, double* part, cudaStream_t s) {
  for (int i = 0; i < count || i == 0;) {
    Batch<N> b;
    const int n = fill(b, tensors, i, count, true, 0);
    const cudaError_t err = launch_dependent(grad_norm_kernel<N>, blocks, THREADS, 0, s, b, part, i == 0);
    if (err != cudaSuccess) return err;
    i += std::max(n, 1);
  }
  return cudaSuccess;
}

template <int N>
cudaError_t launch_step(StepArgs a, const moe_adamw_tensor_t* tensors, int count, int state_bits, cudaStream_t s) {
  for (int i = 0; i < count || i == 0;) {
    Batch<N> b;
    const int n = fill(b, tensors, i, count, false, state_bits);
    // 8-bit states: as many blocks as fit, since what a block computes once would be a fifth of the instructions of a piece. 32 bits,
    // bound by memory: a block for each piece, which spread better (201 million parameters: 902 us, 1047 in runs).
    a.blocks = std::max(b.chunk0[n], 1u);
    if (state_bits == 8) a.blocks = std::min(a.blocks, static_cast<unsigned>(step_blocks(8) * device_sm_count()));
    a.last = i + n >= count;
    const cudaError_t err = launch_dependent(state_bits == 8 ? adamw_kernel<8, N> : adamw_kernel<32, N>, a.blocks, THREADS, state_bits == 8 ? Ahead::BYTES : 0, s, b, a);
    if (err != cudaSuccess) return err;
    i += std::max(n, 1);
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_norm_workspace_bytes() { return NORM_BLOCKS * sizeof(double); }

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_grad_norm(const moe_adamw_tensor_t* tensors, int count, float max_norm, float* norm, void* ws,
                           size_t ws_bytes, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (!(max_norm > 0.f) || std::isinf(max_norm) || !norm || !element_aligned(norm, 4) || !aligned_to(ws, 8)) return MOE_ERR_INVALID_ARG;
  moe_status_t st = check_tensors(tensors, count, true, 0);
  if (st != MOE_OK) return st;
  if (ws_bytes < grad_norm_workspace_bytes()) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!ws) return MOE_ERR_INVALID_ARG;
  st = check_device();
  if (st != MOE_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(ws);
  unsigned most = 1;  // blocks: no more than the largest launch has pieces
  for (int i = 0; i < count; i += MAX_TENSORS) {
    unsigned chunks = 0;
    for (int k = i; k < std::min(count, i + MAX_TENSORS); ++k) chunks += static_cast<unsigned>((tensors[k].n + CHUNK - 1) / CHUNK);
    most = std::max(most, chunks);
  }
  const int blocks = static_cast<int>(std::min<unsigned>(most, NORM_BLOCKS));
  cudaError_t err = count <= FEW_TENSORS ? launch_norm<FEW_TENSORS>(tensors, count, blocks, part, s)
                                           : launch_norm<MAX_TENSORS>(tensors, count, blocks, part, s);
  if (err == cudaSuccess)
    err = launch_dependent(grad_norm_end_kernel, 1, 256, 0, s, static_cast<const double*>(part), blocks, max_norm, norm);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

moe_status_t moe_adamw_step(const moe_adamw_tensor_t* tensors, int count, int state_bits, double lr, double beta1,
                            double beta2, double eps, uint32_t seed, int32_t* steps, const float* lr_scale,
                            const float* grad_scale, moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (state_bits != 32 && state_bits != 8) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(lr) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || std::isinf(eps))
    return MOE_ERR_INVALID_ARG;
  if (!steps || !element_aligned(steps, 4) || !element_aligned(lr_scale, 4) || !element_aligned(grad_scale, 4))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = check_tensors(tensors, count, false, state_bits);
  if (st != MOE_OK) return st;
  st = check_device();
  if (st != MOE_OK) return st;
  StepArgs a{};
  a.lr = static_cast<float>(lr);
  a.b1 = static_cast<float>(beta1);
  a.omb1 = static_cast<float>(1.0 - beta1);
  a.b2 = static_cast<float>(beta2);
  a.omb2 = static_cast<float>(1.0 - beta2);
  a.log_b1 = static_cast<float>(std::log(beta1));
  a.log_b2 = static_cast<float>(std::log(beta2));
  a.eps = eps > 0.0 ? std::max(static_cast<float>(eps), 1.17549435e-38f) : 0.f;  // the quotient takes subnormals for 0
  a.seed = seed;
  a.steps = steps;
  a.lr_scale = lr_scale;
  a.grad_scale = grad_scale;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = count <= FEW_TENSORS ? launch_step<FEW_TENSORS>(a, tensors, count, state_bits, s)
                                               : launch_step<MAX_TENSORS>(a, tensors, count, state_bits, s);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

}  // extern "C"
