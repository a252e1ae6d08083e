// Pieces of rows shared by the norm kernels: typed chunks, weights, sums over the threads of a row,
// asynchronous copies.
#pragma once

#include "common.cuh"

namespace moe {
namespace {

// VB consecutive elements of a row: one 16-byte access, or one element where the rows or bases
// are not 16-byte aligned.
template <typename T, int VB>
struct Chunk;
template <>
struct Chunk<bf16, 8> {
  uint4 v;
  __device__ __forceinline__ void from_shared(uint32_t a) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  }
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
  __device__ __forceinline__ void from_shared(uint32_t a) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  }
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
  // not __ldg: an output may lie over the rows, and the join reads back what it has stored
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ void unpack(float (&f)[1]) const { f[0] = v; }
  static __device__ __forceinline__ void store(float* p, const float (&f)[1]) { *p = f[0]; }
};

// VB consecutive weights from column c: fp32 or bf16, `fill` where there are none.
template <int VB>
__device__ __forceinline__ void load_weight(const void* w, bool w_bf16, int c, float fill, float (&o)[VB]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < VB; ++i) o[i] = fill;
  } else if constexpr (VB == 1) {
    o[0] = w_bf16 ? __bfloat162float(static_cast<const bf16*>(w)[c]) : __ldg(static_cast<const float*>(w) + c);
  } else if (w_bf16) {
#pragma unroll
    for (int i = 0; i < VB; i += 4) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const bf16*>(w) + c + i));
      o[i] = bf16_lo(q.x);
      o[i + 1] = bf16_hi(q.x);
      o[i + 2] = bf16_lo(q.y);
      o[i + 3] = bf16_hi(q.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VB; i += 4) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + c + i));
      o[i] = q.x;
      o[i + 1] = q.y;
      o[i + 2] = q.z;
      o[i + 3] = q.w;
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the TPR threads of a row. For rows wider than a warp, `buf` is one of two alternating
// buffers: a thread that is a reduction ahead writes the other one.
template <int TPR>
__device__ __forceinline__ float row_sum(float a, float* buf) {
  a = warp_sum(a);
  if constexpr (TPR == 32) {
    return a;
  } else {
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = a;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < TPR / 32; w += 4) {
      const float4 q = *reinterpret_cast<const float4*>(buf + w);
      s += (q.x + q.y) + (q.z + q.w);
    }
    return s;
  }
}

// ... of a and b: the lower half of the warp adds up a, the upper half b
template <int TPR>
__device__ __forceinline__ float2 row_sum(float a, float b, float* buf) {
  const bool up = (threadIdx.x & 16) != 0;
  float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR == 32) {
    return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
  } else {
    if ((threadIdx.x & 15) == 0) buf[(up ? TPR / 32 : 0) + (threadIdx.x >> 5)] = v;
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < TPR / 32; w += 4) {
      const float4 p = *reinterpret_cast<const float4*>(buf + w), q = *reinterpret_cast<const float4*>(buf + TPR / 32 + w);
      s.x += (p.x + p.y) + (p.z + p.w);
      s.y += (q.x + q.y) + (q.z + q.w);
    }
    return s;
  }
}

// threads of a block: a row's TPR, or four rows of one warp each
__host__ __device__ constexpr int block_threads(int tpr) { return tpr == 32 ? 128 : tpr; }

// Asynchronous 16-byte copy global -> shared, and the group it is waited for by.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Two fp32 values that one instruction takes together.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pair(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 both(float x) { return pair(x, x); }
__device__ __forceinline__ float2 parts(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dtype_ok(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F32; }
int dtype_bytes(int t) { return t == MOE_DTYPE_BF16 ? 2 : 4; }
bool element_aligned(const void* p, int es) { return (reinterpret_cast<uintptr_t>(p) & (es - 1)) == 0; }

}  // namespace
}  // namespace moe
