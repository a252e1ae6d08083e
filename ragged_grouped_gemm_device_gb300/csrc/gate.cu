// The router's gate: softmax over the experts, the top_k experts of each token and their weights,
// per-expert counts, the balance and z losses, and the gradient of all of it.
//
//   p = softmax(l_t);  lse_t = log sum_e exp(l_te);  ids = top_k experts by logit, ties to the lower id
//   w_j = p_ids[j], or with MOE_GATE_RENORM p_ids[j] / sum_i p_ids[i]
//   counts_e = slots routed to e;  N = tokens that take part;  P_e = sum_t p_te
//   L_bal = E sum_e (counts_e / (top_k N)) (P_e / N);  L_z = sum_t lse_t^2 / N
// The gradient treats the counts as constants (they are step functions of the logits):
//   dl_e = p_e (c_e - sum_i p_i c_i - s + 2 dL_z lse / N) + [e = ids[j]] w_j (dw_j - s')
// with c_e = dL_bal E counts_e / (top_k N^2); without renormalisation s = sum_j w_j dw_j and
// s' = 0, with it s = 0 and s' = sum_j w_j dw_j.
//
// One warp a token, its logits in registers: expert e = 32 j + lane is element j of lane e % 32.
// Each logit is read once by the forward and once by the backward. The per-expert sums over the
// tokens of a warp stay in registers (lane and element own an expert), a block adds its warps'
// sums in order and leaves one partial row in the workspace, and a second kernel adds those in
// block order: no floating-point atomics, so results do not depend on scheduling.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "trace.h"

namespace moe {
namespace {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int MAX_E = 1024;
constexpr int MAX_TOPK = 32;
// Blocks at most, and so rows of partial sums: four for each of the 152 SMs. A constant, because
// the size of the workspace is host arithmetic.
constexpr int MAX_BLOCKS = 608;
constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

// Unsigned key with the order of the floats. A logit of -inf or NaN gets 0, below every other
// value: it is never selected.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (!(f > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(f == 0.f ? 0.f : f);  // -0 and +0 tie
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

struct GateArgs {
  const void* logits;
  long long ld;
  const uint8_t* mask;  // nullable [T]
  int T, k, E;
  bool renorm;
  int32_t* ids;
  float* weights;
  float* lse;           // nullable
  float* part;          // nullable: per block [P_e (E) | counts_e (E) | sum lse^2 | tokens], 4-byte words
};

constexpr int part_words(int E) { return 2 * E + 2; }

template <typename T, int NV>
__global__ void __launch_bounds__(THREADS) gate_fwd_kernel(const GateArgs a) {
  extern __shared__ float sh[];  // [WARPS][E] probability sums, then [E] counts
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool stats = a.part != nullptr;
  int* s_cnt = reinterpret_cast<int*>(sh + WARPS * a.E);
  if (stats) {
    for (int e = threadIdx.x; e < a.E; e += THREADS) s_cnt[e] = 0;
    __syncthreads();
  }
  float psum[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) psum[j] = 0.f;
  float z = 0.f;
  int tokens = 0;
  for (long long t = static_cast<long long>(blockIdx.x) * WARPS + warp; t < a.T;
       t += static_cast<long long>(gridDim.x) * WARPS) {
    int32_t* ids = a.ids + t * a.k;
    float* wt = a.weights + t * a.k;
    const bool on = a.mask == nullptr || __ldg(a.mask + t) != 0;  // warp-uniform
    float v[NV];
    float m = -INFINITY;
    if (on) {
      const T* row = static_cast<const T*>(a.logits) + t * a.ld;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e = 32 * j + lane;
        v[j] = e < a.E ? load_logit(row + e) : -INFINITY;
        m = fmaxf(m, v[j]);  // ignores NaN
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
    }
    const float base = m > -INFINITY ? m : 0.f;
    float p[NV];
    float sum = 0.f;
    if (on) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        p[j] = __expf(v[j] - base);
        sum += p[j];
      }
      sum = warp_sum(sum);
    }
    // a token without any logit above -inf takes no part, like a masked one; one with a NaN
    // does, and its probabilities are NaN
    if (!on || sum == 0.f) {
      if (lane < a.k) {
        ids[lane] = -1;
        wt[lane] = 0.f;
      }
      if (a.lse != nullptr && lane == 0) a.lse[t] = -INFINITY;
      continue;
    }
    const float inv = 1.0f / sum;
    const float lse = base + logf(sum);
    if (a.lse != nullptr && lane == 0) a.lse[t] = lse;
    if (stats) {
#pragma unroll
      for (int j = 0; j < NV; ++j) psum[j] = fmaf(p[j], inv, psum[j]);
      z = fmaf(lse, lse, z);
      ++tokens;
    }
    // top_k: k rounds of a warp-wide maximum; ties go to the lower expert
    uint32_t key[NV];
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      key[j] = order_key(v[j]);
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    }
    int my_id = -1;
    float my_e = 0.f;
    for (int r = 0; r < a.k; ++r) {
      const uint32_t top = __reduce_max_sync(FULL, best);
      if (top == 0u) break;  // warp-uniform: fewer than k selectable experts
      const int id = static_cast<int>(__reduce_min_sync(FULL, best == top ? static_cast<unsigned>(32 * at + lane) : FULL));
      if (lane == r) {
        my_id = id;
        const uint32_t b = (top & 0x80000000u) ? (top & 0x7fffffffu) : ~top;  // the logit again
        my_e = __expf(__uint_as_float(b) - base);
      }
      if (lane == (id & 31)) {
        best = 0u;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (32 * j + lane == id) key[j] = 0u;
          if (key[j] > best) {
            best = key[j];
            at = j;
          }
        }
      }
    }
    const float norm = a.renorm ? warp_sum(my_e) : sum;
    // a NaN anywhere in the row makes every weight of the row NaN, renormalised or not
    const float w = sum != sum ? sum : my_e / norm;
    if (lane < a.k) {
      ids[lane] = my_id;
      wt[lane] = my_id >= 0 ? w : 0.f;
      if (stats && my_id >= 0) atomicAdd(s_cnt + my_id, 1);
    }
  }
  if (!stats) return;
  __shared__ float s_z[WARPS];
  __shared__ int s_n[WARPS];
  float* mine = sh + warp * a.E;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (32 * j + lane < a.E) mine[32 * j + lane] = psum[j];
  if (lane == 0) {
    s_z[warp] = z;
    s_n[warp] = tokens;
  }
  __syncthreads();
  float* out = a.part + static_cast<size_t>(blockIdx.x) * part_words(a.E);
  int* iout = reinterpret_cast<int*>(out);
  for (int e = threadIdx.x; e < a.E; e += THREADS) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) s += sh[w * a.E + e];
    out[e] = s;
    iout[a.E + e] = s_cnt[e];
  }
  if (threadIdx.x == 0) {
    float sz = 0.f;
    int n = 0;
    for (int w = 0; w < WARPS; ++w) {
      sz += s_z[w];
      n += s_n[w];
    }
    out[2 * a.E] = sz;
    iout[2 * a.E + 1] = n;
  }
}

// Adds the blocks' partial rows in order: one block, thread e over the blocks (coalesced over
// the experts), then the two losses from the totals.
__global__ void __launch_bounds__(1024) gate_stats_kernel(const float* __restrict__ part, int blocks, int k, int E,
                                                          int32_t* __restrict__ counts, int32_t* __restrict__ n_valid,
                                                          float* __restrict__ prob_sum, float* __restrict__ loss) {
  __shared__ float s_p[32][33];
  __shared__ int s_c[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int words = part_words(E);
  const int* ipart = reinterpret_cast<const int*>(part);
  float z = 0.f;
  int n = 0;
  if (threadIdx.x < 32) {
    for (int b = cx; b < blocks; b += 32) {
      z += part[static_cast<size_t>(b) * words + 2 * E];
      n += ipart[static_cast<size_t>(b) * words + 2 * E + 1];
    }
    z = warp_sum(z);
    n = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(n)));
  }
  float bal = 0.f;  // sum of counts_e P_e (first warp)
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + cx;
    float p = 0.f;
    int c = 0;
    if (e < E)
      for (int b = ry; b < blocks; b += 32) {
        p += part[static_cast<size_t>(b) * words + e];
        c += ipart[static_cast<size_t>(b) * words + E + e];
      }
    s_p[ry][cx] = p;
    s_c[ry][cx] = c;
    __syncthreads();
    if (ry == 0) {
      p = 0.f;
      c = 0;
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        p += s_p[r][cx];
        c += s_c[r][cx];
      }
      if (e < E) {
        prob_sum[e] = p;
        counts[e] = c;
      }
      bal = fmaf(static_cast<float>(c), p, bal);
    }
    __syncthreads();
  }
  if (threadIdx.x < 32) {
    bal = warp_sum(bal);
    if (threadIdx.x == 0) {
      const float nf = static_cast<float>(n);
      *n_valid = n;
      loss[0] = n > 0 ? static_cast<float>(E) / (static_cast<float>(k) * nf) * (bal / nf) : 0.f;
      loss[1] = n > 0 ? z / nf : 0.f;
    }
  }
}

struct GateBwdArgs {
  const void* logits;
  long long ld;
  const float* lse;
  const int32_t* ids;
  const float* weights;
  const int32_t* counts;   // nullable with d_loss
  const int32_t* n_valid;
  const float* d_weights;  // nullable [T, k]
  const float* d_loss;     // nullable [2]
  int T, k, E;
  bool renorm;
  void* dlogits;
  long long ldd;
};

template <typename T, int NV>
__global__ void __launch_bounds__(THREADS) gate_bwd_kernel(const GateBwdArgs a) {
  extern __shared__ float sh[];  // [WARPS][E] what the selected experts of the warp's token get on top
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* mine = sh + warp * a.E;
  float c[NV];
  float cz = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) c[j] = 0.f;
  if (a.d_loss != nullptr) {
    const int n = __ldg(a.n_valid);
    if (n > 0) {
      const float nf = static_cast<float>(n);
      const float cb = __ldg(a.d_loss) * static_cast<float>(a.E) / (static_cast<float>(a.k) * nf) / nf;
      cz = 2.0f * __ldg(a.d_loss + 1) / nf;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (32 * j + lane < a.E) c[j] = cb * static_cast<float>(__ldg(a.counts + 32 * j + lane));
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (32 * j + lane < a.E) mine[32 * j + lane] = 0.f;
  __syncwarp();
  for (long long t = static_cast<long long>(blockIdx.x) * WARPS + warp; t < a.T;
       t += static_cast<long long>(gridDim.x) * WARPS) {
    T* out = static_cast<T*>(a.dlogits) + t * a.ldd;
    const float lse = __ldg(a.lse + t);
    if (lse == -INFINITY) {  // the token took no part (warp-uniform)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (32 * j + lane < a.E) store_logit(out + 32 * j + lane, 0.f);
      continue;
    }
    int id = -1;
    float w = 0.f, dw = 0.f;
    if (lane < a.k && a.d_weights != nullptr) {
      id = __ldg(a.ids + t * a.k + lane);
      w = __ldg(a.weights + t * a.k + lane);
      dw = __ldg(a.d_weights + t * a.k + lane);
      if (id < 0 || id >= a.E) id = -1;
    }
    const float s = warp_sum(id >= 0 ? w * dw : 0.f);
    if (id >= 0) mine[id] = w * (a.renorm ? dw - s : dw);
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    float p[NV];
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = 32 * j + lane;
      p[j] = e < a.E ? __expf(load_logit(row + e) - lse) : 0.f;
      dot = fmaf(p[j], c[j], dot);
    }
    dot = warp_sum(dot) + (a.renorm ? 0.f : s);  // warp_sum orders the writes of `mine` too
    __syncwarp();
    const float shift = fmaf(cz, lse, -dot);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = 32 * j + lane;
      if (e < a.E) store_logit(out + e, fmaf(p[j], c[j] + shift, mine[e]));
    }
    __syncwarp();
    if (id >= 0) mine[id] = 0.f;
    __syncwarp();
  }
}

template <typename T, int NV>
void launch_fwd(const GateArgs& a, int blocks, cudaStream_t s) {
  const size_t smem = a.part != nullptr ? sizeof(float) * (WARPS + 1) * a.E : 0;
  gate_fwd_kernel<T, NV><<<blocks, THREADS, smem, s>>>(a);
}
template <typename T, int NV>
void launch_bwd(const GateBwdArgs& a, int blocks, cudaStream_t s) {
  gate_bwd_kernel<T, NV><<<blocks, THREADS, sizeof(float) * WARPS * a.E, s>>>(a);
}

#define MOE_GATE_BY_WIDTH(fn, T, args, blocks, s)        \
  do {                                                   \
    if (args.E <= 32) fn<T, 1>(args, blocks, s);         \
    else if (args.E <= 64) fn<T, 2>(args, blocks, s);    \
    else if (args.E <= 128) fn<T, 4>(args, blocks, s);   \
    else if (args.E <= 256) fn<T, 8>(args, blocks, s);   \
    else if (args.E <= 512) fn<T, 16>(args, blocks, s);  \
    else fn<T, 32>(args, blocks, s);                     \
  } while (0)

int blocks_for(int T) { return static_cast<int>(std::max(1LL, std::min<long long>((static_cast<long long>(T) + WARPS - 1) / WARPS, MAX_BLOCKS))); }

bool dtype_ok(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F32; }
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

moe_status_t launched() {
  const cudaError_t err = cudaGetLastError();
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

}  // namespace

size_t gate_workspace_bytes(int T, int E) {
  return static_cast<size_t>(blocks_for(T)) * part_words(E) * sizeof(float);
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_gate_fwd(const void* logits, int dtype, long long ld, const uint8_t* token_mask, int T, int top_k,
                          int E, int flags, int32_t* ids, float* weights, float* lse, int32_t* counts,
                          int32_t* n_valid, float* prob_sum, float* loss, void* ws, size_t ws_bytes,
                          moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (T < 0 || top_k < 1 || E < 1 || ld < 0 || !dtype_ok(dtype) || (flags & ~MOE_GATE_RENORM)) return MOE_ERR_INVALID_ARG;
  if (top_k > MAX_TOPK || E > MAX_E || top_k > E) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (static_cast<long long>(T) * top_k >= (1LL << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && (!logits || !ids || !weights)) return MOE_ERR_INVALID_ARG;
  const bool stats = counts != nullptr;
  if (stats != (n_valid != nullptr) || stats != (prob_sum != nullptr) || stats != (loss != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, dtype == MOE_DTYPE_BF16 ? 2 : 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(lse, 4) ||
      !aligned(counts, 4) || !aligned(n_valid, 4) || !aligned(prob_sum, 4) || !aligned(loss, 4) || !aligned(ws, 4))
    return MOE_ERR_INVALID_ARG;
  if (stats) {
    if (ws_bytes < gate_workspace_bytes(T, E)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!ws) return MOE_ERR_INVALID_ARG;
  }
  moe_status_t st = check_device();
  if (st != MOE_OK || (T == 0 && !stats)) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  GateArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.mask = token_mask;
  a.T = T;
  a.k = top_k;
  a.E = E;
  a.renorm = (flags & MOE_GATE_RENORM) != 0;
  a.ids = ids;
  a.weights = weights;
  a.lse = lse;
  a.part = stats ? static_cast<float*>(ws) : nullptr;
  const int blocks = blocks_for(T);
  if (dtype == MOE_DTYPE_BF16) MOE_GATE_BY_WIDTH(launch_fwd, bf16, a, blocks, s);
  else MOE_GATE_BY_WIDTH(launch_fwd, float, a, blocks, s);
  if ((st = launched()) != MOE_OK || !stats) return st;
  gate_stats_kernel<<<1, 1024, 0, s>>>(a.part, blocks, top_k, E, counts, n_valid, prob_sum, loss);
  return launched();
}

moe_status_t moe_gate_bwd(const void* logits, int dtype, long long ld, const float* lse, const int32_t* ids,
                          const float* weights, const int32_t* counts, const int32_t* n_valid, const float* d_weights,
                          const float* d_loss, int T, int top_k, int E, int flags, void* dlogits, long long ldd,
                          moe_stream_t stream) {
  MOE_TRACE_CALL();
  if (T < 0 || top_k < 1 || E < 1 || ld < 0 || ldd < E || !dtype_ok(dtype) || (flags & ~MOE_GATE_RENORM))
    return MOE_ERR_INVALID_ARG;
  if (top_k > MAX_TOPK || E > MAX_E || top_k > E) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (static_cast<long long>(T) * top_k >= (1LL << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && (!logits || !lse || !dlogits)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && d_weights && (!ids || !weights)) return MOE_ERR_INVALID_ARG;
  if (d_loss && (!counts || !n_valid)) return MOE_ERR_INVALID_ARG;
  const int es = dtype == MOE_DTYPE_BF16 ? 2 : 4;
  if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(lse, 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(counts, 4) || !aligned(n_valid, 4) || !aligned(d_weights, 4) || !aligned(d_loss, 4))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = check_device();
  if (st != MOE_OK || T == 0) return st;
  GateBwdArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.lse = lse;
  a.ids = ids;
  a.weights = weights;
  a.counts = counts;
  a.n_valid = n_valid;
  a.d_weights = d_weights;
  a.d_loss = d_loss;
  a.T = T;
  a.k = top_k;
  a.E = E;
  a.renorm = (flags & MOE_GATE_RENORM) != 0;
  a.dlogits = dlogits;
  a.ldd = ldd;
  const int blocks = blocks_for(T);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MOE_DTYPE_BF16) MOE_GATE_BY_WIDTH(launch_bwd, bf16, a, blocks, s);
  else MOE_GATE_BY_WIDTH(launch_bwd, float, a, blocks, s);
  return launched();
}

}  // extern "C"
