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
// G lanes a token (8, 16 or 32: several tokens a warp when there are few experts), eight consecutive
// experts a lane, its logits in registers: each logit is read once by the forward and once by
// the backward, 16 bytes at a time where the rows allow it. Each lane sorts its eight (logit,
// expert) keys with a 19-comparator network; a round of the top_k is then one maximum over the
// lanes' heads and a step in the winner's list. Neither kernel is bound by memory: of many tokens the
// forward keeps 58% of the issue slots busy and 14% of the memory, and waits for the loads of a token
// between one token's work and the next's, on the 16 warps that its registers leave an SM. So the
// instructions of a token are what the layout minimises (rescanning a lane's values in each round
// instead of sorting once took four times as long). The sorted lists lie in shared
// memory, where taking a list's next head is one load instead of a shift of eight registers.
// Measured: 131072 tokens x 256 experts, top 8 of bf16 logits, 51 us without statistics (67 MB of
// logits, 1.3 TB/s) and 59 with them; its gradient 31.5 us (4.3 TB/s of logits read and gradient
// written); 16 tokens x 128 experts 2.5 us, where the launch and the chain of rounds are the time.
// The per-expert sums over the tokens of a lane group stay in registers (lane and element own
// an expert), a block adds its groups' sums in order and leaves one partial row in the workspace,
// and a second kernel adds those in block order: no floating-point atomics, so results do not
// depend on scheduling.
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
// Blocks of the backward at most, five for each SM: what fits of one list on 32 lanes (131072 x 256 bf16:
// 31.5 us; twice as many 32.2, four times 35.3; more blocks on an SM with fewer registers 33 to 46). Of the
// other layouts fewer fit (two to four, by their registers) and the rest run after them.
constexpr int BWD_BLOCKS = 760;
constexpr unsigned FULL = 0xffffffffu;

// Eight consecutive logits from expert e0 of a row; -inf past the last expert. VEC: the row is
// 16-byte aligned and E a multiple of 8.
template <bool VEC>
__device__ __forceinline__ void load8(const float* row, int e0, int E, float (&v)[8]) {
  if constexpr (VEC) {
    if (e0 < E) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + e0)), b = __ldg(reinterpret_cast<const float4*>(row + e0) + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = -INFINITY;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e0 + j < E ? __ldg(row + e0 + j) : -INFINITY;
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const bf16* row, int e0, int E, float (&v)[8]) {
  if constexpr (VEC) {
    if (e0 < E) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(row + e0));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_lo(w[j]);
        v[2 * j + 1] = bf16_hi(w[j]);
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = -INFINITY;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e0 + j < E ? __bfloat162float(row[e0 + j]) : -INFINITY;
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(float* row, int e0, int E, const float (&v)[8]) {
  if constexpr (VEC) {
    if (e0 >= E) return;
    reinterpret_cast<float4*>(row + e0)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(row + e0)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e0 + j < E) row[e0 + j] = v[j];
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(bf16* row, int e0, int E, const float (&v)[8]) {
  if constexpr (VEC) {
    if (e0 < E)
      *reinterpret_cast<uint4*>(row + e0) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e0 + j < E) row[e0 + j] = __float2bfloat16_rn(v[j]);
  }
}

// e^x without the subnormal range's scaling instructions (results below 2^-126 are 0)
__device__ __forceinline__ float exp_f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}

// Unsigned number with the order of the floats; NaN orders as -inf, -0 as 0.
__device__ __forceinline__ uint32_t order_bits(float f) {
  const int b = __float_as_int(fmaxf(f, -INFINITY) + 0.f);
  return static_cast<uint32_t>(b ^ ((b >> 31) | static_cast<int>(0x80000000u)));
}
__device__ __forceinline__ float order_value(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k); }

// Keys that order by logit, then by lower expert, and are unique and not 0. A bf16 logit has 16
// bits, so that one 32-bit word holds it with the expert; an fp32 logit takes 64.
template <typename T>
struct Key;
template <>
struct Key<bf16> {
  typedef uint32_t type;
  static __device__ __forceinline__ type make(float f, int e) {
    // of a bf16 value the low 16 order bits are all zeros or all ones
    return (order_bits(f) & 0xffff0000u) | static_cast<uint32_t>(0xffff - e);
  }
  static __device__ __forceinline__ int expert(type k) { return 0xffff - static_cast<int>(k & 0xffffu); }
  static __device__ __forceinline__ float value(type k) {
    return order_value((k & 0x80000000u) ? (k & 0xffff0000u) : (k | 0xffffu));
  }
  template <int G>
  static __device__ __forceinline__ type group_max(type k) {
    if constexpr (G == 32) {
      return __reduce_max_sync(FULL, k);
    } else {
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) k = max(k, __shfl_xor_sync(FULL, k, o));
      return k;
    }
  }
};
template <>
struct Key<float> {
  typedef unsigned long long type;
  static __device__ __forceinline__ type make(float f, int e) {
    return (static_cast<type>(order_bits(f)) << 32) | static_cast<uint32_t>(0xffff - e);
  }
  static __device__ __forceinline__ int expert(type k) { return 0xffff - static_cast<int>(k & 0xffffu); }
  static __device__ __forceinline__ float value(type k) { return order_value(static_cast<uint32_t>(k >> 32)); }
  template <int G>
  static __device__ __forceinline__ type group_max(type k) {
    if constexpr (G == 32) {
      const uint32_t hi = static_cast<uint32_t>(k >> 32);
      const uint32_t top = __reduce_max_sync(FULL, hi);
      const uint32_t lo = __reduce_max_sync(FULL, hi == top ? static_cast<uint32_t>(k) : 0u);
      return (static_cast<type>(top) << 32) | lo;
    } else {
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) k = max(k, __shfl_xor_sync(FULL, k, o));
      return k;
    }
  }
};

// Descending order of eight keys: Batcher's odd-even merge sort.
template <typename K>
__device__ __forceinline__ void sort8(K (&k)[8]) {
  constexpr int net[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                              {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
  for (int i = 0; i < 19; ++i) {
    const K a = k[net[i][0]], b = k[net[i][1]];
    k[net[i][0]] = max(a, b);
    k[net[i][1]] = min(a, b);
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
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
  unsigned* ticket;     // with part: the statistics kernel's block counter, cleared here
};

constexpr int part_words(int E) { return 2 * E + 2; }
__host__ __device__ constexpr int count_bytes(int E) { return (4 * E + 15) & ~15; }
constexpr int LIST = 9;  // a lane's eight sorted keys and a 0; odd, so that lanes use different banks

// NL lists of eight experts a lane: expert 8 (G l + lane_in_group) + j.
template <typename T, int NL, int G, bool VEC>
__global__ void __launch_bounds__(THREADS) gate_fwd_kernel(GateArgs a) {
  grid_wait();
  a.logits = after_wait(a.logits);
  a.mask = after_wait(a.mask);
  typedef Key<T> KT;
  typedef typename KT::type K;
  constexpr int GROUPS = 32 / G;           // tokens a warp
  constexpr int NS = 32 / G;               // slots a lane keeps (top_k <= 32)
  // [E] counts, then the lists, over which the block's sums are staged at the end
  extern __shared__ __align__(16) uint8_t fsh[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gl = lane % G, grp = warp * GROUPS + lane / G;
  const bool stats = a.part != nullptr;
  int* s_cnt = reinterpret_cast<int*>(fsh);
  uint8_t* body = fsh + count_bytes(a.E);
  K* list = reinterpret_cast<K*>(body) + threadIdx.x * (NL * LIST);
  if (stats) {
    for (int e = threadIdx.x; e < a.E; e += THREADS) s_cnt[e] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
    __syncthreads();
  }
#pragma unroll
  for (int l = 0; l < NL; ++l) list[l * LIST + 8] = 0;
  float psum[NL][8];
#pragma unroll
  for (int l = 0; l < NL; ++l)
#pragma unroll
    for (int j = 0; j < 8; ++j) psum[l][j] = 0.f;
  float z = 0.f;
  int tokens = 0;
  // warp-uniform loop: the shuffles need every lane
  for (long long t0 = (static_cast<long long>(blockIdx.x) * WARPS + warp) * GROUPS; t0 < a.T;
       t0 += static_cast<long long>(gridDim.x) * WARPS * GROUPS) {
    const long long t = t0 + lane / G;
    const bool in = t < a.T;
    // the row is loaded whether the token takes part or not: the two loads then wait together
    const T* row = static_cast<const T*>(a.logits) + (in ? t : 0) * a.ld;
    float v[NL][8];
#pragma unroll
    for (int l = 0; l < NL; ++l) load8<VEC>(row, in ? 8 * (G * l + gl) : a.E, a.E, v[l]);
    const bool live = in && (a.mask == nullptr || __ldg(a.mask + t) != 0);
    float m = -INFINITY;
#pragma unroll
    for (int l = 0; l < NL; ++l)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, v[l][j]);  // ignores NaN
    m = group_max<G>(m);
    const float base = m > -INFINITY ? m : 0.f;
    K head[NL];
    float sum = 0.f;
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      K key[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        key[j] = KT::make(v[l][j], 8 * (G * l + gl) + j);
        v[l][j] = exp_f(v[l][j] - base);
        sum += v[l][j];
      }
      sort8(key);
      head[l] = key[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) list[l * LIST + j] = key[j];
    }
    sum = group_sum<G>(sum);
    // a token without any logit above -inf takes no part, like a masked one; one with a NaN
    // does, and its probabilities are NaN
    const bool part = live && !(sum == 0.f);
    const float lse = part ? base + logf(sum) : -INFINITY;
    if (a.lse != nullptr && gl == 0 && in) a.lse[t] = lse;
    if (stats && part) {
      const float inv = 1.0f / sum;
#pragma unroll
      for (int l = 0; l < NL; ++l)
#pragma unroll
        for (int j = 0; j < 8; ++j) psum[l][j] = fmaf(v[l][j], inv, psum[l][j]);
      z = fmaf(lse, lse, z);
      ++tokens;
    }
    int my_id[NS];
    float my_e[NS];
    int next[NL];
#pragma unroll
    for (int l = 0; l < NL; ++l) next[l] = l * LIST + 1;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      K mine = 0;
      // a round takes the group's largest key. Keys are unique and the group has at least twice as
      // many as there are rounds, so an empty list's 0 never wins
      for (int r = 0; r < G && s * G + r < a.k; ++r) {
        K best = head[0];
#pragma unroll
        for (int l = 1; l < NL; ++l) best = max(best, head[l]);
        const K top = KT::template group_max<G>(best);
        if (gl == r) mine = top;
#pragma unroll
        for (int l = 0; l < NL; ++l)
          if (head[l] == top) head[l] = list[next[l]++];
      }
      const float logit = KT::value(mine);
      const bool chosen = part && mine != 0 && logit > -INFINITY;
      my_id[s] = chosen ? KT::expert(mine) : -1;
      my_e[s] = chosen ? exp_f(logit - base) : 0.f;
    }
    float norm = sum;
    if (a.renorm) {
      norm = 0.f;
#pragma unroll
      for (int s = 0; s < NS; ++s) norm += my_e[s];
      norm = group_sum<G>(norm);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int slot = s * G + gl;
      if (!in || slot >= a.k) continue;
      // a NaN anywhere in the row makes every weight of the row NaN, renormalised or not
      const float w = sum != sum ? sum : my_e[s] / norm;
      a.ids[t * a.k + slot] = my_id[s];
      a.weights[t * a.k + slot] = my_id[s] >= 0 ? w : 0.f;
      if (stats && my_id[s] >= 0) atomicAdd(s_cnt + my_id[s], 1);
    }
  }
  if (!stats) return;
  __shared__ float s_z[WARPS * GROUPS];
  __shared__ int s_n[WARPS * GROUPS];
  float* sh = reinterpret_cast<float*>(body);  // [WARPS * GROUPS][E] probability sums
  float* mine = sh + grp * a.E;
  __syncthreads();  // every list has been read
#pragma unroll
  for (int l = 0; l < NL; ++l)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (8 * (G * l + gl) + j < a.E) mine[8 * (G * l + gl) + j] = psum[l][j];
  if (gl == 0) {
    s_z[grp] = z;
    s_n[grp] = tokens;
  }
  __syncthreads();
  float* out = a.part + static_cast<size_t>(blockIdx.x) * part_words(a.E);
  int* iout = reinterpret_cast<int*>(out);
  for (int e = threadIdx.x; e < a.E; e += THREADS) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS * GROUPS; ++w) s += sh[w * a.E + e];
    out[e] = s;
    iout[a.E + e] = s_cnt[e];
  }
  if (threadIdx.x == 0) {
    float sz = 0.f;
    int n = 0;
    for (int w = 0; w < WARPS * GROUPS; ++w) {
      sz += s_z[w];
      n += s_n[w];
    }
    out[2 * a.E] = sz;
    iout[2 * a.E + 1] = n;
  }
}

__device__ __forceinline__ float warp_sum(float v) { return group_sum<32>(v); }

// Adds the blocks' partial rows in a fixed order: eight experts a block, 128 threads an expert over
// the rows (a 32-byte sector a row). The last block to finish adds the blocks' shares of the
// balance loss in block order and writes the losses.
constexpr int STAT_COLS = 8;
__global__ void __launch_bounds__(1024) gate_stats_kernel(const float* part, int blocks, int k, int E,
                                                          int32_t* __restrict__ counts, int32_t* __restrict__ n_valid,
                                                          float* __restrict__ prob_sum, float* __restrict__ loss,
                                                          unsigned* ticket, float* share) {
  __shared__ float s_p[32][STAT_COLS];
  __shared__ int s_c[32][STAT_COLS];
  __shared__ float s_z[32];
  __shared__ int s_n[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cx = threadIdx.x % STAT_COLS, ry = threadIdx.x / STAT_COLS;
  const int words = part_words(E);
  const int e = blockIdx.x * STAT_COLS + cx;
  grid_wait();  // launched ahead of the end of the forward kernel
  part = after_wait(part);
  const int* ipart = reinterpret_cast<const int*>(part);
  // every load at once (a loop of a run-time length waits for each round of them)
  constexpr int ROUNDS = (MAX_BLOCKS + 1024 / STAT_COLS - 1) / (1024 / STAT_COLS);
  static_assert(MAX_BLOCKS <= 1024, "one thread a block");
  float pv[ROUNDS], z = 0.f;
  int cv[ROUNDS], n = 0;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int b = ry + i * (1024 / STAT_COLS);
    const bool on = e < E && b < blocks;
    pv[i] = on ? part[static_cast<size_t>(b) * words + e] : 0.f;
    cv[i] = on ? ipart[static_cast<size_t>(b) * words + E + e] : 0;
  }
  if (threadIdx.x < blocks) {
    z = part[static_cast<size_t>(threadIdx.x) * words + 2 * E];
    n = ipart[static_cast<size_t>(threadIdx.x) * words + 2 * E + 1];
  }
  float p = 0.f;
  int c = 0;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    p += pv[i];
    c += cv[i];
  }
  z = warp_sum(z);
  n = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(n)));
  if (lane == 0) {
    s_z[warp] = z;
    s_n[warp] = n;
  }
#pragma unroll
  for (int o = STAT_COLS; o < 32; o <<= 1) {
    p += __shfl_xor_sync(FULL, p, o);
    c += __shfl_xor_sync(FULL, c, o);
  }
  if (lane < STAT_COLS) {
    s_p[warp][lane] = p;
    s_c[warp][lane] = c;
  }
  __syncthreads();
  if (warp != 0) return;
  p = 0.f;
  c = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r) {  // lane group g adds warps 8g..8g+7
    p += s_p[(lane / STAT_COLS) * 8 + r][cx];
    c += s_c[(lane / STAT_COLS) * 8 + r][cx];
  }
#pragma unroll
  for (int o = STAT_COLS; o < 32; o <<= 1) {
    p += __shfl_xor_sync(FULL, p, o);
    c += __shfl_xor_sync(FULL, c, o);
  }
  const bool mine = lane < STAT_COLS && e < E;
  if (mine) {
    prob_sum[e] = p;
    counts[e] = c;
  }
  const float bal = warp_sum(mine ? static_cast<float>(c) * p : 0.f);
  unsigned last = 0u;
  if (lane == 0) {
    share[blockIdx.x] = bal;
    __threadfence();
    last = atomicAdd(ticket, 1u) == gridDim.x - 1 ? 1u : 0u;
  }
  if (__shfl_sync(FULL, last, 0) == 0u) return;
  __threadfence();
  z = warp_sum(s_z[lane]);
  n = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(s_n[lane])));
  float total = 0.f;
  for (int b = lane; b < static_cast<int>(gridDim.x); b += 32) total += __ldcg(share + b);
  total = warp_sum(total);
  if (lane == 0) {
    const float nf = static_cast<float>(n);
    *n_valid = n;
    loss[0] = n > 0 ? static_cast<float>(E) / (static_cast<float>(k) * nf) * (total / nf) : 0.f;
    loss[1] = n > 0 ? z / nf : 0.f;
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

template <typename T, int NL, int G, bool VEC>
__global__ void __launch_bounds__(THREADS) gate_bwd_kernel(GateBwdArgs a) {
  grid_wait();
  a.logits = after_wait(a.logits);
  a.lse = after_wait(a.lse);
  a.ids = after_wait(a.ids);
  a.weights = after_wait(a.weights);
  a.counts = after_wait(a.counts);
  a.n_valid = after_wait(a.n_valid);
  a.d_weights = after_wait(a.d_weights);
  a.d_loss = after_wait(a.d_loss);
  constexpr int GROUPS = 32 / G;
  constexpr int NS = 32 / G;
  extern __shared__ __align__(16) float bsh[];  // [WARPS * GROUPS][8 G NL] what a token's selected experts get on top
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gl = lane % G;
  float* mine = bsh + (warp * GROUPS + lane / G) * (8 * G * NL);
  float c[NL][8];
  float cz = 0.f;
#pragma unroll
  for (int l = 0; l < NL; ++l)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[l][j] = 0.f;
      mine[8 * (G * l + gl) + j] = 0.f;
    }
  if (a.d_loss != nullptr) {
    const int n = __ldg(a.n_valid);
    if (n > 0) {
      const float nf = static_cast<float>(n);
      const float cb = __ldg(a.d_loss) * static_cast<float>(a.E) / (static_cast<float>(a.k) * nf) / nf;
      cz = 2.0f * __ldg(a.d_loss + 1) / nf;
#pragma unroll
      for (int l = 0; l < NL; ++l)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = 8 * (G * l + gl) + j;
          if (e < a.E) c[l][j] = cb * static_cast<float>(__ldg(a.counts + e));
        }
    }
  }
  __syncwarp();
  for (long long t0 = (static_cast<long long>(blockIdx.x) * WARPS + warp) * GROUPS; t0 < a.T;
       t0 += static_cast<long long>(gridDim.x) * WARPS * GROUPS) {
    const long long t = t0 + lane / G;
    const bool in = t < a.T;
    // every load of the token before any of them is waited for
    const T* row = static_cast<const T*>(a.logits) + (in ? t : 0) * a.ld;
    float p[NL][8];
#pragma unroll
    for (int l = 0; l < NL; ++l) load8<VEC>(row, in ? 8 * (G * l + gl) : a.E, a.E, p[l]);
    const float lse = in ? __ldg(a.lse + t) : -INFINITY;
    int id[NS];
    float w[NS], dw[NS], s = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int slot = i * G + gl;
      id[i] = -1;
      w[i] = dw[i] = 0.f;
      if (in && slot < a.k && a.d_weights != nullptr) {
        id[i] = __ldg(a.ids + t * a.k + slot);
        w[i] = __ldg(a.weights + t * a.k + slot);
        dw[i] = __ldg(a.d_weights + t * a.k + slot);
      }
    }
    const bool part = lse != -INFINITY;  // else the token took no part: its gradient is 0
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      if (!part || id[i] < 0 || id[i] >= a.E) id[i] = -1;
      else s = fmaf(w[i], dw[i], s);
    }
    float dot = 0.f;
#pragma unroll
    for (int l = 0; l < NL; ++l)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // lse is rounded to fp32, so p is off by its last place as well: 6e-5 of p where |lse| is 1e3
        p[l][j] = part ? exp_f(p[l][j] - lse) : 0.f;
        dot = fmaf(p[l][j], c[l][j], dot);
      }
    // without renormalisation only the sum of the two is wanted
    if (a.renorm) {
      s = group_sum<G>(s);
      dot = group_sum<G>(dot);
    } else {
      dot = group_sum<G>(dot + s);
      s = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (id[i] >= 0) mine[id[i]] = w[i] * (dw[i] - s);
    __syncwarp();
    const float shift = part ? fmaf(cz, lse, -dot) : 0.f;
    T* out = static_cast<T*>(a.dlogits) + (in ? t : 0) * a.ldd;
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      const float4* add = reinterpret_cast<const float4*>(mine + 8 * (G * l + gl));
      const float4 x = add[0], y = add[1];
      const float top[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) p[l][j] = part ? fmaf(p[l][j], c[l][j] + shift, top[j]) : 0.f;
      store8<VEC>(out, in ? 8 * (G * l + gl) : a.E, a.E, p[l]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (id[i] >= 0) mine[id[i]] = 0.f;
    __syncwarp();
  }
}

template <typename T, int NL, int G, bool VEC>
moe_status_t launch_fwd(const GateArgs& a, int blocks, cudaStream_t s) {
  constexpr int lists = THREADS * NL * LIST * static_cast<int>(sizeof(typename Key<T>::type));
  constexpr int widest = 8 * G * NL;
  constexpr int most = count_bytes(widest) + std::max(lists, WARPS * (32 / G) * widest * 4);
  const int smem = count_bytes(a.E) + std::max(lists, WARPS * (32 / G) * a.E * 4);
  if (most > 48 * 1024) {
    const cudaError_t err = ensure_max_dynamic_smem(reinterpret_cast<const void*>(gate_fwd_kernel<T, NL, G, VEC>), most);
    if (err != cudaSuccess) return cuda_fail(err);
  }
  const cudaError_t err =
      launch_dependent(gate_fwd_kernel<T, NL, G, VEC>, blocks, THREADS, smem, s, a);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}
template <typename T, int NL, int G, bool VEC>
moe_status_t launch_bwd(const GateBwdArgs& a, int blocks, cudaStream_t s) {
  const cudaError_t err = launch_dependent(gate_bwd_kernel<T, NL, G, VEC>, blocks,
                                              THREADS, sizeof(float) * WARPS * 32 * 8 * NL, s, a);
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
}

// Lanes a token and lists a lane. The forward gives many tokens eight lanes each (16 above 256
// experts) and so up to four lists a lane: what a token costs besides its experts (sums, rounds,
// addresses) is then shared by more tokens of the warp. 131072 x 256 bf16 without statistics takes
// 51 us with 4 lists on 8 lanes, 56 with 2 on 16 and 62 with 1 on 32. Few tokens (less than one for
// each warp of the grid) take as many lanes as hold eight experts each, which keeps more warps at
// work, and so do rows that are read one element at a time. The backward has no rounds and waits
// for its loads: always full width (34 us then, against 44 on 8 lanes).
struct Width {
  int lists, lanes;
};
Width width_for(int E, bool many) {
  if (E <= 64) return {1, 8};
  if (E <= 128) return many ? Width{2, 8} : Width{1, 16};
  if (E <= 256) return many ? Width{4, 8} : Width{1, 32};
  if (E <= 512) return many ? Width{4, 16} : Width{2, 32};
  return {4, 32};
}

template <typename T, bool VEC>
moe_status_t by_width_fwd(const GateArgs& a, Width w, int blocks, cudaStream_t s) {
  if constexpr (VEC) {
    if (w.lists == 2 && w.lanes == 8) return launch_fwd<T, 2, 8, VEC>(a, blocks, s);
    if (w.lists == 4 && w.lanes == 8) return launch_fwd<T, 4, 8, VEC>(a, blocks, s);
    if (w.lists == 4 && w.lanes == 16) return launch_fwd<T, 4, 16, VEC>(a, blocks, s);
  }
  if (w.lanes == 8) return launch_fwd<T, 1, 8, VEC>(a, blocks, s);
  if (w.lanes == 16) return launch_fwd<T, 1, 16, VEC>(a, blocks, s);
  if (w.lists == 1) return launch_fwd<T, 1, 32, VEC>(a, blocks, s);
  if (w.lists == 2) return launch_fwd<T, 2, 32, VEC>(a, blocks, s);
  return launch_fwd<T, 4, 32, VEC>(a, blocks, s);
}
template <typename T, bool VEC>
moe_status_t by_width_bwd(const GateBwdArgs& a, Width w, int blocks, cudaStream_t s) {
  if (w.lanes == 8) return launch_bwd<T, 1, 8, VEC>(a, blocks, s);
  if (w.lanes == 16) return launch_bwd<T, 1, 16, VEC>(a, blocks, s);
  if (w.lists == 1) return launch_bwd<T, 1, 32, VEC>(a, blocks, s);
  if (w.lists == 2) return launch_bwd<T, 2, 32, VEC>(a, blocks, s);
  return launch_bwd<T, 4, 32, VEC>(a, blocks, s);
}

// blocks for tokens of `lanes` lanes each
int blocks_for(int T, int lanes, int most) {
  const int per = WARPS * (32 / lanes);
  return static_cast<int>(std::max(1LL, std::min<long long>((static_cast<long long>(T) + per - 1) / per, most)));
}

bool dtype_ok(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F32; }
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// rows that start on 16-byte boundaries and hold whole groups of eight experts
bool rows16(const void* p, long long ld, int E, int dtype) {
  return aligned(p, 16) && E % 8 == 0 && ld % (dtype == MOE_DTYPE_BF16 ? 8 : 4) == 0;
}

}  // namespace

// the blocks' partial rows, then the statistics kernel's block counter and shares
size_t gate_workspace_bytes(int T, int E) {
  return (static_cast<size_t>(blocks_for(T, 32, MAX_BLOCKS)) * part_words(E) + 1 + MAX_E / STAT_COLS) * sizeof(float);
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
  const bool vec = rows16(logits, ld, E, dtype);
  const Width w = width_for(E, vec && T >= MAX_BLOCKS * WARPS);
  // four lists a lane leave registers for two blocks on an SM
  const int blocks = blocks_for(T, w.lanes, w.lists == 4 ? MAX_BLOCKS / 2 : MAX_BLOCKS);
  a.ticket = stats ? static_cast<unsigned*>(ws) + static_cast<size_t>(blocks) * part_words(E) : nullptr;
  if (dtype == MOE_DTYPE_BF16) st = vec ? by_width_fwd<bf16, true>(a, w, blocks, s) : by_width_fwd<bf16, false>(a, w, blocks, s);
  else st = vec ? by_width_fwd<float, true>(a, w, blocks, s) : by_width_fwd<float, false>(a, w, blocks, s);
  if (st != MOE_OK || !stats) return st;
  const cudaError_t err = launch_dependent(gate_stats_kernel, (E + STAT_COLS - 1) / STAT_COLS, 1024, 0, s, a.part, blocks,
                                           top_k, E, counts, n_valid, prob_sum, loss, a.ticket,
                                           reinterpret_cast<float*>(a.ticket + 1));
  return err == cudaSuccess ? MOE_OK : cuda_fail(err);
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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool vec = rows16(logits, ld, E, dtype) && rows16(dlogits, ldd, E, dtype);
  const Width w = width_for(E, false);
  const int blocks = blocks_for(T, w.lanes, BWD_BLOCKS);
  if (dtype == MOE_DTYPE_BF16) return vec ? by_width_bwd<bf16, true>(a, w, blocks, s) : by_width_bwd<bf16, false>(a, w, blocks, s);
  return vec ? by_width_bwd<float, true>(a, w, blocks, s) : by_width_bwd<float, false>(a, w, blocks, s);
}

}  // extern "C"
