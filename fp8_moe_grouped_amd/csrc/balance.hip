// Balance losses of a router and their gradient.  A token counts unless all its
// logits are -inf; n is the number of those, p = softmax(x[t, :]), lse[t] the
// logarithm of the sum of its exponentials, counts[e] the slots of expert e, S their sum.
//
//   probs[e]  = sum_t p[t, e] / n
//   losses[0] = E sum_e (counts[e] / S) probs[e],   losses[1] = sum_t lse[t]^2 / n
//   dx[t, e]  = p[t, e] (a (c[e] - sum_f p[t, f] c[f]) + b lse[t]) + add[t, e],
//               a = dlosses[0] E / (n S), b = dlosses[1] 2 / n
//
// The gradient takes c[e] = counts[e] - S / E: since sum_f p[t, f] = 1 the value is the
// same, and a nearly even load does not cancel in it.
//
// The forward reads the logits once.  A lane keeps its experts' sums over the tokens that
// its lanes take in registers; they are joined over the wave, the block (LDS) and the grid
// (partial sums in the workspace), each in a fixed order.
#include "logits.hpp"
#include "moe_launch.hpp"

#include <algorithm>

namespace fp8gmm {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxBlocks = 256;                     // of the forward, a partial sum each
constexpr int kOneBlock = 64;                       // tokens that one block takes by itself

__host__ __device__ constexpr int padded(int E) { return (E + 63) & ~63; }

// A token's exponentials in x (0 outside), their sum, and what was taken off the logits.  The sum is 0
// only where all logits are -inf: a finite maximum adds 1, NaN and +inf make it NaN.
template <int L, int V, typename TX>
__device__ __forceinline__ void exponentials(float (&x)[V], int E, int at, float& top, float& total) {
  constexpr int C = 16 / (int)sizeof(TX);
  top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (expert_of<L, C>(at, i) >= E) x[i] = -__builtin_inff();
    top = __builtin_fmaxf(top, x[i]);
  }
  top = lanes_max<L>(top);
  top = top == -__builtin_inff() ? 0.f : top;
  total = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = expf(x[i] - top);
    total += x[i];
  }
  total = lanes_sum<L>(total);
}

// What the losses come from: one thread an expert (E <= kThreads) with its sums over all tokens.
__device__ __forceinline__ void write_losses(int tid, int E, float prob, int count, float z, int n,
                                             float* __restrict__ losses, int* __restrict__ counts,
                                             float* __restrict__ probs, int* __restrict__ tokens, bool counted) {
  __shared__ double joint[2][kWaves];
  const float mean = n > 0 ? prob / (float)n : 0.f;
  if (tid < E) {
    probs[tid] = mean;
    if (counted) counts[tid] = count;
  }
  const double c = tid < E ? (double)max(count, 0) : 0.0;
  const auto plus = [](double a, double b) { return a + b; };
  const double dot = reduce<64>(tid < E ? c * (double)mean : 0.0, plus), slots = reduce<64>(c, plus);
  if ((tid & 63) == 0) {
    joint[0][tid >> 6] = dot;
    joint[1][tid >> 6] = slots;
  }
  __syncthreads();
  if (tid == 0) {
    double d = 0.0, s = 0.0;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
      d += joint[0][w];
      s += joint[1][w];
    }
    losses[0] = s > 0.0 && n > 0 ? (float)((double)E * d / s) : 0.f;
    losses[1] = n > 0 ? z / (float)n : 0.f;
    tokens[0] = n;
  }
}

// ONE: the grid is one block, which writes the results itself.  Otherwise partial sums: probs f32 [blocks][Ep],
// counts i32 [blocks][Ep], then z f32 [blocks] and n i32 [blocks].
template <int L, int V, typename TX, bool ONE>
__global__ __launch_bounds__(kThreads) void balance_kernel(const TX* __restrict__ logits, const int* __restrict__ ids,
                                                           int T, int E, int slots, float* __restrict__ losses,
                                                           int* __restrict__ counts, float* __restrict__ probs,
                                                           int* __restrict__ tokens, float* __restrict__ part) {
  constexpr int C = 16 / (int)sizeof(TX);
  __shared__ __attribute__((aligned(16))) float sums[kWaves][L * V];
  __shared__ int hist[1024];
  __shared__ float zs[kWaves];
  __shared__ int ns[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, at = lane % L, sub = lane / L;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), blocks = gridDim.x, b = blockIdx.x;
  const bool wide = E % C == 0;
  hist[tid] = 0;
  __syncthreads();
  if (ids) {
    const int each = (slots + blocks - 1) / blocks, end = min((b + 1) * each, slots);
    for (int s = b * each + tid; s < end; s += kThreads) {
      const int id = ids[s];
      if (id >= 0 && id < E) atomicAdd(hist + id, 1);   // integers: the order does not matter
    }
  }
  float acc[V] = {}, z = 0.f;
  int n = 0;
  for (int t0 = (b * kWaves + wave) * (64 / L); t0 < T; t0 += blocks * kWaves * (64 / L)) {
    const int t = t0 + sub;
    const bool here = t < T;
    float x[V], top, total;
    load_logits<L, V>(logits + (size_t)t * E, E, at, here, wide, x);
    exponentials<L, V, TX>(x, E, at, top, total);
    const bool some = here && total != 0.f;
    const float share = some ? 1.f / total : 0.f, lse = some ? top + logf(total) : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += x[i] * share;
    z += lse * lse;
    n += some;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (L == 16) {                                  // the wave's four rows of lanes
      acc[i] += other_rows<16>(acc[i], (lane & 16) != 0);
      acc[i] += other_rows<32>(acc[i], (lane & 32) != 0);
    }
    if (sub == 0) sums[wave][expert_of<L, C>(at, i)] = acc[i];
  }
  z = lanes_sum<64>(at == 0 ? z : 0.f);
  n = reduce<64>((uint32_t)(at == 0 ? n : 0), [](uint32_t u, uint32_t v) { return u + v; });
  if (lane == 0) {
    zs[wave] = z;
    ns[wave] = n;
  }
  __syncthreads();
  float prob = 0.f;
  z = 0.f;
  n = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (tid < E) prob += sums[w][tid];
    z += zs[w];
    n += ns[w];
  }
  if (ONE) {
    write_losses(tid, E, prob, ids ? hist[tid] : tid < E ? counts[tid] : 0, z, n, losses, counts, probs, tokens,
                 ids != nullptr);
    return;
  }
  const int Ep = padded(E);
  int* const part_c = reinterpret_cast<int*>(part + (size_t)blocks * Ep);
  float* const part_z = reinterpret_cast<float*>(part_c + (size_t)blocks * Ep);
  if (tid < Ep) {
    part[(size_t)b * Ep + tid] = prob;
    part_c[(size_t)b * Ep + tid] = hist[tid];
  }
  if (tid == 0) {
    part_z[b] = z;
    reinterpret_cast<int*>(part_z + blocks)[b] = n;
  }
}

// Joins the blocks' partial sums: one block, groups of Ep threads take every group-th partial.
__global__ __launch_bounds__(kThreads) void balance_join_kernel(const float* __restrict__ part, int blocks, int E,
                                                                float* __restrict__ losses, int* __restrict__ counts,
                                                                float* __restrict__ probs, int* __restrict__ tokens,
                                                                bool counted) {
  __shared__ float sums[kThreads];
  __shared__ int hist[kThreads];
  __shared__ float zs[kWaves];
  __shared__ int ns[kWaves];
  const int tid = threadIdx.x, Ep = padded(E), groups = kThreads / Ep, group = tid / Ep, e = tid % Ep;
  const int* const part_c = reinterpret_cast<const int*>(part + (size_t)blocks * Ep);
  const float* const part_z = reinterpret_cast<const float*>(part_c + (size_t)blocks * Ep);
  float prob = 0.f;
  int count = 0;
  if (group < groups)
    for (int b = group; b < blocks; b += groups) {
      prob += part[(size_t)b * Ep + e];
      count += part_c[(size_t)b * Ep + e];
    }
  sums[tid] = prob;
  hist[tid] = count;
  float z = tid < blocks ? part_z[tid] : 0.f;       // blocks <= kMaxBlocks <= kThreads
  int n = tid < blocks ? reinterpret_cast<const int*>(part_z + blocks)[tid] : 0;
  z = lanes_sum<64>(z);
  n = reduce<64>((uint32_t)n, [](uint32_t u, uint32_t v) { return u + v; });
  if ((tid & 63) == 0) {
    zs[tid >> 6] = z;
    ns[tid >> 6] = n;
  }
  __syncthreads();
  prob = 0.f;
  count = 0;
  if (tid < E)
    for (int g = 0; g < groups; ++g) {
      prob += sums[g * Ep + tid];
      count += hist[g * Ep + tid];
    }
  z = 0.f;
  n = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    z += zs[w];
    n += ns[w];
  }
  write_losses(tid, E, prob, counted ? count : tid < E ? counts[tid] : 0, z, n, losses, counts, probs, tokens, counted);
}

template <int L, int V, typename TX>
__global__ __launch_bounds__(256) void balance_bwd_kernel(const float* __restrict__ dlosses,
                                                          const TX* __restrict__ logits,
                                                          const int* __restrict__ counts,
                                                          const int* __restrict__ tokens, int T, int E, const TX* add,
                                                          TX* dlogits) {
  constexpr int C = 16 / (int)sizeof(TX);
  const int lane = threadIdx.x & 63, at = lane % L, sub = lane / L;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (blockIdx.x * 4 + wave) * (64 / L) + sub;
  const bool here = t < T, wide = E % C == 0;
  float x[V], old[V], c[V], top, total;
  load_logits<L, V>(logits + (size_t)t * E, E, at, here, wide, x);
  if (add) load_logits<L, V>(add + (size_t)t * E, E, at, here, wide, old);
  double slots = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = expert_of<L, C>(at, i);
    c[i] = e < E ? (float)max(counts[e], 0) : 0.f;
    slots += (double)c[i];
  }
  slots = reduce<L>(slots, [](double a, double b) { return a + b; });
  const float mean = (float)(slots / E);
  const int n = tokens[0];
  const float a = n > 0 && slots > 0.0 ? (float)((double)dlosses[0] * E / ((double)n * slots)) : 0.f;
  const float b = n > 0 ? dlosses[1] * 2.f / (float)n : 0.f;
  exponentials<L, V, TX>(x, E, at, top, total);
  const bool some = total != 0.f;
  const float share = 1.f / total, lse = top + logf(total);
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] -= mean;
    x[i] *= share;
    dot += x[i] * c[i];
  }
  dot = lanes_sum<L>(dot);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = some ? x[i] * (a * (c[i] - dot) + b * lse) : 0.f;
    if (add) x[i] += old[i];
  }
  if (here) store_logits<L, V>(dlogits + (size_t)t * E, E, at, wide, x);
}

int balance_blocks(int T) { return T <= kOneBlock ? 1 : std::min((T + 63) / 64, kMaxBlocks); }

template <int L, int V, typename TX>
hipError_t balance_impl(const TX* logits, const int* ids, int T, int E, int k, float* losses, int* counts, float* probs,
                        int* tokens, float* part, hipStream_t stream) {
  const int blocks = balance_blocks(T), slots = T * k;
  if (blocks == 1) {
    hipLaunchKernelGGL((balance_kernel<L, V, TX, true>), dim3(1), dim3(kThreads), 0, stream, logits, ids, T, E, slots,
                       losses, counts, probs, tokens, part);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((balance_kernel<L, V, TX, false>), dim3(blocks), dim3(kThreads), 0, stream, logits, ids, T, E,
                     slots, losses, counts, probs, tokens, part);
  const hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  hipLaunchKernelGGL(balance_join_kernel, dim3(1), dim3(kThreads), 0, stream, part, blocks, E, losses, counts, probs,
                     tokens, ids != nullptr);
  return hipGetLastError();
}

// The lanes of a token, from its experts; a lane holds whole 16-byte chunks (4 logits in f32, 8 in bf16).
#define BY_EXPERTS(RUN)                                   \
  constexpr int C = 16 / (int)sizeof(TX);                 \
  if (E <= 16 * C) return RUN(16, C);                     \
  if (E <= 128) return RUN(16, 8); /* f32 alone */        \
  if (E <= 256) return RUN(16, 16);                       \
  if (E <= 64 * C) return RUN(64, C);                     \
  if (E <= 512) return RUN(64, 8); /* f32 alone */        \
  return RUN(64, 16);

template <typename TX>
hipError_t balance_pick(const TX* logits, const int* ids, int T, int E, int k, float* losses, int* counts, float* probs,
                        int* tokens, float* part, hipStream_t stream) {
#define RUN(L, V) (balance_impl<L, V, TX>(logits, ids, T, E, k, losses, counts, probs, tokens, part, stream))
  BY_EXPERTS(RUN)
#undef RUN
}

template <int L, int V, typename TX>
hipError_t balance_bwd_impl(const float* dlosses, const TX* logits, const int* counts, const int* tokens, int T, int E,
                            const TX* add, TX* dlogits, hipStream_t stream) {
  hipLaunchKernelGGL((balance_bwd_kernel<L, V, TX>), dim3((T + 256 / L - 1) / (256 / L)), dim3(256), 0, stream,
                     dlosses, logits, counts, tokens, T, E, add, dlogits);
  return hipGetLastError();
}

template <typename TX>
hipError_t balance_bwd_pick(const float* dlosses, const TX* logits, const int* counts, const int* tokens, int T, int E,
                            const TX* add, TX* dlogits, hipStream_t stream) {
#define RUN(L, V) (balance_bwd_impl<L, V, TX>(dlosses, logits, counts, tokens, T, E, add, dlogits, stream))
  BY_EXPERTS(RUN)
#undef RUN
}

}  // namespace

size_t balance_workspace_bytes(int T, int E) {
  const size_t blocks = balance_blocks(T);
  return blocks == 1 ? 0 : 8 * blocks * (padded(E) + 1);
}

hipError_t launch_balance(const void* logits, bool bf16, const int* ids, int T, int E, int k, float* losses,
                          int* counts, float* probs, int* tokens, void* ws, hipStream_t stream) {
  float* const part = static_cast<float*>(ws);
  if (bf16)
    return balance_pick(static_cast<const uint16_t*>(logits), ids, T, E, k, losses, counts, probs, tokens, part, stream);
  return balance_pick(static_cast<const float*>(logits), ids, T, E, k, losses, counts, probs, tokens, part, stream);
}

hipError_t launch_balance_bwd(const float* dlosses, const void* logits, bool bf16, const int* counts,
                              const int* tokens, int T, int E, const void* add, void* dlogits, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  if (bf16)
    return balance_bwd_pick(dlosses, static_cast<const uint16_t*>(logits), counts, tokens, T, E,
                            static_cast<const uint16_t*>(add), static_cast<uint16_t*>(dlogits), stream);
  return balance_bwd_pick(dlosses, static_cast<const float*>(logits), counts, tokens, T, E,
                          static_cast<const float*>(add), static_cast<float*>(dlogits), stream);
}

}  // namespace fp8gmm
