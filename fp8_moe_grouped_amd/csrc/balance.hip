// Balance losses of a router and their gradient.  A token counts unless all its
// logits are -inf; n is the number of those, p = softmax(x[t, :]), lse[t] the
// logarithm of the sum of its exponentials, counts[e] the slots of expert e, S their sum.
//
//   probs[e]  = sum_t p[t, e] / n
//   losses[0] = E sum_e (counts[e] / S) probs[e],   losses[1] = sum_t lse[t]^2 / n
//   dx[t, e]  = p[t, e] (a (c[e] - sum_f p[t, f] c[f]) + b lse[t]) + add[t, e],
//               a = dlosses[0] E / (n S), b = dlosses[1] 2 / n
//
// The gradient takes c[e] = counts[e] - S / E, in f64: since sum_f p[t, f] = 1 the value is the
// same, and a nearly even load does not cancel in it.
//
// The forward reads the logits once.  A lane keeps its experts' sums over the tokens that
// its lanes take in registers; they are joined over the wave, the block (LDS) and the grid
// (partial sums in the workspace), each in a fixed order.  Its bytes are few (16384 x 256 in
// bf16: 9 MB, 1.7 us at a copy's rate): what bounds it is a launch, the loads' latency and the
// exponentials, 5.6 us of the kernel (4.6 at least) and 4.2 of the join's, 9.4 a call.
#include "logits.hpp"
#include "moe_launch.hpp"

#include <algorithm>

namespace fp8gmm {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxBlocks = 256;                     // of the forward, a partial sum each
constexpr int kBackwardBlocks = 2;                  // of the gradient, a CU
constexpr int kJoin = 32;                           // experts that a block of the join takes

__host__ __device__ constexpr int padded(int E) { return (E + 63) & ~63; }

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

// A token's logits x become 2^(x log2(e) - below) with below = log2(e) max x; `total` is their sum: 0 only where all
// logits are -inf, as a finite maximum adds 1 and NaN or +inf make it NaN.  The product and the difference round once
// together, and what `below` was rounded by is the same in all terms, so a term is as exact as exp(x - max x).
template <int L, int V>
__device__ __forceinline__ void exponentials(float (&x)[V], float& total, float& lse) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < V; ++i) top = __builtin_fmaxf(top, x[i]);
  top = lanes_max<L>(top);
  top = top == -__builtin_inff() ? 0.f : top;
  const float below = top * kLog2e;
  if (__builtin_amdgcn_ballot_w64(__builtin_fabsf(below) > 0x1p16f)) {   // `below` is 2^-8 off or more: from distances
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __builtin_amdgcn_exp2f((x[i] - top) * kLog2e);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], kLog2e, -below));
  }
  total = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) total += x[i];
  total = lanes_sum<L>(total);
  lse = top + kLn2 * __builtin_amdgcn_logf(total);
}

// Sum over the wave's four rows of 16 lanes: a lane keeps V / 4 of its V values, the columns from kept(lane), and adds
// the other rows' of those.  An exchange of rows brings two registers' halves together, so each level halves them.
template <int V>
__device__ __forceinline__ void rows_sum(const float (&v)[V], float (&out)[V / 4]) {
  float half[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i + V / 2]), false, false);
    half[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(half[i]), __float_as_uint(half[i + V / 4]), false, false);
    out[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
}
template <int V>
__device__ __forceinline__ int kept(int lane) { return (lane & 16 ? V / 2 : 0) + (lane & 32 ? V / 4 : 0); }

// What a part of the experts gives the losses, one thread an expert (`inside`) of a whole wave: counts times mean
// probabilities and counts, summed over the wave.
struct Share {
  double dot, slots;
};
__device__ __forceinline__ Share write_expert(bool inside, int e, float prob, int count, int n,
                                              int* __restrict__ counts, float* __restrict__ probs, bool counted) {
  const float mean = n > 0 ? prob / (float)n : 0.f;
  if (inside) {
    probs[e] = mean;
    if (counted) counts[e] = count;
  }
  const double c = inside ? (double)max(count, 0) : 0.0;
  const auto plus = [](double a, double b) { return a + b; };
  return {reduce<64>(inside ? c * (double)mean : 0.0, plus), reduce<64>(c, plus)};
}
__device__ __forceinline__ void write_losses(int E, const Share& s, float z, int n, float* __restrict__ losses,
                                             int* __restrict__ tokens) {
  losses[0] = s.slots > 0.0 && n > 0 ? (float)((double)E * s.dot / s.slots) : 0.f;
  losses[1] = n > 0 ? z / (float)n : 0.f;
  tokens[0] = n;
}

// The workspace of a grid of several blocks: each block's sums, then the join's.
struct Partial {
  float* probs;                                     // [blocks][Ep]
  int* counts;                                      // [blocks][Ep]
  float* z;                                         // [blocks]
  int* n;                                           // [blocks]
  double* shares;                                   // [Ep / kJoin][2]
  unsigned* done;
};
__host__ __device__ inline Partial partial_of(void* ws, int blocks, int E) {
  Partial p;
  const size_t Ep = padded(E);
  p.shares = static_cast<double*>(ws);
  p.probs = reinterpret_cast<float*>(p.shares + 2 * (Ep / kJoin));
  p.counts = reinterpret_cast<int*>(p.probs + blocks * Ep);
  p.z = reinterpret_cast<float*>(p.counts + blocks * Ep);
  p.n = reinterpret_cast<int*>(p.z + blocks);
  p.done = reinterpret_cast<unsigned*>(p.n + blocks);
  return p;
}

// ONE: the grid is one block, which writes the results itself.
template <int L, int V, typename TX, bool WIDE, bool ONE>
__global__ __launch_bounds__(kThreads) void balance_kernel(const TX* __restrict__ logits, const int* __restrict__ ids,
                                                           int T, int E, int slots, float* __restrict__ losses,
                                                           int* __restrict__ counts, float* __restrict__ probs,
                                                           int* __restrict__ tokens, void* __restrict__ ws) {
  constexpr int C = 16 / (int)sizeof(TX);
  __shared__ __attribute__((aligned(16))) float sums[kWaves][L * V];
  __shared__ int hist[1024];
  __shared__ float zs[kWaves];
  __shared__ int ns[kWaves];
  __shared__ Share shares[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, at = lane % L, sub = lane / L;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), blocks = gridDim.x, b = blockIdx.x;
  // the first tokens' logits and slots are on their way while the histogram is cleared
  const int step = blocks * kWaves * (64 / L);
  int t = (b * kWaves + wave) * (64 / L) + sub;
  const int each = (slots + blocks - 1) / blocks, end = min((b + 1) * each, slots);
  int s = b * each + tid;
  int id = ids && s < end ? ids[s] : -1;
  Chunks<V, TX> next;
  load_chunks<L, V, true>(logits + (size_t)t * E, E, at, t < T, WIDE, next);
  hist[tid] = 0;
  __syncthreads();
  while (s < end && ids) {
    const int now = id;
    s += kThreads;
    id = s < end ? ids[s] : -1;
    if (now >= 0 && now < E) atomicAdd(hist + now, 1);   // integers: the order does not matter
  }
  float acc[V] = {}, z = 0.f;
  int n = 0;
  while (t - sub < T) {
    float x[V], total, lse;
    unpack<V>(next, x);
    t += step;
    load_chunks<L, V, true>(logits + (size_t)t * E, E, at, t < T, WIDE, next);
    exponentials<L, V>(x, total, lse);
    const bool some = total != 0.f;                 // 0 past the last token too
    const float share = some ? 1.f / total : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += x[i] * share;
    z += some ? lse * lse : 0.f;
    n += some;
  }
  if constexpr (L == 16) {
    float mine[V / 4];
    rows_sum<V>(acc, mine);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) sums[wave][expert_of<L, C>(at, kept<V>(lane) + i)] = mine[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) sums[wave][expert_of<L, C>(at, i)] = acc[i];
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
    const bool inside = tid < E;
    const Share one = write_expert(inside, tid, prob, ids || !inside ? hist[tid] : counts[tid], n, counts, probs,
                                   ids != nullptr);
    if (lane == 0) shares[wave] = one;
    __syncthreads();
    if (tid == 0) {
      Share all = shares[0];
      for (int w = 1; w < kWaves; ++w) {
        all.dot += shares[w].dot;
        all.slots += shares[w].slots;
      }
      write_losses(E, all, z, n, losses, tokens);
    }
    return;
  }
  const int Ep = padded(E);
  const Partial part = partial_of(ws, blocks, E);
  if (tid < Ep) {
    part.probs[(size_t)b * Ep + tid] = prob;
    part.counts[(size_t)b * Ep + tid] = hist[tid];
  }
  if (tid == 0) {
    part.z[b] = z;
    part.n[b] = n;
    if (b == 0) *part.done = 0;                     // the join's, which runs after this grid
  }
}

// Joins the blocks' sums for kJoin experts a block; the block that is done last writes the losses.  A chain of
// latencies: every thread's loads go out at once, sums stay in registers but for one step through LDS.
__global__ __launch_bounds__(kThreads) void balance_join_kernel(void* __restrict__ ws, int blocks, int E,
                                                                float* __restrict__ losses, int* __restrict__ counts,
                                                                float* __restrict__ probs, int* __restrict__ tokens,
                                                                bool counted) {
  constexpr int kGroups = kThreads / kJoin, kEach = kMaxBlocks / kGroups;
  static_assert(kJoin == 32, "two groups a wave");
  __shared__ float sums[kWaves][kJoin];
  __shared__ int hist[kWaves][kJoin];
  __shared__ float zs[kMaxBlocks / 64];
  __shared__ int ns[kMaxBlocks / 64];
  const Partial part = partial_of(ws, blocks, E);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, Ep = padded(E), group = tid / kJoin, col = tid % kJoin;
  const int e = blockIdx.x * kJoin + col;
  const bool upper = (lane & 32) != 0;
  float p[kEach], z = 0.f;
  int c[kEach], n = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = group + i * kGroups;
    p[i] = b < blocks ? part.probs[(size_t)b * Ep + e] : 0.f;
    c[i] = b < blocks ? part.counts[(size_t)b * Ep + e] : 0;
  }
  if (tid < blocks) {
    z = part.z[tid];
    n = part.n[tid];
  }
  const int given = !counted && tid < kJoin && e < E ? counts[e] : 0;
#pragma unroll
  for (int i = 1; i < kEach; ++i) {
    p[0] += p[i];
    c[0] += c[i];
  }
  sums[wave][col] = p[0] + other_rows<32>(p[0], upper);
  hist[wave][col] = c[0] + (int)other_rows<32>((uint32_t)c[0], upper);
  if (wave < kMaxBlocks / 64) {
    z = lanes_sum<64>(z);
    n = reduce<64>((uint32_t)n, [](uint32_t u, uint32_t v) { return u + v; });
    if (lane == 0) {
      zs[wave] = z;
      ns[wave] = n;
    }
  }
  __syncthreads();
  if (tid >= 64) return;
  float prob = 0.f;
  int count = 0;
#pragma unroll
  for (int w = 0; w < kWaves / 2; ++w) {            // a half of the waves' sums for each half of this wave
    prob += sums[w + (upper ? kWaves / 2 : 0)][col];
    count += hist[w + (upper ? kWaves / 2 : 0)][col];
  }
  prob += other_rows<32>(prob, upper);
  count += (int)other_rows<32>((uint32_t)count, upper);
  z = 0.f;
  n = 0;
#pragma unroll
  for (int w = 0; w < kMaxBlocks / 64; ++w) {
    z += zs[w];
    n += ns[w];
  }
  const Share one = write_expert(tid < kJoin && e < E, e, prob, counted ? count : given, n, counts, probs, counted);
  unsigned before = 0;
  if (tid == 0) {
    __hip_atomic_store(part.shares + 2 * blockIdx.x, one.dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(part.shares + 2 * blockIdx.x + 1, one.slots, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // The device's other blocks read the shares with atomic loads alone, so that the stores have arrived is all that
    // the count needs: a release of the agent's scope would write the whole L2 back.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    before = __hip_atomic_fetch_add(part.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if ((unsigned)__builtin_amdgcn_readfirstlane((int)before) + 1 != gridDim.x) return;
  const int joins = gridDim.x;                      // at most 32
  const auto plus = [](double a, double b) { return a + b; };
  const auto of = [&](int k) {
    const double* s = part.shares + 2 * min(tid, joins - 1) + k;
    const double v = __hip_atomic_load(s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return reduce<64>(tid < joins ? v : 0.0, plus);
  };
  const Share all{of(0), of(1)};
  if (tid == 0) write_losses(E, all, z, n, losses, tokens);
}

// Reads the logits (and add) once and writes the gradient: 16384 x 256 f32 with add, 50 MB, in 12.8 us, 9.5 at a copy's
// rate; blocks that take several tokens each load the next ones' while they compute, two blocks a CU (one or three
// 13.1 and 13.4 us a call against 12.7, four 15.4).  Few tokens (10007 x 160 bf16, 6.8 us) wait for the counts: a lane's V
// loads of them, behind a condition each, follow one another and hold up the logits that were asked for before them.
template <int L, int V, typename TX, bool WIDE>
__global__ __launch_bounds__(256) void balance_bwd_kernel(const float* __restrict__ dlosses,
                                                          const TX* __restrict__ logits,
                                                          const int* __restrict__ counts,
                                                          const int* __restrict__ tokens, int T, int E, const TX* add,
                                                          TX* dlogits) {
  constexpr int C = 16 / (int)sizeof(TX);
  const int lane = threadIdx.x & 63, at = lane % L, sub = lane / L;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int step = gridDim.x * 4 * (64 / L);
  int t = (blockIdx.x * 4 + wave) * (64 / L) + sub;
  Chunks<V, TX> next, next_add;
  load_chunks<L, V, true>(logits + (size_t)t * E, E, at, t < T, WIDE, next);
  if (add) load_chunks<L, V, false>(add + (size_t)t * E, E, at, t < T, WIDE, next_add);
  float c[V];
  int count[V];
  uint64_t slots = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = expert_of<L, C>(at, i);
    count[i] = e < E ? max(counts[e], 0) : 0;
    slots += (uint32_t)count[i];
  }
  const double S = reduce<L>((double)slots, [](double a, double b) { return a + b; }), mean = S / (double)E;
  const float n = (float)tokens[0];
  const float a = n > 0.f && S > 0.0 ? dlosses[0] * (float)E / n / (float)S : 0.f;
  const float b = n > 0.f ? dlosses[1] * 2.f / n : 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = (float)((double)count[i] - mean);   // loads past 2^24 are no f32 numbers
  while (t - sub < T) {
    const int now = t;
    float x[V], old[V], total, lse, dot = 0.f;
    unpack<V>(next, x);
    if (add) unpack<V>(next_add, old);
    t += step;
    load_chunks<L, V, true>(logits + (size_t)t * E, E, at, t < T, WIDE, next);
    if (add) load_chunks<L, V, false>(add + (size_t)t * E, E, at, t < T, WIDE, next_add);
    exponentials<L, V>(x, total, lse);
    const bool some = total != 0.f;
    const float share = 1.f / total;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] *= share;
      dot += x[i] * c[i];
    }
    const float centre = a * lanes_sum<L>(dot), far = b * lse;
    if (__builtin_amdgcn_ballot_w64(__builtin_fabsf(far) == __builtin_inff())) {   // logits near f32's largest: p first
#pragma unroll
      for (int i = 0; i < V; ++i)
        x[i] = some ? __builtin_fmaf(x[i] * b, lse, x[i] * __builtin_fmaf(a, c[i], -centre)) : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = some ? x[i] * __builtin_fmaf(a, c[i], far - centre) : 0.f;
    }
    if (add)
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] += old[i];
    if (now < T) store_logits<L, V>(dlogits + (size_t)now * E, E, at, WIDE, x);
  }
}

// One block by itself for few tokens, which a launch of its own to join others would double: 512 x 128 10.0 us, joined
// 10.5; 512 x 256 13.3 and 10.6, 1024 x 16 12.8 and 10.4.
int balance_blocks(int T, int E) {
  return T <= 512 && T * E <= 65536 ? 1 : std::min((T + 63) / 64, kMaxBlocks);
}

template <int L, int V, typename TX, bool WIDE>
hipError_t balance_impl(const TX* logits, const int* ids, int T, int E, int k, float* losses, int* counts, float* probs,
                        int* tokens, void* ws, hipStream_t stream) {
  const int blocks = balance_blocks(T, E), slots = T * k;
  if (blocks == 1) {
    hipLaunchKernelGGL((balance_kernel<L, V, TX, WIDE, true>), dim3(1), dim3(kThreads), 0, stream, logits, ids, T, E, slots,
                       losses, counts, probs, tokens, ws);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((balance_kernel<L, V, TX, WIDE, false>), dim3(blocks), dim3(kThreads), 0, stream, logits, ids, T, E,
                     slots, losses, counts, probs, tokens, ws);
  const hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  hipLaunchKernelGGL(balance_join_kernel, dim3((E + kJoin - 1) / kJoin), dim3(kThreads), 0, stream, ws, blocks, E,
                     losses, counts, probs, tokens, ids != nullptr);
  return hipGetLastError();
}

// The lanes of a token, from its experts; a lane holds whole 16-byte chunks (4 logits in f32, 8 in bf16), which rows
// of other sizes do not keep together.
#define BY_EXPERTS(RUN)                                                       \
  constexpr int C = 16 / (int)sizeof(TX);                                     \
  if (E % C == 0) {                                                           \
    BY_LANES(RUN, true)                                                       \
  }                                                                           \
  BY_LANES(RUN, false)
#define BY_LANES(RUN, WIDE)                             \
  if (E <= 16 * C) return RUN(16, C, WIDE);             \
  if (E <= 128) return RUN(16, 8, WIDE); /* f32 alone */ \
  if (E <= 256) return RUN(16, 16, WIDE);               \
  if (E <= 64 * C) return RUN(64, C, WIDE);             \
  if (E <= 512) return RUN(64, 8, WIDE); /* f32 alone */ \
  return RUN(64, 16, WIDE);

template <typename TX>
hipError_t balance_pick(const TX* logits, const int* ids, int T, int E, int k, float* losses, int* counts, float* probs,
                        int* tokens, void* ws, hipStream_t stream) {
#define RUN(L, V, WIDE) (balance_impl<L, V, TX, WIDE>(logits, ids, T, E, k, losses, counts, probs, tokens, ws, stream))
  BY_EXPERTS(RUN)
#undef RUN
}

template <int L, int V, typename TX, bool WIDE>
hipError_t balance_bwd_impl(const float* dlosses, const TX* logits, const int* counts, const int* tokens, int T, int E,
                            const TX* add, TX* dlogits, hipStream_t stream) {
  const int blocks = std::min((T + 256 / L - 1) / (256 / L), kBackwardBlocks * device_cu_count());
  hipLaunchKernelGGL((balance_bwd_kernel<L, V, TX, WIDE>), dim3(blocks), dim3(256), 0, stream, dlosses, logits, counts,
                     tokens, T, E, add, dlogits);
  return hipGetLastError();
}

template <typename TX>
hipError_t balance_bwd_pick(const float* dlosses, const TX* logits, const int* counts, const int* tokens, int T, int E,
                            const TX* add, TX* dlogits, hipStream_t stream) {
#define RUN(L, V, WIDE) (balance_bwd_impl<L, V, TX, WIDE>(dlosses, logits, counts, tokens, T, E, add, dlogits, stream))
  BY_EXPERTS(RUN)
#undef RUN
}

}  // namespace

size_t balance_workspace_bytes(int T, int E) {
  const size_t blocks = balance_blocks(T, E);
  return blocks == 1 ? 0 : 16 * (size_t)(padded(E) / kJoin) + 8 * blocks * (padded(E) + 1) + 8;
}

hipError_t launch_balance(const void* logits, bool bf16, const int* ids, int T, int E, int k, float* losses,
                          int* counts, float* probs, int* tokens, void* ws, hipStream_t stream) {
  if (bf16)
    return balance_pick(static_cast<const uint16_t*>(logits), ids, T, E, k, losses, counts, probs, tokens, ws, stream);
  return balance_pick(static_cast<const float*>(logits), ids, T, E, k, losses, counts, probs, tokens, ws, stream);
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
