// Routing of a mixture-of-experts layer: the k largest of each token's E router
// logits, their softmax weights, and the stable sort of the T*k (token, choice)
// slots by expert that the grouped matmuls' group_sizes describe.
//
//   ids[t, :]    = the k largest x[t, e], largest first, ties to the lowest e;
//                  a logit of -inf is masked: never chosen (id -1, weight 0)
//   weights[t,j] = exp(x[t, ids_j] - m) / sum exp(x - m), the sum over the chosen
//                  (renormalize) or over all E logits
//   group_sizes[e] = slots with id e;  row_of_slot[t*k + j] = the slot's row in
//                  expert order (slots of one expert keep their order; -1 if
//                  masked);  slot_of_row = its inverse (-1 past the last row)
//
// Gradient, with s = sum_j w_j dw_j over the chosen and p the softmax over all:
//   dx[t, ids_j] = w_j (dw_j - s), 0 elsewhere          (renormalize)
//   dx[t, e]     = [e = ids_j] w_j dw_j - p_e s         (otherwise)
//
// A wave holds one token's logits, as keys whose unsigned order is the logits'
// order, and takes the maximum k times.  A token's choices are distinct, so the
// wave counts them into its LDS histogram without conflicts, and the count
// before the increment is the slot's rank among the wave's slots of that
// expert.  Waves of a block and then blocks are joined by prefix sums of the
// histograms: the order of slots never depends on timing.
#include "common.hpp"
#include "launch.hpp"

#include <algorithm>

namespace fp8gmm {
namespace {

constexpr int kThreads = 1024;                      // 16 waves
constexpr int kWaves = kThreads / 64;
constexpr int kTokensPerWave = 4;
constexpr int kTokensPerBlock = kWaves * kTokensPerWave;   // per chunk
constexpr int kMaxBlocks = 512;                     // longer batches give a block several chunks
constexpr uint32_t kKeyMasked = 0x007FFFFFu;        // key of -inf

// Unsigned order of the keys = order of the floats; -0 equals +0, NaN is above +inf.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);     // -0 + 0 = +0
  const uint32_t key = u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
  return x != x ? 0xFFFFFFFFu : key;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}
// Maximum over the wave, in a scalar register (rotations within rows of 16, then the four rows).
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = dpp_max<0x128>(v);
  v = dpp_max<0x124>(v);
  v = dpp_max<0x122>(v);
  v = dpp_max<0x121>(v);
  const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16));
  const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48));
  return max(a, b);
}

__device__ __forceinline__ float wave_fsum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

__device__ __forceinline__ float load_logit(const float* x) { return *x; }
__device__ __forceinline__ float load_logit(const uint16_t* x) { return __uint_as_float((uint32_t)*x << 16); }

// The k choices of one token: lane j < k returns choice j.  V logits per lane,
// logit e = 64 * i + lane in x[i].
template <int V>
__device__ __forceinline__ void choose(const float (&x)[V], int E, int k, bool renorm, int lane, int& id, float& w) {
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = 64 * i + lane < E ? order_key(x[i]) : 0u;
  uint32_t top = 0;
  id = -1;
  uint32_t mine = kKeyMasked;
  for (int j = 0; j < k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = max(m, key[i]);
    m = wave_umax(m);
    if (j == 0) top = m;
    if (m <= kKeyMasked) break;                     // only masked logits are left
    bool found = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint64_t hit = __ballot(key[i] == m);
      if (!found && hit != 0) {                     // the lowest index of the largest value
        const int at = __ffsll((unsigned long long)hit) - 1;
        if (lane == at) key[i] = 0;
        if (lane == j) {
          id = 64 * i + at;
          mine = m;
        }
        found = true;
      }
    }
  }
  const float big = key_value(top);
  float total;
  const float e = id >= 0 ? expf(key_value(mine) - big) : 0.f;
  if (renorm) {
    total = wave_fsum(e);
  } else {
    total = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (64 * i + lane < E) total += expf(x[i] - big);
    total = wave_fsum(total);
  }
  w = id >= 0 ? e / total : 0.f;
}

// hist holds a block's slots per expert as 16 bits (a block has fewer than 2^16
// tokens, and a token chooses an expert once): [blocks][Ep], Ep = E rounded up to 8.
// ONE: the grid is one block, which places the slots itself.
template <int V, typename TX, bool ONE>
__global__ __launch_bounds__(kThreads) void route_topk_kernel(const TX* __restrict__ logits, int T, int E, int k,
                                                             int renorm, int chunks, int* __restrict__ ids,
                                                             float* __restrict__ weights, int* __restrict__ row_of_slot,
                                                             uint16_t* __restrict__ hist, int* __restrict__ group_sizes,
                                                             int* __restrict__ slot_of_row) {
  extern __shared__ int smem[];
  int* const seen = smem;                           // [E] slots of earlier chunks (ONE: first row of the expert)
  int* const cnt = smem + E;                        // [kWaves][E]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int e = tid; e < E; e += kThreads) seen[e] = 0;
  for (int c = 0; c < chunks; ++c) {
    const int t0 = (blockIdx.x * chunks + c) * kTokensPerBlock + wave * kTokensPerWave;
    for (int i = tid; i < kWaves * E; i += kThreads) cnt[i] = 0;
    float x[kTokensPerWave][V];
#pragma unroll
    for (int q = 0; q < kTokensPerWave; ++q)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = 64 * i + lane;
        x[q][i] = (t0 + q < T && e < E) ? load_logit(logits + (size_t)(t0 + q) * E + e) : 0.f;
      }
    __syncthreads();
    int id[kTokensPerWave], rank[kTokensPerWave];
#pragma unroll
    for (int q = 0; q < kTokensPerWave; ++q) {
      id[q] = -1;
      rank[q] = 0;
      if (t0 + q < T) {
        float w;
        choose<V>(x[q], E, k, renorm != 0, lane, id[q], w);
        if (lane < k) {
          const size_t at = (size_t)(t0 + q) * k + lane;
          ids[at] = id[q];
          weights[at] = w;
          if (id[q] >= 0) {
            rank[q] = cnt[wave * E + id[q]];
            cnt[wave * E + id[q]] = rank[q] + 1;
          }
        }
      }
    }
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) {       // counts -> first rank of each wave
      int s = seen[e];
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        const int n = cnt[v * E + e];
        cnt[v * E + e] = s;
        s += n;
      }
      seen[e] = s;
    }
    __syncthreads();
    if (ONE) {
      const int n = tid < E ? seen[tid] : 0;        // E <= kThreads
      if (tid < E) group_sizes[tid] = n;
      __shared__ int part[kWaves];
      const int incl = wave_incl_scan(n);
      if (lane == 63) part[wave] = incl;
      __syncthreads();
      int before = 0, all = 0;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        if (v < wave) before += part[v];
        all += part[v];
      }
      if (tid < E) seen[tid] = before + incl - n;
      __syncthreads();
      for (int r = all + tid; r < T * k; r += kThreads) slot_of_row[r] = -1;
#pragma unroll
      for (int q = 0; q < kTokensPerWave; ++q)
        if (t0 + q < T && lane < k) {
          const int slot = (t0 + q) * k + lane;
          const int row = id[q] < 0 ? -1 : seen[id[q]] + cnt[wave * E + id[q]] + rank[q];
          row_of_slot[slot] = row;
          if (row >= 0) slot_of_row[row] = slot;
        }
    } else {
#pragma unroll
      for (int q = 0; q < kTokensPerWave; ++q)
        if (t0 + q < T && lane < k && id[q] >= 0)   // rank within the block for now
          row_of_slot[(size_t)(t0 + q) * k + lane] = cnt[wave * E + id[q]] + rank[q];
    }
    __syncthreads();
  }
  if (!ONE) {
    const int Ep = (E + 7) & ~7;
    for (int e = tid; e < Ep; e += kThreads) hist[(size_t)blockIdx.x * Ep + e] = (uint16_t)(e < E ? seen[e] : 0);
  }
}

// Places the slots of block b: an expert's first row, plus its slots in earlier
// blocks, plus the rank within the block that route_topk_kernel left in row_of_slot.
__global__ __launch_bounds__(kThreads) void route_place_kernel(const int* __restrict__ ids,
                                                              const uint16_t* __restrict__ hist, int T, int E, int k,
                                                              int chunks, int* __restrict__ group_sizes,
                                                              int* __restrict__ row_of_slot,
                                                              int* __restrict__ slot_of_row) {
  extern __shared__ int smem[];
  const int Ep = (E + 7) & ~7, ne = Ep / 8;
  int* const first = smem;                          // [Ep] slots in earlier blocks, then the block's first rows
  int* const total = smem + Ep;                     // [Ep]
  __shared__ int part[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = blockIdx.x, nb = gridDim.x;
  for (int e = tid; e < 2 * Ep; e += kThreads) smem[e] = 0;
  __syncthreads();
  // thread (segment, 8 experts): the histogram's rows segment, segment + nseg, ...
  const int nseg = kThreads / ne, seg = tid / ne, e0 = (tid % ne) * 8;
  if (seg < nseg) {
    int before[8] = {}, all[8] = {};
#pragma unroll 4
    for (int r = seg; r < nb; r += nseg) {
      const v4i h = *reinterpret_cast<const v4i*>(hist + (size_t)r * Ep + e0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int n = (int)(((uint32_t)h[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
        all[i] += n;
        if (r < b) before[i] += n;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {                   // sums of whole numbers: any order gives the same
      if (before[i]) atomicAdd(&first[e0 + i], before[i]);
      if (all[i]) atomicAdd(&total[e0 + i], all[i]);
    }
  }
  __syncthreads();
  const int n = tid < E ? total[tid] : 0;           // E <= kThreads
  if (b == 0 && tid < E) group_sizes[tid] = n;
  const int incl = wave_incl_scan(n);
  if (lane == 63) part[wave] = incl;
  __syncthreads();
  int offset = 0, rows = 0;
#pragma unroll
  for (int v = 0; v < kWaves; ++v) {
    if (v < wave) offset += part[v];
    rows += part[v];
  }
  if (tid < E) first[tid] += offset + incl - n;
  __syncthreads();
  const int s0 = b * chunks * kTokensPerBlock * k;  // T * k < 2^24, and a block starts below T
  const int s1 = min(s0 + chunks * kTokensPerBlock * k, T * k);
  for (int s = s0 + tid; s < s1; s += kThreads) {
    const int id = ids[s];
    const int row = id < 0 ? -1 : first[id] + row_of_slot[s];
    row_of_slot[s] = row;
    if (row >= 0) slot_of_row[row] = s;
    if (s >= rows) slot_of_row[s] = -1;             // no slot is placed there
  }
}

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.f); }

// One wave per token.  Lane j < k holds choice j; its share of the gradient is
// handed to the lane that holds the logit.
template <int V, typename TX>
__global__ __launch_bounds__(256) void route_bwd_kernel(const float* __restrict__ dweights,
                                                        const TX* __restrict__ logits, const int* __restrict__ ids,
                                                        const float* __restrict__ weights, int T, int E, int k,
                                                        int renorm, TX* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= T) return;
  int id = -1;
  float w = 0.f, dw = 0.f;
  if (lane < k) {
    const size_t at = (size_t)t * k + lane;
    id = ids[at];
    if (id >= 0 && id < E) {                        // a masked choice's gradient is not read
      w = weights[at];
      dw = dweights[at];
    }
  }
  const float inner = wave_fsum(w * dw);
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = 0.f;
  const float here = w * (renorm ? dw - inner : dw);
  for (int j = 0; j < k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, here), j));
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e == 64 * i + lane) d[i] += v;
  }
  if (!renorm) {
    float x[V], top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 64 * i + lane;
      x[i] = e < E ? load_logit(logits + (size_t)t * E + e) : -__builtin_inff();
      top = __builtin_fmaxf(top, x[i]);
    }
    top = wave_max(top);
    if (top != -__builtin_inff()) {                 // a token without experts has no gradient
      float total = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[i] = expf(x[i] - top);
        total += x[i];
      }
      total = wave_fsum(total);
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] -= x[i] / total * inner;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 64 * i + lane;
    if (e < E) store_logit(dlogits + (size_t)t * E + e, d[i]);
  }
}

int route_blocks(int T, int& chunks) {
  const int nc = (T + kTokensPerBlock - 1) / kTokensPerBlock;
  chunks = std::max(1, (nc + kMaxBlocks - 1) / kMaxBlocks);   // 1 for no tokens
  return (nc + chunks - 1) / chunks;
}

template <int V, typename TX>
hipError_t route_impl(const TX* logits, int T, int E, int k, int renorm, int* ids, float* weights, int* group_sizes,
                      int* row_of_slot, int* slot_of_row, uint16_t* hist, hipStream_t stream) {
  int chunks;
  const int nb = route_blocks(T, chunks);
  const size_t lds = sizeof(int) * (size_t)E * (kWaves + 1);
  if (nb <= 1) {
    hipLaunchKernelGGL((route_topk_kernel<V, TX, true>), dim3(1), dim3(kThreads), lds, stream, logits, T, E, k, renorm,
                       1, ids, weights, row_of_slot, hist, group_sizes, slot_of_row);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((route_topk_kernel<V, TX, false>), dim3(nb), dim3(kThreads), lds, stream, logits, T, E, k, renorm,
                     chunks, ids, weights, row_of_slot, hist, group_sizes, slot_of_row);
  hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  hipLaunchKernelGGL(route_place_kernel, dim3(nb), dim3(kThreads), sizeof(int) * 2 * (size_t)((E + 7) & ~7), stream,
                     ids, hist, T, E, k, chunks, group_sizes, row_of_slot, slot_of_row);
  return hipGetLastError();
}

template <typename TX>
hipError_t route_pick(const TX* logits, int T, int E, int k, int renorm, int* ids, float* weights, int* group_sizes,
                      int* row_of_slot, int* slot_of_row, uint16_t* hist, hipStream_t stream) {
#define ROUTE(V) \
  route_impl<V, TX>(logits, T, E, k, renorm, ids, weights, group_sizes, row_of_slot, slot_of_row, hist, stream)
  if (E <= 64) return ROUTE(1);
  if (E <= 128) return ROUTE(2);
  if (E <= 256) return ROUTE(4);
  if (E <= 512) return ROUTE(8);
  return ROUTE(16);
#undef ROUTE
}

template <typename TX>
hipError_t route_bwd_pick(const float* dweights, const TX* logits, const int* ids, const float* weights, int T, int E,
                          int k, int renorm, TX* dlogits, hipStream_t stream) {
#define ROUTE(V)                                                                                                     \
  hipLaunchKernelGGL((route_bwd_kernel<V, TX>), dim3((T + 3) / 4), dim3(256), 0, stream, dweights, logits, ids, weights, \
                     T, E, k, renorm, dlogits)
  if (E <= 64) ROUTE(1);
  else if (E <= 128) ROUTE(2);
  else if (E <= 256) ROUTE(4);
  else if (E <= 512) ROUTE(8);
  else ROUTE(16);
#undef ROUTE
  return hipGetLastError();
}

}  // namespace

size_t route_workspace_bytes(int T, int E) {
  int chunks;
  const int nb = T > 0 ? route_blocks(T, chunks) : 0;
  return nb <= 1 ? 0 : sizeof(uint16_t) * (size_t)nb * ((E + 7) & ~7);
}

hipError_t launch_route(const void* logits, bool bf16, int T, int E, int k, bool renorm, int* ids, float* weights,
                        int* group_sizes, int* row_of_slot, int* slot_of_row, void* ws, hipStream_t stream) {
  uint16_t* hist = static_cast<uint16_t*>(ws);
  if (bf16)
    return route_pick(static_cast<const uint16_t*>(logits), T, E, k, renorm, ids, weights, group_sizes, row_of_slot,
                      slot_of_row, hist, stream);
  return route_pick(static_cast<const float*>(logits), T, E, k, renorm, ids, weights, group_sizes, row_of_slot,
                    slot_of_row, hist, stream);
}

hipError_t launch_route_bwd(const float* dweights, const void* logits, bool bf16, const int* ids, const float* weights,
                            int T, int E, int k, bool renorm, void* dlogits, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  if (bf16)
    return route_bwd_pick(dweights, static_cast<const uint16_t*>(logits), ids, weights, T, E, k, renorm,
                          static_cast<uint16_t*>(dlogits), stream);
  return route_bwd_pick(dweights, static_cast<const float*>(logits), ids, weights, T, E, k, renorm,
                        static_cast<float*>(dlogits), stream);
}

}  // namespace fp8gmm
