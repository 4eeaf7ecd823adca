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
// A token's logits lie in a row of 16 lanes (four tokens a wave) or, for more than
// 256 experts or 16 choices, in the whole wave; each becomes a key that holds its
// order and its expert, so that keys are distinct and the lower expert wins a tie.
// A lane sorts its keys once with a network; k times the largest head over the
// lanes is taken and its lane's list moves up.  (Searching all keys k times, one
// token a wave, was bound by its instructions: 18 us for 16384 x 256 bf16, k = 8,
// against 7.2 us now, of which 2 us are the bytes.)
//
// A token's choices are distinct, so a wave counts them into its LDS histogram
// without conflicts, and the count before the increment is the slot's rank among
// the wave's slots of that expert.  Waves of a block and then blocks are joined by
// prefix sums of the histograms: the order of slots never depends on timing.
#include "logits.hpp"
#include "moe_launch.hpp"

#include <algorithm>
#include <type_traits>
#include <utility>

namespace fp8gmm {
namespace {

constexpr int kThreads = 1024;                      // 16 waves
constexpr int kWaves = kThreads / 64;
constexpr int kTokensPerWave = 4;
constexpr int kTokensPerBlock = kWaves * kTokensPerWave;   // per chunk
constexpr int kMaxBlocks = 512;                     // longer batches give a block several chunks
constexpr int kByteChunks = 3;                      // 192 tokens
static_assert(kByteChunks * kTokensPerBlock < 256, "a block's count fits a byte");
// A wave of route_place_kernel joins its share of the rows, up to 32 of 512, or a row a lane where a row is one chunk.
static_assert(64 * kByteChunks * kTokensPerBlock < 65536, "a wave's sums of bytes fit 16 bits");
__host__ __device__ constexpr int hist_row(int E) { return (E + 15) & ~15; }

// The wave's lanes see each other's LDS writes past this point: LDS serves a wave in order, and
// the compiler may neither move nor forward accesses across it.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Keys: larger for the larger logit, then for the lower expert.  -0 equals +0, NaN is above +inf;
// a masked logit (-inf) is at or below kMasked, a place past the experts is kNone.
template <typename TX>
struct Order;

// bf16: the bits as an unsigned number, the complement of the expert below them.
template <>
struct Order<uint16_t> {
  using Key = uint32_t;
  static constexpr Key kMasked = 0x007FFFFFu, kNone = 0;
  static __device__ __forceinline__ Key key(float x, int e) {
    const uint32_t u = __float_as_uint(x + 0.0f);   // -0 + 0 = +0
    const uint32_t o = x != x ? 0xFFFF0000u : u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
    return (o & 0xFFFF0000u) | (uint32_t)(0xFFFF - e);
  }
  static __device__ __forceinline__ int expert(Key k) { return 0xFFFF - (int)(k & 0xFFFFu); }
  static __device__ __forceinline__ float value(Key k) {
    return __uint_as_float(k & 0x80000000u ? (k & 0x7FFF0000u) : ~(k | 0xFFFFu));
  }
  static __device__ __forceinline__ Key larger(Key a, Key b) { return max(a, b); }
  static __device__ __forceinline__ Key smaller(Key a, Key b) { return min(a, b); }
};

// f32: the value in f64, whose mantissa has 29 bits to spare for the expert (a negative key grows
// with its distance from zero, so it takes the expert itself); infinities and NaN become finite
// numbers beyond the f32 range, so that maximum and minimum instructions order them.
template <>
struct Order<float> {
  using Key = double;
  static constexpr Key kInf = 0x1p200, kNan = 0x1p300, kMasked = -0x1p200, kNone = -0x1p400;
  static __device__ __forceinline__ Key key(float x, int e) {
    double d = __builtin_fmin(__builtin_fmax((double)(x + 0.0f), -kInf), kInf);
    d = x != x ? kNan : d;
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, d) | (uint64_t)(uint32_t)(d < 0 ? e : 1023 - e));
  }
  static __device__ __forceinline__ int expert(Key k) {
    const int low = (int)(__builtin_bit_cast(uint64_t, k) & 1023);
    return k < 0 ? low : 1023 - low;
  }
  static __device__ __forceinline__ float value(Key k) {
    const double d = __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~1023ull);
    return d == kNan ? __builtin_nanf("") : (float)d;   // 2^200 overflows to infinity
  }
  static __device__ __forceinline__ Key larger(Key a, Key b) { return __builtin_fmax(a, b); }
  static __device__ __forceinline__ Key smaller(Key a, Key b) { return __builtin_fmin(a, b); }
};

// Batcher's odd-even merge sort of n = 4, 8 or 16 as a list of exchanges.
struct Network {
  int n = 0;
  uint8_t a[64] = {}, b[64] = {};
};
constexpr Network network(int n) {
  Network w;
  for (int p = 1; p < n; p *= 2)
    for (int k = p; k >= 1; k /= 2)
      for (int j = k % p; j + k < n; j += 2 * k)
        for (int i = 0; i < k && i + j + k < n; ++i)
          if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            w.a[w.n] = (uint8_t)(i + j);
            w.b[w.n] = (uint8_t)(i + j + k);
            ++w.n;
          }
  return w;
}
template <typename O, int V, int... I>
__device__ __forceinline__ void sort_down(typename O::Key (&s)[V], std::integer_sequence<int, I...>) {
  constexpr Network w = network(V);
  auto exchange = [&](auto& x, auto& y) {
    const auto big = O::larger(x, y), small = O::smaller(x, y);
    x = big;
    y = small;
  };
  (exchange(s[w.a[I]], s[w.b[I]]), ...);
}

// The k choices of a token: lane j < k of its lanes returns choice j.  A lane's list never moves up
// more than k - 1 places, so its first D = min(V, k's bound) keys are all that is read.
template <int L, int V, int D, typename TX>
__device__ __forceinline__ void choose(const float (&x)[V], int E, int k, bool renorm, int at, int& id, float& w) {
  using O = Order<TX>;
  using Key = typename O::Key;
  constexpr int C = 16 / (int)sizeof(TX);
  float big = -__builtin_inff(), total = 0.f;
  if (!renorm) {                                    // over all logits, before their registers become keys
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (expert_of<L, C>(at, i) < E) big = __builtin_fmaxf(big, x[i]);
    big = lanes_max<L>(big);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (expert_of<L, C>(at, i) < E) total += expf(x[i] - big);
    total = lanes_sum<L>(total);
  }
  Key s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = expert_of<L, C>(at, i);
    s[i] = e < E ? O::key(x[i], e) : O::kNone;
  }
  sort_down<O>(s, std::make_integer_sequence<int, network(V).n>{});
  Key top = O::kNone, mine = O::kNone;
  for (int j = 0; j < k; ++j) {
    const Key m = reduce<L>(s[0], [](Key a, Key b) { return O::larger(a, b); });
    if (j == 0) top = m;
    if (at == j) mine = m;
    const bool taken = s[0] == m;
#pragma unroll
    for (int i = 0; i < D; ++i) {                   // copies: a conditional of two elements would index the array
      const Key own = s[i], next = i + 1 < D ? Key(s[i + 1]) : O::kNone;
      s[i] = taken ? next : own;
    }
  }
  id = mine > O::kMasked ? O::expert(mine) : -1;
  if (renorm) big = O::value(top);
  const float e = id >= 0 ? expf(O::value(mine) - big) : 0.f;
  if (renorm) total = lanes_sum<L>(e);
  w = id >= 0 ? e / total : 0.f;
}

// hist holds a block's slots per expert, at most one a token: bytes for up to
// kByteChunks chunks a block, 16 bits beyond; a row of 16-byte multiples a block.
// ONE: the grid is one block, of as many waves as its tokens need, which places the
// slots itself.
template <int L, int V, int D, typename TX, bool ONE>
__global__ __launch_bounds__(kThreads) void route_topk_kernel(const TX* __restrict__ logits, int T, int E, int k,
                                                             int renorm, int chunks, int* __restrict__ ids,
                                                             float* __restrict__ weights, int* __restrict__ row_of_slot,
                                                             void* __restrict__ hist, int* __restrict__ group_sizes,
                                                             int* __restrict__ slot_of_row) {
  constexpr int kRounds = kTokensPerWave * L / 64;  // tokens of a wave, 64 / L at a time
  extern __shared__ int smem[];
  int* const seen = smem;                           // [E] slots of earlier chunks (ONE: first row of the expert)
  int* const cnt = smem + E;                        // [waves][E]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int threads = blockDim.x, waves = threads >> 6;
  const int at = lane % L, sub = lane / L;
  const bool wide = E % (16 / (int)sizeof(TX)) == 0;
  for (int e = tid; e < E; e += threads) seen[e] = 0;
  for (int c = 0; c < chunks; ++c) {
    const int t0 = (blockIdx.x * chunks + c) * kTokensPerBlock + wave * kTokensPerWave + sub;
    float x[V];
    load_logits<L, V>(logits + (size_t)t0 * E, E, at, t0 < T, wide, x);
    for (int i = tid; i < waves * E; i += threads) cnt[i] = 0;
    __syncthreads();
    int id[kRounds], rank[kRounds];
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
      const int t = t0 + q * (64 / L);
      float w;
      if (q > 0) load_logits<L, V>(logits + (size_t)t * E, E, at, t < T, wide, x);
      choose<L, V, D, TX>(x, E, k, renorm != 0, at, id[q], w);
      rank[q] = 0;
      const bool mine = t < T && at < k;
      if (mine) {
        const size_t slot = (size_t)t * k + at;
        ids[slot] = id[q];
        weights[slot] = w;
      }
#pragma unroll
      for (int v = 0; v < 64 / L; ++v) {            // one token after the other
        if (mine && id[q] >= 0 && sub == v) {
          rank[q] = cnt[wave * E + id[q]];
          cnt[wave * E + id[q]] = rank[q] + 1;
        }
        wave_lds_order();
      }
    }
    __syncthreads();
    for (int e = tid; e < E; e += threads) {        // counts -> first rank of each wave
      int s = seen[e];
      if (ONE) {                                    // one wave to 16
        for (int v = 0; v < waves; ++v) {
          const int n = cnt[v * E + e];
          cnt[v * E + e] = s;
          s += n;
        }
      } else {
        int n[kWaves];
#pragma unroll
        for (int v = 0; v < kWaves; ++v) n[v] = cnt[v * E + e];
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
          cnt[v * E + e] = s;
          s += n[v];
        }
      }
      seen[e] = s;
    }
    __syncthreads();
    if (ONE) {
      int all = 0;
      if (wave == 0)                                // slots per expert -> first row of the expert
        for (int base = 0; base < E; base += 64) {
          const int e = base + lane, n = e < E ? seen[e] : 0;
          const int upto = all + wave_scan_dpp(n);
          if (e < E) {
            group_sizes[e] = n;
            seen[e] = upto - n;
          }
          all = __builtin_amdgcn_readlane(upto, 63);
        }
      __syncthreads();
      // rows past the last slot's: as many as there are masked choices
      if (wave == 0)
        for (int r = all + lane; r < T * k; r += 64) slot_of_row[r] = -1;
#pragma unroll
      for (int q = 0; q < kRounds; ++q) {
        const int t = t0 + q * (64 / L);
        if (t < T && at < k) {
          const int slot = t * k + at;
          const int row = id[q] < 0 ? -1 : seen[id[q]] + cnt[wave * E + id[q]] + rank[q];
          row_of_slot[slot] = row;
          if (row >= 0) slot_of_row[row] = slot;
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < kRounds; ++q) {
        const int t = t0 + q * (64 / L);
        if (t < T && at < k && id[q] >= 0)          // rank within the block for now
          row_of_slot[(size_t)t * k + at] = cnt[wave * E + id[q]] + rank[q];
      }
      __syncthreads();
    }
  }
  if (!ONE) {
    const int Ep = hist_row(E);
    for (int e = tid; e < Ep; e += threads) {
      const int n = e < E ? seen[e] : 0;
      const size_t at = (size_t)blockIdx.x * Ep + e;
      if (chunks <= kByteChunks) static_cast<uint8_t*>(hist)[at] = (uint8_t)n;
      else static_cast<uint16_t*>(hist)[at] = (uint16_t)n;
    }
  }
}

// Places the slots of block b: an expert's first row, plus its slots in earlier
// blocks, plus the rank within the block that route_topk_kernel left in row_of_slot.
// Every block sums the whole histogram instead of a launch between that would scan
// it: 64 KB at 16384 x 256, from L2, in bytes and two counts an addition (as 16 bits,
// one count an addition and LDS atomics, at least 6.5 us in a kernel trace; now 6.0).
//
// Thread (segment, chunk of 16 bytes) adds the rows segment, segment + segments, ..
template <typename H>
__global__ __launch_bounds__(kThreads) void route_place_kernel(const int* __restrict__ ids, const H* __restrict__ hist,
                                                              int T, int E, int k, int chunks, int chunk_lanes,
                                                              int* __restrict__ group_sizes,
                                                              int* __restrict__ row_of_slot,
                                                              int* __restrict__ slot_of_row) {
  constexpr int C = 16 / (int)sizeof(H);            // counts of a chunk
  extern __shared__ __attribute__((aligned(16))) int smem[];
  const int Ep = hist_row(E);
  int* const first = smem;                          // [Ep] the block's first rows
  int* const sums = smem + Ep;                      // [partial sums][2][Ep]
  __shared__ int part[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = blockIdx.x, nb = gridDim.x;
  const int s0 = b * chunks * kTokensPerBlock * k;  // T * k < 2^24, and a block starts below T
  const int s1 = min(s0 + chunks * kTokensPerBlock * k, T * k);
  const int mine = s0 + tid;                        // the first slot's loads run while the histogram is summed
  const int id0 = mine < s1 ? ids[mine] : -1, rank0 = mine < s1 ? row_of_slot[mine] : 0;
  // chunk_lanes: the chunks of a row, rounded up to a power of two
  const int g = tid & (chunk_lanes - 1), seg = tid / chunk_lanes, segs = kThreads / chunk_lanes;
  const bool here = g * C < Ep;
  // bytes: counts 0 and 2 of a word in acc[2j] and 1 and 3 in acc[2j + 1], 16 bits each; 16 bits: one count each
  uint32_t acc[2][8] = {};                          // rows before b, all rows
  if (here)
    for (int r0 = seg; r0 < nb; r0 += 4 * segs) {
      v4i h[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = r0 + u * segs;
        h[u] = r < nb ? *reinterpret_cast<const v4i*>(hist + (size_t)r * Ep + C * g) : (v4i){0, 0, 0, 0};
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t earlier = r0 + u * segs < b ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t w = (uint32_t)h[u][j / 2];
          const uint32_t c = sizeof(H) == 1 ? (j & 1 ? w >> 8 : w) & 0x00FF00FFu : (j & 1 ? w >> 16 : w & 0xFFFFu);
          acc[0][j] += c & earlier;
          acc[1][j] += c;
        }
      }
    }
  // segments of a wave, to all its lanes (uniform branches; shuffles through LDS took half of the kernel)
  auto join = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i / 8][i % 8] += f(acc[i / 8][i % 8]);
  };
  if (chunk_lanes <= 8) join([](uint32_t v) { return dpp_row<0x128>(v); });
  if (chunk_lanes <= 4) join([](uint32_t v) { return dpp_row<0x124>(v); });
  if (chunk_lanes <= 2) join([](uint32_t v) { return dpp_row<0x122>(v); });
  if (chunk_lanes <= 1) join([](uint32_t v) { return dpp_row<0x121>(v); });
  if (chunk_lanes <= 16) join([&](uint32_t v) { return other_rows<16>(v, (lane & 16) != 0); });
  if (chunk_lanes <= 32) join([&](uint32_t v) { return other_rows<32>(v, (lane & 32) != 0); });
  const int rows_of_sums = min(segs, kWaves), at = min(seg, tid / 64);
  if (here && (chunk_lanes >= 64 || lane < chunk_lanes))
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v4i* const out = reinterpret_cast<v4i*>(sums + (2 * at + i) * Ep + C * g);
      const uint32_t(&a)[8] = acc[i];
#pragma unroll
      for (int j = 0; j < C / 4; ++j)
        out[j] = sizeof(H) == 1 ? (v4i){(int)(a[2 * j] & 0xFFFF), (int)(a[2 * j + 1] & 0xFFFF), (int)(a[2 * j] >> 16),
                                        (int)(a[2 * j + 1] >> 16)}
                                : (v4i){(int)a[4 * j % 8], (int)a[(4 * j + 1) % 8], (int)a[(4 * j + 2) % 8],
                                        (int)a[(4 * j + 3) % 8]};
    }
  __syncthreads();
  int before = 0, n = 0;
  if (tid < E) {                                    // E <= kThreads
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      if (w < rows_of_sums) {
        before += sums[2 * w * Ep + tid];
        n += sums[(2 * w + 1) * Ep + tid];
      }
    if (b == 0) group_sizes[tid] = n;
  }
  const int incl = wave_scan_dpp(n);
  if (lane == 63) part[wave] = incl;
  __syncthreads();
  int offset = 0, rows = 0;
#pragma unroll
  for (int v = 0; v < kWaves; ++v) {
    if (v < wave) offset += part[v];
    rows += part[v];
  }
  if (tid < E) first[tid] = before + offset + incl - n;
  __syncthreads();
  for (int s = mine; s < s1; s += kThreads) {
    const int id = s == mine ? id0 : ids[s], rank = s == mine ? rank0 : row_of_slot[s];
    const int row = id < 0 ? -1 : first[id] + rank;
    row_of_slot[s] = row;
    if (row >= 0) slot_of_row[row] = s;
    if (s >= rows) slot_of_row[s] = -1;             // no slot is placed there
  }
}

// Gradient: 16384 x 160 f32 in 7.2 us, 4.1 us of them bytes (one token a wave with
// comparisons for each choice: 11.4).  Lanes share tokens as above: lane j < k holds
// choice j and puts its term into the token's row in LDS (the wave's own, so no
// barrier), which the lanes then read as their chunks.
template <int L, int V, typename TX>
__global__ __launch_bounds__(256) void route_bwd_kernel(const float* __restrict__ dweights,
                                                        const TX* __restrict__ logits, const int* __restrict__ ids,
                                                        const float* __restrict__ weights, int T, int E, int k,
                                                        int renorm, TX* __restrict__ dlogits) {
  constexpr int C = 16 / (int)sizeof(TX);
  __shared__ __attribute__((aligned(16))) float rows[4][64 * V];
  const int lane = threadIdx.x & 63, at = lane % L, sub = lane / L;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (blockIdx.x * 4 + wave) * (64 / L) + sub;
  const bool here = t < T, wide = E % C == 0;
  float* const row = rows[wave] + sub * L * V;
  int id = -1;
  float w = 0.f, dw = 0.f;
  if (here && at < k) {
    const size_t s = (size_t)t * k + at;
    id = ids[s];
    w = weights[s];
    dw = dweights[s];
    if (id < 0 || id >= E) {                        // a masked choice's gradient does not count
      id = -1;
      w = dw = 0.f;
    }
  }
  float x[V];
  if (!renorm) load_logits<L, V>(logits + (size_t)t * E, E, at, here, wide, x);
#pragma unroll
  for (int i = 0; i < V; i += 4) *reinterpret_cast<v4f*>(row + expert_of<L, C>(at, i)) = (v4f){0.f, 0.f, 0.f, 0.f};
  const float inner = lanes_sum<L>(w * dw);
  wave_lds_order();
  if (id >= 0) atomicAdd(row + id, w * (renorm ? dw - inner : dw));   // experts of a token are distinct
  wave_lds_order();
  float d[V];
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const v4f v = *reinterpret_cast<const v4f*>(row + expert_of<L, C>(at, i));
#pragma unroll
    for (int c = 0; c < 4; ++c) d[i + c] = v[c];
  }
  if (!renorm) {
    float top = -__builtin_inff(), total = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (expert_of<L, C>(at, i) < E) top = __builtin_fmaxf(top, x[i]);
    top = lanes_max<L>(top);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool counts = expert_of<L, C>(at, i) < E && x[i] != -__builtin_inff();
      x[i] = counts ? expf(x[i] - top) : 0.f;
      total += x[i];
    }
    total = lanes_sum<L>(total);
    const bool some = total != 0.f;                 // 0: a token without experts, no gradient (NaN with only NaN ones)
    const float share = inner / total;
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = some ? d[i] - x[i] * share : 0.f;
  }
  if (!here) return;
  store_logits<L, V>(dlogits + (size_t)t * E, E, at, wide, d);
}

int route_blocks(int T, int& chunks) {
  const int nc = (T + kTokensPerBlock - 1) / kTokensPerBlock;
  chunks = std::max(1, (nc + kMaxBlocks - 1) / kMaxBlocks);   // 1 for no tokens
  return (nc + chunks - 1) / chunks;
}

template <int L, int V, int D, typename TX>
hipError_t route_impl(const TX* logits, int T, int E, int k, int renorm, int* ids, float* weights, int* group_sizes,
                      int* row_of_slot, int* slot_of_row, void* hist, hipStream_t stream) {
  int chunks;
  const int nb = route_blocks(T, chunks);
  if (nb <= 1) {
    const int waves = std::max(1, (T + kTokensPerWave - 1) / kTokensPerWave);
    hipLaunchKernelGGL((route_topk_kernel<L, V, D, TX, true>), dim3(1), dim3(64 * waves), sizeof(int) * E * (waves + 1),
                       stream, logits, T, E, k, renorm, 1, ids, weights, row_of_slot, hist, group_sizes, slot_of_row);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((route_topk_kernel<L, V, D, TX, false>), dim3(nb), dim3(kThreads), sizeof(int) * E * (kWaves + 1),
                     stream, logits, T, E, k, renorm, chunks, ids, weights, row_of_slot, hist, group_sizes,
                     slot_of_row);
  hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  const int Ep = hist_row(E), C = chunks <= kByteChunks ? 16 : 8;
  int chunk_lanes = 1;
  while (chunk_lanes * C < Ep) chunk_lanes *= 2;
  const size_t place_lds = sizeof(int) * (size_t)Ep * (1 + 2 * std::min(kThreads / chunk_lanes, kWaves));
  if (chunks <= kByteChunks)
    hipLaunchKernelGGL(route_place_kernel<uint8_t>, dim3(nb), dim3(kThreads), place_lds, stream, ids,
                       static_cast<const uint8_t*>(hist), T, E, k, chunks, chunk_lanes, group_sizes, row_of_slot,
                       slot_of_row);
  else
    hipLaunchKernelGGL(route_place_kernel<uint16_t>, dim3(nb), dim3(kThreads), place_lds, stream, ids,
                       static_cast<const uint16_t*>(hist), T, E, k, chunks, chunk_lanes, group_sizes, row_of_slot,
                       slot_of_row);
  return hipGetLastError();
}

// A lane holds whole 16-byte chunks: 4 logits in f32, 8 in bf16.
template <typename TX>
hipError_t route_pick(const TX* logits, int T, int E, int k, int renorm, int* ids, float* weights, int* group_sizes,
                      int* row_of_slot, int* slot_of_row, void* hist, hipStream_t stream) {
  constexpr int C = 16 / (int)sizeof(TX);
#define ROUTE(L, V)                                                                                                    \
  (k <= 8 ? route_impl<L, V, V < 8 ? V : 8, TX>(logits, T, E, k, renorm, ids, weights, group_sizes, row_of_slot,       \
                                                slot_of_row, hist, stream)                                             \
          : route_impl<L, V, V, TX>(logits, T, E, k, renorm, ids, weights, group_sizes, row_of_slot, slot_of_row, hist, \
                                    stream))
  if (k <= 16) {
    if (E <= 16 * C) return ROUTE(16, C);
    if (E <= 128) return ROUTE(16, 8);              // f32 alone: 16 * C is 128 in bf16
    if (E <= 256) return ROUTE(16, 16);
  }
  if (E <= 64 * C) return ROUTE(64, C);
  if (E <= 512) return ROUTE(64, 8);                // f32 alone
  return ROUTE(64, 16);
#undef ROUTE
}

template <typename TX>
hipError_t route_bwd_pick(const float* dweights, const TX* logits, const int* ids, const float* weights, int T, int E,
                          int k, int renorm, TX* dlogits, hipStream_t stream) {
  constexpr int C = 16 / (int)sizeof(TX);
#define ROUTE(L, V)                                                                                               \
  hipLaunchKernelGGL((route_bwd_kernel<L, V, TX>), dim3((T + 256 / L - 1) / (256 / L)), dim3(256), 0, stream,      \
                     dweights, logits, ids, weights, T, E, k, renorm, dlogits)
  if (k <= 16 && E <= 16 * C) ROUTE(16, C);
  else if (k <= 16 && E <= 128) ROUTE(16, 8);       // f32 alone: 16 * C is 128 in bf16
  else if (k <= 16 && E <= 256) ROUTE(16, 16);
  else if (E <= 64 * C) ROUTE(64, C);
  else if (E <= 512) ROUTE(64, 8);                  // f32 alone
  else ROUTE(64, 16);
#undef ROUTE
  return hipGetLastError();
}

}  // namespace

size_t route_workspace_bytes(int T, int E) {
  int chunks;
  const int nb = T > 0 ? route_blocks(T, chunks) : 0;
  return nb <= 1 ? 0 : (chunks <= kByteChunks ? 1 : 2) * (size_t)nb * hist_row(E);
}

hipError_t launch_route(const void* logits, bool bf16, int T, int E, int k, bool renorm, int* ids, float* weights,
                        int* group_sizes, int* row_of_slot, int* slot_of_row, void* ws, hipStream_t stream) {
  if (bf16)
    return route_pick(static_cast<const uint16_t*>(logits), T, E, k, renorm, ids, weights, group_sizes, row_of_slot,
                      slot_of_row, ws, stream);
  return route_pick(static_cast<const float*>(logits), T, E, k, renorm, ids, weights, group_sizes, row_of_slot,
                    slot_of_row, ws, stream);
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
