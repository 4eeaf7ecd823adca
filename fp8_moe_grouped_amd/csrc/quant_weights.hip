// Master weights w [G, K, N] to the FP8 calls' codes and scales, one scale per output
// channel over all K:
//   scale[g, n] = f32(max(max_k |w|, 1e-12) / 448),   code = e4m3fn(f32(w / scale))
//
// The quotient never passes 448 by more than a rounding, which the conversion brings back,
// so nothing is clamped and a NaN stays one.
//
// Bound by HBM: 5 bytes an element in f32.  A strip of 64 columns or more keeps reads and codes in
// whole half-lines or more: with 16 columns the codes' 16-byte pieces took as long as half of
// the reads (8 x 7168 x 4096 f32: 357 us, 228 without the stores).  128 columns of 7168 rows are
// 3.7 MB, eight times a CU's registers, so a strip's rows are shared by blocks that exchange
// their maxima (229 us in a row of calls, 5.1 TB/s; two passes over the weights 960).  Weights of
// one round of blocks (8 x 768 x 2048 bf16, 12.3 us) wait for HBM twice: in the compiled
// kernels a block's first two loads arrive before the rest go out.
#include "moe_common.hpp"
#include "moe_launch.hpp"

#include <type_traits>

namespace fp8gmm {
namespace {

// x / s, correctly rounded, from r = 1/s: two corrections, each with the exact remainder (the first brings the
// quotient within a step of the truth, where the second rounds it as a division would).  The remainder comes negated,
// which keeps the sign of a zero.  s is finite and at least 1e-12 / 448; remainders are subnormal only where the code is
// 0 whatever they are.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = div_by_scale(x, s, r);
  return __builtin_fmaf(-__builtin_fmaf(q, s, -x), r, q);
}

typedef uint16_t v8u __attribute__((ext_vector_type(8)));

// A chunk of 16 bytes: 4 f32 or 8 bf16.
template <typename TW>
__device__ __forceinline__ float element(const v4i& w, int c) {
  if constexpr (sizeof(TW) == 4) return __uint_as_float((uint32_t)w[c]);
  else return c & 1 ? bf16_hi((uint32_t)w[c / 2]) : bf16_lo((uint32_t)w[c / 2]);
}

// Largest magnitude over the lanes that hold the same chunk of a row: every LPR-th of the wave.
template <int LPR>
__device__ __forceinline__ float same_columns_max(float v) {
  const auto f = [](float a, float b) { return __builtin_fmaxf(a, b); };
  if (LPR <= 4) v = f(v, dpp_row<0x124>(v));        // rotations by 4 and 8 within 16 lanes
  if (LPR <= 8) v = f(v, dpp_row<0x128>(v));
  if (LPR <= 16) v = f(v, other_rows<16>(v, (threadIdx.x & 16) != 0));
  if (LPR <= 32) v = f(v, other_rows<32>(v, (threadIdx.x & 32) != 0));
  return v;
}

constexpr int kTogether = 4;                        // strips side by side that one XCD takes

// A block keeps M chunks a thread, a strip of LPR chunks x kRows * M rows, in its registers, so that the weights are
// read once.  Where that is not all of K (parts > 1), the strip's blocks tell each other their columns' largest
// magnitudes through `words` [total][parts][columns], zero at first: the magnitude's bits and one, published and read as
// one word, so that no other order matters.  The blocks of a strip follow each other on one XCD and
// run at the same time; where a thread waited in vain for `polls` looks, it reads the rows of that block instead and looks
// once for each of the rest, so every wait ends.
template <typename TW, int THREADS, int LPR, int M>
__global__ __launch_bounds__(THREADS, 4) void quant_weights_fp8_kernel(const TW* __restrict__ w, int K, int N, int strips,
                                                                       int total, int parts, int each, int polls,
                                                                       uint32_t* __restrict__ words,
                                                                       uint8_t* __restrict__ codes,
                                                                       float* __restrict__ scales) {
  constexpr int C = 16 / (int)sizeof(TW), kRows = THREADS / LPR, kWaves = THREADS / 64, kColumns = LPR * C;
  __shared__ __attribute__((aligned(16))) float tops[kWaves][kColumns];
  const int tid = threadIdx.x, col = tid % LPR * C, wave = tid >> 6;
  // Blocks go to the 8 XCDs in turn: an XCD takes a strip's parts one after the other, and every 8th group of strips,
  // so that all work on neighbouring columns (an XCD with an expert of its own: 270 us instead of 243).
  const long long b = linear_block();
  const int slot = (int)(b / 8), turn = slot / parts, part = slot % parts;
  const int strip = (turn / kTogether * 8 + (int)(b % 8)) * kTogether + turn % kTogether;
  if (strip >= total) return;
  const int g = strip / strips, n = strip % strips * kColumns + col;
  const int first = part * each, end = min(K, first + each);
  // A wave's rows are inside or outside together.  Its addresses are a uniform part and 32 bits of each lane
  // (at most 16 rows of N < 2^24), so that M of them need no registers.
  const int row = first + tid / LPR, wave_row = __builtin_amdgcn_readfirstlane(row);
  const size_t base = (size_t)g * K * N + (size_t)wave_row * N + (n - col);
  const uint32_t lane_at = (uint32_t)(row - wave_row) * (uint32_t)N + (uint32_t)col;
  const char* const from = reinterpret_cast<const char*>(w + base);
  v4i x[M];
#pragma unroll
  for (int i = 0; i < M; ++i)
    if (wave_row + i * kRows < end)
      x[i] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(from + (size_t)i * kRows * N * sizeof(TW) +
                                                                     lane_at * (uint32_t)sizeof(TW)));
    else
      x[i] = (v4i){0, 0, 0, 0};
  float top[C] = {};
  const auto largest = [&] {
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c) top[c] = __builtin_fmaxf(top[c], __builtin_fabsf(element<TW>(x[i], c)));
  };
  if constexpr (C == 4) {
    largest();
  } else {                                          // magnitudes are ordered as their bits are, two at a time
    v8u t = {};
    const v8u most = 0x7F80;
#pragma unroll
    for (int i = 0; i < M; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(v8u, x[i]) & (uint16_t)0x7FFF);
    bool nan = false;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      nan = nan || t[c] > most[c];
      top[c] = __uint_as_float((uint32_t)t[c] << 16);
    }
    if (nan) {                                      // which does not count
#pragma unroll
      for (int c = 0; c < C; ++c) top[c] = 0.f;
      largest();
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    top[c] = same_columns_max<LPR>(top[c]);
    if ((tid & 63) < LPR) tops[wave][col + c] = top[c];
  }
  __syncthreads();
  constexpr int kGroups = THREADS / kColumns < kWaves ? THREADS / kColumns : kWaves;
  if (parts > 1) {                                  // group 0 has the block's own, each group some of the others'
    const int column = tid % kColumns, group = tid / kColumns;
    float most = 0.f;
    if (group < kGroups) {
      uint32_t* const mine = words + (size_t)strip * parts * kColumns + column;
      const auto publish = [&](int q, float top) {
        __hip_atomic_store(mine + q * kColumns, __float_as_uint(top) + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      };
      if (group == 0) {
#pragma unroll
        for (int v = 0; v < kWaves; ++v) most = __builtin_fmaxf(most, tops[v][column]);
        publish(part, most);
      }
      int looks = polls;
      for (int o = 1 + group; o < parts; o += kGroups) {
        const int q = part + o < parts ? part + o : part + o - parts;
        uint32_t word = 0;
        for (int tries = 0; tries < looks && !word; ++tries) {
          word = __hip_atomic_load(mine + q * kColumns, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          if (!word) __builtin_amdgcn_s_sleep(4);
        }
        if (word) {
          most = __builtin_fmaxf(most, __uint_as_float(word - 1));
        } else {
          looks = min(looks, 1);
          const TW* const others = w + (size_t)g * K * N + (n - col) + column;
          const int stop = min(K, (q + 1) * each);
          float there = 0.f;
#pragma unroll 2                                    // 4 or 8: their registers cost every call 5 or 8 %
          for (int k = q * each; k < stop; ++k) {
            float v;
            if constexpr (C == 4) v = others[(size_t)k * N];
            else v = __uint_as_float((uint32_t)others[(size_t)k * N] << 16);
            there = __builtin_fmaxf(there, __builtin_fabsf(v));
          }
          most = __builtin_fmaxf(most, there);
          publish(q, there);
        }
      }
    }
    __syncthreads();
    if (group < kGroups) tops[group][column] = most;
    __syncthreads();
  }
  const int rows_of_tops = parts > 1 ? kGroups : kWaves;
  float scale[C], inverse[C];
  bool finite = true;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float t = kAmaxFloor;
#pragma unroll
    for (int v = 0; v < kWaves; ++v)
      if (v < rows_of_tops) t = __builtin_fmaxf(t, tops[v][col + c]);
    scale[c] = t / kE4M3Max;
    inverse[c] = 1.f / scale[c];
    finite = finite && __builtin_isfinite(scale[c]);
    if (row == 0) scales[(size_t)g * N + n + c] = scale[c];
  }
  const auto put = [&](auto fast) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      if (wave_row + i * kRows >= end) continue;
      int q[C / 4];
#pragma unroll
      for (int c = 0; c < C; c += 4) {
        float e[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float v = element<TW>(x[i], c + d);
          if constexpr (!decltype(fast)::value) e[d] = v / scale[c + d];
          else if constexpr (C == 4) e[d] = quotient(v, scale[c + d], inverse[c + d]);
          else e[d] = div_by_scale(v, scale[c + d], inverse[c + d]);   // enough for bf16 values and their scales
        }
        const int low = __builtin_amdgcn_cvt_pk_fp8_f32(e[0], e[1], 0, false);
        q[c / 4] = __builtin_amdgcn_cvt_pk_fp8_f32(e[2], e[3], low, true);
      }
      uint8_t* const to = codes + base + (size_t)i * kRows * N + lane_at;
      if constexpr (C == 4) *reinterpret_cast<int*>(to) = q[0];
      else *reinterpret_cast<v2i*>(to) = (v2i){q[0], q[C / 4 - 1]};
    }
  };
  if (finite) put(std::true_type{});
  else put(std::false_type{});
}

__global__ __launch_bounds__(256) void clear_words_kernel(v4i* __restrict__ words, long long n) {
  const long long i = linear_block() * 256 + threadIdx.x;
  if (i < n) words[i] = (v4i){0, 0, 0, 0};
}

// A strip's lanes and a thread's chunks, by how many elements a CU has: wide strips for whole lines of codes, narrow
// ones for enough blocks; more chunks where one part less, of one or two, is left to wait for.  Both sides in us:
//   f32   128 columns or 64: 8 x 7168 x 3840 240, 257; 8 x 3200 x 3328 92, 86
//         64 or 32: 2 x 2304 x 896 12.6, 9.9; 4 x 2176 x 1792 21.9, 22.2;   32 or 16: 2 x 768 x 1664 6.7, 5.8;
//         1 x 2048 x 768 10.2, 8.4
//   bf16  128 or 64: 8 x 7168 x 3840 149, 169; 4 x 4096 x 3584 44.6, 42.6;   64 or 32: 8 x 768 x 2048 12.2, 13.4;
//         4 x 6656 x 256 15.4, 11.2
//   16 chunks or 24: 7 x 1280 x 1536 bf16 18.1, 14.9; 4 x 2432 x 2688 29.6, 25.0; but 6 x 3968 x 1920 33.7, 41.7
//   8 or 16: 2 x 1408 x 1408 f32 11.1, 8.5; 1 x 1536 x 2048 bf16 8.7, 7.8; but 1 x 6144 x 768 11.4, 14.6
// A block of 512 threads keeps 384 rows of 128 columns in f32; of 64 and 32 columns there 768 and 1024, of 128 and 64 in
// bf16 768 and 1024 or 1536, of the narrowest 1024 or 2048.  A strip's parts get the same number of rows, within a
// block's step (7 x 4864 x 1920 bf16 51.9 -> 49.1).
// An XCD has room for 64 blocks.  Calls on several streams each fill it with what is ready and may leave each other's
// strips half in: strips of at most kMostParts leave room for two (two of 8 x 16384 x 4096 at once 1.4 ms; in strips of
// 43 parts 150 and more, every block waiting and reading for the others).
constexpr int kThreads = 512;
constexpr int kMostParts = 24;                      // 128 columns or 64: 8 x 16384 x 4096 656, 665
constexpr int kWideRows = 384, kOtherRows = 768;    // of 128 columns in f32, and of any other cut at least
constexpr int kWideK = kMostParts * kWideRows;      // the most that strips of 128 columns in f32 are taken for
static_assert(kMaxK <= kMostParts * kOtherRows, "longer columns have more parts than two calls at once have room for");
template <typename TW, int LPR, int M>
hipError_t run(const TW* w, int G, int K, int N, int polls, uint8_t* codes, float* scales, uint32_t* words,
               hipStream_t stream) {
  constexpr int kRows = kThreads / LPR, kMost = kRows * M;
  static_assert(kMost >= (LPR == 32 ? kWideRows : kOtherRows), "the workspace is counted for these");
  const int strips = N / (LPR * 16 / (int)sizeof(TW)), total = strips * G, parts = (K + kMost - 1) / kMost;
  const int each = ((K + parts - 1) / parts + kRows - 1) / kRows * kRows;   // rows of a part
  if (parts > 1) {
    const long long n = (long long)G * N * parts / 4;
    hipLaunchKernelGGL(clear_words_kernel, linear_grid((n + 255) / 256), dim3(256), 0, stream,
                       reinterpret_cast<v4i*>(words), n);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
  }
  constexpr int kAll = 8 * kTogether;
  hipLaunchKernelGGL((quant_weights_fp8_kernel<TW, kThreads, LPR, M>),
                     linear_grid((long long)((total + kAll - 1) / kAll * kAll) * parts, kThreads), dim3(kThreads), 0, stream, w,
                     K, N, strips, total, parts, each, polls, words, codes, scales);
  return hipGetLastError();
}

template <typename TW>
hipError_t quantize(const TW* w, int G, int K, int N, int polls, uint8_t* codes, float* scales, uint32_t* words,
                    hipStream_t stream) {
  const long long each = (long long)G * K * N / device_cu_count();
  const auto parts = [K](int rows) { return (K + rows - 1) / rows; };
#define RUN(L, M) run<TW, L, M>(w, G, K, N, polls, codes, scales, words, stream)
  if constexpr (sizeof(TW) == 4) {
    if (each >= 1 << 19 && K <= kWideK) return RUN(32, 24);
    if (each >= 1 << 16) return RUN(16, 24);
    if (each >= 1 << 13) return RUN(8, 16);
  } else {
    if (each >= 1 << 18) return RUN(16, 24);
    if (each >= 1 << 15) return parts(1536) <= 2 && parts(1536) < parts(1024) ? RUN(8, 24) : RUN(8, 16);
  }
  return parts(2048) == 1 && parts(1024) == 2 ? RUN(4, 16) : RUN(4, 8);
#undef RUN
}

}  // namespace

size_t quant_weights_workspace_bytes(bool bf16, int G, int K, int N) {
  // the most that any cut of these columns needs: a device with another number of CUs gives the same answer
  const size_t rows = !bf16 && K <= kWideK ? kWideRows : kOtherRows, parts = (K + rows - 1) / rows;
  return parts > 1 ? 4 * (size_t)G * N * parts : 0;
}

hipError_t launch_quant_weights_fp8(const void* w, bool bf16, int G, int K, int N, uint8_t* codes, float* scales,
                                    void* ws, int polls, hipStream_t stream) {
  uint32_t* const words = static_cast<uint32_t*>(ws);
  if (bf16) return quantize(static_cast<const uint16_t*>(w), G, K, N, polls, codes, scales, words, stream);
  return quantize(static_cast<const float*>(w), G, K, N, polls, codes, scales, words, stream);
}

}  // namespace fp8gmm
