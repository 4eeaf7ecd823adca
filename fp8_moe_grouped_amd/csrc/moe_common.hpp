// Device helpers of the kernels around the grouped products (routing, dispatch, combine,
// 4-bit): copies, long grids, reductions and scans over lanes without LDS.  They stand
// apart from common.hpp, whose text belongs to the FP8 kernels' measured traffic.
#pragma once
#include "common.hpp"

namespace fp8gmm {

// ----------------------------------------------------------------- copies to LDS

// Direct copies to LDS, as dma16 and dma4, from a 64-bit address of each lane: 16 bytes or 4.
#define GLOBAL_PTR(p) ((__attribute__((address_space(1))) void*)(p))
__device__ __forceinline__ void copy16(const void* src, void* lds_wave_base) {
  __builtin_amdgcn_global_load_lds(GLOBAL_PTR(const_cast<void*>(src)), LDS_PTR(void, lds_wave_base), 16, 0, 0);
}
__device__ __forceinline__ void copy4(const void* src, void* lds_wave_base) {
  __builtin_amdgcn_global_load_lds(GLOBAL_PTR(const_cast<void*>(src)), LDS_PTR(void, lds_wave_base), 4, 0, 0);
}

// ----------------------------------------------------------------- long grids

// A launch dimension holds fewer than 2^32 threads: longer grids continue in y.  Blocks past the last one exist, so a
// kernel checks its index.
inline dim3 linear_grid(long long blocks, int threads = 256) {
  const long long kWide = (1LL << 31) / threads;
  if (blocks <= kWide) return dim3((unsigned)blocks);
  return dim3((unsigned)kWide, (unsigned)((blocks + kWide - 1) / kWide));
}
__device__ __forceinline__ long long linear_block() { return (long long)blockIdx.y * gridDim.x + blockIdx.x; }

// ----------------------------------------------------------------- reductions and scans

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_row(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_row(float v) {
  return __uint_as_float(dpp_row<CTRL>(__float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp_row(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp_row<CTRL>((uint32_t)u) | (uint64_t)dpp_row<CTRL>((uint32_t)(u >> 32)) << 32);
}
// v of the lane whose row index differs in bit 0 (B = 16) or bit 1 (B = 32): exchanges rows or halves.
template <int B>
__device__ __forceinline__ uint32_t other_rows(uint32_t v, bool upper) {
  if (B == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return upper ? r[0] : r[1];
  }
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return upper ? r[0] : r[1];
}
template <int B>
__device__ __forceinline__ float other_rows(float v, bool upper) {
  return __uint_as_float(other_rows<B>(__float_as_uint(v), upper));
}
template <int B>
__device__ __forceinline__ double other_rows(double v, bool upper) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)other_rows<B>((uint32_t)u, upper) |
                                        (uint64_t)other_rows<B>((uint32_t)(u >> 32), upper) << 32);
}

// Reduction over the rows of 16 lanes (L = 16) or the wave (64), to all of their lanes, without LDS: rotations
// within a row, then exchanges of rows.  Every lane joins the same pairs, so all hold the same sum.
template <int L, typename T, typename F>
__device__ __forceinline__ T reduce(T v, F f) {
  v = f(v, dpp_row<0x128>(v));
  v = f(v, dpp_row<0x124>(v));
  v = f(v, dpp_row<0x122>(v));
  v = f(v, dpp_row<0x121>(v));
  if (L == 64) {
    v = f(v, other_rows<16>(v, (threadIdx.x & 16) != 0));
    v = f(v, other_rows<32>(v, (threadIdx.x & 32) != 0));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  return reduce<L>(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {     // lanes without a source add 0
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
// Inclusive prefix sum across the wave without LDS.
__device__ __forceinline__ int wave_scan_dpp(int v) {
  v = dpp_add<0x111, 0xF>(v);                       // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);                       // row_bcast 15 into rows 1 and 3
  return dpp_add<0x143, 0xC>(v);                    // row_bcast 31 into rows 2 and 3
}

// valid_rows of common.hpp without LDS.  A lane's sum stays at or below M < 2^24, the wave's below 2^30.
__device__ __forceinline__ int valid_rows_dpp(const int* __restrict__ group_sizes, int G, int M) {
  int s = 0;
  for (int g = (int)(threadIdx.x & 63); g < G; g += 64) s = min(s + min(max(group_sizes[g], 0), M), M);
  return min(__builtin_amdgcn_readlane(wave_scan_dpp(s), 63), M);
}

}  // namespace fp8gmm
