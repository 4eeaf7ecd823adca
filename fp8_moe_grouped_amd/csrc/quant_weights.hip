// Master weights w [G, K, N] to the FP8 calls' codes and scales, one scale per output
// channel over all K:
//   scale[g, n] = f32(max(max_k |w|, 1e-12) / 448),   code = e4m3fn(f32(w / scale))
//
// The quotient never passes 448 by more than a rounding, which the conversion brings back,
// so nothing is clamped and a NaN stays one.
#include "moe_common.hpp"
#include "moe_launch.hpp"

namespace fp8gmm {
namespace {

constexpr int kThreads = 256;
constexpr int kColumns = 128;                       // a block's strip
constexpr int kRows = kThreads * 4 / kColumns;

__device__ __forceinline__ v4f load4(const float* p) { return *reinterpret_cast<const v4f*>(p); }
__device__ __forceinline__ v4f load4(const uint16_t* p) {
  const v2i w = *reinterpret_cast<const v2i*>(p);
  return (v4f){bf16_lo((uint32_t)w[0]), bf16_hi((uint32_t)w[0]), bf16_lo((uint32_t)w[1]), bf16_hi((uint32_t)w[1])};
}

template <typename TW>
__global__ __launch_bounds__(kThreads) void quant_weights_fp8_kernel(const TW* __restrict__ w, int K, int N,
                                                                     uint8_t* __restrict__ codes,
                                                                     float* __restrict__ scales) {
  __shared__ __attribute__((aligned(16))) float tops[kRows][kColumns];
  const int tid = threadIdx.x, col = tid % (kColumns / 4) * 4, row = tid / (kColumns / 4);
  const int n = blockIdx.x * kColumns + col;
  const size_t base = (size_t)blockIdx.y * K * N + n;
  v4f top = {0.f, 0.f, 0.f, 0.f};
  for (int k = row; k < K; k += kRows) {
    const v4f x = load4(w + base + (size_t)k * N);
#pragma unroll
    for (int c = 0; c < 4; ++c) top[c] = __builtin_fmaxf(top[c], __builtin_fabsf(x[c]));
  }
  *reinterpret_cast<v4f*>(&tops[row][col]) = top;
  __syncthreads();
  v4f scale;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float t = kAmaxFloor;
#pragma unroll
    for (int r = 0; r < kRows; ++r) t = __builtin_fmaxf(t, tops[r][col + c]);
    scale[c] = t / kE4M3Max;
  }
  if (row == 0) *reinterpret_cast<v4f*>(scales + (size_t)blockIdx.y * N + n) = scale;
  for (int k = row; k < K; k += kRows) {
    const v4f x = load4(w + base + (size_t)k * N);
    int q = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] / scale[0], x[1] / scale[1], 0, false);
    q = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] / scale[2], x[3] / scale[3], q, true);
    *reinterpret_cast<int*>(codes + base + (size_t)k * N) = q;
  }
}

}  // namespace

hipError_t launch_quant_weights_fp8(const void* w, bool bf16, int G, int K, int N, uint8_t* codes, float* scales,
                                    hipStream_t stream) {
  const dim3 grid(N / kColumns, G);
  if (bf16)
    hipLaunchKernelGGL(quant_weights_fp8_kernel<uint16_t>, grid, dim3(kThreads), 0, stream,
                       static_cast<const uint16_t*>(w), K, N, codes, scales);
  else
    hipLaunchKernelGGL(quant_weights_fp8_kernel<float>, grid, dim3(kThreads), 0, stream, static_cast<const float*>(w),
                       K, N, codes, scales);
  return hipGetLastError();
}

}  // namespace fp8gmm
