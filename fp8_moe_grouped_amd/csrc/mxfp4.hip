// Microscaled 4-bit floating point (MXFP4): blocks of 32 values along K share
// one power of two.  With amax the block's largest magnitude,
//
//   power = max(floor(log2 amax) - 2, -127)      (-127 for a block of zeros)
//   scale = the E8M0 byte power + 127            (255, NaN, if the block holds Inf or NaN)
//   code  = e2m1(x / 2^power)                    nearest even, saturating at 6, signed zeros
//
// floor(log2 amax) + 127 is the exponent field of a normal f32, and a block whose
// amax is subnormal is clamped anyway, so the byte is max(field - 2, 0): integer
// arithmetic on the largest magnitude's bits.  The conversion instruction takes
// its scale from an f32's exponent field and rounds as above for every bf16
// value and every scale byte below 255 (field 0 is 2^-127).
//
// Codes [.., rows, K/2] hold the even k of a pair in the low half byte; scales
// [K/128, rows, 4] of weights put the four blocks of 128 k of a row in one word,
// which is what a lane of the scaled matrix instructions takes.
#include "moe_common.hpp"
#include "moe_launch.hpp"

namespace fp8gmm {
namespace {

// E8M0 byte of a block whose largest magnitude has the f32 bits `amax` (sign clear).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int field = (int)(amax >> 23);
  return field == 255 ? 255u : (uint32_t)max(field - 2, 0);
}

// Eight bf16 values in four words -> eight codes.
__device__ __forceinline__ uint32_t cvt_fp4x8(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, w0), s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, w1), s, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, w2), s, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, w3), s, 3);
  return q;
}

template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}

// Activations: one 16-byte chunk (8 values) per lane, four lanes a block of 32.  Scale rows
// are padded to 16 bytes.  Bound by HBM: 5000 x 7168 in 18 us, 91 MB at 5 TB/s.
// ROWS: x is the ragged buffer itself, and rows past the valid prefix are neither read nor
// written (the sizes cost 0.1 to 0.5 us of a product's call; 19661 valid rows of 32768 in a
// 2048 x 7168 product 268 -> 262 us).  Otherwise x holds tokens, all of which are quantized, and row T is written as
// zeros: the product reads it for rows without a token.
template <bool ROWS>
__global__ __launch_bounds__(256) void quant_rows_mxfp4_kernel(const v4i* __restrict__ x,
                                                              const int* __restrict__ group_sizes, int G, int T,
                                                              int nch, uint32_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
  const long long i = linear_block() * 256 + threadIdx.x;
  const long long end = (long long)(ROWS ? valid_rows_dpp(group_sizes, G, T) : T) * nch;
  if (i >= (ROWS ? end : end + nch)) return;
  const v4i v = i < end ? x[i] : (v4i){0, 0, 0, 0};
  uint32_t am = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = (uint32_t)v[e] & 0x7FFF7FFFu;
    am = max(am, max(w << 16, w & 0xFFFF0000u));
  }
  am = quad_max<0xB1>(am);                          // lanes 1 0 3 2
  am = quad_max<0x4E>(am);                          // lanes 2 3 0 1
  const uint32_t b = scale_byte(am);
  codes[i] = cvt_fp4x8(v[0], v[1], v[2], v[3], b);
  if ((threadIdx.x & 3) == 0) {
    const int t = (int)(i / nch), c = (int)(i % nch);
    scales[(size_t)t * ((nch + 63) / 64 * 16) + (c >> 2)] = (uint8_t)b;
  }
}

// Weights: a block turns a tile of 256 k x 128 n.  A lane owns two adjacent
// columns of 32 k, so a block of values lies in one lane; the codes pass through
// LDS so that they leave 128 bytes a row at a time.  Bound by HBM: 8 x 7168 x 2048 in
// 52 us, 297 MB at 5.7 TB/s.
constexpr int kTileK = 256, kTileN = 128;
constexpr int kRow = kTileK / 2 + 16;               // bytes of an LDS row

__global__ __launch_bounds__(256) void quant_weights_mxfp4_kernel(const uint32_t* __restrict__ w, int K, int N,
                                                                 uint8_t* __restrict__ codes,
                                                                 uint32_t* __restrict__ scales) {
  __shared__ __attribute__((aligned(16))) uint8_t lc[kTileN * kRow];
  __shared__ uint8_t ls[kTileK / 128][kTileN][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n0 = blockIdx.x * kTileN, k0 = blockIdx.y * kTileK, g = blockIdx.z;
  const int nb = min(kTileK, K - k0) / 32;          // blocks of 32 along K here: 4 or 8
  const uint32_t* src = w + ((size_t)g * K + k0) * (N / 2) + n0 / 2 + lane;
  for (int b = wave; b < nb; b += 4) {
    uint32_t v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __builtin_nontemporal_load(src + (size_t)(32 * b + i) * (N / 2));
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      lo = max(lo, (v[i] << 16) & 0x7FFFFFFFu);
      hi = max(hi, v[i] & 0x7FFF0000u);
    }
    const uint32_t b0 = scale_byte(lo), b1 = scale_byte(hi);
    const float s0 = __uint_as_float(b0 << 23), s1 = __uint_as_float(b1 << 23);
    v4i q0, q1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a = 0, c = 0;
#define PAIR(p)                                                                                                \
  a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, bf16_lo(v[8 * i + 2 * p]), bf16_lo(v[8 * i + 2 * p + 1]), s0, p); \
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, bf16_hi(v[8 * i + 2 * p]), bf16_hi(v[8 * i + 2 * p + 1]), s1, p);
      PAIR(0) PAIR(1) PAIR(2) PAIR(3)
#undef PAIR
      q0[i] = (int)a;
      q1[i] = (int)c;
    }
    *reinterpret_cast<v4i*>(lc + (2 * lane) * kRow + 16 * b) = q0;
    *reinterpret_cast<v4i*>(lc + (2 * lane + 1) * kRow + 16 * b) = q1;
    ls[b >> 2][2 * lane][b & 3] = (uint8_t)b0;
    ls[b >> 2][2 * lane + 1][b & 3] = (uint8_t)b1;
  }
  __syncthreads();
  uint8_t* dst = codes + ((size_t)g * N + n0) * (K / 2) + k0 / 2;
  const int c = tid & 7;
  if (c < nb)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = (tid >> 3) + 32 * i;
      *reinterpret_cast<v4i*>(dst + (size_t)n * (K / 2) + 16 * c) = *reinterpret_cast<const v4i*>(lc + n * kRow + 16 * c);
    }
  const int kk = tid >> 7, n = tid & 127;
  if (4 * kk < nb)
    scales[((size_t)g * (K / 128) + k0 / 128 + kk) * N + n0 + n] = *reinterpret_cast<const uint32_t*>(ls[kk][n]);
}

// Values of codes: 8 codes in, 16 bytes out per lane; a wave covers 512 k of a
// row, a block 16 rows (the rows whose scales share a 64-byte sector).  Bound by HBM:
// 8 x 2048 x 7168 in 44 us, 297 MB at 6.7 TB/s.
__global__ __launch_bounds__(256) void dequant_mxfp4_kernel(const uint32_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int N, int K,
                                                           v4i* __restrict__ out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nch = K / 8, c = blockIdx.x * 64 + lane;
  const int g = blockIdx.z;
  if (c >= nch) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = blockIdx.y * 16 + 4 * i + wave;   // N is a multiple of 128
    const size_t row = (size_t)g * N + n;
    const uint32_t q = __builtin_nontemporal_load(codes + row * nch + c);
    const uint32_t b = scales[(((size_t)g * (K / 128) + (c >> 4)) * N + n) * 4 + ((c >> 2) & 3)];
    const float s = __uint_as_float(b << 23);
    v4i o;
    o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
    o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
    o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
    o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
    __builtin_nontemporal_store(o, out + row * nch + c);
  }
}

}  // namespace

hipError_t launch_quant_rows_mxfp4(const uint16_t* x, const int* group_sizes, int G, int T, int K, uint8_t* codes,
                                   uint8_t* scales, hipStream_t stream) {
  const int nch = K / 8;
  const long long rows = group_sizes ? T : (long long)T + 1;
  const dim3 grid = linear_grid((rows * nch + 255) / 256);
  const v4i* xv = reinterpret_cast<const v4i*>(x);
  uint32_t* cv = reinterpret_cast<uint32_t*>(codes);
  if (group_sizes)
    hipLaunchKernelGGL(quant_rows_mxfp4_kernel<true>, grid, dim3(256), 0, stream, xv, group_sizes, G, T, nch, cv, scales);
  else
    hipLaunchKernelGGL(quant_rows_mxfp4_kernel<false>, grid, dim3(256), 0, stream, xv, group_sizes, G, T, nch, cv,
                       scales);
  return hipGetLastError();
}

hipError_t launch_quant_weights_mxfp4(const uint16_t* w, int G, int K, int N, uint8_t* codes, uint8_t* scales,
                                      hipStream_t stream) {
  hipLaunchKernelGGL(quant_weights_mxfp4_kernel, dim3(N / kTileN, (K + kTileK - 1) / kTileK, G), dim3(256), 0, stream,
                     reinterpret_cast<const uint32_t*>(w), K, N, codes, reinterpret_cast<uint32_t*>(scales));
  return hipGetLastError();
}

hipError_t launch_dequant_mxfp4(const uint8_t* codes, const uint8_t* scales, int G, int N, int K, uint16_t* out,
                                hipStream_t stream) {
  hipLaunchKernelGGL(dequant_mxfp4_kernel, dim3((K / 8 + 63) / 64, N / 16, G), dim3(256), 0, stream,
                     reinterpret_cast<const uint32_t*>(codes), scales, N, K, reinterpret_cast<v4i*>(out));
  return hipGetLastError();
}

}  // namespace fp8gmm
