// Between the tokens and the ragged buffer of a mixture-of-experts layer: a
// token's row to the k rows of its choices (permute), the experts' rows back to
// the token with the router's weights (combine), and combine's gradient.  With
// row = row_of_slot[t*k + j]:
//
//   permute      out[row]  = x[t]
//   permute_fp8  codes[row], scales[row] = the e4m3 codes and row scale of x[t],
//                as quantize_rows_fp8 gives them for the permuted row
//   combine      out[t]    = bf16( sum_j w[t,j] * y[row] )    f32, j ascending
//   combine_bwd  dy[row]   = bf16( w[t,j] * dout[t] ),  dw[t,j] = sum_h dout[t,h] y[row,h]
//
// A row outside [0, R) (a masked choice holds -1) is neither read nor written
// and counts as zero.  All are bound by HBM: every token's row is read once and
// every expert row is touched once, in 16-byte chunks, with the streaming policy on
// the k times larger side, which is not read again before it has left the caches:
// 4096 x 7168, k = 8: permute 91 us (5.8 TB/s; 106 without the policy), combine 90
// (5.9 TB/s; 104), its gradient 188 (5.3 TB/s; 200).
#include "moe_common.hpp"
#include "moe_launch.hpp"

#include <type_traits>

namespace fp8gmm {
namespace {

// One wave per (token, piece of 64 chunks).
__global__ __launch_bounds__(256) void permute_kernel(const v4i* __restrict__ x, const int* __restrict__ row_of_slot,
                                                      int T, int k, int R, int nch, int pieces,
                                                      v4i* __restrict__ out) {
  const long long unit = linear_block() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (int)(unit / pieces);
  if (t >= T) return;
  const int c = (int)(unit % pieces) * 64 + (threadIdx.x & 63);
  if (c >= nch) return;
  const v4i v = x[(size_t)t * nch + c];
  for (int j = 0; j < k; ++j) {
    const int row = row_of_slot[(size_t)t * k + j];
    if ((unsigned)row < (unsigned)R) __builtin_nontemporal_store(v, out + (size_t)row * nch + c);
  }
}

// One wave per token: the row stays in registers between its amax and its codes.
template <int CPL>
__global__ __launch_bounds__(256) void permute_fp8_kernel(const uint16_t* __restrict__ x,
                                                          const int* __restrict__ row_of_slot, int T, int k, int R,
                                                          int H, uint8_t* __restrict__ codes,
                                                          float* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= T) return;
  const int nch = H >> 3;
  const BufRsrc rsrc = make_rsrc(x + (size_t)t * H, (uint32_t)H * 2u);   // chunks past the row read as zeros
  v4i v[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c)
    v[c] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rsrc, (uint32_t)lane * 16u,
                                                                         (uint32_t)c * 1024u, 0));
  float am = 0.f;
#pragma unroll
  for (int c = 0; c < CPL; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = (uint32_t)v[c][e];
      am = __builtin_fmaxf(am, __builtin_fabsf(bf16_lo(w)));
      am = __builtin_fmaxf(am, __builtin_fabsf(bf16_hi(w)));
    }
  const float s = __builtin_fmaxf(wave_max(am), kAmaxFloor) / kE4M3Max;   // IEEE f32 division
  const float r = 1.0f / s;
  v2i q[CPL];
  auto quantize = [&](auto fast_c) {
    constexpr bool FAST = decltype(fast_c)::value;
    auto quo = [&](float a) { return FAST ? div_by_scale(a, s, r) : a / s; };
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const uint32_t w0 = v[c][0], w1 = v[c][1], w2 = v[c][2], w3 = v[c][3];
      q[c][0] = (int)cvt_e4m3x4(quo(bf16_lo(w0)), quo(bf16_hi(w0)), quo(bf16_lo(w1)), quo(bf16_hi(w1)));
      q[c][1] = (int)cvt_e4m3x4(quo(bf16_lo(w2)), quo(bf16_hi(w2)), quo(bf16_lo(w3)), quo(bf16_hi(w3)));
    }
  };
  if (__builtin_isfinite(s)) quantize(std::true_type{});
  else quantize(std::false_type{});
  for (int j = 0; j < k; ++j) {
    const int row = row_of_slot[(size_t)t * k + j];
    if ((unsigned)row >= (unsigned)R) continue;
    v2i* dst = reinterpret_cast<v2i*>(codes + (size_t)row * H);
#pragma unroll
    for (int c = 0; c < CPL; ++c)
      if (lane + 64 * c < nch) __builtin_nontemporal_store(q[c], dst + lane + 64 * c);
    if (lane == 0) scales[row] = s;
  }
}

// One wave per (token, piece of 64 chunks).
template <bool WEIGHTED>
__global__ __launch_bounds__(256) void combine_kernel(const v4i* __restrict__ y, const int* __restrict__ row_of_slot,
                                                      const float* __restrict__ weights, int T, int k, int R, int nch,
                                                      int pieces, v4i* __restrict__ out) {
  const long long unit = linear_block() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (int)(unit / pieces);
  if (t >= T) return;
  const int c = (int)(unit % pieces) * 64 + (threadIdx.x & 63);
  if (c >= nch) return;
  float a[8] = {};
  for (int j0 = 0; j0 < k; j0 += 8) {               // eight rows' loads in flight
    v4i v[8];
    float w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int row = j0 + u < k ? row_of_slot[(size_t)t * k + j0 + u] : -1;
      v[u] = (v4i){0, 0, 0, 0};
      w[u] = 0.f;
      if ((unsigned)row < (unsigned)R) {
        v[u] = __builtin_nontemporal_load(y + (size_t)row * nch + c);
        w[u] = WEIGHTED ? weights[(size_t)t * k + j0 + u] : 1.f;
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = bf16_lo((uint32_t)v[u][e]), hi = bf16_hi((uint32_t)v[u][e]);
        a[2 * e] = WEIGHTED ? __builtin_fmaf(w[u], lo, a[2 * e]) : a[2 * e] + lo;
        a[2 * e + 1] = WEIGHTED ? __builtin_fmaf(w[u], hi, a[2 * e + 1]) : a[2 * e + 1] + hi;
      }
  }
  v4i o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = (int)pack_bf16x2(a[2 * e], a[2 * e + 1]);
  out[(size_t)t * nch + c] = o;
}

// One block per token, eight of its rows at a time: dout is read once for them, the
// waves share the width and join their dot products in a fixed order.
__global__ __launch_bounds__(256) void combine_bwd_kernel(const v4i* __restrict__ dout, const v4i* __restrict__ y,
                                                          const int* __restrict__ row_of_slot,
                                                          const float* __restrict__ weights, int k, int R, int nch,
                                                          v4i* __restrict__ dy, float* __restrict__ dweights) {
  __shared__ float part[2][4][8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, t = blockIdx.x;
  const v4i* const d = dout + (size_t)t * nch;
  for (int j0 = 0; j0 < k; j0 += 8) {
    int row[8];
    float w[8], dot[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      row[u] = j0 + u < k ? row_of_slot[(size_t)t * k + j0 + u] : -1;
      w[u] = j0 + u < k ? weights[(size_t)t * k + j0 + u] : 0.f;
      dot[u] = 0.f;
    }
    for (int c = tid; c < nch; c += 256) {
      const v4i g = d[c];
      v4i v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        v[u] = (v4i){0, 0, 0, 0};
        if ((unsigned)row[u] < (unsigned)R) v[u] = __builtin_nontemporal_load(y + (size_t)row[u] * nch + c);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if ((unsigned)row[u] >= (unsigned)R) continue;
        v4i r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float g0 = bf16_lo((uint32_t)g[e]), g1 = bf16_hi((uint32_t)g[e]);
          dot[u] = __builtin_fmaf(g0, bf16_lo((uint32_t)v[u][e]), dot[u]);
          dot[u] = __builtin_fmaf(g1, bf16_hi((uint32_t)v[u][e]), dot[u]);
          r[e] = (int)pack_bf16x2(w[u] * g0, w[u] * g1);
        }
        __builtin_nontemporal_store(r, dy + (size_t)row[u] * nch + c);
      }
    }
    float(&p)[4][8] = part[(j0 >> 3) & 1];          // the other half may still be read
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float sum = reduce<64>(dot[u], [](float a, float b) { return a + b; });
      if (lane == u) p[wave][u] = sum;
    }
    __syncthreads();
    if (tid < 8 && j0 + tid < k) dweights[(size_t)t * k + j0 + tid] = (p[0][tid] + p[1][tid]) + (p[2][tid] + p[3][tid]);
  }
}

long long blocks_of(long long units) { return (units + 3) / 4; }

}  // namespace

hipError_t launch_permute(const uint16_t* x, const int* row_of_slot, int T, int k, int R, int H, uint16_t* out,
                          hipStream_t stream) {
  const int nch = H / 8, pieces = (nch + 63) / 64;
  hipLaunchKernelGGL(permute_kernel, linear_grid(blocks_of((long long)T * pieces)), dim3(256), 0, stream,
                     reinterpret_cast<const v4i*>(x), row_of_slot, T, k, R, nch, pieces, reinterpret_cast<v4i*>(out));
  return hipGetLastError();
}

hipError_t launch_permute_fp8(const uint16_t* x, const int* row_of_slot, int T, int k, int R, int H, uint8_t* codes,
                              float* scales, hipStream_t stream) {
  const int cpl = (H / 8 + 63) / 64;
#define PLAUNCH(C)                                                                                               \
  hipLaunchKernelGGL(permute_fp8_kernel<C>, dim3((unsigned)blocks_of(T)), dim3(256), 0, stream, x, row_of_slot, T, k, R, H, \
                     codes, scales)
  if (cpl <= 1) PLAUNCH(1);
  else if (cpl <= 2) PLAUNCH(2);
  else if (cpl <= 4) PLAUNCH(4);
  else if (cpl <= 8) PLAUNCH(8);
  else if (cpl <= 16) PLAUNCH(16);
  else if (cpl <= 32) PLAUNCH(32);
  else return hipErrorInvalidValue;
#undef PLAUNCH
  return hipGetLastError();
}

hipError_t launch_combine(const uint16_t* y, const int* row_of_slot, const float* weights, int T, int k, int R, int H,
                          uint16_t* out, hipStream_t stream) {
  const int nch = H / 8, pieces = (nch + 63) / 64;
  const dim3 grid = linear_grid(blocks_of((long long)T * pieces));
  const v4i* yv = reinterpret_cast<const v4i*>(y);
  v4i* ov = reinterpret_cast<v4i*>(out);
  if (weights)
    hipLaunchKernelGGL(combine_kernel<true>, grid, dim3(256), 0, stream, yv, row_of_slot, weights, T, k, R, nch, pieces,
                       ov);
  else
    hipLaunchKernelGGL(combine_kernel<false>, grid, dim3(256), 0, stream, yv, row_of_slot, weights, T, k, R, nch,
                       pieces, ov);
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, const int* row_of_slot, const float* weights,
                              int T, int k, int R, int H, uint16_t* dy, float* dweights, hipStream_t stream) {
  hipLaunchKernelGGL(combine_bwd_kernel, dim3(T), dim3(256), 0, stream, reinterpret_cast<const v4i*>(dout),
                     reinterpret_cast<const v4i*>(y), row_of_slot, weights, k, R, H / 8, reinterpret_cast<v4i*>(dy),
                     dweights);
  return hipGetLastError();
}

}  // namespace fp8gmm
