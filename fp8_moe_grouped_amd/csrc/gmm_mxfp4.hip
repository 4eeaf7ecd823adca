// Grouped product on microscaled 4-bit operands, for serving.  Row r of expert g
// is token slot_of_row[r] / topk (r itself without slot_of_row); x is quantized
// to MXFP4 once a token (launch_quant_rows_mxfp4), the weights are MXFP4 already:
//
//   y[r, n]   = sum over the blocks b of 32 k of 2^(ea + ew - 254) sum_{k in b} qa[k] qw[g, n, k]
//   out[r, n] = bf16(y[r, n]),  or with SwiGLU over columns [gate | up] of N = 2I:
//   out[r, i] = bf16( silu(y[r, i]) * y[r, I + i] )
//
// The scaled matrix instruction (16x16x128) applies the blocks' powers of two and
// accumulates in f32.  A lane's operand is 32 consecutive k of one row, which is
// one block with one scale byte.  The weight is the first operand, so a lane ends
// with four consecutive columns of one row.
//
// A block owns 16*MA rows x 32 columns of one expert (16 gate and the matching 16
// up columns for SwiGLU); its four waves share the contraction, 256 k (one cache
// line of codes a row) at a time in turn, and join their sums in LDS.
#include "common.hpp"
#include "launch.hpp"

#include <algorithm>

namespace fp8gmm {
namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ v4f mfma_mxfp4(const v4i& a, const v4i& b, const v4f& c, int sa, int sb) {
  const v8i a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, 0, sa, 0, sb);
}

template <int MA, bool SWIGLU>
__global__ __launch_bounds__(64 * kWaves) void gmm_mxfp4_split_kernel(
    const uint8_t* __restrict__ aq, const uint32_t* __restrict__ ascale, const uint8_t* __restrict__ codes,
    const uint32_t* __restrict__ wscale, const int* __restrict__ group_sizes, const int* __restrict__ slot_of_row,
    int topk, int T, int G, int M, int K, int N, uint16_t* __restrict__ out, int* status) {
  constexpr int BM = 16 * MA;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  v4f* const part = reinterpret_cast<v4f*>(smem);   // [kWaves][MA * 2][64]
  int* const t_start = reinterpret_cast<int*>(part + kWaves * MA * 2 * 64);
  int* const t_end = t_start + G;
  int* const t_pre = t_end + G;
  build_group_table(group_sizes, G, M, BM, GroupTable{t_start, t_end, t_pre}, status);
  __syncthreads();

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = t_pre[G], half = N >> 1;
  const int n_tiles = N / 32;
  if ((int)blockIdx.x >= tiles * n_tiles) return;
  const int mt = __builtin_amdgcn_readfirstlane(blockIdx.x % tiles), nt = blockIdx.x / tiles;
  const int g = __builtin_amdgcn_readfirstlane(find_group(t_pre, G, mt));
  const int row0 = __builtin_amdgcn_readfirstlane(t_start[g] + (mt - t_pre[g]) * BM);
  const int rows = __builtin_amdgcn_readfirstlane(min(BM, t_end[g] - row0));

  const int q = lane >> 4, r16 = lane & 15;
  const int kw = K / 128;                           // scale words of a row
  const uint8_t* ap[MA];
  const uint32_t* as[MA];
#pragma unroll
  for (int i = 0; i < MA; ++i) {
    const int row = row0 + min(16 * i + r16, rows - 1);   // rows past the expert's end repeat its last
    int token = row;
    if (slot_of_row) {
      const int slot = slot_of_row[row];
      token = slot < 0 ? T : min(slot / topk, T);   // row T of the quantized activations is zero
    }
    ap[i] = aq + (size_t)token * (K / 2) + 16 * q;
    as[i] = ascale + (size_t)token * kw;
  }
  int col[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) col[j] = SWIGLU ? j * half + nt * 16 + r16 : nt * 32 + 16 * j + r16;
  const uint8_t* bp[2];
  const uint32_t* bs[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    bp[j] = codes + ((size_t)g * N + col[j]) * (K / 2) + 16 * q;
    bs[j] = wscale + (size_t)g * kw * N + col[j];
  }

  v4f acc[MA][2];
#pragma unroll
  for (int i = 0; i < MA; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
  auto block128 = [&](int kb) __attribute__((always_inline)) {
    v4i a[MA], b[2];
    int sa[MA], sb[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      b[j] = *reinterpret_cast<const v4i*>(bp[j] + 64 * kb);
      sb[j] = (int)(bs[j][(size_t)kb * N] >> (8 * q));
    }
#pragma unroll
    for (int i = 0; i < MA; ++i) {
      a[i] = *reinterpret_cast<const v4i*>(ap[i] + 64 * kb);
      sa[i] = (int)(as[i][kb] >> (8 * q));
    }
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma_mxfp4(b[j], a[i], acc[i][j], sb[j], sa[i]);
  };
  for (int kb = 2 * wave; kb < kw; kb += 2 * kWaves) {
    block128(kb);
    if (kb + 1 < kw) block128(kb + 1);
  }

#pragma unroll
  for (int i = 0; i < MA; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) part[(wave * MA * 2 + 2 * i + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // wave w finishes fragments w, w + 4, ..: lane holds row r16, columns 4q + 0..3
  for (int i = wave; i < MA; i += kWaves) {
    v4f y[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      y[j] = part[(2 * i + j) * 64 + lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) y[j] += part[(w * MA * 2 + 2 * i + j) * 64 + lane];
    }
    const int m = 16 * i + r16;
    if (m >= rows) continue;
    if (SWIGLU) {
      float o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)   // hardware reciprocal: the product is rounded to bf16 right after
        o[e] = y[0][e] * __builtin_amdgcn_rcpf(1.0f + __expf(-y[0][e])) * y[1][e];
      const v2i p = {(int)pack_bf16x2(o[0], o[1]), (int)pack_bf16x2(o[2], o[3])};
      *reinterpret_cast<v2i*>(out + (size_t)(row0 + m) * half + nt * 16 + 4 * q) = p;
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const v2i p = {(int)pack_bf16x2(y[j][0], y[j][1]), (int)pack_bf16x2(y[j][2], y[j][3])};
        *reinterpret_cast<v2i*>(out + (size_t)(row0 + m) * N + nt * 32 + 16 * j + 4 * q) = p;
      }
    }
  }
}

}  // namespace

hipError_t launch_gmm_mxfp4(const uint8_t* aq, const uint8_t* ascale, const uint8_t* codes, const uint8_t* wscale,
                            const int* group_sizes, const int* slot_of_row, int topk, int T, int G, int M, int K,
                            int N, bool swiglu, uint16_t* out, int* status, hipStream_t stream) {
  constexpr int MA = 4;
  const long long tiles = std::min<long long>(M, ((long long)M + 16 * MA - 1) / (16 * MA) + G);
  const dim3 grid((unsigned)(tiles * (N / 32)));
  const size_t lds = sizeof(float) * 4 * kWaves * MA * 2 * 64 + sizeof(int) * (3 * (size_t)G + 1);
  const uint32_t* as = reinterpret_cast<const uint32_t*>(ascale);
  const uint32_t* bs = reinterpret_cast<const uint32_t*>(wscale);
  if (swiglu)
    hipLaunchKernelGGL((gmm_mxfp4_split_kernel<MA, true>), grid, dim3(64 * kWaves), lds, stream, aq, as, codes, bs,
                       group_sizes, slot_of_row, topk, T, G, M, K, N, out, status);
  else
    hipLaunchKernelGGL((gmm_mxfp4_split_kernel<MA, false>), grid, dim3(64 * kWaves), lds, stream, aq, as, codes, bs,
                       group_sizes, slot_of_row, topk, T, G, M, K, N, out, status);
  return hipGetLastError();
}

}  // namespace fp8gmm
