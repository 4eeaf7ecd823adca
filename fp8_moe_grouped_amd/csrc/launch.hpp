// Host-side launchers of the library's kernels (internal; the public C ABI is
// include/fp8_moe_grouped.h).  Every launcher enqueues on `stream`, never
// synchronises and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace fp8gmm {

// Largest K handled by the row quantizer (512 bf16 per lane-chunk x 32).
constexpr int kMaxK = 16384;
// Largest number of experts (the group table lives in LDS).
constexpr int kMaxGroups = 1024;
// Largest number of experts a token chooses (a choice lives in a lane).
constexpr int kMaxTopk = 32;
// Largest N of the MXFP4 product and values (one launch dimension holds the rows).
constexpr int kMaxMxfp4N = 1 << 16;
// Largest static row count (keeps the clamped row prefix sums in int32).
constexpr long long kMaxRows = (1LL << 24) - 1;

// Compute units of the current device, looked up once per device id
// (persistent kernels launch one block per CU).
inline int device_cu_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
  if (dev < 64) {
    const int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
  }
  int n = 0;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
  if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

hipError_t launch_quant_rows_e4m3(const uint16_t* lhs, const int* group_sizes, int G, int M, int K,
                                  uint8_t* codes, float* scales, hipStream_t stream);

hipError_t launch_gmm_fp8_fwd(const uint8_t* aq, const float* ascale, const uint8_t* codes, const float* wscale,
                              const int* group_sizes, int G, int M, int K, int N, bool swiglu, uint16_t* out,
                              uint16_t* preact, int* status, hipStream_t stream);

hipError_t launch_gmm_dlhs_fp8(const uint16_t* dout, const uint8_t* codes, const float* scale, const int* group_sizes,
                               int G, int M, int K, int N, uint16_t* dlhs, int* status, hipStream_t stream);

// dLHS with the dSwiGLU epilogue: preact and d_preact are bf16 [M, 2K].
hipError_t launch_gmm_dswiglu_fp8(const uint16_t* dout, const uint8_t* codes, const float* scale,
                                  const int* group_sizes, int G, int M, int K, int N, const uint16_t* preact,
                                  uint16_t* d_preact, int* status, hipStream_t stream);

hipError_t launch_gmm_bf16_dlhs(const uint16_t* dout, const uint16_t* w, const int* group_sizes, int G, int M, int K,
                                int N, uint16_t* dlhs, int* status, hipStream_t stream);

// Ops-level LHS-quantization variants: ascale holds [M, ceil(K/512)] block scales when block512.
hipError_t launch_quant_rows_e4m3_variant(const uint16_t* lhs, const int* group_sizes, int G, int M, int K,
                                          bool block512, bool scale_bf16, uint8_t* codes, float* scales,
                                          hipStream_t stream);
hipError_t launch_gmm_fp8_fwd_variant(const uint8_t* aq, const float* ascale, const uint8_t* codes,
                                      const float* wscale, const int* group_sizes, int G, int M, int K, int N,
                                      bool block512, bool acc_bf16, bool rhs_first, uint16_t* out, int* status,
                                      hipStream_t stream);

// bf16 measurement arm of the forward: the FP8 forward's kernel on bf16 operands.
hipError_t launch_gmm_bf16_fwd(const uint16_t* lhs, const uint16_t* w, const int* group_sizes, int G, int M, int K,
                               int N, bool swiglu, uint16_t* out, int* status, hipStream_t stream);

// tgmm: workspace holds the transposed decoded operands and the scales.
size_t tgmm_workspace_bytes(long long M, long long K, long long N, int G);
hipError_t launch_tgmm_quant(const uint16_t* lhs, const uint16_t* dout, const int* group_sizes, int G, int M, int K,
                             int N, bool grad_e5m2, float* drhs, float* dbg_sl, float* dbg_sd, void* ws,
                             int* status, hipStream_t stream);

// Buffer-wide baseline of the tgmm's operand quantization (every row of the buffer).
size_t tgmm_dense_workspace_bytes(long long M, long long K, long long N, int G);
hipError_t launch_tgmm_dense(const uint16_t* lhs, const uint16_t* dout, const int* group_sizes, int G, int M, int K,
                             int N, bool grad_e5m2, float* drhs, float* dbg_srow, float* dbg_scol, void* ws,
                             int* status, hipStream_t stream);
hipError_t launch_quant_rows_e4m3_all(const uint16_t* lhs, int M, int K, uint8_t* codes, float* scales,
                                      hipStream_t stream);

hipError_t launch_dequant(const uint8_t* codes, const float* scale, int G, long long K, long long N, uint16_t* out,
                          hipStream_t stream);

// Routing: top-k, its softmax weights and the slots' stable sort by expert (logits f32 or bf16).
size_t route_workspace_bytes(int T, int E);
hipError_t launch_route(const void* logits, bool bf16, int T, int E, int k, bool renorm, int* ids, float* weights,
                        int* group_sizes, int* row_of_slot, int* slot_of_row, void* ws, hipStream_t stream);
hipError_t launch_route_bwd(const float* dweights, const void* logits, bool bf16, const int* ids, const float* weights,
                            int T, int E, int k, bool renorm, void* dlogits, hipStream_t stream);

// Tokens to the ragged buffer's R rows and back.
hipError_t launch_permute(const uint16_t* x, const int* row_of_slot, int T, int k, int R, int H, uint16_t* out,
                          hipStream_t stream);
hipError_t launch_permute_fp8(const uint16_t* x, const int* row_of_slot, int T, int k, int R, int H, uint8_t* codes,
                              float* scales, hipStream_t stream);
hipError_t launch_combine(const uint16_t* y, const int* row_of_slot, const float* weights, int T, int k, int R, int H,
                          uint16_t* out, hipStream_t stream);
hipError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, const int* row_of_slot, const float* weights,
                              int T, int k, int R, int H, uint16_t* dy, float* dweights, hipStream_t stream);

// MXFP4: quantizers (the activations' codes and scales have T + 1 rows, the last of zeros), values, product.
hipError_t launch_quant_rows_mxfp4(const uint16_t* x, int T, int K, uint8_t* codes, uint8_t* scales,
                                   hipStream_t stream);
hipError_t launch_quant_weights_mxfp4(const uint16_t* w, int G, int K, int N, uint8_t* codes, uint8_t* scales,
                                      hipStream_t stream);
hipError_t launch_dequant_mxfp4(const uint8_t* codes, const uint8_t* scales, int G, int N, int K, uint16_t* out,
                                hipStream_t stream);
hipError_t launch_gmm_mxfp4(const uint8_t* aq, const uint8_t* ascale, const uint8_t* codes, const uint8_t* wscale,
                            const int* group_sizes, const int* slot_of_row, int topk, int T, int G, int M, int K,
                            int N, bool swiglu, uint16_t* out, int* status, hipStream_t stream);

}  // namespace fp8gmm
