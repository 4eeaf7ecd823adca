// Host-side launchers of the kernels around the grouped products (internal to the library).
#pragma once
#include "launch.hpp"

namespace fp8gmm {

// Largest number of experts a token chooses (a choice lives in a lane).
constexpr int kMaxTopk = 32;
// Largest N of the MXFP4 product and values (one launch dimension holds the rows).
constexpr int kMaxMxfp4N = 1 << 16;

// Routing: top-k, its softmax weights and the slots' stable sort by expert (logits f32 or bf16).
size_t route_workspace_bytes(int T, int E);
hipError_t launch_route(const void* logits, bool bf16, int T, int E, int k, bool renorm, int* ids, float* weights,
                        int* group_sizes, int* row_of_slot, int* slot_of_row, void* ws, hipStream_t stream);
hipError_t launch_route_bwd(const float* dweights, const void* logits, bool bf16, const int* ids, const float* weights,
                            int T, int E, int k, bool renorm, void* dlogits, hipStream_t stream);

// Balance losses (ids NULL: counts is an input) and the logits' gradient (add may be NULL or dlogits).
size_t balance_workspace_bytes(int T, int E);
hipError_t launch_balance(const void* logits, bool bf16, const int* ids, int T, int E, int k, float* losses,
                          int* counts, float* probs, int* tokens, void* ws, hipStream_t stream);
hipError_t launch_balance_bwd(const float* dlosses, const void* logits, bool bf16, const int* counts,
                              const int* tokens, int T, int E, const void* add, void* dlogits, hipStream_t stream);

// Tokens to the ragged buffer's R rows and back.
hipError_t launch_permute(const uint16_t* x, const int* row_of_slot, int T, int k, int R, int H, uint16_t* out,
                          hipStream_t stream);
hipError_t launch_permute_fp8(const uint16_t* x, const int* row_of_slot, int T, int k, int R, int H, uint8_t* codes,
                              float* scales, hipStream_t stream);
hipError_t launch_combine(const uint16_t* y, const int* row_of_slot, const float* weights, int T, int k, int R, int H,
                          uint16_t* out, hipStream_t stream);
hipError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, const int* row_of_slot, const float* weights,
                              int T, int k, int R, int H, uint16_t* dy, float* dweights, hipStream_t stream);

// MXFP4: quantizers, values, product.  launch_quant_rows_mxfp4: with group_sizes, the valid rows of the ragged
// buffer x [T, K]; without, all T tokens and a row of zeros at T (codes and scales have T + 1 rows).
hipError_t launch_quant_rows_mxfp4(const uint16_t* x, const int* group_sizes, int G, int T, int K, uint8_t* codes,
                                   uint8_t* scales, hipStream_t stream);
hipError_t launch_quant_weights_mxfp4(const uint16_t* w, int G, int K, int N, uint8_t* codes, uint8_t* scales,
                                      hipStream_t stream);
hipError_t launch_dequant_mxfp4(const uint8_t* codes, const uint8_t* scales, int G, int N, int K, uint16_t* out,
                                hipStream_t stream);
hipError_t launch_gmm_mxfp4(const uint8_t* aq, const uint8_t* ascale, const uint8_t* codes, const uint8_t* wscale,
                            const int* group_sizes, const int* slot_of_row, int topk, int T, int G, int M, int K,
                            int N, bool swiglu, uint16_t* out, int* status, hipStream_t stream);

// Master weights to e4m3 codes and a scale per output channel.  polls: how often a block looks for another one's
// maxima before it computes them itself, a third of a microsecond each.  By itself a call is as fast with 100 to 20000
// and a tenth to a third slower with 30; four of 8 x 16384 x 4096 f32 at once take 18 ms with 300, 26 with
// 1000 and 280 with 20000.
constexpr int kQuantPolls = 300;
size_t quant_weights_workspace_bytes(bool bf16, int G, int K, int N);
hipError_t launch_quant_weights_fp8(const void* w, bool bf16, int G, int K, int N, uint8_t* codes, float* scales,
                                    void* ws, int polls, hipStream_t stream);

// AdamW's coefficients: c1 and c2 are 1 - beta, decay, up and root lr * weight_decay, lr / (1 - beta1^step) and
// 1 / sqrt(1 - beta2^step).  lr_dev and step_dev replace lr and step.
struct AdamW {
  float b1, c1, b2, c2, eps, decay, up, root;
  double lr, log_beta1, log_beta2, weight_decay;
  int64_t step;
  const float* lr_dev;
  const int64_t* step_dev;
  const float* grad_scale;
};
// 1 - beta^t, on the host and on the device: nothing cancels, so both are a few 2^-53 of it off at any beta (a beta of 0
// has the logarithm -inf, which gives 1).
__host__ __device__ inline double one_minus_power(double log_beta, int64_t t) { return -expm1((double)t * log_beta); }
hipError_t launch_adamw(int tensors, const int64_t* sizes, void* const* params, bool param_bf16,
                        const void* const* grads, bool grad_bf16, float* const* m, float* const* v, const AdamW& how,
                        hipStream_t stream);
hipError_t launch_adamw8(int tensors, const int64_t* sizes, void* const* params, bool param_bf16,
                         const void* const* grads, bool grad_bf16, uint8_t* const* m_codes, float* const* m_scales,
                         uint8_t* const* r_codes, float* const* r_scales, uint64_t seed, const AdamW& how,
                         hipStream_t stream);

}  // namespace fp8gmm
