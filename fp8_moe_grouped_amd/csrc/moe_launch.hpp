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

}  // namespace fp8gmm
