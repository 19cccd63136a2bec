// Host launchers of the 8-bit and mixture-of-experts operators, called by the ABI after validation. They stand apart from
// common.hpp, which every FP4 kernel is compiled with: what was measured on those sources stays valid.
#pragma once

#include "choices.hpp"
#include "common.hpp"

// 8-bit (E4M3, one float32 scale for 128 values along K) operators.
hipError_t fp8_launch_quantize(const uint16_t* X, int64_t M, int64_t K, int64_t ldx, uint8_t* codes, float* scales,
                               hipStream_t stream);
hipError_t fp8_launch_quantize_weights(const uint16_t* W, int64_t N, int64_t K, int64_t ldw, uint8_t* codes,
                                       float* scales, hipStream_t stream);
hipError_t fp8_launch_add_rmsnorm_quantize(const uint16_t* X, int64_t M, int64_t K, int64_t ldx, const uint16_t* R,
                                           int64_t ldr, const uint16_t* G, float eps, uint8_t* codes, float* scales,
                                           uint16_t* H, uint16_t* Y, hipStream_t stream);
hipError_t fp8_launch_linear(const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws, int64_t M,
                             int64_t N, int64_t K, uint16_t* Y, hipStream_t stream);
hipError_t fp8_launch_linear_split(int bm, int bn, const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws,
                                   int64_t M, int64_t N, int64_t K, uint16_t* Y, int dev, hipStream_t stream);

// Mixture of experts for a few tokens.
hipError_t fp4_launch_moe_route(const uint16_t* X, int64_t T, int64_t D, int64_t ldx, const uint16_t* Wr, int64_t E, int k,
                                int renorm, float* logits, int* ids, float* weights, hipStream_t stream);
hipError_t fp4_launch_moe_experts(const uint16_t* X, int64_t T, int64_t D, int64_t ldx, const int* ids,
                                  const float* weights, int k, int64_t E, int64_t I, int block, const uint8_t* W13q,
                                  const uint8_t* W13s, const uint8_t* W2q, const uint8_t* W2s, uint16_t* Y,
                                  uint8_t* workspace, hipStream_t stream);
