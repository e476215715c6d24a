// Launchers of the norm, the router and the int8 layer, beside those of launch.h.
#pragma once

#include "launch.h"

namespace fp8moe {

// Int8 variants: one scale per token row and per weight row.  GEMM1 writes the
// SwiGLU output as bf16 (act [cap][I]), launch_quant_rows_int8 quantises its
// rows (those with sorted_src >= 0; every row if NULL), GEMM2 takes the codes
// and row scales.  tile_m in {16, 32, 64} (streaming kernels) or kTileMaxInt8
// (tile kernels).
constexpr int kTileMaxInt8 = 288;
hipError_t launch_gemm1_int8(const uint8_t* x, const float* x_scale, const uint8_t* w13, const float* w13_scale,
                             const GroupedRows& g, int H, int I, uint16_t* act, int tile_m, bool packed,
                             hipStream_t stream);
hipError_t launch_quant_rows_int8(const uint16_t* in, const int32_t* sorted_src, int64_t rows, int N, uint8_t* q,
                                  float* scale, hipStream_t stream);
// YT: uint16_t (bf16 rows) or float
template <typename YT>
hipError_t launch_gemm2_int8(const uint8_t* q, const float* q_scale, const uint8_t* w2, const float* w2_scale,
                             const float* topk_weights, const GroupedRows& g, int H, int I, YT* Y, int tile_m,
                             bool packed, hipStream_t stream);

// The whole layer without routing for at most kDirectMaxRows routed rows of at
// most kDirectMaxSlots slots a token; act [T*K][I].
constexpr int kDirectMaxRows = 16, kDirectMaxSlots = 8;
hipError_t launch_moe_direct_int8(const uint8_t* x, const float* x_scale, const uint8_t* w13, const float* w13_scale,
                                  const uint8_t* w2, const float* w2_scale, const int32_t* topk_ids,
                                  const float* topk_weights, int T, int H, int I, int E, int K, uint16_t* act,
                                  uint16_t* out, bool packed, hipStream_t stream);
// The tile kernels; GEMM1's takes x of less than 4 GiB (hipErrorInvalidValue).
hipError_t launch_gemm1_int8_tile(const uint8_t* x, const float* x_scale, const uint8_t* w13, const float* w13_scale,
                                  const GroupedRows& g, int H, int I, uint16_t* act, bool packed, hipStream_t stream);
template <typename YT>
hipError_t launch_gemm2_int8_tile(const uint8_t* q, const float* q_scale, const uint8_t* w2, const float* w2_scale,
                                  const float* topk_weights, const GroupedRows& g, int H, int I, YT* Y,
                                  bool packed, hipStream_t stream);

// Residual addition + RMS norm + quantisation (format: FP8MOE_NORM_*), and the
// router's choice of experts (score: FP8MOE_SCORE_*).
hipError_t launch_add_rmsnorm(const uint16_t* x, const void* residual, bool residual_f32, const void* weight,
                              bool weight_f32, float eps, int64_t T, int H, int format, void* residual_out,
                              uint16_t* norm_out, uint8_t* q, void* scale, hipStream_t stream);
hipError_t launch_router_topk(const void* logits, bool bf16, const float* bias, int T, int E, int K, int score,
                              int n_group, int topk_group, int group_top, bool renormalize, float scale,
                              int32_t* ids, float* weights, hipStream_t stream);

// launch_combine over fp32 rows.
hipError_t launch_combine_f32(const float* Y, const int32_t* topk_ids, int T, int H, int E, int K, uint16_t* out,
                              hipStream_t stream);

// launch_route_permute where `inverse` may be false: the caller does not read
// src_to_sorted, which then holds anything where there are many rows (its
// launch is left out).
hipError_t launch_route_permute(const int32_t* ids, int R, int E, int align, int cap,
                                int32_t* counts, int32_t* m_indptr, int32_t* padded_indptr,
                                int32_t* sorted_src, int32_t* src_to_sorted, hipStream_t stream,
                                uint32_t* zero2, bool inverse);

}  // namespace fp8moe
