// Internal interface between the C-ABI entry points of the routed layer
// (experts_api.cu) and its kernels (route.cu, mx_quant.cu, mx_linear.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/lora_delta.h"

namespace lora {

constexpr int kRouteMaxTopK = 32;      // choices of a token: one lane of its warp each
constexpr int kRouteMaxGroups = 32;    // expert groups: one lane each
constexpr int kRouteMaxExperts = 1024; // 32 experts per lane

struct RouteParams {
  const void* logits;      // [T, E]
  const float* bias;       // [E] or nullptr
  int* ids;                // [T, top_k]
  float* weights;          // [T, top_k]
  uint32_t* flags;
  int T, E, top_k;
  int score;               // LORA_SCORE_*
  int num_groups, top_groups, group_score;
  int renormalize;
  float scale;
};

struct GroupParams {
  const int* ids;          // [T * top_k]
  const int* token_slot;   // [T] or nullptr
  int* expert_offsets;     // [E + 1]
  int* row_token;          // [T * top_k]
  int* pair_row;           // [T * top_k]
  int* row_slot;           // [T * top_k] or nullptr
  uint32_t* flags;
  int n, top_k, E;         // n = T * top_k
};

struct CombineParams {
  const void* y;           // [rows_cap, F]
  const int* pair_row;     // [T, top_k]
  const float* weights;    // [T, top_k]
  const void* residual;    // [T, F] or nullptr
  void* out;               // [T, F]
  uint32_t* flags;
  int T, top_k, rows_cap, F;
};

struct MxQuantParams {
  const void* x;           // [x_rows, F] (or [x_rows, 2F] for SILU_MUL)
  const int* row_index;    // [rows] or nullptr
  const int* row_count;    // device, or nullptr
  void* rows_out;          // [rows, F] or nullptr
  uint8_t* codes;          // [rows, F / 2]
  uint8_t* scales;         // [rows, F / 32]
  uint32_t* flags;
  int x_rows, rows, F;
};

struct MxLinearParams {
  const uint8_t* x_codes;
  const uint8_t* x_scales;
  const uint8_t* w_codes;
  const uint8_t* w_scales;
  const int* expert_offsets;  // [experts + 1], or nullptr: one weight for every row
  void* y;
  uint32_t* flags;
  int rows, K, N, experts;
};

cudaError_t route_launch(const RouteParams& p, int type, cudaStream_t stream);
cudaError_t group_launch(const GroupParams& p, cudaStream_t stream);
cudaError_t combine_launch(const CombineParams& p, int type, cudaStream_t stream);
cudaError_t mx_quant_launch(const MxQuantParams& p, int type, int act, cudaStream_t stream);
cudaError_t mx_dequant_launch(const uint8_t* codes, const uint8_t* scales, void* out, int rows,
                              int F, int type, cudaStream_t stream);
cudaError_t mx_linear_launch(const MxLinearParams& p, int type, cudaStream_t stream,
                             const char** why);

}  // namespace lora
