// C-ABI entry points of the routed layer (routing, grouping, MXFP4 quantisation
// and product, combine): host-side validation and launches.  Nothing here
// synchronises with the device or allocates memory.
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "experts.h"

namespace lora {
void set_last_error(const char* msg);  // api.cu
}

namespace {

lora_status fail(lora_status st, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  lora::set_last_error(msg);
  return st;
}

lora_status ok() {
  lora::set_last_error("");
  return LORA_OK;
}

lora_status done(const char* op, cudaError_t err, const char* why = nullptr) {
  if (err == cudaSuccess) return ok();
  if (why != nullptr) return fail(LORA_ERR_UNSUPPORTED, "%s: %s", op, why);
  return fail(LORA_ERR_CUDA, "%s: %s", op, cudaGetErrorString(err));
}

struct Ptr {
  const void* p;
  const char* name;
  unsigned align;
  bool optional;
};

lora_status check_ptrs(const char* op, std::initializer_list<Ptr> ptrs) {
  for (const Ptr& q : ptrs) {
    if (q.p == nullptr) {
      if (!q.optional) return fail(LORA_ERR_INVALID, "%s: %s is NULL", op, q.name);
    } else if (reinterpret_cast<uintptr_t>(q.p) % q.align != 0) {
      return fail(LORA_ERR_INVALID, "%s: %s is not %u-byte aligned", op, q.name, q.align);
    }
  }
  return LORA_OK;
}

lora_status check_type(const char* op, int32_t type) {
  if (type < LORA_TYPE_BF16 || type > LORA_TYPE_F32)
    return fail(LORA_ERR_INVALID, "%s: type = %d is none of LORA_TYPE_*", op, type);
  return LORA_OK;
}

lora_status check_count(const char* op, const char* name, int32_t v) {
  if (v < 0) return fail(LORA_ERR_INVALID, "%s: %s = %d < 0", op, name, v);
  return LORA_OK;
}

lora_status check_multiple(const char* op, const char* name, int32_t v, int32_t of) {
  if (v <= 0 || v % of != 0)
    return fail(LORA_ERR_INVALID, "%s: %s = %d must be a positive multiple of %d", op, name, v, of);
  return LORA_OK;
}

lora_status check_experts(const char* op, int32_t num_experts, int32_t top_k, int32_t T) {
  if (num_experts <= 0)
    return fail(LORA_ERR_INVALID, "%s: num_experts = %d must be positive", op, num_experts);
  if (num_experts > LORA_ROUTE_MAX_EXPERTS)
    return fail(LORA_ERR_UNSUPPORTED, "%s: num_experts = %d > %d", op, num_experts,
                LORA_ROUTE_MAX_EXPERTS);
  if (top_k <= 0) return fail(LORA_ERR_INVALID, "%s: top_k = %d must be positive", op, top_k);
  if ((long long)T * top_k > (1LL << 30))
    return fail(LORA_ERR_UNSUPPORTED, "%s: T * top_k = %lld > 2^30", op, (long long)T * top_k);
  return LORA_OK;
}

#define TRY(call)                          \
  do {                                     \
    const lora_status st_ = (call);        \
    if (st_ != LORA_OK) return st_;        \
  } while (0)

lora_status mx_linear_impl(const char* op, const uint8_t* x_codes, const uint8_t* x_scales,
                           const uint8_t* w_codes, const uint8_t* w_scales,
                           const int32_t* expert_offsets, bool grouped, void* y, int32_t type,
                           int32_t rows, int32_t in_features, int32_t out_features,
                           int32_t num_experts, uint32_t* err_flags, void* stream) {
  TRY(check_type(op, type));
  TRY(check_count(op, grouped ? "rows_cap" : "rows", rows));
  TRY(check_multiple(op, "in_features", in_features, 32));
  TRY(check_multiple(op, "out_features", out_features, 8));
  TRY(check_experts(op, num_experts, 1, 0));
  if (in_features > (1 << 24) || (long long)num_experts * out_features > (1LL << 30) ||
      rows > (1 << 28))
    return fail(LORA_ERR_UNSUPPORTED,
                "%s: at most 2^24 input features, 2^30 weight rows and 2^28 rows", op);
  // tiles of 16 rows x 128 features are counted in 32 bits
  if ((rows / 16LL + num_experts) * (out_features / 128 + 1) > (1LL << 30))
    return fail(LORA_ERR_UNSUPPORTED, "%s: rows * out_features is too large", op);
  if (rows == 0) return ok();
  TRY(check_ptrs(op, {{x_codes, "x_codes", 16, false},
                      {x_scales, "x_scales", 16, false},
                      {w_codes, "w_codes", 16, false},
                      {w_scales, "w_scales", 16, false},
                      {y, "y", 16, false},
                      {expert_offsets, "expert_offsets", 4, !grouped},
                      {err_flags, "err_flags", 4, true}}));
  lora::MxLinearParams p = {};
  p.x_codes = x_codes; p.x_scales = x_scales; p.w_codes = w_codes; p.w_scales = w_scales;
  p.expert_offsets = expert_offsets; p.y = y; p.flags = err_flags; p.rows = rows;
  p.K = in_features; p.N = out_features; p.experts = num_experts;
  const char* why = nullptr;
  const cudaError_t err =
      lora::mx_linear_launch(p, type, reinterpret_cast<cudaStream_t>(stream), &why);
  return done(op, err, why);
}

}  // namespace

extern "C" {

lora_status lora_route_experts(const void* logits, int32_t type, const float* bias,
                               int32_t* topk_ids, float* topk_weights, int32_t T,
                               int32_t num_experts, int32_t top_k, int32_t score,
                               int32_t num_groups, int32_t top_groups, int32_t group_score,
                               int32_t renormalize, float scale, uint32_t* err_flags,
                               void* stream) {
  const char* op = "lora_route_experts";
  TRY(check_type(op, type));
  TRY(check_count(op, "T", T));
  TRY(check_experts(op, num_experts, top_k, T));
  if (score != LORA_SCORE_SOFTMAX && score != LORA_SCORE_SIGMOID)
    return fail(LORA_ERR_INVALID, "%s: score = %d is none of LORA_SCORE_*", op, score);
  if (group_score != LORA_GROUP_MAX && group_score != LORA_GROUP_TOP_PAIR)
    return fail(LORA_ERR_INVALID, "%s: group_score = %d is none of LORA_GROUP_*", op, group_score);
  if (num_groups <= 0 || num_experts % num_groups != 0)
    return fail(LORA_ERR_INVALID, "%s: num_groups = %d must divide num_experts = %d", op,
                num_groups, num_experts);
  if (top_groups < 1 || top_groups > num_groups)
    return fail(LORA_ERR_INVALID, "%s: top_groups = %d outside [1, num_groups = %d]", op,
                top_groups, num_groups);
  if (top_k > num_experts / num_groups * top_groups)
    return fail(LORA_ERR_INVALID, "%s: top_k = %d > the %d experts of top_groups groups", op,
                top_k, num_experts / num_groups * top_groups);
  if (top_k > LORA_ROUTE_MAX_TOP_K)
    return fail(LORA_ERR_UNSUPPORTED, "%s: top_k = %d > %d", op, top_k, LORA_ROUTE_MAX_TOP_K);
  if (num_groups > LORA_ROUTE_MAX_GROUPS)
    return fail(LORA_ERR_UNSUPPORTED, "%s: num_groups = %d > %d", op, num_groups,
                LORA_ROUTE_MAX_GROUPS);
  if (T == 0) return ok();
  TRY(check_ptrs(op, {{logits, "logits", 16, false},
                      {bias, "bias", 4, true},
                      {topk_ids, "topk_ids", 4, false},
                      {topk_weights, "topk_weights", 4, false},
                      {err_flags, "err_flags", 4, true}}));
  lora::RouteParams p = {};
  p.logits = logits; p.bias = bias; p.ids = topk_ids; p.weights = topk_weights;
  p.flags = err_flags; p.T = T; p.E = num_experts; p.top_k = top_k; p.score = score;
  // every group is kept: there is nothing to choose between
  p.num_groups = top_groups == num_groups ? 1 : num_groups;
  p.top_groups = top_groups; p.group_score = group_score; p.renormalize = renormalize != 0;
  p.scale = scale;
  return done(op, lora::route_launch(p, type, reinterpret_cast<cudaStream_t>(stream)));
}

lora_status lora_group_experts(const int32_t* topk_ids, const int32_t* token_slot,
                               int32_t* expert_offsets, int32_t* row_token, int32_t* pair_row,
                               int32_t* row_slot, int32_t T, int32_t top_k, int32_t num_experts,
                               uint32_t* err_flags, void* stream) {
  const char* op = "lora_group_experts";
  TRY(check_count(op, "T", T));
  TRY(check_experts(op, num_experts, top_k, T));
  // T = 0 still writes the offsets (all zero)
  TRY(check_ptrs(op, {{topk_ids, "topk_ids", 4, T == 0},
                      {expert_offsets, "expert_offsets", 4, false},
                      {row_token, "row_token", 4, T == 0},
                      {pair_row, "pair_row", 4, T == 0},
                      {token_slot, "token_slot", 4, true},
                      {row_slot, "row_slot", 4, true},
                      {err_flags, "err_flags", 4, true}}));
  if ((token_slot == nullptr) != (row_slot == nullptr) && T > 0)
    return fail(LORA_ERR_INVALID, "%s: token_slot and row_slot go together", op);
  // (pair_row holds the counts of many pairs until their rows are known)
  const uintptr_t in = reinterpret_cast<uintptr_t>(topk_ids), bytes = (uintptr_t)T * top_k * 4;
  const uintptr_t out = reinterpret_cast<uintptr_t>(pair_row);
  if (in < out + bytes && out < in + bytes)
    return fail(LORA_ERR_INVALID, "%s: pair_row overlaps topk_ids", op);
  lora::GroupParams p = {};
  p.ids = topk_ids; p.token_slot = token_slot; p.expert_offsets = expert_offsets;
  p.row_token = row_token; p.pair_row = pair_row; p.row_slot = row_slot; p.flags = err_flags;
  p.n = T * top_k; p.top_k = top_k; p.E = num_experts;
  return done(op, lora::group_launch(p, reinterpret_cast<cudaStream_t>(stream)));
}

lora_status lora_mx_quantize(const void* x, int32_t type, const int32_t* row_index,
                             const int32_t* row_count, void* rows_out, uint8_t* codes,
                             uint8_t* scales, int32_t x_rows, int32_t rows, int32_t features,
                             int32_t activation, uint32_t* err_flags, void* stream) {
  const char* op = "lora_mx_quantize";
  TRY(check_type(op, type));
  TRY(check_count(op, "x_rows", x_rows));
  TRY(check_count(op, "rows", rows));
  TRY(check_multiple(op, "features", features, 32));
  if (features > (1 << 24)) return fail(LORA_ERR_UNSUPPORTED, "%s: features > 2^24", op);
  if (activation != LORA_ACT_NONE && activation != LORA_ACT_SILU_MUL)
    return fail(LORA_ERR_INVALID, "%s: activation = %d is none of LORA_ACT_*", op, activation);
  if (row_index == nullptr && x_rows < rows)
    return fail(LORA_ERR_INVALID, "%s: rows = %d > x_rows = %d without row_index", op, rows, x_rows);
  if (rows == 0) return ok();
  TRY(check_ptrs(op, {{x, "x", 16, x_rows == 0},
                      {codes, "codes", 16, false},
                      {scales, "scales", 16, false},
                      {rows_out, "rows_out", 16, true},
                      {row_index, "row_index", 4, true},
                      {row_count, "row_count", 4, true},
                      {err_flags, "err_flags", 4, true}}));
  lora::MxQuantParams p = {};
  p.x = x; p.row_index = row_index; p.row_count = row_count; p.rows_out = rows_out;
  p.codes = codes; p.scales = scales; p.flags = err_flags; p.x_rows = x_rows; p.rows = rows;
  p.F = features;
  return done(op, lora::mx_quant_launch(p, type, activation, reinterpret_cast<cudaStream_t>(stream)));
}

lora_status lora_mx_dequantize(const uint8_t* codes, const uint8_t* scales, void* out,
                               int32_t type, int32_t rows, int32_t features, void* stream) {
  const char* op = "lora_mx_dequantize";
  TRY(check_type(op, type));
  TRY(check_count(op, "rows", rows));
  TRY(check_multiple(op, "features", features, 32));
  if (features > (1 << 24)) return fail(LORA_ERR_UNSUPPORTED, "%s: features > 2^24", op);
  if (rows == 0) return ok();
  TRY(check_ptrs(op, {{codes, "codes", 16, false},
                      {scales, "scales", 16, false},
                      {out, "out", 16, false}}));
  return done(op, lora::mx_dequant_launch(codes, scales, out, rows, features, type,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

lora_status lora_mx_linear(const uint8_t* x_codes, const uint8_t* x_scales,
                           const uint8_t* w_codes, const uint8_t* w_scales, void* y, int32_t type,
                           int32_t rows, int32_t in_features, int32_t out_features,
                           uint32_t* err_flags, void* stream) {
  return mx_linear_impl("lora_mx_linear", x_codes, x_scales, w_codes, w_scales, nullptr, false, y,
                        type, rows, in_features, out_features, 1, err_flags, stream);
}

lora_status lora_mx_expert_linear(const uint8_t* x_codes, const uint8_t* x_scales,
                                  const uint8_t* w_codes, const uint8_t* w_scales,
                                  const int32_t* expert_offsets, void* y, int32_t type,
                                  int32_t rows_cap, int32_t in_features, int32_t out_features,
                                  int32_t num_experts, uint32_t* err_flags, void* stream) {
  return mx_linear_impl("lora_mx_expert_linear", x_codes, x_scales, w_codes, w_scales,
                        expert_offsets, true, y, type, rows_cap, in_features, out_features,
                        num_experts, err_flags, stream);
}

lora_status lora_combine_experts(const void* y_sorted, int32_t type, const int32_t* pair_row,
                                 const float* topk_weights, const void* residual, void* out,
                                 int32_t T, int32_t top_k, int32_t rows_cap, int32_t features,
                                 uint32_t* err_flags, void* stream) {
  const char* op = "lora_combine_experts";
  TRY(check_type(op, type));
  TRY(check_count(op, "T", T));
  TRY(check_count(op, "rows_cap", rows_cap));
  if (top_k <= 0) return fail(LORA_ERR_INVALID, "%s: top_k = %d must be positive", op, top_k);
  TRY(check_multiple(op, "features", features, 8));
  // (blocks of 1024 columns are the grid's second dimension)
  if (T > (1 << 30) || features > 65535 * 1024)
    return fail(LORA_ERR_UNSUPPORTED, "%s: at most 2^30 tokens of 65535 * 1024 features", op);
  if (T == 0) return ok();
  TRY(check_ptrs(op, {{y_sorted, "y_sorted", 16, rows_cap == 0},
                      {pair_row, "pair_row", 4, false},
                      {topk_weights, "topk_weights", 4, false},
                      {residual, "residual", 16, true},
                      {out, "out", 16, false},
                      {err_flags, "err_flags", 4, true}}));
  lora::CombineParams p = {};
  p.y = y_sorted; p.pair_row = pair_row; p.weights = topk_weights; p.residual = residual;
  p.out = out; p.flags = err_flags; p.T = T; p.top_k = top_k; p.rows_cap = rows_cap;
  p.F = features;
  return done(op, lora::combine_launch(p, type, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
