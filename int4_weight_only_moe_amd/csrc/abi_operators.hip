// Exported C entry points of the operators beside the layer: host-side
// validation, sizes, and kernel launches. As in abi.hip every check runs
// before the first HIP call.
#include <algorithm>
#include <cmath>

#include "../../include/moe_w4a16.h"
#include "operators.h"

namespace {

constexpr int32_t kMaxExperts = 1024;
constexpr int32_t kMaxTopK = 16;
constexpr int32_t kMaxSequences = 65535;
constexpr int32_t kMaxAdapters = 1024;
constexpr int32_t kMaxGroups = 64;
constexpr int32_t kMaxWidth = 1 << 20;
constexpr int32_t kMaxRows = 1 << 24;

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

int check_balance(int32_t M, int32_t E, int32_t k, const int32_t* offsets, int32_t S) {
  if (M < 0 || E <= 0 || k <= 0 || S <= 0 || (!offsets && S != 1)) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || k > E || k > kMaxTopK || S > kMaxSequences) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)M * k >= (int64_t(1) << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_lora(int32_t M, int32_t L, int32_t K, int32_t N, int32_t r) {
  if (M < 0 || L <= 0 || K <= 0 || N <= 0 || r <= 0) return MOE_ERR_INVALID_ARG;
  if (L > kMaxAdapters || r > moe::kLoraMaxRank || r % 8 != 0 || K % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (K > kMaxWidth || N > kMaxWidth || M > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A matrix of the projection's output side (bf16 or fp32, any alignment of
// its elements).
bool side_ok(const void* p, int64_t ld, int32_t width, int32_t dtype) {
  return ld >= width && aligned(p, dtype == MOE_DTYPE_F32 ? 4 : 2);
}
// A bf16 matrix of the projection's input side: 16-byte aligned rows.
bool rows_ok(const void* p, int64_t ld, int32_t width) { return ld >= width && ld % 8 == 0 && aligned(p, 16); }

int check_scored(int32_t M, int32_t E, int32_t k, int32_t scoring, float scale) {
  if (M < 0 || E <= 0 || k <= 0 || (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID) ||
      !std::isfinite(scale))
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || k > E || k > kMaxTopK || (int64_t)M * k >= (int64_t(1) << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_norm(int32_t M, int32_t N, int32_t dtype) {
  if (M < 0 || N <= 0 || (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32)) return MOE_ERR_INVALID_ARG;
  if (N > moe::kNormMaxWidth || M > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Two matrices that may be the same one: then with the same row stride.
bool same_or_apart(const void* a, int64_t ld_a, const void* b, int64_t ld_b, bool may) {
  return !a || a != b || (may && ld_a == ld_b);
}

int check_grads(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n) {
  if (n < 0 || (n > 0 && (!grads || !sizes || !dtypes))) return MOE_ERR_INVALID_ARG;
  if (n > moe::kClipMaxTensors) return MOE_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < n; ++i) {
    if (sizes[i] < 0 || (dtypes[i] != MOE_DTYPE_BF16 && dtypes[i] != MOE_DTYPE_F32) || (sizes[i] > 0 && !grads[i]) ||
        !aligned(grads[i], dtypes[i] == MOE_DTYPE_F32 ? 4 : 2))
      return MOE_ERR_INVALID_ARG;
    if (sizes[i] > (int64_t(1) << 40)) return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

// The memory of a non-empty tensor of the call.
struct Extent {
  uintptr_t lo, hi;
  int32_t i;
};
Extent extent_of(const void* p, int64_t size, int32_t dtype, int32_t i) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + (uintptr_t)size * (dtype == MOE_DTYPE_F32 ? 4 : 2), i};
}

// Whether no out overlaps another out or another entry's gradient (its own may
// be the same memory, not a part of it).
bool outs_apart(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* dtypes, int32_t n) {
  Extent out[moe::kClipMaxTensors];
  int32_t m = 0;
  for (int32_t i = 0; i < n; ++i)
    if (sizes[i] > 0) out[m++] = extent_of(outs[i], sizes[i], dtypes[i], i);
  std::sort(out, out + m, [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
  for (int32_t j = 1; j < m; ++j)
    if (out[j].lo < out[j - 1].hi) return false;
  for (int32_t i = 0; i < n; ++i) {
    if (sizes[i] == 0) continue;
    const Extent g = extent_of(grads[i], sizes[i], dtypes[i], i);
    // the first out that ends behind the gradient's start; outs do not overlap, so ends ascend too
    int32_t j = (int32_t)(std::upper_bound(out, out + m, g.lo, [](uintptr_t v, const Extent& e) { return v < e.hi; }) - out);
    for (; j < m && out[j].lo < g.hi; ++j)
      if (out[j].i != i || out[j].lo != g.lo) return false;
  }
  return true;
}

int check_outs(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* dtypes, int32_t n,
               const double* sumsq, float max_norm, const float* norm) {
  if (!(max_norm >= 0.0f) || !aligned(sumsq, 8) || !aligned(norm, 4) || (n > 0 && !outs)) return MOE_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if ((sizes[i] > 0 && !outs[i]) || !aligned(outs[i], dtypes[i] == MOE_DTYPE_F32 ? 4 : 2)) return MOE_ERR_INVALID_ARG;
  return outs_apart(grads, outs, sizes, dtypes, n) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

int64_t moe_balance_workspace_bytes(int32_t M, int32_t E, int32_t S) {
  if (M < 0 || E <= 0 || S <= 0 || E > kMaxExperts || S > kMaxSequences || M >= (int32_t(1) << 30)) return -1;
  return moe::balance_layout(M, E, S).total;
}

int moe_balance_loss(const float* logits, const int32_t* topk_ids, int32_t M, int32_t E, int32_t top_k,
                     const int32_t* seq_offsets, int32_t S, const uint8_t* row_valid, int32_t* expert_counts,
                     float* prob_sums, int32_t* seq_tokens, float* loss, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  const int st = check_balance(M, E, top_k, seq_offsets, S);
  if (st != MOE_OK) return st;
  if ((M > 0 && (!logits || !topk_ids)) || !expert_counts || !prob_sums || !seq_tokens || !loss || !workspace)
    return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(seq_offsets, 4) || !aligned(expert_counts, 4) ||
      !aligned(prob_sums, 4) || !aligned(seq_tokens, 4) || !aligned(loss, 4) || !aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe::balance_layout(M, E, S).total) return MOE_ERR_WORKSPACE;
  moe::BalanceArgs a{};
  a.logits = logits; a.topk_ids = topk_ids; a.offsets = seq_offsets; a.valid = row_valid;
  a.M = M; a.E = E; a.k = top_k; a.S = S;
  a.counts = expert_counts; a.prob_sums = prob_sums; a.tokens = seq_tokens; a.loss = loss;
  a.ws = (uint8_t*)workspace;
  return hip_status(moe::launch_balance_loss(a, (hipStream_t)stream));
}

int moe_balance_loss_backward(const float* logits, int32_t M, int32_t E, int32_t top_k, const int32_t* seq_offsets,
                              int32_t S, const uint8_t* row_valid, const int32_t* expert_counts,
                              const int32_t* seq_tokens, const float* grad_loss, float* grad_logits, void* stream) {
  const int st = check_balance(M, E, top_k, seq_offsets, S);
  if (st != MOE_OK || M == 0) return st;
  if (!logits || !expert_counts || !seq_tokens || !grad_loss || !grad_logits) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(seq_offsets, 4) || !aligned(expert_counts, 4) || !aligned(seq_tokens, 4) ||
      !aligned(grad_loss, 4) || !aligned(grad_logits, 4))
    return MOE_ERR_INVALID_ARG;
  moe::BalanceArgs a{};
  a.logits = logits; a.offsets = seq_offsets; a.valid = row_valid;
  a.M = M; a.E = E; a.k = top_k; a.S = S;
  a.counts = const_cast<int32_t*>(expert_counts); a.tokens = const_cast<int32_t*>(seq_tokens);
  a.dloss = grad_loss; a.grad = grad_logits;
  return hip_status(moe::launch_balance_backward(a, (hipStream_t)stream));
}

int64_t moe_lora_workspace_bytes(int32_t M, int32_t L, int32_t K, int32_t N, int32_t rank, int32_t backward) {
  if (check_lora(M, L, K, N, rank) != MOE_OK) return -1;
  return moe::lora_layout(M, L, K, N, rank, backward != 0).total;
}

int moe_lora_forward(const uint16_t* x_bf16, int64_t ldx, const int32_t* adapter_ids, int32_t M, int32_t L, int32_t K,
                     int32_t N, int32_t rank, const uint16_t* a_bf16, const uint16_t* b_bf16, const float* scales,
                     const void* base, int64_t ld_base, void* out, int64_t ld_out, int32_t out_dtype, float* h,
                     void* workspace, int64_t workspace_bytes, void* stream) {
  const int st = check_lora(M, L, K, N, rank);
  if (st != MOE_OK) return st;
  if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!x_bf16 || !adapter_ids || !a_bf16 || !b_bf16 || !out || !workspace) return MOE_ERR_INVALID_ARG;
  if (!rows_ok(x_bf16, ldx, K) || (base && !side_ok(base, ld_base, N, out_dtype)) ||
      !side_ok(out, ld_out, N, out_dtype) || (base == out && ld_base != ld_out))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(adapter_ids, 4) || !aligned(a_bf16, 16) || !aligned(b_bf16, 16) || !aligned(scales, 4) ||
      !aligned(h, 16) || !aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe::lora_layout(M, L, K, N, rank, false).total) return MOE_ERR_WORKSPACE;
  moe::LoraArgs a{};
  a.x = x_bf16; a.ldx = ldx; a.ids = adapter_ids;
  a.M = M; a.L = L; a.K = K; a.N = N; a.r = rank; a.y_f32 = out_dtype == MOE_DTYPE_F32;
  a.a = a_bf16; a.b = b_bf16; a.scales = scales;
  a.base = base; a.ld_base = ld_base; a.out = out; a.ld_out = ld_out; a.h = h;
  a.ws = (uint8_t*)workspace;
  return hip_status(moe::launch_lora_forward(a, (hipStream_t)stream));
}

int moe_lora_backward(const void* grad_out, int64_t ld_grad_out, int32_t out_dtype, const uint16_t* x_bf16,
                      int64_t ldx, const int32_t* adapter_ids, const float* h, int32_t M, int32_t L, int32_t K,
                      int32_t N, int32_t rank, const uint16_t* a_bf16, const uint16_t* b_bf16, const float* scales,
                      const uint16_t* dx_base, int64_t ld_dx_base, uint16_t* dx, int64_t ld_dx, float* grad_a,
                      float* grad_b, void* workspace, int64_t workspace_bytes, void* stream) {
  const int st = check_lora(M, L, K, N, rank);
  if (st != MOE_OK) return st;
  if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (!a_bf16 || !b_bf16 || !grad_a || !grad_b || !workspace) return MOE_ERR_INVALID_ARG;
  if (M > 0) {
    if (!grad_out || !x_bf16 || !adapter_ids || !h || (dx_base && !dx)) return MOE_ERR_INVALID_ARG;
    if (!side_ok(grad_out, ld_grad_out, N, out_dtype) || !rows_ok(x_bf16, ldx, K) ||
        (dx_base && !rows_ok(dx_base, ld_dx_base, K)) || (dx && !rows_ok(dx, ld_dx, K)) ||
        (dx && dx_base == dx && ld_dx_base != ld_dx))
      return MOE_ERR_INVALID_ARG;
  }
  if (!aligned(adapter_ids, 4) || !aligned(h, 16) || !aligned(a_bf16, 16) || !aligned(b_bf16, 16) ||
      !aligned(scales, 4) || !aligned(grad_a, 16) || !aligned(grad_b, 16) || !aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe::lora_layout(M, L, K, N, rank, true).total) return MOE_ERR_WORKSPACE;
  moe::LoraArgs a{};
  a.x = x_bf16; a.ldx = ldx; a.ids = adapter_ids;
  a.M = M; a.L = L; a.K = K; a.N = N; a.r = rank; a.y_f32 = out_dtype == MOE_DTYPE_F32;
  a.a = a_bf16; a.b = b_bf16; a.scales = scales; a.h = const_cast<float*>(h);
  a.dout = grad_out; a.ld_dout = ld_grad_out;
  a.dx_base = dx_base; a.ld_dx_base = ld_dx_base; a.dx = dx; a.ld_dx = ld_dx; a.da = grad_a; a.db = grad_b;
  a.ws = (uint8_t*)workspace;
  return hip_status(moe::launch_lora_backward(a, (hipStream_t)stream));
}

int moe_route_scored(const float* logits, int32_t M, int32_t E, int32_t top_k, int32_t scoring, const float* bias,
                     int32_t n_groups, int32_t top_groups, int32_t group_top, int32_t renormalise, float scale,
                     const uint8_t* row_valid, int32_t block_m, int32_t* topk_ids, float* topk_weights,
                     int32_t* sorted_token_ids, int32_t* block_expert_ids, int32_t* expert_offsets,
                     int32_t* num_tokens_post_pad, int64_t cap, void* stream) {
  const int st = check_scored(M, E, top_k, scoring, scale);
  if (st != MOE_OK) return st;
  if (n_groups <= 0 || top_groups <= 0 || top_groups > n_groups || (group_top != 1 && group_top != 2))
    return MOE_ERR_INVALID_ARG;
  if (n_groups > kMaxGroups || E % n_groups != 0 || group_top > E / n_groups ||
      (int64_t)top_groups * (E / n_groups) < top_k)
    return MOE_ERR_UNSUPPORTED;
  const bool grouping = sorted_token_ids || block_expert_ids || expert_offsets || num_tokens_post_pad;
  if (grouping && moe_route_align_capacity(M, E, top_k, block_m) < 0) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_weights) return MOE_ERR_INVALID_ARG;
  if (grouping && (!sorted_token_ids || !block_expert_ids || !expert_offsets || !num_tokens_post_pad))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) ||
      !aligned(sorted_token_ids, 4) || !aligned(block_expert_ids, 4) || !aligned(expert_offsets, 4) ||
      !aligned(num_tokens_post_pad, 4))
    return MOE_ERR_INVALID_ARG;
  if (grouping && (cap < moe_route_align_capacity(M, E, top_k, block_m) || cap % block_m != 0))
    return MOE_ERR_CAPACITY;
  moe::ScoredArgs a{};
  a.logits = logits; a.bias = bias; a.valid = row_valid;
  a.M = M; a.E = E; a.k = top_k;
  a.sigmoid = scoring == MOE_SCORE_SIGMOID; a.renorm = renormalise != 0; a.scale = scale;
  a.groups = n_groups; a.top_groups = top_groups; a.group_top = group_top;
  a.ids = topk_ids; a.weights = topk_weights;
  if (grouping) {
    a.block_m = block_m; a.sorted_ids = sorted_token_ids; a.block_expert = block_expert_ids;
    a.offsets = expert_offsets; a.npp = num_tokens_post_pad; a.cap = cap;
  }
  return hip_status(moe::launch_route_scored(a, (hipStream_t)stream));
}

int moe_route_scored_backward(const float* logits, int32_t M, int32_t E, int32_t top_k, int32_t scoring,
                              int32_t renormalise, float scale, const int32_t* topk_ids, const float* grad_weights,
                              const float* grad_base, float* grad_logits, void* stream) {
  const int st = check_scored(M, E, top_k, scoring, scale);
  if (st != MOE_OK || M == 0) return st;
  if (!logits || !topk_ids || !grad_weights || !grad_logits) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(grad_weights, 4) || !aligned(grad_base, 4) ||
      !aligned(grad_logits, 4))
    return MOE_ERR_INVALID_ARG;
  moe::ScoredBackwardArgs a{};
  a.logits = logits; a.M = M; a.E = E; a.k = top_k;
  a.sigmoid = scoring == MOE_SCORE_SIGMOID; a.renorm = renormalise != 0; a.scale = scale;
  a.ids = topk_ids; a.dweights = grad_weights; a.base = grad_base; a.grad = grad_logits;
  return hip_status(moe::launch_route_scored_backward(a, (hipStream_t)stream));
}

int moe_add_rms_norm(const uint16_t* x_bf16, int64_t ldx, const void* residual, int64_t ld_residual, int32_t res_dtype,
                     int32_t M, int32_t N, const uint16_t* weight_bf16, double eps, void* residual_out,
                     int64_t ld_residual_out, uint16_t* out_bf16, int64_t ld_out, uint8_t* out8_e4m3, int64_t ld_out8,
                     float* scales, int32_t quant_group, float* rstd, void* stream) {
  const int st = check_norm(M, N, res_dtype);
  if (st != MOE_OK) return st;
  if (!std::isfinite(eps) || eps < 0.0) return MOE_ERR_INVALID_ARG;
  if (out8_e4m3 && quant_group <= 0) return MOE_ERR_INVALID_ARG;
  if (out8_e4m3 && quant_group != N &&
      ((quant_group != 32 && quant_group != 64 && quant_group != 128) || N % quant_group != 0))
    return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  const bool f32 = res_dtype == MOE_DTYPE_F32;
  if ((!x_bf16 && !residual) || (!residual && f32) || !weight_bf16 || (!out_bf16 && !out8_e4m3) ||
      !out8_e4m3 != !scales)
    return MOE_ERR_INVALID_ARG;
  if ((x_bf16 && !side_ok(x_bf16, ldx, N, MOE_DTYPE_BF16)) ||
      (residual && !side_ok(residual, ld_residual, N, res_dtype)) ||
      (residual_out && !side_ok(residual_out, ld_residual_out, N, res_dtype)) ||
      (out_bf16 && !side_ok(out_bf16, ld_out, N, MOE_DTYPE_BF16)) || (out8_e4m3 && ld_out8 < N))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(weight_bf16, 2) || !aligned(scales, 4) || !aligned(rstd, 4)) return MOE_ERR_INVALID_ARG;
  if (!same_or_apart(residual_out, ld_residual_out, residual, ld_residual, true) ||
      !same_or_apart(residual_out, ld_residual_out, x_bf16, ldx, !f32) ||
      !same_or_apart(out_bf16, ld_out, x_bf16, ldx, true) ||
      !same_or_apart(out_bf16, ld_out, residual_out, ld_residual_out, false) ||
      !same_or_apart(out_bf16, ld_out, residual, ld_residual, false))
    return MOE_ERR_INVALID_ARG;
  moe::NormArgs a{};
  a.x = x_bf16; a.ldx = ldx; a.res = residual; a.ld_res = ld_residual; a.f32 = f32;
  a.M = M; a.N = N; a.w = weight_bf16; a.eps = eps;
  a.res_out = residual_out; a.ld_res_out = ld_residual_out; a.out = out_bf16; a.ld_out = ld_out;
  a.out8 = out8_e4m3; a.ld_out8 = ld_out8; a.scales = scales; a.group = quant_group; a.rstd = rstd;
  return hip_status(moe::launch_norm(a, (hipStream_t)stream));
}

int64_t moe_add_rms_norm_workspace_bytes(int32_t M, int32_t N) {
  if (check_norm(M, N, MOE_DTYPE_BF16) != MOE_OK) return -1;
  return (int64_t)moe::norm_backward_parts(M, N) * N * 4;
}

int moe_add_rms_norm_backward(const uint16_t* grad_out_bf16, int64_t ld_grad_out, const void* h, int64_t ld_h,
                              int32_t res_dtype, const float* rstd, int32_t M, int32_t N, const uint16_t* weight_bf16,
                              const void* grad_residual, int64_t ld_grad_residual, void* grad_h, int64_t ld_grad_h,
                              float* grad_weight, void* workspace, int64_t workspace_bytes, void* stream) {
  const int st = check_norm(M, N, res_dtype);
  if (st != MOE_OK) return st;
  const bool f32 = res_dtype == MOE_DTYPE_F32;
  if (grad_weight) {
    if (!aligned(grad_weight, 4) || !workspace || !aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_add_rms_norm_workspace_bytes(M, N)) return MOE_ERR_WORKSPACE;
  }
  if (M > 0) {
    if (!grad_out_bf16 || !h || !rstd || !weight_bf16 || (!grad_h && !grad_weight) || (grad_residual && !grad_h))
      return MOE_ERR_INVALID_ARG;
    if (!side_ok(grad_out_bf16, ld_grad_out, N, MOE_DTYPE_BF16) || !side_ok(h, ld_h, N, res_dtype) ||
        (grad_residual && !side_ok(grad_residual, ld_grad_residual, N, res_dtype)) ||
        (grad_h && !side_ok(grad_h, ld_grad_h, N, res_dtype)) || !aligned(rstd, 4) || !aligned(weight_bf16, 2))
      return MOE_ERR_INVALID_ARG;
    if (!same_or_apart(grad_h, ld_grad_h, grad_residual, ld_grad_residual, true) ||
        !same_or_apart(grad_h, ld_grad_h, h, ld_h, true) ||
        !same_or_apart(grad_h, ld_grad_h, grad_out_bf16, ld_grad_out, !f32))
      return MOE_ERR_INVALID_ARG;
  } else if (!grad_weight) {
    return MOE_OK;
  }
  moe::NormBackwardArgs a{};
  a.dout = grad_out_bf16; a.ld_dout = ld_grad_out; a.h = h; a.ld_h = ld_h; a.f32 = f32; a.rstd = rstd;
  a.M = M; a.N = N; a.w = weight_bf16; a.dres = grad_residual; a.ld_dres = ld_grad_residual;
  a.dh = grad_h; a.ld_dh = ld_grad_h; a.dw = grad_weight; a.parts = (float*)workspace;
  return hip_status(moe::launch_norm_backward(a, (hipStream_t)stream));
}

int64_t moe_grad_norm_workspace_bytes(int32_t n) {
  if (n < 0 || n > moe::kClipMaxTensors) return -1;
  return (moe::clip_parts(n) + 2) * 8;
}

int moe_grad_sumsq(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n, double* sumsq,
                   void* workspace, int64_t workspace_bytes, void* stream) {
  const int st = check_grads(grads, sizes, dtypes, n);
  if (st != MOE_OK) return st;
  if (!sumsq || !workspace || !aligned(sumsq, 8) || !aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_grad_norm_workspace_bytes(n)) return MOE_ERR_WORKSPACE;
  moe::ClipArgs a{};
  a.grads = grads; a.sizes = sizes; a.dtypes = dtypes; a.n = n; a.sumsq = sumsq; a.parts = (double*)workspace;
  return hip_status(moe::launch_grad_sumsq(a, (hipStream_t)stream));
}

int moe_grad_clip(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                  const double* sumsq, float max_norm, float* norm, void* stream) {
  int st = check_grads(grads, sizes, dtypes, n);
  if (st != MOE_OK) return st;
  if (!sumsq) return MOE_ERR_INVALID_ARG;
  st = check_outs(grads, outs, sizes, dtypes, n, sumsq, max_norm, norm);
  if (st != MOE_OK) return st;
  moe::ClipArgs a{};
  a.grads = grads; a.outs = outs; a.sizes = sizes; a.dtypes = dtypes; a.n = n;
  a.sumsq = const_cast<double*>(sumsq); a.max_norm = max_norm; a.norm = norm;
  return hip_status(moe::launch_grad_clip(a, (hipStream_t)stream));
}

int moe_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* dtypes,
                       int32_t n, float max_norm, double* sumsq, float* norm, void* workspace, int64_t workspace_bytes,
                       void* stream) {
  int st = check_grads(grads, sizes, dtypes, n);
  if (st != MOE_OK) return st;
  st = check_outs(grads, outs, sizes, dtypes, n, sumsq, max_norm, norm);
  if (st != MOE_OK) return st;
  if (!workspace || !aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_grad_norm_workspace_bytes(n)) return MOE_ERR_WORKSPACE;
  moe::ClipArgs a{};
  a.grads = grads; a.outs = outs; a.sizes = sizes; a.dtypes = dtypes; a.n = n; a.sumsq = sumsq;
  a.max_norm = max_norm; a.norm = norm; a.parts = (double*)workspace;
  return hip_status(moe::launch_clip_grad_norm(a, (hipStream_t)stream));
}

}  // extern "C"
