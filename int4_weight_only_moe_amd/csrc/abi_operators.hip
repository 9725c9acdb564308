// Exported C entry points of the operators beside the layer: host-side
// validation, sizes, and kernel launches. As in abi.hip every check runs
// before the first HIP call.
#include "../../include/moe_w4a16.h"
#include "operators.h"

namespace {

constexpr int32_t kMaxExperts = 1024;
constexpr int32_t kMaxTopK = 16;
constexpr int32_t kMaxSequences = 65535;
constexpr int32_t kMaxAdapters = 1024;
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

}  // extern "C"
