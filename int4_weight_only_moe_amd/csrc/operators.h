// Internal declarations of the operators beside the layer: the balance loss
// of the router (balance.hip), low-rank adapters (lora.hip), routing by scores
// (route_scored.hip), the norm with the residual's addition (norm.hip) and the
// gradient norm with clipping (clip.hip). The entry points are in
// abi_operators.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- balance loss ---------------------------------------------------------
// Rows are summed in chunks of balance_chunk_rows(M) rows, one workgroup
// each. A chunk writes one partial per sequence it touches; the partial of
// (chunk c, sequence s) has slot c + s, which is unique because going down
// the rows every step from one partial to the next raises c or s.
int balance_chunk_rows(int64_t M);
struct BalanceLayout {
  int64_t chunks, slots;
  int64_t sums_off, counts_off, tokens_off, loss_off, ticket_off, total;
};
BalanceLayout balance_layout(int64_t M, int64_t E, int64_t S);

struct BalanceArgs {
  const float* logits;       // [M, E]
  const int32_t* topk_ids;   // [M, k], forward only
  const int32_t* offsets;    // [S + 1], or null: one sequence of all rows
  const uint8_t* valid;      // [M], or null: every row counts
  int M, E, k, S;
  int32_t* counts;           // [S, E]
  float* prob_sums;          // [S, E], forward only
  int32_t* tokens;           // [S]
  float* loss;               // [S], forward only
  const float* dloss;        // [S], backward only
  float* grad;               // [M, E], backward only
  uint8_t* ws;
};
hipError_t launch_balance_loss(const BalanceArgs& a, hipStream_t stream);
hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t stream);

// ---- low-rank adapters ----------------------------------------------------
constexpr int kLoraTile = 64;     // rows of one adapter that a workgroup takes together
constexpr int kLoraMaxRank = 128;

struct LoraArgs {
  // x [M, K] bf16; y: the projection's output side [M, N] (bf16 or fp32)
  const uint16_t* x;
  int64_t ldx;
  const int32_t* ids;        // [M]
  int M, L, K, N, r;
  bool y_f32;
  const uint16_t* a;         // [L, r, K]
  const uint16_t* b;         // [L, N, r]
  const float* scales;       // [L] or null
  // forward
  const void* base;          // [M, N] or null
  int64_t ld_base;
  void* out;                 // [M, N]
  int64_t ld_out;
  float* h;                  // [M, r]; null in a forward that keeps none
  // backward
  const void* dout;          // [M, N]
  int64_t ld_dout;
  const uint16_t* dx_base;   // [M, K] or null
  int64_t ld_dx_base;
  uint16_t* dx;              // [M, K] or null
  int64_t ld_dx;
  float* da;                 // [L, r, K]
  float* db;                 // [L, N, r]
  uint8_t* ws;
};

// Workspace of one call. Forward: the grouping (not for a small batch, which
// its kernels group themselves) and the partial products of each split of K.
// Backward adds the transposed weights, dh, the rank-major factors of the
// weight gradients and their partial sums.
constexpr int kLoraSmallRows = 256;  // rows up to which a forward needs no grouping launch
struct LoraLayout {
  int64_t cap;                                  // padded rows the grouping may reach
  int tiles;                                    // workgroups' tiles: cap / 64, or a small batch's bound
  int splits;                                   // of the contraction (forward K, backward N)
  bool small;
  int64_t sorted_off, block_off, offs_off, part_off, h_off;
  int64_t at_off, bt_off, n_pad;                // backward: A^T [L, K, r], B^T [L, r, n_pad]
  int64_t dh_off, dht_off, ht_off;              // backward: dh [M, r]; bf16 parts of dh and s*h, rank-major
  int64_t a_slots_off, b_slots_off;             // backward: partial gradients [slots][r * K], [slots][N * r]
  int a_chunk, b_chunk;                         // positions per partial of dA and dB
  int64_t total;
};
LoraLayout lora_layout(int64_t M, int64_t L, int64_t K, int64_t N, int64_t r, bool backward);

hipError_t launch_lora_forward(const LoraArgs& a, hipStream_t stream);
hipError_t launch_lora_backward(const LoraArgs& a, hipStream_t stream);

// ---- routing by scores ------------------------------------------------------
struct ScoredArgs {
  const float* logits;       // [M, E]
  const float* bias;         // [E] or null
  const uint8_t* valid;      // [M] or null
  int M, E, k;
  bool sigmoid, renorm;
  float scale;
  int groups, top_groups, group_top;
  int32_t* ids;              // [M, k]
  float* weights;            // [M, k]
  // grouping, or all null
  int block_m;
  int32_t* sorted_ids;       // [cap]
  int32_t* block_expert;     // [cap / block_m]
  int32_t* offsets;          // [E + 1]
  int32_t* npp;              // [1]
  int64_t cap;
};
hipError_t launch_route_scored(const ScoredArgs& a, hipStream_t stream);

struct ScoredBackwardArgs {
  const float* logits;
  int M, E, k;
  bool sigmoid, renorm;
  float scale;
  const int32_t* ids;
  const float* dweights;
  const float* base;         // [M, E], null, or grad
  float* grad;               // [M, E]
};
hipError_t launch_route_scored_backward(const ScoredBackwardArgs& a, hipStream_t stream);

// ---- norm -------------------------------------------------------------------
constexpr int kNormMaxWidth = 32768;
struct NormArgs {
  const uint16_t* x;         // [M, N] or null
  int64_t ldx;
  const void* res;           // [M, N] or null
  int64_t ld_res;
  bool f32;                  // the stream's type
  int M, N;
  const uint16_t* w;         // [N]
  double eps;
  void* res_out;             // [M, N] or null
  int64_t ld_res_out;
  uint16_t* out;             // [M, N] or null
  int64_t ld_out;
  uint8_t* out8;             // [M, N] or null
  int64_t ld_out8;
  float* scales;             // [M, N / group]
  int group;
  float* rstd;               // [M] or null
};
hipError_t launch_norm(const NormArgs& a, hipStream_t stream);

struct NormBackwardArgs {
  const uint16_t* dout;      // [M, N]
  int64_t ld_dout;
  const void* h;             // [M, N]
  int64_t ld_h;
  bool f32;
  const float* rstd;         // [M]
  int M, N;
  const uint16_t* w;         // [N]
  const void* dres;          // [M, N] or null
  int64_t ld_dres;
  void* dh;                  // [M, N] or null
  int64_t ld_dh;
  float* dw;                 // [N] or null
  float* parts;              // [norm_backward_parts(M, N), N]
};
int norm_backward_parts(int64_t M, int64_t N);  // rows of partial weight gradients
hipError_t launch_norm_backward(const NormBackwardArgs& a, hipStream_t stream);

// ---- gradient norm and clipping ----------------------------------------------
constexpr int kClipMaxTensors = 8192;
constexpr int kClipTensorsPerLaunch = 96;
constexpr int kSumsqBlocks = 2048;        // partial sums of a launch
struct ClipArgs {
  const void* const* grads;
  void* const* outs;         // clip only
  const int64_t* sizes;
  const int32_t* dtypes;
  int n;
  double* sumsq;
  float max_norm;            // clip only
  float* norm;               // clip only, or null
  double* parts;             // up to kSumsqBlocks a launch, and a sum of them
};
inline int64_t clip_launches(int64_t n) { return ceil_div(n, kClipTensorsPerLaunch); }
inline int64_t clip_parts(int64_t n) { return (n ? clip_launches(n) : 1) * kSumsqBlocks; }
hipError_t launch_grad_sumsq(const ClipArgs& a, hipStream_t stream);
hipError_t launch_grad_clip(const ClipArgs& a, hipStream_t stream);
hipError_t launch_clip_grad_norm(const ClipArgs& a, hipStream_t stream);

}  // namespace moe
