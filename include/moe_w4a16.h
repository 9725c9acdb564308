/*
 * moe_w4a16.h - C ABI of the MI355X (gfx950) weight-only INT4 MoE layer.
 *
 * The layer is the one "The Throughput Lever: Quantifying the MoE GEMM and
 * Mapping the Road to B300" identifies as the throughput lever of its MoE
 * serving stack (section "Phase 3: The INT4 Marlin MoE Throughput Lever"):
 * an INT4, group-size-32 (section "Building the Benchmark"), weight-only
 * Mixture-of-Experts grouped GEMM run over a dense token batch of
 * M = streams x q_len tokens (section "What It Means for the Engine"), each
 * token routed to its top-k experts (section "The Result: Two Regimes").
 *
 * One layer call is two entry points on one stream:
 *   moe_route_align   top-k routing + per-expert grouping of the M*k
 *                     (token, slot) assignments, padded to the tile size;
 *   moe_w4a16_forward FC1 (gate/up) with SiLU(gate)*up, FC2, and the
 *                     routing-weighted sum of each token's k expert outputs.
 * Weights are converted once by moe_w4a16_repack from the canonical GPTQ-style
 * format into the device layout the kernels stream.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers unless marked "host". The caller allocates
 *     and frees every buffer; the library allocates nothing, keeps no pointer
 *     after returning and has no mutable global state.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Calls only enqueue work: no host synchronisation, no device-to-host
 *     copy, so a layer call can be captured in a HIP graph. Buffers must stay
 *     alive until the stream has executed the work.
 *   - Arguments are validated on the host before anything is launched; on an
 *     error nothing is launched and no output is touched. Launch failures
 *     return MOE_ERR_HIP. A device fault surfaces at the caller's next
 *     synchronisation. No C++ exception crosses this interface.
 *   - M = 0 is valid: the call returns MOE_OK and launches nothing (except
 *     where an output does not depend on M: the operators at the end say so).
 *   - bf16 and fp16 values travel as uint16_t bit patterns.
 *
 * Canonical weight format (input of moe_w4a16_repack, a reading of the
 * "GPTQ-format" INT4 weights of "Building the Benchmark"):
 *   qweight uint8 [E, N, K/2]: byte i of a row holds input channel 2i in its
 *           low nibble and 2i+1 in its high nibble; nibble u encodes q = u - 8.
 *   scales  fp16  [E, N, K/32]: W[e, n, c] = q[e, n, c] * scales[e, n, c/32].
 *   W13 (kind 0): N = 2*I, K = H; rows [0, I) gate, rows [I, 2I) up.
 *   W2  (kind 1): N = H,   K = I.
 *
 * Limits (MOE_ERR_UNSUPPORTED otherwise): 1 <= E <= 1024, 1 <= top_k <= min(E, 16),
 * H and I multiples of 128, block_m in {16, 32, 64, 128}, M*top_k*max(H, I) < 2^31,
 * and one expert's repacked W13 or W2 (moe_w4a16_packed_bytes with E = 1,
 * less its trailer) below 2^31 bytes (H*I below about 1.9e9; the repack and size
 * calls apply the same per-tensor limit, and -1 / MOE_ERR_UNSUPPORTED past it).
 *
 * MXFP4 expert weights (the moe_mxfp4_* entry points at the end): "From
 * 1,060 to 4,016 tok/s on one B300, and why it wasn't the kernels" serves a
 * MoE whose experts are MXFP4 (opening section; its MoE kernels are MXFP4,
 * section "Finding 2: the MoE autotuner only saw decode shapes"). The same
 * routing, grouping, layer structure and bf16 activations, with the weights
 * in the OCP Microscaling (MX) v1.0 MXFP4 format: FP4 e2m1 codes and one E8M0
 * scale per 32 input channels.
 *
 * Operators beside the layer (moe_balance_*, moe_lora_* at the end): what
 * trains the router and adapts the frozen weights to a task or a request; and
 * what stands between the layer and the rest of a model (moe_route_scored*,
 * moe_add_rms_norm*, moe_grad_*).
 */
#ifndef MOE_W4A16_H
#define MOE_W4A16_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1, /* null pointer, negative size, misaligned pointer */
    MOE_ERR_UNSUPPORTED = -2, /* a size outside the limits above */
    MOE_ERR_CAPACITY = -3,    /* cap smaller than moe_route_align_capacity() */
    MOE_ERR_WORKSPACE = -4,   /* workspace smaller than the call's ..._workspace_bytes() */
    MOE_ERR_HIP = -5,         /* a HIP launch failed */
    MOE_ERR_SCRATCH = -6      /* batch too large for moe_w4a16_layer_noalloc's static scratch */
};

/* Version of this interface (bumped on any signature or layout change). */
int32_t moe_w4a16_abi_version(void);

/* Static, human-readable text for a status code (host). */
const char* moe_w4a16_status_string(int status);

/*
 * moe_route_align_capacity (host): entries of sorted_token_ids a call with
 * these sizes may write, rounded up to a multiple of block_m:
 *   roundup(M*k + min(E, M*k)*(block_m - 1), block_m).
 * Every expert's list is padded to a multiple of block_m, so the padded total
 * never exceeds this. Returns -1 on invalid sizes.
 */
int64_t moe_route_align_capacity(int32_t M, int32_t E, int32_t top_k, int32_t block_m);

/*
 * moe_route_align: top-k routing and per-expert grouping of one token batch.
 *
 * Routing ("The Result: Two Regimes": each token activates its top-k
 * experts; softmax over the experts, keep the k largest, renormalise):
 *   logits        fp32 [M, E] row-major, finite.
 *   topk_ids      out int32 [M, top_k]: the k experts with the largest logits,
 *                 largest first; equal logits go to the lower expert index,
 *                 -0.0 equals +0.0.
 *   topk_weights  out fp32 [M, top_k]: exp(L_j - L_0) / sum_i exp(L_i - L_0)
 *                 over the kept logits (equal to softmax-then-renormalise).
 * Grouping (the grouped GEMM of "Phase 3: The INT4 Marlin MoE Throughput
 * Lever" runs each expert over the tokens routed to it). Assignment
 * f = t*top_k + j:
 *   expert_offsets     out int32 [E+1]: exclusive prefix sum of the per-expert
 *                      counts, each rounded up to a multiple of block_m.
 *   num_tokens_post_pad out int32 [1]: expert_offsets[E] (NPP).
 *   sorted_token_ids   out int32 [cap]: entries [off[e], off[e+1]) list the
 *                      assignments of expert e in ascending f, then the
 *                      sentinel M*top_k up to the end of the range. Entries at
 *                      positions >= NPP are unspecified.
 *   block_expert_ids   out int32 [cap/block_m]: expert of each block_m-row
 *                      block; entries >= NPP/block_m are unspecified.
 * cap must be >= moe_route_align_capacity(M, E, top_k, block_m) and a multiple
 * of block_m. The integer outputs are deterministic (identical on every call).
 */
int moe_route_align(const float* logits, int32_t M, int32_t E, int32_t top_k, int32_t block_m,
                    int32_t* topk_ids, float* topk_weights,
                    int32_t* sorted_token_ids, int32_t* block_expert_ids,
                    int32_t* expert_offsets, int32_t* num_tokens_post_pad,
                    int64_t cap, void* stream);

/*
 * moe_w4a16_packed_bytes (host): size of the repacked weights of E experts
 * of an [N, K] INT4 matrix with the given group size: E*N*K*9/16 (nibbles plus
 * fp16 scales) + E*N (one int8 exponent shift per weight row, derived from its
 * scales, used by the large-batch kernels). Returns -1 unless group == 32,
 * N % 32 == 0 and K % 128 == 0.
 */
int64_t moe_w4a16_packed_bytes(int32_t E, int32_t N, int32_t K, int32_t group);

/*
 * moe_w4a16_repack: canonical INT4 weights -> the device layout the forward
 * streams. This is the analogue of the one-time weight repack of "Building
 * the Benchmark" (there into the Marlin layout; here a gfx950 layout of
 * 16-row x 128-channel tiles, each 1 KiB of nibbles followed by its 128 B of
 * scales, ordered so one wave reads one tile with one 16-byte load per lane,
 * and for W13 with gate tile r followed by up tile r).
 *   qweight  uint8 [E, N, K/2], scales_f16 uint16 [E, N, K/32] (canonical).
 *   kind     0 = W13 (N = 2I, K = H), 1 = W2 (N = H, K = I).
 *   packed   out, moe_w4a16_packed_bytes(E, N, K, group) bytes, 16-byte aligned.
 * The map is a bijection: moe_w4a16_unpack inverts it exactly (the row
 * shifts after the tiles are derived data: sigma = clamp(floor(log2(max over
 * the row's groups of |scale|)) - 11, -15, 4), 0 for a row of zero scales).
 */
int moe_w4a16_repack(const uint8_t* qweight, const uint16_t* scales_f16,
                     int32_t E, int32_t N, int32_t K, int32_t group, int32_t kind,
                     void* packed, void* stream);

/* moe_w4a16_unpack: exact inverse of moe_w4a16_repack (used by tests). */
int moe_w4a16_unpack(const void* packed, int32_t E, int32_t N, int32_t K, int32_t group, int32_t kind,
                     uint8_t* qweight, uint16_t* scales_f16, void* stream);

/*
 * moe_w4a16_workspace_bytes (host): scratch the forward needs for M tokens:
 * an fp32 [M, H] accumulator, the bf16 [M*top_k, I] FC1 activations, and
 * the tile table of the tiled grouped GEMM (256 bytes + (2*M*top_k + 16) x
 * 8 bytes); from M*top_k >= 16*E on also fp16 copies of the A rows
 * (max(M*H, M*top_k*I) x 2 bytes) and their exponents (M*top_k x 4 bytes).
 * Each part is padded to 256 bytes. Returns -1 on invalid sizes.
 */
int64_t moe_w4a16_workspace_bytes(int32_t M, int32_t E, int32_t H, int32_t I, int32_t top_k);

/*
 * moe_w4a16_preferred_block_m (host): the block_m the forward runs best with
 * for this batch (a function of the expected tokens per expert, M*top_k/E).
 * It never returns 128: the kernels that take blocks take at most 64 rows,
 * so with block_m = 128 they run each block as its two 64-row halves (and
 * the tiled kernel as one tile). Measured on the 384-expert layer: as fast
 * as the preferred size from 16 assignments per expert (the tiled kernel),
 * 1.5-1.8x slower below (64-row blocks of mostly padding rows).
 */
int32_t moe_w4a16_preferred_block_m(int32_t M, int32_t E, int32_t H, int32_t I, int32_t top_k);

/*
 * moe_w4a16_forward: the expert MLPs and the weighted combine for one batch.
 * "The Throughput Lever: Quantifying the MoE GEMM and Mapping the Road to
 * B300", section "Phase 3: The INT4 Marlin MoE Throughput Lever": the MoE
 * layer's work is a grouped GEMM over the experts with INT4 weights fused into
 * it (there the fused Marlin MoE kernel), run over the dense token batch;
 * section "The Result: Two Regimes": each token's top-k expert outputs are
 * combined with its routing weights.
 * Equivalent to moe_w4a16_fc1 followed by moe_w4a16_fc2 on the same stream.
 *   x_bf16      bf16 [M, H] activations, 16-byte aligned.
 *   topk_weights, sorted_token_ids, block_expert_ids, expert_offsets,
 *   num_tokens_post_pad: the outputs of moe_route_align for the same M, E,
 *               top_k, block_m and cap (read on the device only).
 *   w13_packed  moe_w4a16_repack output of W13 (kind 0), w2_packed of W2 (kind 1).
 *   workspace   >= moe_w4a16_workspace_bytes(M, E, H, I, top_k) bytes,
 *               16-byte aligned; contents on entry do not matter.
 *   out_bf16    out bf16 [M, H]: out[t] = sum_j topk_weights[t, j] *
 *               FC2_e(SiLU(gate_e(x_t)) * up_e(x_t)), e = topk_ids[t, j],
 *               accumulated in fp32 and rounded once to bf16. The FC1
 *               activation is stored as bf16 between the two GEMMs.
 * Numerics by regime. While experts average fewer than 16 assignments
 * (M*top_k < 16*E) each group's partial product uses the exact weights
 * q*s (scale applied to the fp32 product). From 16 on ("The Result: Two
 * Regimes": the compute-heavy regime) the weights enter the matrix core as
 * fp16(q * s * 2^-sigma), one rounding of the exact product (relative error
 * <= 2^-11), and each activation row as an exact fp16 copy scaled by a power
 * of two; the shifts are undone exactly in fp32. Both stay within the
 * layer's error bound against a float64 reference.
 * Float results may differ in the last bits between calls (the k
 * contributions are added with fp32 atomics in arrival order).
 */
int moe_w4a16_forward(const uint16_t* x_bf16, int32_t M, int32_t E, int32_t H, int32_t I,
                      int32_t top_k, int32_t block_m, const float* topk_weights,
                      const int32_t* sorted_token_ids, const int32_t* block_expert_ids,
                      const int32_t* expert_offsets, const int32_t* num_tokens_post_pad, int64_t cap,
                      const void* w13_packed, const void* w2_packed,
                      void* workspace, int64_t workspace_bytes, uint16_t* out_bf16, void* stream);

/*
 * moe_w4a16_fc1: first stage of moe_w4a16_forward. For every assignment f in
 * sorted_token_ids (expert e, token t = f / top_k) it computes
 * h = W13_e x_t, stores act_f = bf16(SiLU(h[0:I]) * h[I:2I]) in the
 * workspace, and clears the fp32 accumulator stage 2 uses.
 */
int moe_w4a16_fc1(const uint16_t* x_bf16, int32_t M, int32_t E, int32_t H, int32_t I,
                  int32_t top_k, int32_t block_m,
                  const int32_t* sorted_token_ids, const int32_t* block_expert_ids,
                  const int32_t* num_tokens_post_pad, int64_t cap,
                  const void* w13_packed, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * moe_w4a16_fc2: second stage. y_f = W2_e act_f; acc[t] += topk_weights[f] * y_f
 * in fp32 (atomics), then out_bf16 = bf16(acc) in one rounding. Must follow
 * moe_w4a16_fc1 with the same workspace on the same stream.
 */
int moe_w4a16_fc2(int32_t M, int32_t E, int32_t H, int32_t I, int32_t top_k, int32_t block_m,
                  const float* topk_weights, const int32_t* sorted_token_ids,
                  const int32_t* block_expert_ids, const int32_t* num_tokens_post_pad, int64_t cap,
                  const void* w2_packed, void* workspace, int64_t workspace_bytes,
                  uint16_t* out_bf16, void* stream);

/*
 * moe_w4a16_layer: one whole layer call, moe_route_align followed by
 * moe_w4a16_forward, with the same arguments, outputs and results (integer
 * outputs identical, out_bf16 within the same tolerance).
 *
 * "The Throughput Lever: Quantifying the MoE GEMM and Mapping the Road to
 * B300", section "The B300 Analysis: When the Bottleneck Flips": at decode
 * sizes fixed per-step costs such as kernel launches dominate once the GEMM
 * runs at HBM speed. Small batches therefore run two kernels instead of
 * four, with the routing and grouping inside the FC1 kernel (one of its
 * workgroups also writes the routing/grouping outputs):
 *   - M = 1: the decode path; every FC1 workgroup routes the
 *     batch, and FC2 is output-stationary (each output tile sums its token's
 *     top_k expert results in slot order in one workgroup: no atomics, and
 *     the bf16 output is then identical on every call);
 *   - M <= 16 and M*top_k <= 256 while few experts are touched and the
 *     batch's x rows fit in 128 KB of LDS (the grouped FC1 would fill at
 *     most 1.75 rounds of the device's CUs; on the 384-expert top-8 layer
 *     M = 2..7), and M = 2 or 3 wherever M*top_k <= 64: a persistent FC1
 *     kernel that routes once per workgroup and splits the work into small
 *     items (not when the tiled grouped GEMM below takes the batch);
 *   - else M = 4 with M*top_k <= 64: the decode path.
 * Up to 16 tokens the output-stationary FC2 follows the FC1 while the
 * M*top_k expert reads stay within 1.2x the expected number of distinct
 * experts (no accumulator and no finalize kernel); otherwise the grouped FC2
 * of moe_w4a16_forward.
 *   stage_events  NULL, or two hipEvent_t that receive the start and end
 *                 timestamps of the FC1-stage kernel itself (on the two-kernel
 *                 paths the routing is part of it), for timing that stage.
 */
int moe_w4a16_layer(const float* logits, const uint16_t* x_bf16, int32_t M, int32_t E, int32_t H, int32_t I,
                    int32_t top_k, int32_t block_m, int32_t* topk_ids, float* topk_weights,
                    int32_t* sorted_token_ids, int32_t* block_expert_ids, int32_t* expert_offsets,
                    int32_t* num_tokens_post_pad, int64_t cap, const void* w13_packed, const void* w2_packed,
                    void* workspace, int64_t workspace_bytes, uint16_t* out_bf16, void* stream,
                    void* const* stage_events);

/*
 * moe_w4a16_layer_noalloc: moe_w4a16_layer without a caller workspace, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation). The workspace is a
 * static device array of MOE_W4A16_NOALLOC_SCRATCH_BYTES inside the library:
 * each GPU the library runs on holds its own copy from the first call on that
 * device until the process ends (the call resolves its address with
 * hipGetSymbolAddress on the current device; `stream` must belong to that
 * device). Arguments, outputs and results are those of moe_w4a16_layer (no
 * stage events). A batch whose moe_w4a16_workspace_bytes exceeds the scratch
 * size returns MOE_ERR_SCRATCH and launches nothing (48 MiB covers, e.g., up
 * to 512 tokens of the 384-expert layer: E = 384, H = 7168, I = 2048, top-8).
 * The call allocates nothing (no hipMalloc, hipFree or allocating library
 * routine). Every call on a GPU shares that GPU's scratch, which keeps the
 * last call's contents (the kernels clear what must start at zero): calls
 * that overlap on one GPU (several streams, several threads) race and must
 * be serialised by the caller.
 */
#define MOE_W4A16_NOALLOC_SCRATCH_BYTES (48ll << 20)
int moe_w4a16_layer_noalloc(const float* logits, const uint16_t* x_bf16, int32_t M, int32_t E, int32_t H,
                            int32_t I, int32_t top_k, int32_t block_m, int32_t* topk_ids, float* topk_weights,
                            int32_t* sorted_token_ids, int32_t* block_expert_ids, int32_t* expert_offsets,
                            int32_t* num_tokens_post_pad, int64_t cap, const void* w13_packed,
                            const void* w2_packed, uint16_t* out_bf16, void* stream);

/*
 * ---- MXFP4 weights --------------------------------------------------------
 * Canonical MXFP4 weight format (input of moe_mxfp4_repack):
 *   qweight     uint8 [E, N, K/2]: byte i of a row holds input channel 2i in
 *               its low nibble and 2i+1 in its high nibble; a nibble is an
 *               FP4 e2m1 code (bit 3 sign, bits 2..1 exponent with bias 1,
 *               bit 0 mantissa: magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6).
 *   scales_e8m0 uint8 [E, N, K/32]: s encodes 2^(s - 127) (255 = NaN).
 *   W[e, n, c] = fp4(qweight code) * 2^(scales_e8m0[e, n, c/32] - 127).
 *   W13 / W2 rows and shapes as for the INT4 format. Limits as above.
 * The device layout is the INT4 one with the codes in canonical byte order
 * and one scale byte per group: 0.53125 bytes per weight (INT4: 0.5625).
 * The kernels widen each code to the exact bf16 value code * 2^(s - 127)
 * (gfx950's FP4 conversion), so scales whose weights leave bf16's range
 * (s >= 253, or subnormal products) are outside the exact-result contract.
 */

/* Bytes of one repacked MXFP4 weight tensor (host); -1 for unsupported shapes. */
int64_t moe_mxfp4_packed_bytes(int32_t E, int32_t N, int32_t K);

/* moe_mxfp4_repack / moe_mxfp4_unpack: as moe_w4a16_repack / _unpack for the
 * MXFP4 format (kind 0 = W13, 1 = W2; 16-byte aligned buffers). */
int moe_mxfp4_repack(const uint8_t* qweight, const uint8_t* scales_e8m0, int32_t E, int32_t N, int32_t K,
                     int32_t kind, void* packed, void* stream);
int moe_mxfp4_unpack(const void* packed, int32_t E, int32_t N, int32_t K, int32_t kind, uint8_t* qweight,
                     uint8_t* scales_e8m0, void* stream);

/* moe_mxfp4_fc1, _fc2, _forward, _layer: the moe_w4a16_* entry points of the
 * same names (same arguments, workspace, routing buffers and semantics) with
 * moe_mxfp4_repack weights. */
int moe_mxfp4_fc1(const uint16_t* x_bf16, int32_t M, int32_t E, int32_t H, int32_t I, int32_t top_k,
                  int32_t block_m, const int32_t* sorted_token_ids, const int32_t* block_expert_ids,
                  const int32_t* num_tokens_post_pad, int64_t cap, const void* w13_packed, void* workspace,
                  int64_t workspace_bytes, void* stream);
int moe_mxfp4_fc2(int32_t M, int32_t E, int32_t H, int32_t I, int32_t top_k, int32_t block_m,
                  const float* topk_weights, const int32_t* sorted_token_ids, const int32_t* block_expert_ids,
                  const int32_t* num_tokens_post_pad, int64_t cap, const void* w2_packed, void* workspace,
                  int64_t workspace_bytes, uint16_t* out_bf16, void* stream);
int moe_mxfp4_forward(const uint16_t* x_bf16, int32_t M, int32_t E, int32_t H, int32_t I, int32_t top_k,
                      int32_t block_m, const float* topk_weights, const int32_t* sorted_token_ids,
                      const int32_t* block_expert_ids, const int32_t* expert_offsets,
                      const int32_t* num_tokens_post_pad, int64_t cap, const void* w13_packed,
                      const void* w2_packed, void* workspace, int64_t workspace_bytes, uint16_t* out_bf16,
                      void* stream);
int moe_mxfp4_layer(const float* logits, const uint16_t* x_bf16, int32_t M, int32_t E, int32_t H, int32_t I,
                    int32_t top_k, int32_t block_m, int32_t* topk_ids, float* topk_weights,
                    int32_t* sorted_token_ids, int32_t* block_expert_ids, int32_t* expert_offsets,
                    int32_t* num_tokens_post_pad, int64_t cap, const void* w13_packed, const void* w2_packed,
                    void* workspace, int64_t workspace_bytes, uint16_t* out_bf16, void* stream,
                    void* const* stage_events);

/*
 * ---- Balance loss of the router -------------------------------------------
 * Beside moe_route_align, for training the router: per-expert counts, the loss
 * that keeps the experts evenly used, and its gradient with respect to the
 * logits. With p = softmax(logits[t, :]) over the E experts, and for each
 * sequence s of T valid tokens
 *   c[s, e] = how often e stands in the tokens' topk_ids,
 *   P[s, e] = sum of p[t, e] over the tokens,
 *   loss[s] = E / (top_k * T^2) * sum_e c[s, e] * P[s, e]
 * (1 when the choices and the probabilities are uniform; T = 0 gives 0). The
 * counts are constants of the gradient:
 *   grad_logits[t, e] = grad_loss[s] * E / (top_k * T^2) * p[t, e] *
 *                       (c[s, e] - sum_j c[s, j] * p[t, j]).
 *
 *   logits      fp32 [M, E]. -inf gives an expert probability 0; a row of
 *               nothing but -inf has all probabilities 0 and no gradient.
 *   topk_ids    int32 [M, top_k] of moe_route_align; entries outside [0, E)
 *               (dropped choices) are not counted.
 *   seq_offsets int32 [S + 1], ascending: sequence s has the rows
 *               [seq_offsets[s], seq_offsets[s + 1]); NULL (S = 1 only): all
 *               rows. What the logits of rows of no sequence hold is not used, and
 *               their rows of grad_logits are left as they were.
 *   row_valid   uint8 [M] or NULL: rows with 0 (padding) are not counted, what
 *               their logits hold is not used; their rows of grad_logits are 0.
 *   expert_counts int32 [S, E], prob_sums fp32 [S, E], seq_tokens int32 [S]
 *               (T), loss fp32 [S]: out, all of it written. With M = 0 too:
 *               zeros.
 *   workspace   >= moe_balance_workspace_bytes(M, E, S) bytes, 16-byte
 *               aligned; contents on entry do not matter. One for a larger M
 *               or S serves smaller ones.
 * The backward call takes expert_counts and seq_tokens as the forward wrote
 * them. A data-parallel job may sum expert_counts, prob_sums and seq_tokens
 * over its ranks before it uses them. Results are identical on every call.
 * Limits: those of moe_route_align, 1 <= S <= 65535.
 */
int64_t moe_balance_workspace_bytes(int32_t M, int32_t E, int32_t S); /* host; -1 on invalid sizes */
int moe_balance_loss(const float* logits, const int32_t* topk_ids, int32_t M, int32_t E, int32_t top_k,
                     const int32_t* seq_offsets, int32_t S, const uint8_t* row_valid, int32_t* expert_counts,
                     float* prob_sums, int32_t* seq_tokens, float* loss, void* workspace, int64_t workspace_bytes,
                     void* stream);
int moe_balance_loss_backward(const float* logits, int32_t M, int32_t E, int32_t top_k, const int32_t* seq_offsets,
                              int32_t S, const uint8_t* row_valid, const int32_t* expert_counts,
                              const int32_t* seq_tokens, const float* grad_loss, float* grad_logits, void* stream);

/*
 * ---- Low-rank adapters of many requests ------------------------------------
 * The expert weights are frozen 4-bit codes; what is trained and what differs
 * from request to request are low-rank adapters. These calls add them to a
 * projection that all requests share: the router's (fp32 logits), the layer
 * as a whole (bf16 out), or any other. Row t of the batch has adapter
 * a = adapter_ids[t], or none if that is outside [0, L):
 *   h[t]   = A_a x[t]
 *   out[t] = base[t] + scales[a] * B_a h[t]            (no adapter: base[t])
 * and backwards, from grad_out,
 *   dh[t]  = scales[a] * B_a^T grad_out[t]
 *   dx[t]  = dx_base[t] + A_a^T dh[t]                  (no adapter: dx_base[t])
 *   grad_a[a] = sum of dh[t] x[t]^T, grad_b[a] = scales[a] * sum of
 *   grad_out[t] h[t]^T over the rows t of adapter a (no rows: zeros).
 *
 *   x_bf16      bf16 [M, K], row stride ldx (elements).
 *   adapter_ids int32 [M], in any order; rows are grouped by adapter inside
 *               the call.
 *   a_bf16      bf16 [L, rank, K], b_bf16 bf16 [L, N, rank]: contiguous. An
 *               adapter of a smaller rank is stored with zero rows of A.
 *   scales      fp32 [L], or NULL: 1.
 *   base, out   [M, N] of out_dtype, row strides ld_base and ld_out. base may
 *               be NULL (zeros) or the same matrix as out (in place: rows
 *               without an adapter are then not touched).
 *   h           fp32 [M, rank]: out, for the backward call (rows without an
 *               adapter are 0), or NULL.
 *   dx_base, dx bf16 [M, K], as base and out; dx may be NULL (then dx_base is).
 *   grad_a, grad_b fp32 [L, rank, K], [L, N, rank]: every element written.
 *               With M = 0 too: zeros.
 *   workspace   >= moe_lora_workspace_bytes(M, L, K, N, rank, backward) bytes;
 *               contents on entry do not matter. One for a larger M serves
 *               smaller ones, a backward call's serves the forward call. A
 *               backward call's has room for all L adapters once more
 *               (2 * L * rank * (K + N) bytes), whichever have rows.
 * out and dx are accumulated in fp32 and rounded once; h and dh are fp32 and
 * enter every result with all their bits (from a magnitude of 2^-102 up; fp32
 * values beyond the largest finite bf16, 3.389e38, count as not finite). A
 * row that is not finite (or whose adapter is not) makes its own row of the
 * results not finite, and its adapter's gradients.
 * Results are identical on every call.
 * x, a, b, dx_base, dx, h, grad_a, grad_b and workspace are 16-byte aligned,
 * ldx, ld_dx_base and ld_dx multiples of 8; base, out and grad_out need their
 * elements' alignment only (16-byte aligned rows of a multiple of 16 bytes are
 * faster). Buffers other than base = out and dx_base = dx must not overlap.
 * Limits: 1 <= L <= 1024; rank a multiple of 8 up to 128; K a multiple of 8;
 * K, N <= 2^20; M <= 2^24.
 */
enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_F32 = 1 };
int64_t moe_lora_workspace_bytes(int32_t M, int32_t L, int32_t K, int32_t N, int32_t rank,
                                 int32_t backward); /* host; -1 on invalid sizes */
int moe_lora_forward(const uint16_t* x_bf16, int64_t ldx, const int32_t* adapter_ids, int32_t M, int32_t L, int32_t K,
                     int32_t N, int32_t rank, const uint16_t* a_bf16, const uint16_t* b_bf16, const float* scales,
                     const void* base, int64_t ld_base, void* out, int64_t ld_out, int32_t out_dtype, float* h,
                     void* workspace, int64_t workspace_bytes, void* stream);
int moe_lora_backward(const void* grad_out, int64_t ld_grad_out, int32_t out_dtype, const uint16_t* x_bf16,
                      int64_t ldx, const int32_t* adapter_ids, const float* h, int32_t M, int32_t L, int32_t K,
                      int32_t N, int32_t rank, const uint16_t* a_bf16, const uint16_t* b_bf16, const float* scales,
                      const uint16_t* dx_base, int64_t ld_dx_base, uint16_t* dx, int64_t ld_dx, float* grad_a,
                      float* grad_b, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * ---- Routing by scores -----------------------------------------------------
 * moe_route_align with the choices that other routers make: scores of all
 * experts, a bias that balances the choice without entering the weights,
 * experts in groups, weights that are renormalised or not, and scaled. For a
 * token's logits l:
 *   s[e] = softmax(l)[e] over the E experts (MOE_SCORE_SOFTMAX), or
 *          1 / (1 + exp(-l[e])) (MOE_SCORE_SIGMOID);
 *   c[e] = s[e] + bias[e];
 *   groups: the experts are n_groups runs of E / n_groups. A group's score is
 *          the sum of its group_top (1 or 2) highest c; only experts of the
 *          top_groups groups of the highest scores are chosen from (equal
 *          scores: the lower group);
 *   topk_ids: the top_k of these experts with the highest c, highest first
 *          (equal c: the lower expert). Without a bias that is the order of the
 *          logits, and where group_top is 1 that of the groups' highest logits;
 *   topk_weights[j] = scale * s[e_j], or with renormalise scale * s[e_j] / sum
 *          of the kept s (softmax: the softmax over the kept logits; sigmoid:
 *          the sum plus 1e-20).
 * The choice is that of c in fp64, however close two experts are.
 *
 *   logits      fp32 [M, E]. An expert whose logit or bias is -inf is absent:
 *               never chosen, and a group of none but such is never chosen
 *               either (a group score leaves them out). Slots that no expert
 *               is left for have id -1 and weight 0, which the grouping, the
 *               layer, the balance loss and the backward call leave out. NaN
 *               counts as the highest value.
 *   bias        fp32 [E] or NULL.
 *   row_valid   uint8 [M] or NULL: all slots of rows with 0 (padding) are -1,
 *               what their logits hold is not used.
 *   grouping outputs as moe_route_align's, whole: sorted_token_ids past the
 *               padded total is M*top_k, block_expert_ids there -1 (all cap and
 *               cap / block_m entries are written). All four NULL: none are
 *               wanted; block_m and cap are then not used.
 * Limits: those of moe_route_align; E a multiple of n_groups, 1 <= n_groups <=
 * 64, 1 <= top_groups <= n_groups, top_k <= top_groups * E / n_groups,
 * group_top <= E / n_groups. Results are identical on every call.
 *
 * moe_route_scored_backward: the logits' gradient from the weights'
 * (grad_weights fp32 [M, top_k]); the choice and the bias have none:
 *   softmax:              s[e] * (g[e] - sum_i g[i] s[i]), g[e_j] = scale * grad_weights[j], else 0
 *   softmax, renormalised: the same with the softmax over the kept logits
 *   sigmoid:              g[j] s (1 - s) at e_j
 *   sigmoid, renormalised: s (1 - s) / S * (g[j] - sum_i g[i] s[i] / S) at e_j, S the sum plus 1e-20
 * plus grad_base (fp32 [M, E], or NULL: zeros), for instance the balance
 * loss's gradient. grad_base may be grad_logits: it is then added to in place.
 * topk_ids are the forward's, those of a row distinct; entries outside [0, E)
 * are left out, a row of none but such has no gradient whatever its logits.
 */
enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };
int moe_route_scored(const float* logits, int32_t M, int32_t E, int32_t top_k, int32_t scoring, const float* bias,
                     int32_t n_groups, int32_t top_groups, int32_t group_top, int32_t renormalise, float scale,
                     const uint8_t* row_valid, int32_t block_m, int32_t* topk_ids, float* topk_weights,
                     int32_t* sorted_token_ids, int32_t* block_expert_ids, int32_t* expert_offsets,
                     int32_t* num_tokens_post_pad, int64_t cap, void* stream);
int moe_route_scored_backward(const float* logits, int32_t M, int32_t E, int32_t top_k, int32_t scoring,
                              int32_t renormalise, float scale, const int32_t* topk_ids, const float* grad_weights,
                              const float* grad_base, float* grad_logits, void* stream);

/*
 * ---- Root-mean-square norm with the residual's addition ---------------------
 * What stands before the layer: the residual stream takes the last sublayer's
 * output (moe_w4a16_forward's, for instance) and is normalised into the next
 * one's x. For each row
 *   h = x + residual, rounded to the stream's type
 *   r = 1 / sqrt(mean(h^2) + eps)
 *   out = bf16(h * r * weight), rounded once
 *   out8 = e4m3(y / s), y = h * r * weight unrounded, s = max(max |y| / 448, 2^-126)
 *          in fp32 over quant_group columns (out8 is what y / s rounds to in
 *          exact arithmetic: nearest, ties to even).
 *
 *   x           bf16 [M, N], row stride ldx (elements), or NULL: 0.
 *   residual    [M, N] of res_dtype (bf16 or fp32), or NULL: 0 (h = x; res_dtype
 *               bf16). Not both NULL.
 *   residual_out [M, N] of res_dtype: h, or NULL. May be the same matrix as
 *               residual (in place), or as x where that has its type.
 *   weight      bf16 [N].
 *   out_bf16    bf16 [M, N], or NULL. May be the same matrix as x.
 *   out8_e4m3   uint8 [M, N] of OCP e4m3 values, scales fp32 [M, N / quant_group]
 *               (contiguous), or both NULL. quant_group 32, 64 or 128, a divisor
 *               of N, or N (a scale a row).
 *   rstd        fp32 [M]: r, for the backward call, or NULL.
 * At least one of out_bf16 and out8_e4m3. A row that holds NaN is NaN, one that
 * holds an infinity has r = 0.
 * out_bf16 and rstd take r in fp32: with eps 0 a row whose root of the mean square
 * is below some 2^-128 has an infinite rstd and no finite out_bf16 (zeros: NaN).
 * Sums are fp64. Results are identical on every call.
 *
 * moe_add_rms_norm_backward, from grad_out (bf16 [M, N]):
 *   n = h * r, u = weight * grad_out
 *   grad_h = grad_residual + r * (u - n * mean(u * n))     (of x and of residual alike)
 *   grad_weight = sum over the rows of grad_out * n
 *   h           the forward's residual_out (or x, where there was no residual).
 *   grad_residual [M, N] of res_dtype, what reaches h beside the norm, or NULL.
 *   grad_h      [M, N] of res_dtype; may be the same matrix as grad_residual
 *               or, where the type is the same, as grad_out or h; or NULL.
 *   grad_weight fp32 [N], every element written (M = 0: zeros), or NULL. Runs of
 *               at most 64 rows are summed in fp32, the runs in fp64.
 *   workspace   >= moe_add_rms_norm_workspace_bytes(M, N) bytes, 16-byte
 *               aligned; contents on entry do not matter. One for a larger M
 *               serves smaller ones. Not used (may be NULL) without grad_weight.
 * All matrices need their elements' alignment only (16-byte aligned rows of a
 * multiple of 8 elements are faster). Other overlaps of buffers are not allowed.
 * Limits: 1 <= N <= 32768, M <= 2^24; eps >= 0 and finite.
 */
int moe_add_rms_norm(const uint16_t* x_bf16, int64_t ldx, const void* residual, int64_t ld_residual, int32_t res_dtype,
                     int32_t M, int32_t N, const uint16_t* weight_bf16, double eps, void* residual_out,
                     int64_t ld_residual_out, uint16_t* out_bf16, int64_t ld_out, uint8_t* out8_e4m3, int64_t ld_out8,
                     float* scales, int32_t quant_group, float* rstd, void* stream);
int64_t moe_add_rms_norm_workspace_bytes(int32_t M, int32_t N); /* host; -1 on invalid sizes */
int moe_add_rms_norm_backward(const uint16_t* grad_out_bf16, int64_t ld_grad_out, const void* h, int64_t ld_h,
                              int32_t res_dtype, const float* rstd, int32_t M, int32_t N, const uint16_t* weight_bf16,
                              const void* grad_residual, int64_t ld_grad_residual, void* grad_h, int64_t ld_grad_h,
                              float* grad_weight, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * ---- Global gradient norm and clipping --------------------------------------
 * Over n gradients at once (the adapters', the router's, the norms'):
 *   sumsq = sum of the squares of all elements, fp64
 *   norm = sqrt(sumsq);  out_i = grad_i * (norm > max_norm ? max_norm / norm : 1)
 * moe_grad_sumsq writes sumsq; a data-parallel job may sum it over its ranks
 * before moe_grad_clip scales. moe_clip_grad_norm does both (a launch less for
 * up to 192 tensors). A sum that is not finite scales nothing (norm says so:
 * leave the step out).
 *
 *   grads, outs, sizes, dtypes: host arrays of n entries, read during the call:
 *               contiguous device tensors (outs_i may be grads_i: in place),
 *               their numbers of elements (0 is valid) and MOE_DTYPE_*. An out
 *               may overlap neither another out nor another entry's gradient
 *               (MOE_ERR_INVALID_ARG). A gradient in place that is not scaled is
 *               not written.
 *   sumsq       fp64 [1] (moe_clip_grad_norm: or NULL). norm fp32 [1], or NULL.
 *   max_norm    >= 0, infinity included.
 *   workspace   >= moe_grad_norm_workspace_bytes(n) bytes, 16-byte aligned;
 *               contents on entry do not matter. One for a larger n serves
 *               smaller ones.
 * Results are identical on every call. n = 0: sumsq and norm are 0.
 * Limits: n <= 8192, 2^40 elements a tensor.
 */
int64_t moe_grad_norm_workspace_bytes(int32_t n); /* host; -1 on invalid sizes */
int moe_grad_sumsq(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n, double* sumsq,
                   void* workspace, int64_t workspace_bytes, void* stream);
int moe_grad_clip(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                  const double* sumsq, float max_norm, float* norm, void* stream);
int moe_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* dtypes,
                       int32_t n, float max_norm, double* sumsq, float* norm, void* workspace, int64_t workspace_bytes,
                       void* stream);

/* Measurement helpers (not part of the layer). They measure what this GPU
 * sustains, so that a layer kernel's rate can be stated as a fraction of the
 * attainable rate as well as of the published peaks ("The Throughput Lever",
 * section "The Result: Two Regimes", measures the layer as a fraction of the
 * memory bandwidth).
 *
 * moe_calib_read_granule (host): the byte multiple moe_calib_hbm_read reads
 *   (32768).
 * moe_calib_hbm_read: reads `bytes` of `buf` once (non-temporal 16-byte loads,
 *   `workgroups` workgroups of 256 threads; each thread writes the XOR of the
 *   32-bit words it read to sink[workgroup * 256 + thread], so the XOR of the
 *   whole sink is the XOR of every word of the buffer). bytes > 0, a multiple
 *   of the granule; buf 16-byte and sink 4-byte aligned; sink holds
 *   workgroups * 256 words; 1 <= workgroups <= 2^20. MOE_ERR_INVALID_ARG
 *   otherwise (nothing launched).
 * moe_calib_mfma_f16: `workgroups` workgroups of 4 waves each issue
 *   iters * 8 v_mfma_f32_16x16x32_f16 on register operands (16384 flops
 *   each; operand values are a fixed hash of lane, element and operand
 *   index). Each thread writes the sum of its accumulators to
 *   sink[workgroup * 256 + thread] (workgroups * 256 floats). iters >= 0;
 *   1 <= workgroups <= 2^20; sink 4-byte aligned. */
int64_t moe_calib_read_granule(void);
int moe_calib_hbm_read(const void* buf, int64_t bytes, int32_t workgroups, uint32_t* sink, void* stream);
int moe_calib_mfma_f16(int64_t iters, int32_t workgroups, float* sink, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_W4A16_H */
