"""MI355X-native weight-only INT4 (group 32) MoE layer.

The layer of "The Throughput Lever: Quantifying the MoE GEMM and Mapping the
Road to B300" (section "Phase 3: The INT4 Marlin MoE Throughput Lever"):
top-k routing, per-expert grouping padded to the tile size, FC1 gate/up with
SiLU*mul and FC2 with the routing-weighted sum, as HIP kernels for gfx950
behind the C ABI of include/moe_w4a16.h, and beside it the router's balance
loss with its gradient (balance_loss, balance_loss_backward), low-rank
adapters of many requests, forward and backward (lora_forward, lora_backward),
and what stands between the layer and the rest of a model: routing by scores
(route_scored, route_scored_backward), the root-mean-square norm with the
residual's addition (add_rms_norm, add_rms_norm_backward) and clipping by the
global gradient norm (grad_sumsq, grad_clip, clip_grad_norm).
This package is the Python binding (ctypes; PyTorch only provides device memory
and streams) plus helpers that allocate the buffers a call needs.
"""
from __future__ import annotations

from contextlib import nullcontext
from dataclasses import dataclass

import torch

from ._binding import (  # noqa: F401
    GROUP, KIND_W13, KIND_W2, MOE_ERR_CAPACITY, MOE_ERR_HIP, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED,
    MOE_ERR_SCRATCH, MOE_ERR_WORKSPACE, MOE_OK, NOALLOC_SCRATCH_BYTES, MoeError, lib, library_path, moe_route_align, moe_route_align_capacity,
    moe_w4a16_abi_version, moe_w4a16_fc1, moe_w4a16_fc2, moe_w4a16_forward, moe_w4a16_layer, moe_w4a16_layer_noalloc, moe_w4a16_packed_bytes,
    moe_w4a16_preferred_block_m, moe_w4a16_repack, moe_w4a16_unpack, moe_w4a16_workspace_bytes,
    moe_mxfp4_fc1, moe_mxfp4_fc2, moe_mxfp4_forward, moe_mxfp4_layer, moe_mxfp4_packed_bytes, moe_mxfp4_repack,
    moe_mxfp4_unpack, status_string, moe_calib_read_granule, moe_calib_hbm_read, moe_calib_mfma_f16,
    MOE_DTYPE_BF16, MOE_DTYPE_F32, moe_balance_loss, moe_balance_loss_backward, moe_balance_workspace_bytes,
    moe_lora_backward, moe_lora_forward, moe_lora_workspace_bytes,
    MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, moe_route_scored, moe_route_scored_backward, moe_add_rms_norm,
    moe_add_rms_norm_backward, moe_add_rms_norm_workspace_bytes, moe_grad_clip, moe_grad_norm_workspace_bytes,
    moe_grad_sumsq, moe_clip_grad_norm,
)

FORMATS = ("int4", "mxfp4")  # weight formats: INT4 g32 + fp16 scales, MXFP4 (e2m1 + E8M0 per 32)


@dataclass
class RouteBuffers:
    """Outputs of moe_route_align for a batch of M tokens."""
    M: int
    E: int
    top_k: int
    block_m: int
    cap: int
    topk_ids: torch.Tensor
    topk_weights: torch.Tensor
    sorted_token_ids: torch.Tensor
    block_expert_ids: torch.Tensor
    expert_offsets: torch.Tensor
    num_tokens_post_pad: torch.Tensor


def alloc_route_buffers(M: int, E: int, top_k: int, block_m: int, device="cuda") -> RouteBuffers:
    cap = moe_route_align_capacity(M, E, top_k, block_m)
    if cap < 0:
        raise ValueError("unsupported routing sizes")
    i32 = dict(dtype=torch.int32, device=device)
    return RouteBuffers(
        M, E, top_k, block_m, cap,
        torch.empty((M, top_k), **i32), torch.empty((M, top_k), dtype=torch.float32, device=device),
        torch.empty(max(cap, 1), **i32), torch.empty(max(cap // block_m, 1), **i32),
        torch.empty(E + 1, **i32), torch.empty(1, **i32))


def route_align(logits: torch.Tensor, rb: RouteBuffers, stream=None) -> RouteBuffers:
    moe_route_align(logits, rb.top_k, rb.block_m, rb.topk_ids, rb.topk_weights, rb.sorted_token_ids,
                    rb.block_expert_ids, rb.expert_offsets, rb.num_tokens_post_pad, cap=rb.cap, stream=stream)
    return rb


def repack(qweight: torch.Tensor, scales_f16: torch.Tensor, kind: int, stream=None) -> torch.Tensor:
    """Repack canonical [E, N, K/2] nibbles + [E, N, K/32] fp16 scales into a new device blob."""
    E, N, K2 = qweight.shape
    nbytes = moe_w4a16_packed_bytes(E, N, 2 * K2)
    if nbytes < 0:
        raise ValueError("unsupported weight shape")
    packed = torch.empty(nbytes, dtype=torch.uint8, device=qweight.device)
    moe_w4a16_repack(qweight, scales_f16, kind, packed, stream=stream)
    return packed


def repack_mxfp4(qweight: torch.Tensor, scales_e8m0: torch.Tensor, kind: int, stream=None) -> torch.Tensor:
    """Repack canonical [E, N, K/2] FP4 codes + [E, N, K/32] E8M0 scales into a new device blob."""
    E, N, K2 = qweight.shape
    nbytes = moe_mxfp4_packed_bytes(E, N, 2 * K2)
    if nbytes < 0:
        raise ValueError("unsupported weight shape")
    packed = torch.empty(nbytes, dtype=torch.uint8, device=qweight.device)
    moe_mxfp4_repack(qweight, scales_e8m0, kind, packed, stream=stream)
    return packed


def _check_fmt(fmt: str) -> None:
    if fmt not in FORMATS:
        raise ValueError(f"fmt must be one of {FORMATS}")


def forward(x: torch.Tensor, rb: RouteBuffers, I: int, w13_packed: torch.Tensor, w2_packed: torch.Tensor,
            workspace: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None,
            fmt: str = "int4") -> torch.Tensor:
    _check_fmt(fmt)
    M, H = x.shape
    if workspace is None:
        workspace = torch.empty(max(moe_w4a16_workspace_bytes(M, rb.E, H, I, rb.top_k), 16),
                                dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    fwd = moe_mxfp4_forward if fmt == "mxfp4" else moe_w4a16_forward
    fwd(x, rb.E, I, rb.top_k, rb.block_m, rb.topk_weights, rb.sorted_token_ids, rb.block_expert_ids,
        rb.expert_offsets, rb.num_tokens_post_pad, w13_packed, w2_packed, workspace, out, cap=rb.cap, stream=stream)
    return out


def layer(logits: torch.Tensor, x: torch.Tensor, rb: RouteBuffers, I: int, w13_packed: torch.Tensor,
          w2_packed: torch.Tensor, workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
          stream=None, stage_events=None, fmt: str = "int4") -> torch.Tensor:
    """Routing + expert MLPs in one call. Two kernels while few experts are
    touched (routing inside FC1, FC2 per token: M = 1 on the decode path,
    up to 16 tokens on the routed FC1), else three up to 16 tokens (routing,
    grouped FC1, FC2 per token), and routing + grouped FC1 + grouped FC2 +
    finalize above. fmt: "int4" (moe_w4a16_repack weights) or "mxfp4"
    (moe_mxfp4_repack weights)."""
    _check_fmt(fmt)
    M, H = x.shape
    if workspace is None:
        workspace = torch.empty(max(moe_w4a16_workspace_bytes(M, rb.E, H, I, rb.top_k), 16),
                                dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    call = moe_mxfp4_layer if fmt == "mxfp4" else moe_w4a16_layer
    call(logits, x, I, rb.top_k, rb.block_m, rb.topk_ids, rb.topk_weights, rb.sorted_token_ids,
         rb.block_expert_ids, rb.expert_offsets, rb.num_tokens_post_pad, w13_packed, w2_packed,
         workspace, out, cap=rb.cap, stream=stream, stage_events=stage_events)
    return out


# ------------------------------------------------------------------ operators beside the layer
def _memory_of(stream, device):
    """A context in which torch allocates for `stream`: what the helpers below
    allocate themselves is used on it, and is reused only in its order."""
    if stream is None:
        return nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


@dataclass
class BalanceBuffers:
    """Outputs of moe_balance_loss for S sequences of up to M tokens in all, and its workspace."""
    M: int
    E: int
    S: int
    expert_counts: torch.Tensor
    prob_sums: torch.Tensor
    seq_tokens: torch.Tensor
    loss: torch.Tensor
    workspace: torch.Tensor


def alloc_balance_buffers(M: int, E: int, S: int = 1, device="cuda") -> BalanceBuffers:
    nbytes = moe_balance_workspace_bytes(M, E, S)
    if nbytes < 0:
        raise ValueError("unsupported sizes")
    i32, f32 = dict(dtype=torch.int32, device=device), dict(dtype=torch.float32, device=device)
    return BalanceBuffers(M, E, S, torch.empty((S, E), **i32), torch.empty((S, E), **f32), torch.empty(S, **i32),
                          torch.empty(S, **f32), torch.empty(nbytes, dtype=torch.uint8, device=device))


def balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor, bufs: BalanceBuffers,
                 seq_offsets: torch.Tensor | None = None, row_valid: torch.Tensor | None = None,
                 stream=None) -> BalanceBuffers:
    """The balance loss of each sequence, its tokens' choices per expert and
    its sums of probabilities. seq_offsets: int32 [S + 1] (None: one sequence
    of all rows); row_valid: bool [M] (None: all rows count)."""
    moe_balance_loss(logits, topk_ids, bufs.expert_counts, bufs.prob_sums, bufs.seq_tokens, bufs.loss, bufs.workspace,
                     seq_offsets=seq_offsets, row_valid=row_valid, stream=stream)
    return bufs


def balance_loss_backward(logits: torch.Tensor, top_k: int, expert_counts: torch.Tensor, seq_tokens: torch.Tensor,
                          grad_loss: torch.Tensor, seq_offsets: torch.Tensor | None = None,
                          row_valid: torch.Tensor | None = None, grad_logits: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """The gradient of sum(grad_loss * loss) with respect to the logits, fp32
    [M, E]. Rows of no sequence are left as they were in grad_logits (zeros
    if it is allocated here)."""
    if grad_logits is None:
        with _memory_of(stream, logits.device):
            grad_logits = torch.empty_like(logits) if seq_offsets is None else torch.zeros_like(logits)
    moe_balance_loss_backward(logits, top_k, expert_counts, seq_tokens, grad_loss, grad_logits,
                              seq_offsets=seq_offsets, row_valid=row_valid, stream=stream)
    return grad_logits


def _lora_workspace(x, lora_a, lora_b, backward, stream):
    M, K = x.shape
    nbytes = moe_lora_workspace_bytes(M, lora_a.shape[0], K, lora_b.shape[1], lora_a.shape[1], backward)
    if nbytes < 0:
        raise ValueError("unsupported adapter sizes")
    with _memory_of(stream, x.device):
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)


def lora_forward(x: torch.Tensor, adapter_ids: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
                 scales: torch.Tensor | None = None, base: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, h: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = base[t] + scales[a] * B_a (A_a x[t]) with a = adapter_ids[t]
    (outside [0, L): no adapter, out[t] = base[t]). x bf16 [M, K]; adapter_ids
    int32 [M]; lora_a bf16 [L, rank, K]; lora_b bf16 [L, N, rank]; base and out
    bf16 or fp32 [M, N] (out allocated like base, else bf16; out=base adds in
    place). h: fp32 [M, rank] to keep A x in for lora_backward."""
    if out is None:
        with _memory_of(stream, x.device):
            out = torch.empty((x.shape[0], lora_b.shape[1]), dtype=base.dtype if base is not None else torch.bfloat16,
                              device=x.device)
    if workspace is None:
        workspace = _lora_workspace(x, lora_a, lora_b, False, stream)
    moe_lora_forward(x, adapter_ids, lora_a, lora_b, out, workspace, scales=scales, base=base, h=h, stream=stream)
    return out


def lora_backward(grad_out: torch.Tensor, x: torch.Tensor, adapter_ids: torch.Tensor, h: torch.Tensor,
                  lora_a: torch.Tensor, lora_b: torch.Tensor, scales: torch.Tensor | None = None,
                  dx_base: torch.Tensor | None = None, need_dx: bool = True, grads: tuple | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> tuple:
    """Gradients of lora_forward: (dx bf16 [M, K] = dx_base + the adapters'
    part, grad_a fp32 like lora_a, grad_b fp32 like lora_b). need_dx=False
    leaves dx out (None). grads: buffers of an earlier call to write into; one
    that is None there is allocated if it is needed."""
    dx, grad_a, grad_b = (None, None, None) if grads is None else grads
    if not need_dx:
        dx = None
    if (need_dx and dx is None) or grad_a is None or grad_b is None:
        with _memory_of(stream, x.device):
            if need_dx and dx is None:
                dx = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
            if grad_a is None:
                grad_a = torch.empty(lora_a.shape, dtype=torch.float32, device=x.device)
            if grad_b is None:
                grad_b = torch.empty(lora_b.shape, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = _lora_workspace(x, lora_a, lora_b, True, stream)
    moe_lora_backward(grad_out, x, adapter_ids, h, lora_a, lora_b, grad_a, grad_b, workspace, scales=scales, dx=dx,
                      dx_base=dx_base, stream=stream)
    return dx, grad_a, grad_b


def route_scored(logits: torch.Tensor, rb: RouteBuffers, scoring: str = "softmax", bias: torch.Tensor | None = None,
                 n_groups: int = 1, top_groups: int = 1, group_top: int = 1, renormalise: bool = True,
                 scale: float = 1.0, row_valid: torch.Tensor | None = None, grouping: bool = True,
                 stream=None) -> RouteBuffers:
    """route_align by scores: softmax or sigmoid of the logits, a bias [E] in
    the choice only, the top_k experts of the top_groups best of n_groups groups
    (by the sum of a group's group_top highest), weights renormalised and
    scaled. row_valid: bool [M] (None: all); padding rows get ids of -1 and
    weights of 0. grouping=False: only topk_ids and topk_weights are written."""
    lists = dict(sorted_token_ids=rb.sorted_token_ids, block_expert_ids=rb.block_expert_ids,
                 expert_offsets=rb.expert_offsets, num_tokens_post_pad=rb.num_tokens_post_pad,
                 cap=rb.cap) if grouping else {}
    moe_route_scored(logits, rb.top_k, rb.topk_ids, rb.topk_weights, scoring=scoring, bias=bias, n_groups=n_groups,
                     top_groups=top_groups, group_top=group_top, renormalise=renormalise, scale=scale,
                     row_valid=row_valid, block_m=rb.block_m, stream=stream, **lists)
    return rb


def route_scored_backward(logits: torch.Tensor, topk_ids: torch.Tensor, grad_weights: torch.Tensor,
                          scoring: str = "softmax", renormalise: bool = True, scale: float = 1.0,
                          grad_base: torch.Tensor | None = None, grad_logits: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """The gradient of sum(grad_weights * topk_weights) with respect to the
    logits plus grad_base (None: zeros), fp32 [M, E]. grad_logits=grad_base adds
    in place."""
    if grad_logits is None:
        with _memory_of(stream, logits.device):
            grad_logits = torch.empty_like(logits)
    moe_route_scored_backward(logits, topk_ids, grad_weights, grad_logits, scoring=scoring, renormalise=renormalise,
                              scale=scale, grad_base=grad_base, stream=stream)
    return grad_logits


@dataclass
class NormBuffers:
    """Outputs of moe_add_rms_norm for M rows of N columns; those that are None
    are not wanted. out8 holds e4m3 values of out / scales."""
    M: int
    N: int
    quant_group: int
    residual_out: torch.Tensor | None
    out: torch.Tensor | None
    out8: torch.Tensor | None
    scales: torch.Tensor | None
    rstd: torch.Tensor | None


def alloc_norm_buffers(M: int, N: int, residual_dtype: torch.dtype | None = None, out: bool = True, rstd: bool = False,
                       quant_group: int = 0, device="cuda") -> NormBuffers:
    """residual_dtype: the stream's type (None: no residual_out; set it to the
    residual itself for an update in place). quant_group: columns that share a
    scale of the 8-bit output (N: a row; 0: no such output)."""
    if quant_group < 0 or (quant_group and N % quant_group):
        raise ValueError("quant_group must divide N")

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=device)

    return NormBuffers(M, N, quant_group, None if residual_dtype is None else empty((M, N), residual_dtype),
                       empty((M, N), torch.bfloat16) if out else None,
                       empty((M, N), torch.float8_e4m3fn) if quant_group else None,
                       empty((M, N // quant_group), torch.float32) if quant_group else None,
                       empty(M, torch.float32) if rstd else None)


def add_rms_norm(x: torch.Tensor | None, weight: torch.Tensor, bufs: NormBuffers, residual: torch.Tensor | None = None,
                 eps: float = 1e-6, stream=None) -> NormBuffers:
    """h = x + residual (either may be None) to bufs.residual_out, its
    root-mean-square norm times weight to bufs.out (bf16) and bufs.out8 with
    bufs.scales, 1 / sqrt(mean(h^2) + eps) to bufs.rstd."""
    moe_add_rms_norm(weight, x, residual, eps, residual_out=bufs.residual_out, out=bufs.out, out8=bufs.out8,
                     scales=bufs.scales, quant_group=bufs.quant_group, rstd=bufs.rstd, stream=stream)
    return bufs


def add_rms_norm_backward(grad_out: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                          grad_residual: torch.Tensor | None = None, need_h: bool = True, need_weight: bool = True,
                          grads: tuple | None = None, workspace: torch.Tensor | None = None, stream=None) -> tuple:
    """Gradients of add_rms_norm: (grad_h like h = grad_residual + the norm's
    part, of x and of the residual alike; grad_weight fp32 [N]). h: the
    forward's residual_out (x, where there was no residual). need_h=False or
    need_weight=False leave one out (None). grads: buffers of an earlier call to
    write into; one that is None there is allocated if it is needed."""
    grad_h, grad_weight = (None, None) if grads is None else grads
    grad_h = grad_h if need_h else None
    grad_weight = grad_weight if need_weight else None
    M, N = h.shape
    with _memory_of(stream, h.device):
        if need_h and grad_h is None:
            grad_h = torch.empty((M, N), dtype=h.dtype, device=h.device)
        if need_weight and grad_weight is None:
            grad_weight = torch.empty(N, dtype=torch.float32, device=h.device)
        if need_weight and workspace is None:
            nbytes = moe_add_rms_norm_workspace_bytes(M, N)
            if nbytes < 0:
                raise ValueError("unsupported sizes")
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=h.device)
    moe_add_rms_norm_backward(grad_out, h, rstd, weight, grad_h, grad_weight, workspace, grad_residual=grad_residual,
                              stream=stream)
    return grad_h, grad_weight


def _grads_workspace(grads, device, workspace, stream):
    if workspace is None:
        nbytes = moe_grad_norm_workspace_bytes(len(grads))
        if nbytes < 0:
            raise ValueError("too many gradients")
        with _memory_of(stream, device):
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace


def grad_sumsq(grads, sumsq: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The sum of the squares of all elements of a sequence of gradients (bf16
    or fp32), float64 [1]. A data-parallel job may add it over its ranks."""
    if not grads and sumsq is None:
        raise ValueError("no gradients, and no sumsq to write to")
    device = sumsq.device if sumsq is not None else grads[0].device
    workspace = _grads_workspace(grads, device, workspace, stream)
    if sumsq is None:
        with _memory_of(stream, device):
            sumsq = torch.empty(1, dtype=torch.float64, device=device)
    moe_grad_sumsq(grads, sumsq, workspace, stream=stream)
    return sumsq


def grad_clip(grads, sumsq: torch.Tensor, max_norm: float, out=None, norm: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """Scales gradients whose norm sqrt(sumsq) is above max_norm down to it, in
    place or into the tensors of out; returns the norm, float32 [1]."""
    if norm is None:
        with _memory_of(stream, sumsq.device):
            norm = torch.empty(1, dtype=torch.float32, device=sumsq.device)
    moe_grad_clip(grads, grads if out is None else out, sumsq, max_norm, norm=norm, stream=stream)
    return norm


def clip_grad_norm(grads, max_norm: float, out=None, workspace: torch.Tensor | None = None,
                   norm: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """grad_sumsq and grad_clip in one call: clips the gradients by their global
    norm, in place or into the tensors of out; returns the norm before, float32 [1]."""
    if not grads:
        raise ValueError("no gradients")
    device = grads[0].device
    workspace = _grads_workspace(grads, device, workspace, stream)
    if norm is None:
        with _memory_of(stream, device):
            norm = torch.empty(1, dtype=torch.float32, device=device)
    moe_clip_grad_norm(grads, grads if out is None else out, max_norm, workspace, norm=norm, stream=stream)
    return norm
