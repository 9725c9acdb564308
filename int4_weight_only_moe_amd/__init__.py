"""MI355X-native weight-only INT4 (group 32) MoE layer.

The layer of "The Throughput Lever: Quantifying the MoE GEMM and Mapping the
Road to B300" (section "Phase 3: The INT4 Marlin MoE Throughput Lever"):
top-k routing, per-expert grouping padded to the tile size, FC1 gate/up with
SiLU*mul and FC2 with the routing-weighted sum, as HIP kernels for gfx950
behind the C ABI of include/moe_w4a16.h, and beside it the router's balance
loss with its gradient (balance_loss, balance_loss_backward) and low-rank
adapters of many requests, forward and backward (lora_forward, lora_backward).
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
