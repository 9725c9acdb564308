"""ctypes binding of libmoe_w4a16.so (the C ABI declared in include/moe_w4a16.h).

Argument marshalling only: every function here checks the tensors it is
given (device, dtype, contiguity, shape), turns them into raw pointers and
calls the entry point of the same name on the caller's current HIP stream.
All the work runs in the library's kernels. There is no fallback: if the
library is not built, or a call returns an error status, an exception is
raised.
"""
from __future__ import annotations

import ctypes
import operator
import os
from array import array

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libmoe_w4a16.so")
_lib = None

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_CAPACITY = -3
MOE_ERR_WORKSPACE = -4
MOE_ERR_HIP = -5
MOE_ERR_SCRATCH = -6

MOE_DTYPE_BF16 = 0
MOE_DTYPE_F32 = 1
_SIDE_DTYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_F32}
_DTYPE_OF = operator.attrgetter("dtype")

MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
_SCORINGS = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}

KIND_W13 = 0
KIND_W2 = 1
GROUP = 32

_i32, _i64, _vp, _cp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_char_p

# name -> (restype, argtypes), in the order of the header
_SIGNATURES = {
    "moe_w4a16_abi_version": (_i32, []),
    "moe_w4a16_status_string": (_cp, [ctypes.c_int]),
    "moe_route_align_capacity": (_i64, [_i32, _i32, _i32, _i32]),
    "moe_route_align": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp]),
    "moe_w4a16_packed_bytes": (_i64, [_i32, _i32, _i32, _i32]),
    "moe_w4a16_repack": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "moe_w4a16_unpack": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_w4a16_workspace_bytes": (_i64, [_i32, _i32, _i32, _i32, _i32]),
    "moe_w4a16_preferred_block_m": (_i32, [_i32, _i32, _i32, _i32, _i32]),
    "moe_w4a16_forward": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                         _i64, _vp, _vp, _vp, _i64, _vp, _vp]),
    "moe_w4a16_fc1": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _vp,
                                     _i64, _vp]),
    "moe_w4a16_fc2": (ctypes.c_int, [_i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp,
                                     _i64, _vp, _vp]),
    "moe_w4a16_layer": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _i64, _vp, _vp, _vp, _i64, _vp, _vp, _vp]),
    "moe_mxfp4_packed_bytes": (_i64, [_i32, _i32, _i32]),
    "moe_mxfp4_repack": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp]),
    "moe_mxfp4_unpack": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
}
_SIGNATURES["moe_balance_workspace_bytes"] = (_i64, [_i32, _i32, _i32])
_SIGNATURES["moe_balance_loss"] = (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                                  _i64, _vp])
_SIGNATURES["moe_balance_loss_backward"] = (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp,
                                                           _vp])
_SIGNATURES["moe_lora_workspace_bytes"] = (_i64, [_i32, _i32, _i32, _i32, _i32, _i32])
_SIGNATURES["moe_lora_forward"] = (ctypes.c_int, [_vp, _i64, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                                  _i64, _vp, _i64, _i32, _vp, _vp, _i64, _vp])
_SIGNATURES["moe_lora_backward"] = (ctypes.c_int, [_vp, _i64, _i32, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                                   _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp])
_f32 = ctypes.c_float
_SIGNATURES["moe_route_scored"] = (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _vp, _i32, _i32, _i32, _i32, _f32, _vp,
                                                  _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp])
_SIGNATURES["moe_route_scored_backward"] = (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _vp, _vp,
                                                           _vp])
_SIGNATURES["moe_add_rms_norm"] = (ctypes.c_int, [_vp, _i64, _vp, _i64, _i32, _i32, _i32, _vp, ctypes.c_double, _vp, _i64,
                                                  _vp, _i64, _vp, _i64, _vp, _i32, _vp, _vp])
_SIGNATURES["moe_add_rms_norm_workspace_bytes"] = (_i64, [_i32, _i32])
_SIGNATURES["moe_add_rms_norm_backward"] = (ctypes.c_int, [_vp, _i64, _vp, _i64, _i32, _vp, _i32, _i32, _vp, _vp, _i64,
                                                           _vp, _i64, _vp, _vp, _i64, _vp])
_SIGNATURES["moe_grad_norm_workspace_bytes"] = (_i64, [_i32])
_SIGNATURES["moe_grad_sumsq"] = (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, _vp, _i64, _vp])
_SIGNATURES["moe_grad_clip"] = (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _f32, _vp, _vp])
_SIGNATURES["moe_clip_grad_norm"] = (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _i64, _vp])
_SIGNATURES["moe_calib_read_granule"] = (_i64, [])
_SIGNATURES["moe_calib_hbm_read"] = (ctypes.c_int, [_vp, _i64, _i32, _vp, _vp])
_SIGNATURES["moe_calib_mfma_f16"] = (ctypes.c_int, [_i64, _i32, _vp, _vp])
_SIGNATURES["moe_w4a16_layer_noalloc"] = (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp,
                                                          _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp])
# the MXFP4 stages take the same arguments as the INT4 ones
for _stage in ("fc1", "fc2", "forward", "layer"):
    _SIGNATURES["moe_mxfp4_" + _stage] = _SIGNATURES["moe_w4a16_" + _stage]


class MoeError(RuntimeError):
    def __init__(self, name: str, status: int):
        super().__init__(f"{name} failed with status {status}: {status_string(status)}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """Load the HIP library (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with `python -m int4_weight_only_moe_amd.build` "
                "(the MoE path has no CPU fallback)")
        handle = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().moe_w4a16_status_string(status).decode()


def _check(name: str, status: int) -> None:
    if status != MOE_OK:
        raise MoeError(name, status)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None, dtype: torch.dtype, what: str) -> int:
    if t is None:
        return 0
    if not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


# ------------------------------------------------------------------ host helpers
def moe_w4a16_abi_version() -> int:
    return lib().moe_w4a16_abi_version()


def moe_route_align_capacity(M: int, E: int, top_k: int, block_m: int) -> int:
    return lib().moe_route_align_capacity(M, E, top_k, block_m)


def moe_w4a16_packed_bytes(E: int, N: int, K: int, group: int = GROUP) -> int:
    return lib().moe_w4a16_packed_bytes(E, N, K, group)


def moe_mxfp4_packed_bytes(E: int, N: int, K: int) -> int:
    return lib().moe_mxfp4_packed_bytes(E, N, K)


def moe_w4a16_workspace_bytes(M: int, E: int, H: int, I: int, top_k: int) -> int:
    return lib().moe_w4a16_workspace_bytes(M, E, H, I, top_k)


def moe_w4a16_preferred_block_m(M: int, E: int, H: int, I: int, top_k: int) -> int:
    return lib().moe_w4a16_preferred_block_m(M, E, H, I, top_k)


# ------------------------------------------------------------------ device calls
def moe_route_align(logits: torch.Tensor, top_k: int, block_m: int, topk_ids: torch.Tensor,
                    topk_weights: torch.Tensor, sorted_token_ids: torch.Tensor,
                    block_expert_ids: torch.Tensor, expert_offsets: torch.Tensor,
                    num_tokens_post_pad: torch.Tensor, cap: int | None = None, stream=None) -> None:
    M, E = logits.shape
    if cap is None:
        cap = sorted_token_ids.numel()
    st = lib().moe_route_align(
        _ptr(logits, torch.float32, "logits"), M, E, top_k, block_m,
        _ptr(topk_ids, torch.int32, "topk_ids"), _ptr(topk_weights, torch.float32, "topk_weights"),
        _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"),
        _ptr(block_expert_ids, torch.int32, "block_expert_ids"),
        _ptr(expert_offsets, torch.int32, "expert_offsets"),
        _ptr(num_tokens_post_pad, torch.int32, "num_tokens_post_pad"), cap, _stream(stream))
    _check("moe_route_align", st)


def moe_w4a16_repack(qweight: torch.Tensor, scales_f16: torch.Tensor, kind: int, packed: torch.Tensor,
                     stream=None) -> None:
    E, N, K2 = qweight.shape
    st = lib().moe_w4a16_repack(
        _ptr(qweight, torch.uint8, "qweight"), _ptr(scales_f16, torch.float16, "scales"),
        E, N, 2 * K2, GROUP, kind, _ptr(packed, torch.uint8, "packed"), _stream(stream))
    _check("moe_w4a16_repack", st)


def moe_w4a16_unpack(packed: torch.Tensor, E: int, N: int, K: int, kind: int, qweight: torch.Tensor,
                     scales_f16: torch.Tensor, stream=None) -> None:
    st = lib().moe_w4a16_unpack(
        _ptr(packed, torch.uint8, "packed"), E, N, K, GROUP, kind,
        _ptr(qweight, torch.uint8, "qweight"), _ptr(scales_f16, torch.float16, "scales"), _stream(stream))
    _check("moe_w4a16_unpack", st)


def moe_mxfp4_repack(qweight: torch.Tensor, scales_e8m0: torch.Tensor, kind: int, packed: torch.Tensor,
                     stream=None) -> None:
    E, N, K2 = qweight.shape
    st = lib().moe_mxfp4_repack(
        _ptr(qweight, torch.uint8, "qweight"), _ptr(scales_e8m0, torch.uint8, "scales_e8m0"),
        E, N, 2 * K2, kind, _ptr(packed, torch.uint8, "packed"), _stream(stream))
    _check("moe_mxfp4_repack", st)


def moe_mxfp4_unpack(packed: torch.Tensor, E: int, N: int, K: int, kind: int, qweight: torch.Tensor,
                     scales_e8m0: torch.Tensor, stream=None) -> None:
    st = lib().moe_mxfp4_unpack(
        _ptr(packed, torch.uint8, "packed"), E, N, K, kind,
        _ptr(qweight, torch.uint8, "qweight"), _ptr(scales_e8m0, torch.uint8, "scales_e8m0"), _stream(stream))
    _check("moe_mxfp4_unpack", st)


def moe_w4a16_forward(x: torch.Tensor, E: int, I: int, top_k: int, block_m: int,
                      topk_weights: torch.Tensor, sorted_token_ids: torch.Tensor,
                      block_expert_ids: torch.Tensor, expert_offsets: torch.Tensor,
                      num_tokens_post_pad: torch.Tensor, w13_packed: torch.Tensor, w2_packed: torch.Tensor,
                      workspace: torch.Tensor, out: torch.Tensor, cap: int | None = None, stream=None,
                      _prefix: str = "moe_w4a16") -> None:
    M, H = x.shape
    if cap is None:
        cap = sorted_token_ids.numel()
    st = getattr(lib(), _prefix + "_forward")(
        _ptr(x, torch.bfloat16, "x"), M, E, H, I, top_k, block_m,
        _ptr(topk_weights, torch.float32, "topk_weights"),
        _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"),
        _ptr(block_expert_ids, torch.int32, "block_expert_ids"),
        _ptr(expert_offsets, torch.int32, "expert_offsets"),
        _ptr(num_tokens_post_pad, torch.int32, "num_tokens_post_pad"), cap,
        _ptr(w13_packed, torch.uint8, "w13_packed"), _ptr(w2_packed, torch.uint8, "w2_packed"),
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        _ptr(out, torch.bfloat16, "out"), _stream(stream))
    _check(_prefix + "_forward", st)


def moe_w4a16_fc1(x: torch.Tensor, E: int, I: int, top_k: int, block_m: int, sorted_token_ids: torch.Tensor,
                  block_expert_ids: torch.Tensor, num_tokens_post_pad: torch.Tensor, w13_packed: torch.Tensor,
                  workspace: torch.Tensor, cap: int | None = None, stream=None, _prefix: str = "moe_w4a16") -> None:
    M, H = x.shape
    if cap is None:
        cap = sorted_token_ids.numel()
    st = getattr(lib(), _prefix + "_fc1")(
        _ptr(x, torch.bfloat16, "x"), M, E, H, I, top_k, block_m,
        _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"),
        _ptr(block_expert_ids, torch.int32, "block_expert_ids"),
        _ptr(num_tokens_post_pad, torch.int32, "num_tokens_post_pad"), cap,
        _ptr(w13_packed, torch.uint8, "w13_packed"), _ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream))
    _check(_prefix + "_fc1", st)


def moe_w4a16_fc2(M: int, E: int, H: int, I: int, top_k: int, block_m: int, topk_weights: torch.Tensor,
                  sorted_token_ids: torch.Tensor, block_expert_ids: torch.Tensor,
                  num_tokens_post_pad: torch.Tensor, w2_packed: torch.Tensor, workspace: torch.Tensor,
                  out: torch.Tensor, cap: int | None = None, stream=None, _prefix: str = "moe_w4a16") -> None:
    if cap is None:
        cap = sorted_token_ids.numel()
    st = getattr(lib(), _prefix + "_fc2")(
        M, E, H, I, top_k, block_m, _ptr(topk_weights, torch.float32, "topk_weights"),
        _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"),
        _ptr(block_expert_ids, torch.int32, "block_expert_ids"),
        _ptr(num_tokens_post_pad, torch.int32, "num_tokens_post_pad"), cap,
        _ptr(w2_packed, torch.uint8, "w2_packed"), _ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _ptr(out, torch.bfloat16, "out"), _stream(stream))
    _check(_prefix + "_fc2", st)


def moe_w4a16_layer(logits: torch.Tensor, x: torch.Tensor, I: int, top_k: int, block_m: int,
                    topk_ids: torch.Tensor, topk_weights: torch.Tensor, sorted_token_ids: torch.Tensor,
                    block_expert_ids: torch.Tensor, expert_offsets: torch.Tensor,
                    num_tokens_post_pad: torch.Tensor, w13_packed: torch.Tensor, w2_packed: torch.Tensor,
                    workspace: torch.Tensor, out: torch.Tensor, cap: int | None = None, stream=None,
                    stage_events=None, _prefix: str = "moe_w4a16") -> None:
    """stage_events: None or a pair of raw hipEvent_t handles (ints)."""
    M, E = logits.shape
    H = x.shape[1]
    if x.shape[0] != M:
        raise ValueError("logits and x must have the same number of rows")
    if cap is None:
        cap = sorted_token_ids.numel()
    ev = None
    if stage_events is not None:
        ev = (ctypes.c_void_p * 2)(int(stage_events[0]), int(stage_events[1]))
    st = getattr(lib(), _prefix + "_layer")(
        _ptr(logits, torch.float32, "logits"), _ptr(x, torch.bfloat16, "x"), M, E, H, I, top_k, block_m,
        _ptr(topk_ids, torch.int32, "topk_ids"), _ptr(topk_weights, torch.float32, "topk_weights"),
        _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"),
        _ptr(block_expert_ids, torch.int32, "block_expert_ids"),
        _ptr(expert_offsets, torch.int32, "expert_offsets"),
        _ptr(num_tokens_post_pad, torch.int32, "num_tokens_post_pad"), cap,
        _ptr(w13_packed, torch.uint8, "w13_packed"), _ptr(w2_packed, torch.uint8, "w2_packed"),
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _ptr(out, torch.bfloat16, "out"),
        _stream(stream), ev)
    _check(_prefix + "_layer", st)


def moe_w4a16_layer_noalloc(logits: torch.Tensor, x: torch.Tensor, I: int, top_k: int, block_m: int,
                            topk_ids: torch.Tensor, topk_weights: torch.Tensor, sorted_token_ids: torch.Tensor,
                            block_expert_ids: torch.Tensor, expert_offsets: torch.Tensor,
                            num_tokens_post_pad: torch.Tensor, w13_packed: torch.Tensor, w2_packed: torch.Tensor,
                            out: torch.Tensor, cap: int | None = None, stream=None) -> None:
    """moe_w4a16_layer with the library's static scratch as the workspace."""
    M, E = logits.shape
    H = x.shape[1]
    if x.shape[0] != M:
        raise ValueError("logits and x must have the same number of rows")
    if cap is None:
        cap = sorted_token_ids.numel()
    st = lib().moe_w4a16_layer_noalloc(
        _ptr(logits, torch.float32, "logits"), _ptr(x, torch.bfloat16, "x"), M, E, H, I, top_k, block_m,
        _ptr(topk_ids, torch.int32, "topk_ids"), _ptr(topk_weights, torch.float32, "topk_weights"),
        _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"),
        _ptr(block_expert_ids, torch.int32, "block_expert_ids"),
        _ptr(expert_offsets, torch.int32, "expert_offsets"),
        _ptr(num_tokens_post_pad, torch.int32, "num_tokens_post_pad"), cap,
        _ptr(w13_packed, torch.uint8, "w13_packed"), _ptr(w2_packed, torch.uint8, "w2_packed"),
        _ptr(out, torch.bfloat16, "out"), _stream(stream))
    _check("moe_w4a16_layer_noalloc", st)


NOALLOC_SCRATCH_BYTES = 48 << 20  # MOE_W4A16_NOALLOC_SCRATCH_BYTES in the header


def moe_mxfp4_forward(*args, **kw) -> None:
    """moe_w4a16_forward with moe_mxfp4_repack weights."""
    moe_w4a16_forward(*args, _prefix="moe_mxfp4", **kw)


def moe_mxfp4_fc1(*args, **kw) -> None:
    """moe_w4a16_fc1 with moe_mxfp4_repack weights."""
    moe_w4a16_fc1(*args, _prefix="moe_mxfp4", **kw)


def moe_mxfp4_fc2(*args, **kw) -> None:
    """moe_w4a16_fc2 with moe_mxfp4_repack weights."""
    moe_w4a16_fc2(*args, _prefix="moe_mxfp4", **kw)


def moe_mxfp4_layer(*args, **kw) -> None:
    """moe_w4a16_layer with moe_mxfp4_repack weights."""
    moe_w4a16_layer(*args, _prefix="moe_mxfp4", **kw)


# ------------------------------------------------------------------ operators beside the layer
def _refuse(t: torch.Tensor, dtype, shape: tuple, what: str, device: torch.device, layout: str):
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{what} must {layout}")


def _shaped(t: torch.Tensor | None, dtype, shape: tuple, what: str, device: torch.device) -> int:
    """The pointer of a contiguous tensor of this type and shape on this device (None: NULL)."""
    if t is None:
        return 0
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device:
        return t.data_ptr()
    _refuse(t, dtype, shape, what, device, "be contiguous")


def _matrix(t: torch.Tensor | None, dtype, shape: tuple, what: str, device: torch.device) -> tuple:
    """(pointer, row stride) of a matrix whose rows are contiguous (None: NULL)."""
    if t is None:
        return 0, 0
    if t.dtype is dtype and t.shape == shape and t.device == device:
        rows, cols = t.stride()
        if cols == 1 or shape[1] <= 1:
            # the stride of a single row says nothing
            return t.data_ptr(), rows if shape[0] > 1 else -(-shape[1] // 8) * 8
    _refuse(t, dtype, shape, what, device, "have contiguous rows")


def _buffer(t: torch.Tensor, what: str, device: torch.device) -> tuple:
    """(pointer, bytes) of a workspace."""
    if t.dtype is not torch.uint8 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous uint8 tensor on {device}")
    return t.data_ptr(), t.numel()


def _on_device(device: torch.device, name: str, stream, *args) -> None:
    """Call an entry point with `device` current, on `stream` or that device's current stream."""
    if device.type != "cuda":
        raise ValueError(f"{name} needs device tensors")
    if stream is None:  # the stream's handle without the object that torch.cuda.current_stream makes
        stream = torch._C._cuda_getCurrentRawStream(device.index)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    fn = getattr(lib(), name)
    if device.index == torch.cuda.current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != MOE_OK:
        raise MoeError(name, status)


def moe_balance_workspace_bytes(M: int, E: int, S: int) -> int:
    return lib().moe_balance_workspace_bytes(M, E, S)


def _balance_inputs(logits, seq_offsets, S, row_valid):
    if logits.dim() != 2:
        raise ValueError("logits must be a matrix [M, E]")
    dev = logits.device
    M, E = logits.shape
    if row_valid is not None and row_valid.dtype == torch.bool:
        row_valid = row_valid.view(torch.uint8)
    return (dev, M, E, _shaped(logits, torch.float32, (M, E), "logits", dev),
            _shaped(seq_offsets, torch.int32, (S + 1,), "seq_offsets", dev),
            _shaped(row_valid, torch.uint8, (M,), "row_valid", dev))


def moe_balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor, expert_counts: torch.Tensor,
                     prob_sums: torch.Tensor, seq_tokens: torch.Tensor, loss: torch.Tensor, workspace: torch.Tensor,
                     seq_offsets: torch.Tensor | None = None, row_valid: torch.Tensor | None = None,
                     stream=None) -> None:
    """row_valid: bool or uint8 [M]. S is the length of `loss`."""
    S = loss.numel()
    dev, M, E, p_logits, p_off, p_valid = _balance_inputs(logits, seq_offsets, S, row_valid)
    k = topk_ids.shape[-1]
    _on_device(dev, "moe_balance_loss", stream, p_logits, _shaped(topk_ids, torch.int32, (M, k), "topk_ids", dev), M, E,
               k, p_off, S, p_valid, _shaped(expert_counts, torch.int32, (S, E), "expert_counts", dev),
               _shaped(prob_sums, torch.float32, (S, E), "prob_sums", dev),
               _shaped(seq_tokens, torch.int32, (S,), "seq_tokens", dev),
               _shaped(loss, torch.float32, (S,), "loss", dev),
               *_buffer(workspace, "workspace", dev))


def moe_balance_loss_backward(logits: torch.Tensor, top_k: int, expert_counts: torch.Tensor,
                              seq_tokens: torch.Tensor, grad_loss: torch.Tensor, grad_logits: torch.Tensor,
                              seq_offsets: torch.Tensor | None = None, row_valid: torch.Tensor | None = None,
                              stream=None) -> None:
    S = seq_tokens.numel()
    dev, M, E, p_logits, p_off, p_valid = _balance_inputs(logits, seq_offsets, S, row_valid)
    _on_device(dev, "moe_balance_loss_backward", stream, p_logits, M, E, top_k, p_off, S, p_valid,
               _shaped(expert_counts, torch.int32, (S, E), "expert_counts", dev),
               _shaped(seq_tokens, torch.int32, (S,), "seq_tokens", dev),
               _shaped(grad_loss, torch.float32, (S,), "grad_loss", dev),
               _shaped(grad_logits, torch.float32, (M, E), "grad_logits", dev))


def moe_lora_workspace_bytes(M: int, L: int, K: int, N: int, rank: int, backward: bool = False) -> int:
    return lib().moe_lora_workspace_bytes(M, L, K, N, rank, int(backward))


def _lora_sizes(x, lora_a, lora_b):
    if x.dim() != 2 or lora_a.dim() != 3 or lora_b.dim() != 3:
        raise ValueError("x must be [M, K], lora_a [L, rank, K] and lora_b [L, N, rank]")
    M, K = x.shape
    L, r, _ = lora_a.shape
    return M, L, K, lora_b.shape[1], r


def _side_dtype(t: torch.Tensor, what: str) -> int:
    if t.dtype not in _SIDE_DTYPES:
        raise ValueError(f"{what} must be bfloat16 or float32, got {t.dtype}")
    return _SIDE_DTYPES[t.dtype]


def moe_lora_forward(x: torch.Tensor, adapter_ids: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
                     out: torch.Tensor, workspace: torch.Tensor, scales: torch.Tensor | None = None,
                     base: torch.Tensor | None = None, h: torch.Tensor | None = None, stream=None) -> None:
    M, L, K, N, r = _lora_sizes(x, lora_a, lora_b)
    dev, bf16, f32 = x.device, torch.bfloat16, torch.float32
    kind = _side_dtype(out, "out")
    px, ldx = _matrix(x, bf16, (M, K), "x", dev)
    pb, ldb = _matrix(base, out.dtype, (M, N), "base", dev)
    po, ldo = _matrix(out, out.dtype, (M, N), "out", dev)
    _on_device(dev, "moe_lora_forward", stream, px, ldx, _shaped(adapter_ids, torch.int32, (M,), "adapter_ids", dev),
               M, L, K, N, r, _shaped(lora_a, bf16, (L, r, K), "lora_a", dev),
               _shaped(lora_b, bf16, (L, N, r), "lora_b", dev), _shaped(scales, f32, (L,), "scales", dev), pb, ldb,
               po, ldo, kind, _shaped(h, f32, (M, r), "h", dev),
               *_buffer(workspace, "workspace", dev))


def moe_lora_backward(grad_out: torch.Tensor, x: torch.Tensor, adapter_ids: torch.Tensor, h: torch.Tensor,
                      lora_a: torch.Tensor, lora_b: torch.Tensor, grad_a: torch.Tensor, grad_b: torch.Tensor,
                      workspace: torch.Tensor, scales: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                      dx_base: torch.Tensor | None = None, stream=None) -> None:
    M, L, K, N, r = _lora_sizes(x, lora_a, lora_b)
    dev, bf16, f32 = x.device, torch.bfloat16, torch.float32
    kind = _side_dtype(grad_out, "grad_out")
    pg, ldg = _matrix(grad_out, grad_out.dtype, (M, N), "grad_out", dev)
    px, ldx = _matrix(x, bf16, (M, K), "x", dev)
    pb, ldb = _matrix(dx_base, bf16, (M, K), "dx_base", dev)
    pd, ldd = _matrix(dx, bf16, (M, K), "dx", dev)
    _on_device(dev, "moe_lora_backward", stream, pg, ldg, kind, px, ldx,
               _shaped(adapter_ids, torch.int32, (M,), "adapter_ids", dev), _shaped(h, f32, (M, r), "h", dev), M, L, K,
               N, r, _shaped(lora_a, bf16, (L, r, K), "lora_a", dev), _shaped(lora_b, bf16, (L, N, r), "lora_b", dev),
               _shaped(scales, f32, (L,), "scales", dev), pb, ldb, pd, ldd,
               _shaped(grad_a, f32, (L, r, K), "grad_a", dev), _shaped(grad_b, f32, (L, N, r), "grad_b", dev),
               *_buffer(workspace, "workspace", dev))


def _scoring(name: str) -> int:
    if name not in _SCORINGS:
        raise ValueError(f"scoring must be one of {tuple(_SCORINGS)}, got {name!r}")
    return _SCORINGS[name]


def moe_route_scored(logits: torch.Tensor, top_k: int, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                     scoring: str = "softmax", bias: torch.Tensor | None = None, n_groups: int = 1,
                     top_groups: int = 1, group_top: int = 1, renormalise: bool = True, scale: float = 1.0,
                     row_valid: torch.Tensor | None = None, block_m: int = 16,
                     sorted_token_ids: torch.Tensor | None = None, block_expert_ids: torch.Tensor | None = None,
                     expert_offsets: torch.Tensor | None = None, num_tokens_post_pad: torch.Tensor | None = None,
                     cap: int | None = None, stream=None) -> None:
    """row_valid: bool or uint8 [M]. The four grouping outputs together or none of them."""
    if logits.dim() != 2:
        raise ValueError("logits must be a matrix [M, E]")
    M, E = logits.shape
    dev, i32, f32 = logits.device, torch.int32, torch.float32
    if row_valid is not None and row_valid.dtype == torch.bool:
        row_valid = row_valid.view(torch.uint8)
    if cap is None:
        cap = 0 if sorted_token_ids is None else sorted_token_ids.numel()
    if sorted_token_ids is not None and sorted_token_ids.numel() < cap:
        raise ValueError("sorted_token_ids must have cap entries")
    if block_expert_ids is not None and block_m > 0 and block_expert_ids.numel() < cap // block_m:
        raise ValueError("block_expert_ids must have cap / block_m entries")

    def flat(t, what):
        return 0 if t is None else _shaped(t, i32, (t.numel(),), what, dev)

    _on_device(dev, "moe_route_scored", stream, _shaped(logits, f32, (M, E), "logits", dev), M, E, top_k,
               _scoring(scoring), _shaped(bias, f32, (E,), "bias", dev), n_groups, top_groups, group_top,
               int(renormalise), scale, _shaped(row_valid, torch.uint8, (M,), "row_valid", dev), block_m,
               _shaped(topk_ids, i32, (M, top_k), "topk_ids", dev),
               _shaped(topk_weights, f32, (M, top_k), "topk_weights", dev), flat(sorted_token_ids, "sorted_token_ids"),
               flat(block_expert_ids, "block_expert_ids"), _shaped(expert_offsets, i32, (E + 1,), "expert_offsets", dev),
               _shaped(num_tokens_post_pad, i32, (1,), "num_tokens_post_pad", dev), cap)


def moe_route_scored_backward(logits: torch.Tensor, topk_ids: torch.Tensor, grad_weights: torch.Tensor,
                              grad_logits: torch.Tensor, scoring: str = "softmax", renormalise: bool = True,
                              scale: float = 1.0, grad_base: torch.Tensor | None = None, stream=None) -> None:
    if logits.dim() != 2 or topk_ids.dim() != 2:
        raise ValueError("logits must be [M, E] and topk_ids [M, top_k]")
    M, E = logits.shape
    k = topk_ids.shape[1]
    dev, f32 = logits.device, torch.float32
    _on_device(dev, "moe_route_scored_backward", stream, _shaped(logits, f32, (M, E), "logits", dev), M, E, k,
               _scoring(scoring), int(renormalise), scale, _shaped(topk_ids, torch.int32, (M, k), "topk_ids", dev),
               _shaped(grad_weights, f32, (M, k), "grad_weights", dev),
               _shaped(grad_base, f32, (M, E), "grad_base", dev),
               _shaped(grad_logits, f32, (M, E), "grad_logits", dev))


def moe_add_rms_norm(weight: torch.Tensor, x: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                     eps: float = 1e-6, residual_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     out8: torch.Tensor | None = None, scales: torch.Tensor | None = None, quant_group: int = 0,
                     rstd: torch.Tensor | None = None, stream=None) -> None:
    """out8: uint8 or float8_e4m3fn [M, N]."""
    first = x if x is not None else residual
    if first is None or first.dim() != 2:
        raise ValueError("x or residual must be a matrix [M, N]")
    M, N = first.shape
    dev, bf16, f32 = first.device, torch.bfloat16, torch.float32
    res_type = residual.dtype if residual is not None else bf16
    kind = _side_dtype(first if residual is None else residual, "residual")
    if out8 is not None and out8.dtype == torch.float8_e4m3fn:
        out8 = out8.view(torch.uint8)
    groups = N // quant_group if quant_group > 0 else 0
    px, ldx = _matrix(x, bf16, (M, N), "x", dev)
    pr, ldr = _matrix(residual, res_type, (M, N), "residual", dev)
    ps, lds = _matrix(residual_out, res_type, (M, N), "residual_out", dev)
    po, ldo = _matrix(out, bf16, (M, N), "out", dev)
    p8, ld8 = _matrix(out8, torch.uint8, (M, N), "out8", dev)
    _on_device(dev, "moe_add_rms_norm", stream, px, ldx, pr, ldr, kind, M, N, _shaped(weight, bf16, (N,), "weight", dev),
               eps, ps, lds, po, ldo, p8, ld8, _shaped(scales, f32, (M, groups), "scales", dev), quant_group,
               _shaped(rstd, f32, (M,), "rstd", dev))


def moe_add_rms_norm_workspace_bytes(M: int, N: int) -> int:
    return lib().moe_add_rms_norm_workspace_bytes(M, N)


def moe_add_rms_norm_backward(grad_out: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                              grad_h: torch.Tensor | None = None, grad_weight: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None, grad_residual: torch.Tensor | None = None,
                              stream=None) -> None:
    if grad_out.dim() != 2:
        raise ValueError("grad_out must be a matrix [M, N]")
    M, N = grad_out.shape
    dev, bf16, f32 = grad_out.device, torch.bfloat16, torch.float32
    kind = _side_dtype(h, "h")
    pg, ldg = _matrix(grad_out, bf16, (M, N), "grad_out", dev)
    ph, ldh = _matrix(h, h.dtype, (M, N), "h", dev)
    pr, ldr = _matrix(grad_residual, h.dtype, (M, N), "grad_residual", dev)
    pd, ldd = _matrix(grad_h, h.dtype, (M, N), "grad_h", dev)
    _on_device(dev, "moe_add_rms_norm_backward", stream, pg, ldg, ph, ldh, kind, _shaped(rstd, f32, (M,), "rstd", dev),
               M, N, _shaped(weight, bf16, (N,), "weight", dev), pr, ldr, pd, ldd,
               _shaped(grad_weight, f32, (N,), "grad_weight", dev),
               *((0, 0) if workspace is None else _buffer(workspace, "workspace", dev)))


def moe_grad_norm_workspace_bytes(n: int) -> int:
    return lib().moe_grad_norm_workspace_bytes(n)


def _grad_arrays(grads, device: torch.device) -> tuple:
    """(pointers, sizes, types) of contiguous bf16 or fp32 tensors, as host arrays
    (filled by map: a list of tensors is gone through six times, but not in Python)."""
    T = torch.Tensor
    kinds = list(map(_SIDE_DTYPES.get, map(_DTYPE_OF, grads)))
    if device.type != "cuda" or None in kinds or not set(map(T.get_device, grads)) <= {device.index} or \
            not all(map(T.is_contiguous, grads)):
        raise ValueError(f"gradients must be contiguous bfloat16 or float32 tensors on {device}")
    return array("Q", map(T.data_ptr, grads)), array("q", map(T.numel, grads)), array("i", kinds)


def _address(values: array) -> int:
    return values.buffer_info()[0]


def moe_grad_sumsq(grads, sumsq: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """grads: a sequence of tensors; sumsq: float64 [1]."""
    dev = sumsq.device
    lists = _grad_arrays(grads, dev)
    _on_device(dev, "moe_grad_sumsq", stream, *map(_address, lists), len(grads),
               _shaped(sumsq, torch.float64, (1,), "sumsq", dev), *_buffer(workspace, "workspace", dev))


def _clip_arrays(grads, outs, device: torch.device) -> tuple:
    """(gradients' pointers, results' pointers, sizes, types) as host arrays."""
    ptrs, sizes, kinds = _grad_arrays(grads, device)
    if outs is grads:
        return ptrs, ptrs, sizes, kinds
    if len(outs) != len(grads):
        raise ValueError("outs must have as many tensors as grads")
    to, osizes, okinds = _grad_arrays(outs, device)
    if osizes != sizes or okinds != kinds:
        raise ValueError("outs must have the sizes and types of grads")
    return ptrs, to, sizes, kinds


def moe_grad_clip(grads, outs, sumsq: torch.Tensor, max_norm: float, norm: torch.Tensor | None = None,
                  stream=None) -> None:
    """outs: a sequence of tensors like grads (the same one: in place)."""
    dev = sumsq.device
    lists = _clip_arrays(grads, outs, dev)
    _on_device(dev, "moe_grad_clip", stream, *map(_address, lists), len(grads),
               _shaped(sumsq, torch.float64, (1,), "sumsq", dev), max_norm,
               _shaped(norm, torch.float32, (1,), "norm", dev))


def moe_clip_grad_norm(grads, outs, max_norm: float, workspace: torch.Tensor, sumsq: torch.Tensor | None = None,
                       norm: torch.Tensor | None = None, stream=None) -> None:
    """moe_grad_sumsq and moe_grad_clip in one call."""
    dev = workspace.device
    lists = _clip_arrays(grads, outs, dev)
    _on_device(dev, "moe_clip_grad_norm", stream, *map(_address, lists), len(grads), max_norm,
               _shaped(sumsq, torch.float64, (1,), "sumsq", dev), _shaped(norm, torch.float32, (1,), "norm", dev),
               *_buffer(workspace, "workspace", dev))


# ------------------------------------------------------------------ measurement helpers
def moe_calib_read_granule() -> int:
    return lib().moe_calib_read_granule()


def moe_calib_hbm_read(buf: torch.Tensor, sink: torch.Tensor, stream=None) -> None:
    """Read every byte of `buf` once (attainable HBM read rate); sink: int32
    [workgroups * 256], its XOR = the XOR of buf's 32-bit words."""
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous device tensor")
    nbytes = buf.numel() * buf.element_size()
    st = lib().moe_calib_hbm_read(buf.data_ptr(), nbytes, sink.numel() // 256,
                                  _ptr(sink, torch.int32, "sink"), _stream(stream))
    _check("moe_calib_hbm_read", st)


def moe_calib_mfma_f16(iters: int, sink: torch.Tensor, stream=None) -> None:
    """iters * 8 fp16 MFMAs per wave, 4 waves per workgroup, sink.numel() // 256
    workgroups (attainable matrix-core rate); sink: float32 [workgroups * 256]."""
    st = lib().moe_calib_mfma_f16(iters, sink.numel() // 256, _ptr(sink, torch.float32, "sink"), _stream(stream))
    _check("moe_calib_mfma_f16", st)
