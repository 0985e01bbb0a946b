"""MI355X-native MoE normal-mode layout / dispatch / combine.

Thin Python binding of ``libmoe.so`` (the HIP kernels behind the C ABI of
``include/moe.h``). Functions carry the C names; they only marshal torch tensors
(device pointers, sizes, the current HIP stream) into the C calls, allocate
outputs the caller did not pass, and turn negative status codes into
exceptions. Every step of the computation runs in the library's kernels; there
is no other code path. Importing this package fails if the library is not built
(``python combine_moe_layout_02_amd/build.py``).
"""

import ctypes
import functools
import os
from typing import NamedTuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_OK = 0
MOE_ERR_ARG = -1
MOE_ERR_ALIGN = -2
MOE_ERR_WINDOW = -3
MOE_ERR_UNSUPPORTED = -4
MOE_ERR_HIP = -5
MOE_ERR_SCRATCH = -6
MOE_NOALLOC_SCRATCH_BYTES = 1 << 20

MOE_QUANT_NONE = 0
MOE_QUANT_FP8_E4M3_DYN = 1
MOE_QUANT_INT8_DYN = 2

MOE_MX_E2M1 = 1  # 4-bit codes, blocks of 32 with an E8M0 scale
MOE_MX_E4M3 = 2  # 8-bit codes

MOE_MX_PLAIN = 0
MOE_MX_GATED = 1

MOE_BF16 = 1  # element types of a norm's weight and of the router's logits
MOE_FP32 = 2

MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1

MOE_LAYOUT_AUTO = 0
MOE_LAYOUT_MULTI = 1
MOE_LAYOUT_SINGLE = 2

EXPORTED = (
    "moe_slot_bytes", "moe_window_bytes", "moe_slot_offsets", "moe_layout", "moe_layout_ex", "moe_dispatch",
    "moe_dispatch_workspace_bytes", "moe_dispatch_ws", "moe_dispatch_noalloc",
    "moe_layout_dispatch", "moe_layout_dispatch_ex", "moe_layout_dispatch_workspace_bytes",
    "moe_layout_ws", "moe_dispatch_planned", "moe_layout_dispatch_ws", "moe_combine", "moe_combine_scatter", "moe_combine_staged",
    "moe_unpack", "moe_unpack_padded", "moe_dedup_window_bytes", "moe_rank_rows", "moe_dispatch_dedup",
    "moe_expand_dedup", "moe_status_string", "moe_plan_layout", "moe_plan_dispatch_ws",
    "moe_plan_layout_dispatch", "moe_plan_combine", "moe_plan_layout_ws", "moe_plan_dispatch_planned", "moe_plan_run",
    "moe_combine_backward", "moe_combine_backward_mx", "moe_dispatch_backward", "moe_combine_checkpoint",
    "moe_mx_row_bytes", "moe_mx_quantize", "moe_mx_dequantize", "moe_mx_product",
    "moe_row_quantize", "moe_row_dequantize", "moe_scaled_product", "moe_rms_norm", "moe_rms_norm_backward",
    "moe_rms_norm_backward_workspace_bytes", "moe_balance_loss", "moe_balance_loss_backward",
    "moe_balance_loss_workspace_bytes",
)

# include/moe_probe.h: bandwidth probes for the measurement, not part of the path
PROBES = ("moe_probe_fill", "moe_probe_read", "moe_probe_copy")


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with `python combine_moe_layout_02_amd/build.py` "
            "(hipcc, gfx950). There is no fallback implementation."
        )
    lib = ctypes.CDLL(_LIB_PATH)
    missing = [name for name in EXPORTED + PROBES if not hasattr(lib, name)]
    if missing:
        raise ImportError(f"{_LIB_PATH} is stale (missing {missing}); rebuild it with "
                          "`python combine_moe_layout_02_amd/build.py`")
    P, I32, I64, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    sig = {
        "moe_slot_bytes": (I64, [I32]),
        "moe_window_bytes": (I64, [I32, I32, I32]),
        "moe_slot_offsets": (ctypes.c_int, [I32, I32, P, P, P, P]),
        "moe_layout": (ctypes.c_int, [P, I32, I32, I32, I32, I32] + [P] * 9 + [P]),
        "moe_layout_ex": (ctypes.c_int, [P, I32, I32, I32, I32, I32] + [P] * 9 + [I32, P]),
        "moe_dispatch": (ctypes.c_int, [P, P, I32, I32, I32, I32, I32, P, I64, P]),
        "moe_dispatch_workspace_bytes": (I64, [I32, I32, I32]),
        "moe_dispatch_ws": (ctypes.c_int, [P, P, I32, I32, I32, I32, I32, P, I64, P, I64, P]),
        "moe_dispatch_noalloc": (ctypes.c_int, [P, P, I32, I32, I32, I32, I32, P, I64, P]),
        "moe_layout_dispatch": (ctypes.c_int, [P, I32, I32, I32, I32, I32] + [P] * 9 +
                                [P, I32, I32, I32, P, I64, P]),
        "moe_layout_dispatch_ex": (ctypes.c_int, [P, I32, I32, I32, I32, I32] + [P] * 9 +
                                   [P, I32, I32, I32, P, I64, I32, P]),
        "moe_layout_dispatch_workspace_bytes": (I64, [I32, I32, I32, I32, I32, I32, I32]),
        "moe_layout_ws": (ctypes.c_int, [P, I32, I32, I32, I32, I32] + [P] * 9 + [I32, I32, P, I64, P]),
        "moe_dispatch_planned": (ctypes.c_int, [P, P, I32, I32, I32, I32, I32, I32, P, I64, P, I64, P]),
        "moe_layout_dispatch_ws": (ctypes.c_int, [P, I32, I32, I32, I32, I32] + [P] * 9 +
                                   [P, I32, I32, I32, P, I64, I32, P, I64, P]),
        "moe_combine": (ctypes.c_int, [P, I64, I64, P, P, I32, I32, I32, P, P]),
        "moe_combine_scatter": (ctypes.c_int, [P, I64, I64, P, P, I32, I32, I32, P, I64, I64, P]),
        "moe_combine_staged": (ctypes.c_int, [P, I64, I64, P, P, I32, I32, I32, P, P]),
        "moe_unpack": (ctypes.c_int, [P, I64, P, I32, I32, I32, I32, P, P, P, P]),
        "moe_dedup_window_bytes": (I64, [I32, I32, I32, I32]),
        "moe_rank_rows": (ctypes.c_int, [P, I32, I32, I32, I32, I32, P, P, P, P, P]),
        "moe_dispatch_dedup": (ctypes.c_int, [P, P, P, I32, I32, I32, I32, I32, I32, I32, P, I64, P]),
        "moe_expand_dedup": (ctypes.c_int, [P, I64, P, P, P, I32, I32, I32, I32, I32, P, P, P, P]),
        "moe_unpack_padded": (ctypes.c_int, [P, I64, P, I32, I32, I32, I32, I32, I32, I64,
                                             P, P, P, P, P, P]),
        "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "moe_plan_layout": (ctypes.c_int, [P, P, I32, I32, I32, I32, I32] + [P] * 9 + [I32]),
        "moe_plan_dispatch_ws": (ctypes.c_int, [P, P, P, I32, I32, I32, I32, I32, P, I64, P, I64]),
        "moe_plan_layout_ws": (ctypes.c_int, [P, P, I32, I32, I32, I32, I32] + [P] * 9 + [I32, I32, P, I64]),
        "moe_plan_dispatch_planned": (ctypes.c_int, [P, P, P, I32, I32, I32, I32, I32, I32, P, I64, P, I64]),
        "moe_plan_layout_dispatch": (ctypes.c_int, [P, P, I32, I32, I32, I32, I32] + [P] * 9 +
                                     [P, I32, I32, I32, P, I64, I32]),
        "moe_plan_combine": (ctypes.c_int, [P, P, I64, I64, P, P, I32, I32, I32, P]),
        "moe_plan_run": (ctypes.c_int, [P, P]),
        "moe_combine_backward": (ctypes.c_int, [P, P, I64, I64, P, P, I32, I32, I32, P, I64, P, P]),
        "moe_combine_backward_mx": (ctypes.c_int, [P, P, P, I64, P, P, I32, I32, I32, P, I64, P, P]),
        "moe_dispatch_backward": (ctypes.c_int, [P, I64, I64, P, I32, I32, I32, P, P]),
        "moe_combine_checkpoint": (ctypes.c_int, [P, I64, I64, P, P, I32, I32, I32, P, P, P, P]),
        "moe_mx_row_bytes": (I64, [I32, I32]),
        "moe_mx_quantize": (ctypes.c_int, [P, I64, P, I64, I32, I32, P, P, P]),
        "moe_mx_dequantize": (ctypes.c_int, [P, P, P, I64, I32, I32, P, I64, P]),
        "moe_mx_product": (ctypes.c_int, [P, P, I64, P, I32, P, P, I32, I32, I32, P, I64, P]),
        "moe_row_quantize": (ctypes.c_int, [P, I64, P, I64, I32, I32, P, P, P]),
        "moe_row_dequantize": (ctypes.c_int, [P, P, P, I64, I32, I32, P, I64, P]),
        "moe_scaled_product": (ctypes.c_int, [P, P, I64, P, I32, P, P, I32, I32, I32, P, I64, P]),
        "moe_rms_norm": (ctypes.c_int, [P, I64, P, I64, P, I32, F32, I64, I32, I32, P, I64, P, P, P, P]),
        "moe_rms_norm_backward_workspace_bytes": (I64, [I64, I32]),
        "moe_rms_norm_backward": (ctypes.c_int, [P, I64, P, I64, P, I32, F32, P, I64, I64, I32, P, P, P, I64, P]),
        "moe_balance_loss_workspace_bytes": (I64, [I32, I32]),
        "moe_balance_loss": (ctypes.c_int, [P, I64, I32, P, I32, I32, I32, I32, F32, P, P, P, P, I64, P]),
        "moe_balance_loss_backward": (ctypes.c_int, [P, P, I64, I32, P, P, P, I32, I32, I32, I32, F32, P, P]),
        "moe_probe_fill": (ctypes.c_int, [P, I64, P]),
        "moe_probe_read": (ctypes.c_int, [P, I64, P, P]),
        "moe_probe_copy": (ctypes.c_int, [P, P, I64, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


class MoeError(RuntimeError):
    """A HIP launch error reported by the library."""


def moe_status_string(status):
    return _lib.moe_status_string(int(status)).decode()


def _check(status):
    if status == MOE_OK:
        return
    msg = f"{moe_status_string(status)} (status {status})"
    if status == MOE_ERR_HIP:
        raise MoeError(msg)
    raise ValueError(msg)


# The raw handle of the current stream without building a torch Stream object (about 2 us per
# call less); torch.cuda.current_stream is the fallback where that accessor is missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev, stream):
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if _raw_stream is not None:
        return _raw_stream(dev.index if dev.index is not None else torch.cuda.current_device())
    return torch.cuda.current_stream(dev).cuda_stream


def _ptr(t):
    return t.data_ptr()


def _need(t, name, dtype=None, ndim=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_layout(out, S, K, E, P, C, dev):
    """The nine Layout buffers: device, dtype, shape and contiguity."""
    shapes = ((S, P), (P,), (E,), (P, C), (E, C), (P + 1,), (E + 1,), (S, K), (1,))
    for i, (t, shp) in enumerate(zip(out, shapes)):
        dtype = torch.bool if i == 0 else torch.int32
        if (not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != dtype
                or t.shape != shp or not t.is_contiguous()):
            name = Layout._fields[i]
            _need(t, name, dtype, device=dev)
            raise ValueError(f"{name} must have shape {shp}, got {tuple(t.shape)}")


def moe_slot_bytes(H):
    v = _lib.moe_slot_bytes(int(H))
    if v < 0:
        _check(int(v))
    return int(v)


def moe_window_bytes(S, K, H):
    v = _lib.moe_window_bytes(int(S), int(K), int(H))
    if v < 0:
        _check(int(v))
    return int(v)


def moe_slot_offsets(H, quant=MOE_QUANT_NONE):
    vals = [ctypes.c_int64() for _ in range(4)]
    _check(_lib.moe_slot_offsets(int(H), int(quant), *[ctypes.byref(v) for v in vals]))
    keys = ("payload_bytes", "scale_off", "triple_off", "tail_end")
    return {k: v.value for k, v in zip(keys, vals)}


class Layout(NamedTuple):
    is_token_in_rank: torch.Tensor  # bool [S, P]
    num_tokens_per_rank: torch.Tensor  # int32 [P]
    num_tokens_per_expert: torch.Tensor  # int32 [E]
    rank_prefix_matrix: torch.Tensor  # int32 [P, C]
    expert_prefix_matrix: torch.Tensor  # int32 [E, C]
    rank_slot_base: torch.Tensor  # int32 [P + 1]
    expert_slot_base: torch.Tensor  # int32 [E + 1]
    slot_idx: torch.Tensor  # int32 [S, K]
    status: torch.Tensor  # int32 [1]


def empty_layout(S, K, E, P, C, device):
    """Output buffers for moe_layout (allocation only)."""
    i32 = dict(dtype=torch.int32, device=device)
    return Layout(
        torch.empty((S, P), dtype=torch.bool, device=device),
        torch.empty(P, **i32), torch.empty(E, **i32), torch.empty((P, C), **i32),
        torch.empty((E, C), **i32), torch.empty(P + 1, **i32), torch.empty(E + 1, **i32),
        torch.empty((S, K), **i32), torch.empty(1, **i32),
    )


def moe_layout(topk_idx, num_experts, num_ranks, num_channels, out=None, stream=None, path=None):
    """Routing layout of topk_idx (int32 [S, K]) for E experts over P ranks and C channels.
    path: None (moe_layout: the form is chosen by size) or a MOE_LAYOUT_* value (moe_layout_ex)."""
    _need(topk_idx, "topk_idx", torch.int32, 2)
    S, K = topk_idx.shape
    E, P, C = int(num_experts), int(num_ranks), int(num_channels)
    dev = topk_idx.device
    if out is None:
        out = empty_layout(S, K, E, P, C, dev)
    _need_layout(out, S, K, E, P, C, dev)
    if path is None:
        _check(_lib.moe_layout(_ptr(topk_idx), S, K, E, P, C, *[_ptr(t) for t in out],
                               _stream(dev, stream)))
    else:
        _check(_lib.moe_layout_ex(_ptr(topk_idx), S, K, E, P, C, *[_ptr(t) for t in out], int(path),
                                  _stream(dev, stream)))
    return out


def moe_dispatch(x, slot_idx, window, quant=MOE_QUANT_NONE, src_rank=0, stream=None):
    """Pack bf16 rows x [S, H] into the window slots named by slot_idx [S, K]."""
    _need(x, "x", torch.bfloat16, 2)
    _need(slot_idx, "slot_idx", torch.int32, 2, x.device)
    _need(window, "window", device=x.device)
    S, H = x.shape
    if slot_idx.shape[0] != S:
        raise ValueError("slot_idx must have one row per token of x")
    K = slot_idx.shape[1]
    nbytes = window.numel() * window.element_size()
    _check(_lib.moe_dispatch(_ptr(x), _ptr(slot_idx), S, H, K, int(quant), int(src_rank),
                             _ptr(window), nbytes, _stream(x.device, stream)))
    return window


def moe_dispatch_workspace_bytes(S, K, quant=MOE_QUANT_NONE):
    v = _lib.moe_dispatch_workspace_bytes(int(S), int(K), int(quant))
    if v < 0:
        _check(int(v))
    return int(v)


def moe_dispatch_ws(x, slot_idx, window, workspace, quant=MOE_QUANT_NONE, src_rank=0, stream=None):
    """moe_dispatch with a caller workspace (a device buffer of at least
    moe_dispatch_workspace_bytes(S, K, quant) bytes, or None when that size is 0): the same window
    bytes, written by the planned pack where it applies."""
    _need(x, "x", torch.bfloat16, 2)
    _need(slot_idx, "slot_idx", torch.int32, 2, x.device)
    _need(window, "window", device=x.device)
    S, H = x.shape
    if slot_idx.shape[0] != S:
        raise ValueError("slot_idx must have one row per token of x")
    K = slot_idx.shape[1]
    if workspace is None:
        ws_ptr, ws_bytes = None, 0
    else:
        _need(workspace, "workspace", device=x.device)
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    nbytes = window.numel() * window.element_size()
    _check(_lib.moe_dispatch_ws(_ptr(x), _ptr(slot_idx), S, H, K, int(quant), int(src_rank), _ptr(window),
                                nbytes, ws_ptr, ws_bytes, _stream(x.device, stream)))
    return window


def moe_dispatch_noalloc(x, slot_idx, window, quant=MOE_QUANT_NONE, src_rank=0, stream=None):
    """moe_dispatch_ws with the library's fixed device scratch instead of a workspace (allocates
    nothing; calls that overlap on one GPU race on that scratch). ValueError with MOE_ERR_SCRATCH
    when the table needs more than MOE_NOALLOC_SCRATCH_BYTES."""
    _need(x, "x", torch.bfloat16, 2)
    _need(slot_idx, "slot_idx", torch.int32, 2, x.device)
    _need(window, "window", device=x.device)
    S, H = x.shape
    if slot_idx.shape[0] != S:
        raise ValueError("slot_idx must have one row per token of x")
    K = slot_idx.shape[1]
    nbytes = window.numel() * window.element_size()
    _check(_lib.moe_dispatch_noalloc(_ptr(x), _ptr(slot_idx), S, H, K, int(quant), int(src_rank), _ptr(window),
                                     nbytes, _stream(x.device, stream)))
    return window


def moe_layout_dispatch(topk_idx, num_experts, num_ranks, num_channels, x, window,
                        quant=MOE_QUANT_NONE, src_rank=0, out=None, stream=None, path=None):
    """moe_layout and moe_dispatch in one call (one kernel for small tables); returns the Layout.
    path: None (moe_layout_dispatch) or a MOE_LAYOUT_* value (moe_layout_dispatch_ex)."""
    _need(topk_idx, "topk_idx", torch.int32, 2)
    dev = topk_idx.device
    _need(x, "x", torch.bfloat16, 2, dev)
    _need(window, "window", device=dev)
    S, K = topk_idx.shape
    if x.shape[0] != S:
        raise ValueError("x must have one row per token of topk_idx")
    H = x.shape[1]
    E, P, C = int(num_experts), int(num_ranks), int(num_channels)
    if out is None:
        out = empty_layout(S, K, E, P, C, dev)
    _need_layout(out, S, K, E, P, C, dev)
    nbytes = window.numel() * window.element_size()
    if path is None:
        _check(_lib.moe_layout_dispatch(_ptr(topk_idx), S, K, E, P, C, *[_ptr(t) for t in out],
                                        _ptr(x), H, int(quant), int(src_rank), _ptr(window), nbytes,
                                        _stream(dev, stream)))
    else:
        _check(_lib.moe_layout_dispatch_ex(_ptr(topk_idx), S, K, E, P, C, *[_ptr(t) for t in out],
                                           _ptr(x), H, int(quant), int(src_rank), _ptr(window), nbytes,
                                           int(path), _stream(dev, stream)))
    return out


def moe_layout_dispatch_workspace_bytes(S, K, E, P, C, quant=MOE_QUANT_NONE, path=MOE_LAYOUT_AUTO):
    v = _lib.moe_layout_dispatch_workspace_bytes(int(S), int(K), int(E), int(P), int(C), int(quant), int(path))
    if v < 0:
        _check(int(v))
    return int(v)


def _ws_arg(workspace, dev):
    if workspace is None:
        return None, 0
    _need(workspace, "workspace", device=dev)
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def moe_layout_ws(topk_idx, num_experts, num_ranks, num_channels, workspace, quant=MOE_QUANT_NONE,
                  out=None, stream=None, path=MOE_LAYOUT_AUTO):
    """moe_layout with a caller workspace (moe_layout_dispatch_workspace_bytes(...) bytes, or None when
    that is 0): two kernels, and in bf16 the pack plan for moe_dispatch_planned."""
    _need(topk_idx, "topk_idx", torch.int32, 2)
    dev = topk_idx.device
    S, K = topk_idx.shape
    E, P, C = int(num_experts), int(num_ranks), int(num_channels)
    if out is None:
        out = empty_layout(S, K, E, P, C, dev)
    _need_layout(out, S, K, E, P, C, dev)
    ws_ptr, ws_bytes = _ws_arg(workspace, dev)
    _check(_lib.moe_layout_ws(_ptr(topk_idx), S, K, E, P, C, *[_ptr(t) for t in out], int(quant), int(path),
                              ws_ptr, ws_bytes, _stream(dev, stream)))
    return out


def moe_dispatch_planned(x, slot_idx, window, workspace, num_channels, quant=MOE_QUANT_NONE, src_rank=0,
                         stream=None):
    """The pack of the table moe_layout_ws just laid out, from the plan it left in `workspace`."""
    _need(x, "x", torch.bfloat16, 2)
    dev = x.device
    _need(slot_idx, "slot_idx", torch.int32, 2, dev)
    _need(window, "window", device=dev)
    S, H = x.shape
    if slot_idx.shape[0] != S:
        raise ValueError("slot_idx must have one row per token of x")
    K = slot_idx.shape[1]
    ws_ptr, ws_bytes = _ws_arg(workspace, dev)
    nbytes = window.numel() * window.element_size()
    _check(_lib.moe_dispatch_planned(_ptr(x), _ptr(slot_idx), S, H, K, int(num_channels), int(quant),
                                     int(src_rank), _ptr(window), nbytes, ws_ptr, ws_bytes, _stream(dev, stream)))
    return window


def moe_layout_dispatch_ws(topk_idx, num_experts, num_ranks, num_channels, x, window, workspace,
                           quant=MOE_QUANT_NONE, src_rank=0, out=None, stream=None, path=MOE_LAYOUT_AUTO):
    """moe_layout_dispatch with a caller workspace (at least moe_layout_dispatch_workspace_bytes(...)
    bytes, or None when that size is 0): two layout kernels, the pack plan written by the layout."""
    _need(topk_idx, "topk_idx", torch.int32, 2)
    dev = topk_idx.device
    _need(x, "x", torch.bfloat16, 2, dev)
    _need(window, "window", device=dev)
    S, K = topk_idx.shape
    if x.shape[0] != S:
        raise ValueError("x must have one row per token of topk_idx")
    H = x.shape[1]
    E, P, C = int(num_experts), int(num_ranks), int(num_channels)
    if out is None:
        out = empty_layout(S, K, E, P, C, dev)
    _need_layout(out, S, K, E, P, C, dev)
    ws_ptr, ws_bytes = _ws_arg(workspace, dev)
    nbytes = window.numel() * window.element_size()
    _check(_lib.moe_layout_dispatch_ws(_ptr(topk_idx), S, K, E, P, C, *[_ptr(t) for t in out], _ptr(x), H,
                                       int(quant), int(src_rank), _ptr(window), nbytes, int(path), ws_ptr,
                                       ws_bytes, _stream(dev, stream)))
    return out


def moe_combine(expert_out, slot_idx, topk_weights, row_stride_bytes=None, expert_rows=None,
                hidden=None, y=None, stream=None):
    """y[t] = bf16(sum_k w[t,k] * expert_out[slot_idx[t,k]]) with fp32 accumulation.

    expert_out is either a bf16 [R, H] tensor (row stride 2H, R rows) or any device
    buffer with explicit row_stride_bytes, expert_rows and hidden (for example the
    dispatch window with row_stride_bytes = moe_slot_bytes(H)).
    """
    _need(slot_idx, "slot_idx", torch.int32, 2)
    dev = slot_idx.device
    _need(expert_out, "expert_out", device=dev)
    _need(topk_weights, "topk_weights", torch.float32, 2, dev)
    S, K = slot_idx.shape
    if tuple(topk_weights.shape) != (S, K):
        raise ValueError("topk_weights must match slot_idx")
    if row_stride_bytes is None:
        if expert_out.dtype != torch.bfloat16 or expert_out.dim() != 2:
            raise ValueError("pass row_stride_bytes/expert_rows/hidden for a non-[R, H] bf16 buffer")
        expert_rows, H = expert_out.shape
        row_stride_bytes = 2 * H
    else:
        if expert_rows is None or hidden is None:
            raise ValueError("expert_rows and hidden are required with row_stride_bytes")
        H = int(hidden)
        if int(expert_rows) * int(row_stride_bytes) > expert_out.numel() * expert_out.element_size():
            raise ValueError("expert_rows * row_stride_bytes exceeds the expert_out buffer")
    if y is None:
        y = torch.empty((S, H), dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, 2, dev)
    if tuple(y.shape) != (S, H):
        raise ValueError(f"y must have shape {(S, H)}")
    _check(_lib.moe_combine(_ptr(expert_out), int(row_stride_bytes), int(expert_rows),
                            _ptr(slot_idx), _ptr(topk_weights), S, H, K, _ptr(y),
                            _stream(dev, stream)))
    return y


def moe_combine_scatter(expert_out, expand_idx, num_rows, S, K, staging=None, staging_stride_bytes=None,
                        stream=None):
    """First pass of the two-pass combine: bf16 expert rows [R, H] (row s for slot s) to staging
    row t*K + k by their triples expand_idx [R, 3]; rows at or past the device count num_rows are
    skipped. staging defaults to a new bf16 [S*K, H] tensor (stride 2H)."""
    _need(expert_out, "expert_out", torch.bfloat16, 2)
    dev = expert_out.device
    _need(expand_idx, "expand_idx", torch.int32, 2, dev)
    _need(num_rows, "num_rows", torch.int32, device=dev)
    R, H = expert_out.shape
    S, K = int(S), int(K)
    if tuple(expand_idx.shape) != (R, 3):
        raise ValueError("expand_idx must be [rows of expert_out, 3]")
    if staging is None:
        staging = torch.empty((S * K, H), dtype=torch.bfloat16, device=dev)
    _need(staging, "staging", device=dev)
    stride = 2 * H if staging_stride_bytes is None else int(staging_stride_bytes)
    _check(_lib.moe_combine_scatter(_ptr(expert_out), 2 * H, R, _ptr(expand_idx), _ptr(num_rows), S, K,
                                    H, _ptr(staging), stride, staging.numel() * staging.element_size(),
                                    _stream(dev, stream)))
    return staging


def moe_combine_staged(staging, slot_idx, topk_weights, hidden, staging_stride_bytes=None, y=None,
                       stream=None):
    """Second pass of the two-pass combine: y[t] reduces staging rows t*K .. t*K+K-1 (entries with
    slot_idx < 0 skipped) with the arithmetic of moe_combine."""
    _need(slot_idx, "slot_idx", torch.int32, 2)
    dev = slot_idx.device
    _need(staging, "staging", device=dev)
    _need(topk_weights, "topk_weights", torch.float32, 2, dev)
    S, K = slot_idx.shape
    H = int(hidden)
    stride = 2 * H if staging_stride_bytes is None else int(staging_stride_bytes)
    if tuple(topk_weights.shape) != (S, K):
        raise ValueError("topk_weights must match slot_idx")
    if y is None:
        y = torch.empty((S, H), dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, 2, dev)
    if tuple(y.shape) != (S, H):
        raise ValueError(f"y must have shape {(S, H)}")
    _check(_lib.moe_combine_staged(_ptr(staging), stride, staging.numel() * staging.element_size(),
                                   _ptr(slot_idx), _ptr(topk_weights), S, H, K, _ptr(y),
                                   _stream(dev, stream)))
    return y


def moe_probe_fill(dst, stream=None):
    """Write-only bandwidth probe over the whole device tensor dst (measurement only)."""
    _need(dst, "dst")
    _check(_lib.moe_probe_fill(_ptr(dst), dst.numel() * dst.element_size(), _stream(dst.device, stream)))


def moe_probe_read(src, sink, stream=None):
    """Read-only bandwidth probe over the whole device tensor src; sink is a device int32 [1]."""
    _need(src, "src")
    _need(sink, "sink", torch.int32, device=src.device)
    _check(_lib.moe_probe_read(_ptr(src), src.numel() * src.element_size(), _ptr(sink),
                               _stream(src.device, stream)))


def moe_probe_copy(src, dst, stream=None):
    """Copy probe: dst = src, both device tensors of the same byte size."""
    _need(src, "src")
    _need(dst, "dst", device=src.device)
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != n:
        raise ValueError("src and dst must have the same byte size")
    _check(_lib.moe_probe_copy(_ptr(src), _ptr(dst), n, _stream(src.device, stream)))


MOE_PLAN_BYTES = 320  # sizeof(moe_plan)


class Plan:
    """A pre-validated call (include/moe.h, moe_plan_*): the arguments were checked once when the
    plan was made; run() enqueues the call on the current (or given) stream without checking them
    again. The tensors the plan was made from are kept referenced here, so they stay allocated for
    the plan's lifetime; they must keep their shapes (do not resize them)."""

    __slots__ = ("_buf", "_addr", "_dev", "_keep", "_run", "_stream_of")

    def __init__(self, dev, keep):
        self._buf = ctypes.create_string_buffer(MOE_PLAN_BYTES)
        self._addr = ctypes.addressof(self._buf)
        self._dev = dev.index if dev.index is not None else torch.cuda.current_device()
        self._keep = keep
        self._run = _lib.moe_plan_run
        self._stream_of = _raw_stream

    def run(self, stream=None):
        if stream is None and self._stream_of is not None:
            rc = self._run(self._addr, self._stream_of(self._dev))
        else:
            rc = self._run(self._addr, _stream(torch.device("cuda", self._dev), stream))
        if rc:
            _check(rc)


def plan_layout(topk_idx, num_experts, num_ranks, num_channels, out, path=MOE_LAYOUT_AUTO):
    """Plan of moe_layout_ex on these buffers (out: a Layout)."""
    _need(topk_idx, "topk_idx", torch.int32, 2)
    S, K = topk_idx.shape
    E, P, C = int(num_experts), int(num_ranks), int(num_channels)
    dev = topk_idx.device
    _need_layout(out, S, K, E, P, C, dev)
    plan = Plan(dev, (topk_idx, out))
    _check(_lib.moe_plan_layout(plan._addr, _ptr(topk_idx), S, K, E, P, C, *[_ptr(t) for t in out], int(path)))
    return plan


def plan_dispatch_ws(x, slot_idx, window, workspace, quant=MOE_QUANT_NONE, src_rank=0):
    """Plan of moe_dispatch_ws on these buffers."""
    _need(x, "x", torch.bfloat16, 2)
    _need(slot_idx, "slot_idx", torch.int32, 2, x.device)
    _need(window, "window", device=x.device)
    S, H = x.shape
    if slot_idx.shape[0] != S:
        raise ValueError("slot_idx must have one row per token of x")
    K = slot_idx.shape[1]
    if workspace is None:
        ws_ptr, ws_bytes = None, 0
    else:
        _need(workspace, "workspace", device=x.device)
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    plan = Plan(x.device, (x, slot_idx, window, workspace))
    _check(_lib.moe_plan_dispatch_ws(plan._addr, _ptr(x), _ptr(slot_idx), S, H, K, int(quant), int(src_rank),
                                     _ptr(window), window.numel() * window.element_size(), ws_ptr, ws_bytes))
    return plan


def plan_layout_ws(topk_idx, num_experts, num_ranks, num_channels, out, workspace, quant=MOE_QUANT_NONE,
                   path=MOE_LAYOUT_AUTO):
    """Plan of moe_layout_ws on these buffers (out: a Layout)."""
    _need(topk_idx, "topk_idx", torch.int32, 2)
    S, K = topk_idx.shape
    E, P, C = int(num_experts), int(num_ranks), int(num_channels)
    dev = topk_idx.device
    _need_layout(out, S, K, E, P, C, dev)
    ws_ptr, ws_bytes = _ws_arg(workspace, dev)
    plan = Plan(dev, (topk_idx, out, workspace))
    _check(_lib.moe_plan_layout_ws(plan._addr, _ptr(topk_idx), S, K, E, P, C, *[_ptr(t) for t in out], int(quant),
                                   int(path), ws_ptr, ws_bytes))
    return plan


def plan_dispatch_planned(x, slot_idx, window, workspace, num_channels, quant=MOE_QUANT_NONE, src_rank=0):
    """Plan of moe_dispatch_planned on these buffers."""
    _need(x, "x", torch.bfloat16, 2)
    _need(slot_idx, "slot_idx", torch.int32, 2, x.device)
    _need(window, "window", device=x.device)
    S, H = x.shape
    if slot_idx.shape[0] != S:
        raise ValueError("slot_idx must have one row per token of x")
    K = slot_idx.shape[1]
    ws_ptr, ws_bytes = _ws_arg(workspace, x.device)
    plan = Plan(x.device, (x, slot_idx, window, workspace))
    _check(_lib.moe_plan_dispatch_planned(plan._addr, _ptr(x), _ptr(slot_idx), S, H, K, int(num_channels), int(quant),
                                          int(src_rank), _ptr(window), window.numel() * window.element_size(),
                                          ws_ptr, ws_bytes))
    return plan


def plan_layout_dispatch(topk_idx, num_experts, num_ranks, num_channels, x, window, out, quant=MOE_QUANT_NONE,
                         src_rank=0, path=MOE_LAYOUT_AUTO):
    """Plan of moe_layout_dispatch_ex on these buffers (out: a Layout)."""
    _need(topk_idx, "topk_idx", torch.int32, 2)
    dev = topk_idx.device
    _need(x, "x", torch.bfloat16, 2, dev)
    _need(window, "window", device=dev)
    S, K = topk_idx.shape
    if x.shape[0] != S:
        raise ValueError("x must have one row per token of topk_idx")
    E, P, C = int(num_experts), int(num_ranks), int(num_channels)
    _need_layout(out, S, K, E, P, C, dev)
    plan = Plan(dev, (topk_idx, x, window, out))
    _check(_lib.moe_plan_layout_dispatch(plan._addr, _ptr(topk_idx), S, K, E, P, C, *[_ptr(t) for t in out],
                                         _ptr(x), x.shape[1], int(quant), int(src_rank), _ptr(window),
                                         window.numel() * window.element_size(), int(path)))
    return plan


def plan_combine(expert_out, slot_idx, topk_weights, y):
    """Plan of moe_combine of a bf16 [R, H] expert_out into y (bf16 [S, H])."""
    _need(slot_idx, "slot_idx", torch.int32, 2)
    dev = slot_idx.device
    _need(expert_out, "expert_out", torch.bfloat16, 2, dev)
    _need(topk_weights, "topk_weights", torch.float32, 2, dev)
    _need(y, "y", torch.bfloat16, 2, dev)
    S, K = slot_idx.shape
    R, H = expert_out.shape
    if tuple(topk_weights.shape) != (S, K) or tuple(y.shape) != (S, H):
        raise ValueError("topk_weights must match slot_idx and y must be [S, H]")
    plan = Plan(dev, (expert_out, slot_idx, topk_weights, y))
    _check(_lib.moe_plan_combine(plan._addr, _ptr(expert_out), 2 * H, R, _ptr(slot_idx), _ptr(topk_weights), S, H,
                                 K, _ptr(y)))
    return plan


def moe_dedup_window_bytes(S, K, P, H):
    v = _lib.moe_dedup_window_bytes(int(S), int(K), int(P), int(H))
    if v < 0:
        _check(int(v))
    return int(v)


class RankRows(NamedTuple):
    rank_row_idx: torch.Tensor  # int32 [S, K]
    rank_token_base: torch.Tensor  # int32 [P + 1]


def moe_rank_rows(topk_idx, layout, num_experts, num_ranks, num_channels, out=None, stream=None):
    """Per-rank deduplicated rows of the routing table, from moe_layout's rank_prefix_matrix and
    num_tokens_per_rank (layout is the Layout moe_layout returned)."""
    _need(topk_idx, "topk_idx", torch.int32, 2)
    dev = topk_idx.device
    S, K = topk_idx.shape
    E, P, C = int(num_experts), int(num_ranks), int(num_channels)
    _need(layout.rank_prefix_matrix, "rank_prefix_matrix", torch.int32, 2, dev)
    _need(layout.num_tokens_per_rank, "num_tokens_per_rank", torch.int32, 1, dev)
    if tuple(layout.rank_prefix_matrix.shape) != (P, C) or layout.num_tokens_per_rank.shape[0] != P:
        raise ValueError("layout does not match num_ranks / num_channels")
    if out is None:
        out = RankRows(torch.empty((S, K), dtype=torch.int32, device=dev),
                       torch.empty(P + 1, dtype=torch.int32, device=dev))
    _need(out.rank_row_idx, "rank_row_idx", torch.int32, 2, dev)
    _need(out.rank_token_base, "rank_token_base", torch.int32, 1, dev)
    if tuple(out.rank_row_idx.shape) != (S, K) or out.rank_token_base.shape[0] != P + 1:
        raise ValueError("rank_row_idx must be [S, K] and rank_token_base [P + 1]")
    _check(_lib.moe_rank_rows(_ptr(topk_idx), S, K, E, P, C, _ptr(layout.rank_prefix_matrix),
                              _ptr(layout.num_tokens_per_rank), _ptr(out.rank_row_idx),
                              _ptr(out.rank_token_base), _stream(dev, stream)))
    return out


def moe_dispatch_dedup(x, rank_row_idx, topk_idx, num_experts, num_ranks, window, quant=MOE_QUANT_NONE,
                       src_rank=0, stream=None):
    """One row per (token, destination rank) into the rows named by rank_row_idx (bf16, or the
    token's dynamic fp8 / INT8 codes and scale)."""
    _need(x, "x", torch.bfloat16, 2)
    dev = x.device
    _need(rank_row_idx, "rank_row_idx", torch.int32, 2, dev)
    _need(topk_idx, "topk_idx", torch.int32, 2, dev)
    _need(window, "window", device=dev)
    S, H = x.shape
    K = topk_idx.shape[1]
    if tuple(topk_idx.shape) != (S, K) or tuple(rank_row_idx.shape) != (S, K):
        raise ValueError("rank_row_idx and topk_idx must be [S, K] with S rows of x")
    nbytes = window.numel() * window.element_size()
    _check(_lib.moe_dispatch_dedup(_ptr(x), _ptr(rank_row_idx), _ptr(topk_idx), S, H, K,
                                   int(num_experts), int(num_ranks), int(quant), int(src_rank),
                                   _ptr(window), nbytes, _stream(dev, stream)))
    return window


def moe_expand_dedup(window, rank_row_idx, slot_idx, num_slots, num_ranks, H, quant=MOE_QUANT_NONE,
                     out=None, stream=None):
    """Receive-side expansion of the deduplicated rows to the expert-major rows of slot_idx:
    returns Unpacked(expand_x [S*K, H] bf16 or uint8 codes, expand_scales fp32 [S*K] or None,
    expand_idx int32 [S*K, 3]) as moe_unpack would. num_slots is the device count N
    (layout.expert_slot_base[E:])."""
    _need(window, "window")
    dev = window.device
    _need(rank_row_idx, "rank_row_idx", torch.int32, 2, dev)
    _need(slot_idx, "slot_idx", torch.int32, 2, dev)
    _need(num_slots, "num_slots", torch.int32, device=dev)
    S, K = slot_idx.shape
    H, quant = int(H), int(quant)
    rows = S * K
    if tuple(rank_row_idx.shape) != (S, K):
        raise ValueError("rank_row_idx must match slot_idx")
    if out is None:
        if quant == MOE_QUANT_NONE:
            ex, sc = torch.empty((rows, H), dtype=torch.bfloat16, device=dev), None
        else:
            ex = torch.empty((rows, H), dtype=torch.uint8, device=dev)
            sc = torch.empty(rows, dtype=torch.float32, device=dev)
        out = Unpacked(ex, sc, torch.empty((rows, 3), dtype=torch.int32, device=dev))
    ex, sc, idx = out
    _need(ex, "expand_x", device=dev)
    _need(idx, "expand_idx", torch.int32, 2, dev)
    payload = moe_slot_offsets(H, quant)["payload_bytes"]
    if ex.numel() * ex.element_size() < rows * payload or tuple(idx.shape) != (rows, 3):
        raise ValueError("expand_x must hold S*K rows of payload bytes and expand_idx [S*K, 3]")
    if sc is not None:
        _need(sc, "expand_scales", torch.float32, device=dev)
        if sc.numel() < rows:
            raise ValueError("expand_scales must hold S*K values")
    nbytes = window.numel() * window.element_size()
    _check(_lib.moe_expand_dedup(_ptr(window), nbytes, _ptr(rank_row_idx), _ptr(slot_idx),
                                 _ptr(num_slots), S, K, int(num_ranks), H, quant, _ptr(ex),
                                 None if sc is None else _ptr(sc), _ptr(idx), _stream(dev, stream)))
    return out


class Unpacked(NamedTuple):
    expand_x: torch.Tensor  # [S*K, H] bf16, or uint8 codes for the quantised modes
    expand_scales: torch.Tensor  # fp32 [S*K] (quantised modes) or None
    expand_idx: torch.Tensor  # int32 [S*K, 3]


def moe_unpack(window, num_slots, S, K, H, quant=MOE_QUANT_NONE, out=None, stream=None):
    """Compact rows, triples and scales of the first N window slots (N read on the device from
    num_slots, e.g. layout.expert_slot_base[E:]). Rows N..S*K-1 of the outputs are left as is."""
    _need(window, "window")
    dev = window.device
    _need(num_slots, "num_slots", torch.int32, device=dev)
    S, K, H, quant = int(S), int(K), int(H), int(quant)
    rows = S * K
    if out is None:
        if quant == MOE_QUANT_NONE:
            ex = torch.empty((rows, H), dtype=torch.bfloat16, device=dev)
            sc = None
        else:
            ex = torch.empty((rows, H), dtype=torch.uint8, device=dev)
            sc = torch.empty(rows, dtype=torch.float32, device=dev)
        out = Unpacked(ex, sc, torch.empty((rows, 3), dtype=torch.int32, device=dev))
    ex, sc, idx = out
    _need(ex, "expand_x", device=dev)
    _need(idx, "expand_idx", torch.int32, 2, dev)
    payload = moe_slot_offsets(H, quant)["payload_bytes"]
    if ex.numel() * ex.element_size() < rows * payload or tuple(idx.shape) != (rows, 3):
        raise ValueError("expand_x must hold S*K rows of payload bytes and expand_idx [S*K, 3]")
    if sc is not None:
        _need(sc, "expand_scales", torch.float32, device=dev)
        if sc.numel() < rows:
            raise ValueError("expand_scales must hold S*K values")
    nbytes = window.numel() * window.element_size()
    _check(_lib.moe_unpack(_ptr(window), nbytes, _ptr(num_slots), S, K, H, quant, _ptr(ex),
                           None if sc is None else _ptr(sc), _ptr(idx), _stream(dev, stream)))
    return out


class PaddedUnpacked(NamedTuple):
    expand_x: torch.Tensor  # [R, H] bf16, or uint8 codes for the quantised modes
    expand_scales: torch.Tensor  # fp32 [R] (quantised modes) or None
    expand_idx: torch.Tensor  # int32 [R, 3], (-1, -1, -1) on padding rows
    expert_row_base: torch.Tensor  # int32 [E + 1], aligned first row of each expert
    status: torch.Tensor  # int32 [1], 1 if the aligned rows exceeded R


def moe_unpack_padded(window, expert_slot_base, S, K, H, quant=MOE_QUANT_NONE, expert_alignment=1,
                      out_rows=None, out=None, stream=None):
    """Unpack into exactly out_rows rows (default S*K) with each expert's block starting at a
    multiple of expert_alignment; padding rows are zero with triple -1. expert_slot_base is the
    layout's device tensor [E + 1]; nothing is read back to the host."""
    _need(window, "window")
    dev = window.device
    _need(expert_slot_base, "expert_slot_base", torch.int32, 1, dev)
    S, K, H, quant = int(S), int(K), int(H), int(quant)
    E = expert_slot_base.shape[0] - 1
    R = S * K if out_rows is None else int(out_rows)
    if out is None:
        if quant == MOE_QUANT_NONE:
            ex = torch.empty((R, H), dtype=torch.bfloat16, device=dev)
            sc = None
        else:
            ex = torch.empty((R, H), dtype=torch.uint8, device=dev)
            sc = torch.empty(R, dtype=torch.float32, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        out = PaddedUnpacked(ex, sc, torch.empty((R, 3), **i32), torch.empty(E + 1, **i32),
                             torch.empty(1, **i32))
    ex, sc, idx, base, status = out
    _need(ex, "expand_x", device=dev)
    _need(idx, "expand_idx", torch.int32, 2, dev)
    _need(base, "expert_row_base", torch.int32, 1, dev)
    _need(status, "status", torch.int32, device=dev)
    payload = moe_slot_offsets(H, quant)["payload_bytes"]
    if ex.numel() * ex.element_size() < R * payload or tuple(idx.shape) != (R, 3):
        raise ValueError("expand_x must hold out_rows rows of payload bytes and expand_idx [out_rows, 3]")
    if base.shape[0] != E + 1 or status.numel() < 1:
        raise ValueError("expert_row_base must have E + 1 entries and status one")
    if sc is not None:
        _need(sc, "expand_scales", torch.float32, device=dev)
        if sc.numel() < R:
            raise ValueError("expand_scales must hold out_rows values")
    nbytes = window.numel() * window.element_size()
    _check(_lib.moe_unpack_padded(_ptr(window), nbytes, _ptr(expert_slot_base), E, S, K, H, quant,
                                  int(expert_alignment), R, _ptr(ex), None if sc is None else _ptr(sc),
                                  _ptr(idx), _ptr(base), _ptr(status), _stream(dev, stream)))
    return out


# ---------------------------------------------------------------- gradients and MX rows


class MxRows(NamedTuple):
    """Rows in microscaled blocks: codes uint8 [..., R, moe_mx_row_bytes(H, format)] and scales uint8
    [..., R, H / 32]."""

    codes: torch.Tensor
    scales: torch.Tensor


# The current device's index without torch.cuda's lazy initialisation check (tensors on a device exist already).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

# These calls take about as long on the host as a small kernel on the GPU, so each argument is first tested by the
# cheapest accesses that accept it; the reason for a refusal is looked for only after that. Devices are indices here.
_Tensor, _empty = torch.Tensor, torch.empty
_bf16, _fp32, _int32, _uint8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _launch(dev, stream, fn, *args):
    """fn(*args, stream handle) with dev as the current device: a null stream is the current device's."""
    if stream is not None and isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError(f"stream is on cuda:{stream.device_index}, expected cuda:{dev}")  # its kernels run there
    if dev == _current_device():
        rc = fn(*args, _raw_stream(dev) if stream is None and _raw_stream is not None
                else _stream(torch.device("cuda", dev), stream))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(torch.device("cuda", dev), stream))
    if rc:
        _check(rc)


def _out(rows, columns, dtype, dev, stream):
    """A new output for a call on `stream`, from that stream's memory (the current stream's without one)."""
    if stream is None:
        return _empty(rows, columns, dtype=dtype, device=dev)
    with torch.cuda.stream(_torch_stream(stream, dev)):
        return _empty(rows, columns, dtype=dtype, device=dev)


def _torch_stream(stream, dev):
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = _stream(None, stream)
    return torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)


def _dense(t, name, dtype, shape, dev):
    """Pointer of a contiguous device tensor of exactly this shape."""
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    _need(t, name, dtype, len(shape), torch.device("cuda", dev))
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _matrix(t, name, dtype):
    """Device and shape of a two-dimensional device tensor of this type, whatever its strides."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev, shape = t.get_device(), t.shape
    if dev < 0:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype is not dtype or len(shape) != 2:
        raise ValueError(f"{name} must be {dtype} with 2 dims, got {t.dtype} {tuple(shape)}")
    return dev, shape[0], shape[1]


def _width(t, name):
    """The row length of a two-dimensional tensor; type and device are checked with the rest of it."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have 2 dims, got {len(shape)}")
    return shape[1]


def _rows_arg(t, name, H, dev):
    """Pointer, row stride in bytes and row count of bf16 rows: a [R, H] tensor whose rows are each
    contiguous, at any stride."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a device tensor on cuda:{dev}, got {t.device}")
    shape = t.shape
    if t.dtype is not _bf16 or len(shape) != 2 or shape[1] != H:
        raise ValueError(f"{name} must be bfloat16 [rows, {H}], got {t.dtype} {tuple(shape)}")
    n = shape[0]
    if n == 0:
        raise ValueError(f"{name} has no rows")
    if t.is_contiguous():
        return t.data_ptr(), 2 * H, n
    step, col = t.stride()
    if col != 1 or n > 1 and step < H:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), 2 * step if n > 1 else 2 * H, n


def _table_arg(slot_idx):
    """Device, S, K and pointer of the table."""
    if isinstance(slot_idx, _Tensor) and slot_idx.dtype is _int32 and slot_idx.is_contiguous():
        dev, shape = slot_idx.get_device(), slot_idx.shape
        if dev >= 0 and len(shape) == 2:
            return dev, shape[0], shape[1], slot_idx.data_ptr()
    _need(slot_idx, "slot_idx", torch.int32, 2)
    raise ValueError("slot_idx must be a device tensor")


def _mx_width(H, format):
    """Code bytes of a row; the library's error for an H or a format that has none."""
    if 32 <= H <= 16384 and H % 32 == 0:
        if format == MOE_MX_E2M1:
            return H // 2
        if format == MOE_MX_E4M3:
            return H
    return moe_mx_row_bytes(H, format)


def _mx_args(mx, name, rows, H, format, dev):
    codes, scales = mx
    return (_dense(codes, name + ".codes", _uint8, (rows, _mx_width(H, format)), dev),
            _dense(scales, name + ".scales", _uint8, (rows, H // 32), dev))


def _gradient_outs(S, K, H, rows, topk_weights, d_expert_out, d_topk_weights, dev, stream):
    if d_expert_out is None:
        d_expert_out = _out(rows, H, _bf16, dev, stream)
    d_ptr, d_stride, d_count = _rows_arg(d_expert_out, "d_expert_out", H, dev)
    if d_count != rows:
        raise ValueError(f"d_expert_out must have {rows} rows")
    if d_topk_weights is None:
        d_topk_weights = torch.empty_like(topk_weights) if stream is None else _out(S, K, _fp32, dev, stream)
        return d_expert_out, d_ptr, d_stride, d_topk_weights, d_topk_weights.data_ptr()
    return (d_expert_out, d_ptr, d_stride, d_topk_weights,
            _dense(d_topk_weights, "d_topk_weights", _fp32, (S, K), dev))


def moe_combine_backward(dy, expert_out, slot_idx, topk_weights, d_expert_out=None, d_topk_weights=None,
                         stream=None):
    """The combine's gradient: (d_expert_out, d_topk_weights) of dy (bf16 [S, H]) with the forward's
    expert_out (bf16 [R, H], any row stride), slot_idx and topk_weights. Rows of d_expert_out that no
    entry names keep their contents (undefined where it is allocated here)."""
    dev, S, K, table = _table_arg(slot_idx)
    weights = _dense(topk_weights, "topk_weights", _fp32, (S, K), dev)
    H = _width(dy, "dy")
    dy_ptr = _dense(dy, "dy", _bf16, (S, H), dev)
    ptr, stride, rows = _rows_arg(expert_out, "expert_out", H, dev)
    d_expert_out, d_ptr, d_stride, d_topk_weights, dw_ptr = _gradient_outs(S, K, H, rows, topk_weights,
                                                                           d_expert_out, d_topk_weights, dev, stream)
    _launch(dev, stream, _lib.moe_combine_backward, dy_ptr, ptr, stride, rows, table, weights, S, H, K, d_ptr,
            d_stride, dw_ptr)
    return d_expert_out, d_topk_weights


def moe_combine_checkpoint(expert_out, slot_idx, topk_weights, y=None, checkpoint=None, stream=None):
    """moe_combine that also keeps the rows it reads in 8 bits: (y, MxRows in MOE_MX_E4M3 [R, H]). Rows that
    no entry names keep their contents (undefined where the checkpoint is allocated here)."""
    dev, S, K, table = _table_arg(slot_idx)
    weights = _dense(topk_weights, "topk_weights", _fp32, (S, K), dev)
    H = _width(expert_out, "expert_out")
    ptr, stride, rows = _rows_arg(expert_out, "expert_out", H, dev)
    if y is None:
        y = _out(S, H, _bf16, dev, stream)
    y_ptr = _dense(y, "y", _bf16, (S, H), dev)
    if checkpoint is None:
        checkpoint = _mx_empty(rows, H, MOE_MX_E4M3, dev, stream)
    codes, scales = _mx_args(checkpoint, "checkpoint", rows, H, MOE_MX_E4M3, dev)
    _launch(dev, stream, _lib.moe_combine_checkpoint, ptr, stride, rows, table, weights, S, H, K, y_ptr, codes,
            scales)
    return y, MxRows(*checkpoint)


def moe_combine_backward_mx(dy, checkpoint, slot_idx, topk_weights, d_expert_out=None, d_topk_weights=None,
                            stream=None):
    """moe_combine_backward with the rows of a checkpoint (MxRows in MOE_MX_E4M3) in place of expert_out."""
    dev, S, K, table = _table_arg(slot_idx)
    weights = _dense(topk_weights, "topk_weights", _fp32, (S, K), dev)
    H = _width(dy, "dy")
    dy_ptr = _dense(dy, "dy", _bf16, (S, H), dev)
    _, rows, _ = _matrix(checkpoint[1], "checkpoint.scales", torch.uint8)
    codes, scales = _mx_args(checkpoint, "checkpoint", rows, H, MOE_MX_E4M3, dev)
    d_expert_out, d_ptr, d_stride, d_topk_weights, dw_ptr = _gradient_outs(S, K, H, rows, topk_weights,
                                                                           d_expert_out, d_topk_weights, dev, stream)
    _launch(dev, stream, _lib.moe_combine_backward_mx, dy_ptr, codes, scales, rows, table, weights, S, H, K, d_ptr,
            d_stride, dw_ptr)
    return d_expert_out, d_topk_weights


def moe_dispatch_backward(d_rows, slot_idx, dx=None, stream=None):
    """The dispatch's gradient: dx[t] = bf16(sum_k d_rows[slot_idx[t, k]]) of d_rows (bf16 [R, H], any row
    stride), fp32 accumulation."""
    dev, S, K, table = _table_arg(slot_idx)
    H = _width(d_rows, "d_rows")
    ptr, stride, rows = _rows_arg(d_rows, "d_rows", H, dev)
    if dx is None:
        dx = _out(S, H, _bf16, dev, stream)
    dx_ptr = _dense(dx, "dx", _bf16, (S, H), dev)
    _launch(dev, stream, _lib.moe_dispatch_backward, ptr, stride, rows, table, S, H, K, dx_ptr)
    return dx


def moe_mx_row_bytes(H, format):
    v = _lib.moe_mx_row_bytes(int(H), int(format))
    if v < 0:
        _check(int(v))
    return int(v)


def _mx_empty(rows, H, format, dev, stream):
    return MxRows(_out(rows, _mx_width(H, format), _uint8, dev, stream), _out(rows, H // 32, _uint8, dev, stream))


def _count_arg(num_rows, dev):
    if num_rows is None:
        return None
    if (isinstance(num_rows, _Tensor) and num_rows.dtype is _int32 and num_rows.get_device() == dev
            and num_rows.numel() > 0 and num_rows.is_contiguous()):
        return num_rows.data_ptr()
    _need(num_rows, "num_rows", torch.int32, device=torch.device("cuda", dev))
    if num_rows.numel() < 1:
        raise ValueError("num_rows must hold a count")
    return num_rows.data_ptr()


_CALL_ROWS = 1 << 20  # MOE_MAX_OUT_ROWS: the rows that one call of the library converts at most


def _row_parts(name, ptr, stride, codes, width, scales, scale_bytes, count, num_rows, n, H, kind, dev, stream):
    """bf16 rows to codes (width bytes a row) and scales, or back, more rows than one call converts: call after call, all on
    the one stream. kind: the codes' format or quant."""
    quantize, fn = name.endswith("_quantize"), getattr(_lib, name)
    # a call checks its own part alone for outputs over inputs or over one another
    spans = ((ptr, (n - 1) * stride + 2 * H), (codes, n * width), (scales, n * scale_bytes), (count or 0, 4 if count else 0))
    for i, j in (((0, 1), (0, 2), (1, 2), (1, 3), (2, 3)) if quantize else ((0, 1), (0, 2), (0, 3))):
        (x, x_bytes), (y, y_bytes) = spans[i], spans[j]
        if y_bytes and x < y + y_bytes and y < x + x_bytes:
            raise ValueError(f"{name}: outputs must not overlap inputs or one another")
    with torch.cuda.stream(torch.cuda.current_stream(dev) if stream is None else _torch_stream(stream, dev)):
        for at in range(0, n, _CALL_ROWS):
            rows, left = min(_CALL_ROWS, n - at), None
            if count is not None:
                left = num_rows.reshape(-1)[:1].long().sub(at).clamp(0, rows).int()
            r, c, s = ptr + at * stride, codes + at * width, scales + at * scale_bytes
            left_ptr = None if left is None else left.data_ptr()
            if quantize:
                _launch(dev, stream, fn, r, stride, left_ptr, rows, H, kind, c, s)
            else:
                _launch(dev, stream, fn, c, s, left_ptr, rows, H, kind, r, stride)


def moe_mx_quantize(rows, format, num_rows=None, out=None, stream=None):
    """MxRows of bf16 rows [R, H] (any row stride), R without a limit. num_rows: None, or the device count of rows
    to take (e.g. layout.expert_slot_base[E:]); the outputs' other rows keep their contents."""
    dev, n, H = _matrix(rows, "rows", torch.bfloat16)
    if out is None:
        out = _mx_empty(n, H, format, dev, stream)
        codes, scales = out[0].data_ptr(), out[1].data_ptr()
    else:
        codes, scales = _mx_args(out, "out", n, H, format, dev)
    count = _count_arg(num_rows, dev)
    if n:
        ptr, stride, _ = _rows_arg(rows, "rows", H, dev)
        if n > _CALL_ROWS:
            _row_parts("moe_mx_quantize", ptr, stride, codes, _mx_width(H, format), scales, H // 32, count, num_rows, n, H, format, dev, stream)
        else:
            _launch(dev, stream, _lib.moe_mx_quantize, ptr, stride, count, n, H, format, codes, scales)
    return MxRows(*out)


def moe_mx_dequantize(mx, format, num_rows=None, out=None, stream=None):
    """The values of MxRows [R, ...] as bf16 rows [R, H] (out: any row stride), R without a limit."""
    dev, n, blocks = _matrix(mx[1], "mx.scales", torch.uint8)
    H = 32 * blocks
    codes, scales = _mx_args(mx, "mx", n, H, format, dev)
    if out is None:
        out = _out(n, H, _bf16, dev, stream)
    count = _count_arg(num_rows, dev)
    if n:
        ptr, stride, rows = _rows_arg(out, "out", H, dev)
        if rows != n:
            raise ValueError(f"out must have {n} rows")
        if n > _CALL_ROWS:
            _row_parts("moe_mx_dequantize", ptr, stride, codes, _mx_width(H, format), scales, H // 32, count, num_rows, n, H, format, dev, stream)
        else:
            _launch(dev, stream, _lib.moe_mx_dequantize, codes, scales, count, n, H, format, ptr, stride)
    return out


def moe_mx_product(a, w, group_base, epilogue=MOE_MX_PLAIN, out=None, stream=None):
    """The experts' product of MX E2M1 rows a (MxRows [R, ...]) with weights w (MxRows [G, O, ...]): row r of
    group g (group_base int32 [G + 1] on the device, e.g. layout.expert_slot_base) gives bf16 [O], or
    [O / 2] of silu(gate) * up with MOE_MX_GATED. Rows outside every group keep their contents (undefined
    where out is allocated here)."""
    dev, n, blocks = _matrix(a[1], "a.scales", torch.uint8)
    H = 32 * blocks
    a_codes, a_scales = _mx_args(a, "a", n, H, MOE_MX_E2M1, dev)
    w_codes, w_scales = w
    shape = w_codes.shape if isinstance(w_codes, _Tensor) else ()
    if len(shape) != 3:
        raise ValueError(f"w must be codes [G, O, {H // 2}] and scales [G, O, {blocks}]")
    G, O, _ = shape
    wc_ptr = _dense(w_codes, "w.codes", torch.uint8, (G, O, H // 2), dev)
    ws_ptr = _dense(w_scales, "w.scales", torch.uint8, (G, O, blocks), dev)
    base_ptr = _dense(group_base, "group_base", torch.int32, (G + 1,), dev)
    width = O // 2 if epilogue == MOE_MX_GATED else O
    if out is None:
        out = _out(n, width, _bf16, dev, stream)
        out_stride = 2 * width
    else:
        if (not isinstance(out, torch.Tensor) or out.dtype is not torch.bfloat16 or out.get_device() != dev
                or out.shape != (n, width)):
            raise ValueError(f"out must be bfloat16 {(n, width)} on cuda:{dev}")
        if width > 1 and out.stride(1) != 1 or n > 1 and out.stride(0) < width:
            raise ValueError("out must have contiguous rows that do not overlap")
        out_stride = 2 * out.stride(0) if n > 1 else 2 * width
    if n:
        _launch(dev, stream, _lib.moe_mx_product, a_codes, a_scales, n, base_ptr, G, wc_ptr, ws_ptr, O, H, epilogue,
                out.data_ptr(), out_stride)
    return out


# ---------------------------------------------------------------- the layer in 8 bits


class ScaledRows(NamedTuple):
    """Rows in 8 bits with one scale a row: codes uint8 [..., R, H] (INT8 codes may be int8) and scales fp32 [..., R],
    as moe_unpack leaves them in expand_x and expand_scales."""

    codes: torch.Tensor
    scales: torch.Tensor


_int8 = torch.int8


def _line(n, dtype, dev, stream):
    """A new output of n values for a call on `stream`."""
    if stream is None:
        return _empty(n, dtype=dtype, device=dev)
    with torch.cuda.stream(_torch_stream(stream, dev)):
        return _empty(n, dtype=dtype, device=dev)


def _code_type(codes):
    return _int8 if isinstance(codes, _Tensor) and codes.dtype is _int8 else _uint8


def _row8_args(rows8, name, shape, dev):
    """Pointers of the codes [*shape] and scales [*shape[:-1]]."""
    codes, scales = rows8
    return (_dense(codes, name + ".codes", _code_type(codes), shape, dev),
            _dense(scales, name + ".scales", _fp32, shape[:-1], dev))


def _row8_matrix(rows8, name):
    """Device, shape and pointers of the codes [R, H] and scales [R]."""
    codes, scales = rows8
    kind = _code_type(codes)
    dev, n, H = _matrix(codes, name + ".codes", kind)
    if not codes.is_contiguous():
        _dense(codes, name + ".codes", kind, (n, H), dev)
    return dev, n, H, codes.data_ptr(), _dense(scales, name + ".scales", _fp32, (n,), dev)


def _row8_empty(rows, H, dev, stream):
    return ScaledRows(_out(rows, H, _uint8, dev, stream), _line(rows, _fp32, dev, stream))


def _some_rows(t, name, n, H, dev):
    """Pointer and row stride in bytes of bf16 rows [n, H], of which there may be none."""
    if not isinstance(t, _Tensor) or t.shape != (n, H):
        raise ValueError(f"{name} must be bfloat16 {(n, H)}")
    if t.dtype is _bf16 and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr(), 2 * H
    if n == 0:
        raise ValueError(f"{name} must be bfloat16 on cuda:{dev}, got {t.dtype} on {t.device}")
    return _rows_arg(t, name, H, dev)[:2]


def _row_matrix(t, name):
    """Device, shape, pointer and row stride in bytes of bf16 rows [R, H], of which there may be none."""
    if isinstance(t, _Tensor) and t.dtype is _bf16 and t.is_contiguous():
        dev, shape = t.get_device(), t.shape
        if dev >= 0 and len(shape) == 2:
            n, H = shape
            return dev, n, H, t.data_ptr(), 2 * H
    dev, n, H = _matrix(t, name, _bf16)
    return dev, n, H, *_some_rows(t, name, n, H, dev)


def moe_row_quantize(rows, quant, num_rows=None, out=None, stream=None):
    """ScaledRows of bf16 rows [R, H] (any row stride), R without a limit, in MOE_QUANT_INT8_DYN or MOE_QUANT_FP8_E4M3_DYN, as
    moe_dispatch computes them. num_rows: None, or the device count of rows to take (e.g. layout.expert_slot_base[E:]); the
    outputs' other rows keep their contents (undefined where they are allocated here)."""
    dev, n, H, ptr, stride = _row_matrix(rows, "rows")
    if out is None:
        out = _row8_empty(n, H, dev, stream)
        codes, scales = out[0].data_ptr(), out[1].data_ptr()
    else:
        codes, scales = _row8_args(out, "out", (n, H), dev)
    count = _count_arg(num_rows, dev)
    if n > _CALL_ROWS:
        _row_parts("moe_row_quantize", ptr, stride, codes, H, scales, 4, count, num_rows, n, H, quant, dev, stream)
    else:
        _launch(dev, stream, _lib.moe_row_quantize, ptr, stride, count, n, H, quant, codes, scales)
    return ScaledRows(*out)


def moe_row_dequantize(rows8, quant, num_rows=None, out=None, stream=None):
    """The values of ScaledRows [R, H] as bf16 rows (out: any row stride), R without a limit."""
    dev, n, H, codes, scales = _row8_matrix(rows8, "rows8")
    if out is None:
        out = _out(n, H, _bf16, dev, stream)
        ptr, stride = out.data_ptr(), 2 * H
    else:
        ptr, stride = _some_rows(out, "out", n, H, dev)
    count = _count_arg(num_rows, dev)
    if n > _CALL_ROWS:
        _row_parts("moe_row_dequantize", ptr, stride, codes, H, scales, 4, count, num_rows, n, H, quant, dev, stream)
    else:
        _launch(dev, stream, _lib.moe_row_dequantize, codes, scales, count, n, H, quant, ptr, stride)
    return out


def moe_scaled_product(a, w, group_base, epilogue=MOE_MX_PLAIN, out=None, stream=None):
    """The experts' product of INT8 rows a (ScaledRows [R, H], e.g. of moe_unpack's expand_x and expand_scales) with
    INT8 weights w (ScaledRows [G, O, H], a scale for each output): row r of group g (group_base int32 [G + 1] on the
    device, e.g. layout.expert_slot_base; [0, R] with G = 1 for a shared expert) gives bf16 [O], or [O / 2] of
    silu(gate) * up with MOE_MX_GATED. Rows outside every group keep their contents (undefined where out is allocated
    here)."""
    dev, n, H, a_ptr, as_ptr = _row8_matrix(a, "a")
    w_codes = w[0]
    shape = w_codes.shape if isinstance(w_codes, _Tensor) else ()
    if len(shape) != 3 or shape[2] != H:
        raise ValueError(f"w must be codes [G, O, {H}] and scales [G, O]")
    G, O, _ = shape
    w_ptr, ws_ptr = _row8_args(w, "w", (G, O, H), dev)
    base_ptr = _dense(group_base, "group_base", _int32, (G + 1,), dev)
    width = O // 2 if epilogue == MOE_MX_GATED else O
    if out is None:
        out = _out(n, width, _bf16, dev, stream)
        out_stride = 2 * width
    else:
        if not isinstance(out, _Tensor) or out.dtype is not _bf16 or out.get_device() != dev or out.shape != (n, width):
            raise ValueError(f"out must be bfloat16 {(n, width)} on cuda:{dev}")
        if n and (width > 1 and out.stride(1) != 1 or n > 1 and out.stride(0) < width):
            raise ValueError("out must have contiguous rows that do not overlap")
        out_stride = 2 * out.stride(0) if n > 1 else 2 * width
    _launch(dev, stream, _lib.moe_scaled_product, a_ptr, as_ptr, n, base_ptr, G, w_ptr, ws_ptr, O, H, epilogue,
            out.data_ptr(), out_stride)
    return out


class RmsNorm(NamedTuple):
    out: torch.Tensor  # bf16 [S, H]; None with a quant unless it was passed
    sum: torch.Tensor  # bf16 [S, H]: what was normed, x + residual, or x itself without a residual
    rows8: ScaledRows  # the normed rows in 8 bits; None with MOE_QUANT_NONE


def _weight_arg(weight, H, dev):
    """Pointer and moe_float of a norm's weight."""
    kind = weight.dtype if isinstance(weight, _Tensor) else None
    if kind is _bf16:
        return _dense(weight, "weight", _bf16, (H,), dev), MOE_BF16
    return _dense(weight, "weight", _fp32, (H,), dev), MOE_FP32


def moe_rms_norm(x, weight, eps=1e-6, residual=None, quant=MOE_QUANT_NONE, out=None, sum=None, rows8=None, stream=None):
    """The root-mean-square norm of bf16 rows x [S, H], or of x + residual, times weight (bf16 or fp32 [H]): bf16 rows,
    with a quant (MOE_QUANT_INT8_DYN, MOE_QUANT_FP8_E4M3_DYN) rows in 8 bits instead, and both where out is passed too.
    x, residual and sum may have any row stride; sum may be x or residual itself (an addition in place)."""
    dev, n, H, ptr, stride = _row_matrix(x, "x")
    res_ptr, res_stride, sum_ptr, sum_stride, out_ptr, codes, scales = None, 0, None, 0, None, None, None
    if residual is not None:
        res_ptr, res_stride = _some_rows(residual, "residual", n, H, dev)
        if sum is None:
            sum = _out(n, H, _bf16, dev, stream)
            sum_ptr, sum_stride = sum.data_ptr(), 2 * H
        else:
            sum_ptr, sum_stride = _some_rows(sum, "sum", n, H, dev)
    elif sum is not None:
        raise ValueError("sum is written only with a residual")
    else:
        sum = x
    w_ptr, kind = _weight_arg(weight, H, dev)
    if quant == MOE_QUANT_NONE:
        if rows8 is not None:
            raise ValueError("rows8 is written only with a quant")
        if out is None:
            out = _out(n, H, _bf16, dev, stream)
            out_ptr = out.data_ptr()
    elif rows8 is None:
        rows8 = _row8_empty(n, H, dev, stream)
        codes, scales = rows8[0].data_ptr(), rows8[1].data_ptr()
    else:
        codes, scales = _row8_args(rows8, "rows8", (n, H), dev)
        rows8 = ScaledRows(*rows8)
    if out is not None and out_ptr is None:
        out_ptr = _dense(out, "out", _bf16, (n, H), dev)
    _launch(dev, stream, _lib.moe_rms_norm, ptr, stride, res_ptr, res_stride, w_ptr, kind, eps, n, H, quant, sum_ptr,
            sum_stride, out_ptr, codes, scales)
    return RmsNorm(out, sum, rows8)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(name, a, b):
    """The library's answer to a size query of two numbers (never of objects, whose values may change)."""
    v = getattr(_lib, name)(a, b)
    if v < 0:
        _check(int(v))
    return int(v)


def moe_rms_norm_backward_workspace_bytes(rows, H):
    return _workspace_bytes("moe_rms_norm_backward_workspace_bytes", int(rows), int(H))


def _workspace(workspace, need, dev, stream):
    """A call's workspace with its pointer and bytes: one is allocated where none is passed and the call needs one."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = _line(need, _uint8, dev, stream)
        return workspace, workspace.data_ptr(), need
    _need(workspace, "workspace", device=torch.device("cuda", dev))
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def moe_rms_norm_backward(dy, sum, weight, eps=1e-6, d_sum=None, dx=None, d_weight=None, workspace=None, stream=None):
    """The gradients of moe_rms_norm's bf16 output: (dx bf16 [S, H], for x and the residual alike, and d_weight fp32 [H])
    of dy, the rows that the forward normed (its sum), weight and eps. d_sum: the gradient that reaches the sum on its
    other ways, added to dx. dy, sum and d_sum may have any row stride. workspace: a device buffer of at least
    moe_rms_norm_backward_workspace_bytes(S, H) bytes, or None to have one allocated."""
    dev, n, H, ptr, stride = _row_matrix(sum, "sum")
    dy_ptr, dy_stride = _some_rows(dy, "dy", n, H, dev)
    ds_ptr, ds_stride = (None, 0) if d_sum is None else _some_rows(d_sum, "d_sum", n, H, dev)
    w_ptr, kind = _weight_arg(weight, H, dev)
    if dx is None:
        dx = _out(n, H, _bf16, dev, stream)
        dx_ptr = dx.data_ptr()
    else:
        dx_ptr = _dense(dx, "dx", _bf16, (n, H), dev)
    if d_weight is None:
        d_weight = _line(H, _fp32, dev, stream)
        dw_ptr = d_weight.data_ptr()
    else:
        dw_ptr = _dense(d_weight, "d_weight", _fp32, (H,), dev)
    workspace, ws_ptr, ws_bytes = _workspace(workspace, _workspace_bytes("moe_rms_norm_backward_workspace_bytes", n, H), dev, stream)
    _launch(dev, stream, _lib.moe_rms_norm_backward, dy_ptr, dy_stride, ptr, stride, w_ptr, kind, eps, ds_ptr, ds_stride,
            n, H, dx_ptr, dw_ptr, ws_ptr, ws_bytes)
    return dx, d_weight


class BalanceLoss(NamedTuple):
    loss: torch.Tensor  # fp32 [1]
    num_tokens_per_expert: torch.Tensor  # int32 [E], the layout's
    num_tokens: torch.Tensor  # int32 [1], tokens with a valid entry


def _router_args(logits, topk_idx):
    """Device, S, K, E, and the logits' pointer, row stride in bytes and type, and the entries' pointer."""
    dev, S, K, table = _table_arg(topk_idx)
    if isinstance(logits, _Tensor) and logits.dtype is _bf16:
        size, kind = 2, MOE_BF16
    else:
        size, kind = 4, MOE_FP32
    at, rows, E = _matrix(logits, "logits", _bf16 if kind == MOE_BF16 else _fp32)
    if at != dev or rows != S:
        raise ValueError(f"logits must have {S} rows on cuda:{dev}")
    if logits.is_contiguous():
        return dev, S, K, E, logits.data_ptr(), size * E, kind, table
    step, col = logits.stride()
    if E > 1 and col != 1 or S > 1 and step < E:
        raise ValueError("logits must have contiguous rows that do not overlap")
    return dev, S, K, E, logits.data_ptr(), size * (step if S > 1 else E), kind, table


def moe_balance_loss_workspace_bytes(S, E):
    return _workspace_bytes("moe_balance_loss_workspace_bytes", int(S), int(E))


def moe_balance_loss(logits, topk_idx, coef, score=MOE_SCORE_SOFTMAX, out=None, workspace=None, stream=None):
    """BalanceLoss of the router's logits (bf16 or fp32 [S, E], any row stride) and its choice topk_idx (int32 [S, K], -1
    for padding and dropped entries): coef * E / (N * T) * sum_e count_e * sum_t score[t, e] over the T tokens that have a
    valid entry, N of those in all. score: MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID. workspace: a device buffer of at
    least moe_balance_loss_workspace_bytes(S, E) bytes, or None to have one allocated."""
    dev, S, K, E, ptr, stride, kind, table = _router_args(logits, topk_idx)
    if out is None:
        out = BalanceLoss(_line(1, _fp32, dev, stream), _line(E, _int32, dev, stream), _line(1, _int32, dev, stream))
        loss, counts, tokens = out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr()
    else:
        out = BalanceLoss(*out)
        loss = _dense(out.loss, "loss", _fp32, (1,), dev)
        counts = _dense(out.num_tokens_per_expert, "num_tokens_per_expert", _int32, (E,), dev)
        tokens = _dense(out.num_tokens, "num_tokens", _int32, (1,), dev)
    workspace, ws_ptr, ws_bytes = _workspace(workspace, _workspace_bytes("moe_balance_loss_workspace_bytes", S, E), dev, stream)
    _launch(dev, stream, _lib.moe_balance_loss, ptr, stride, kind, table, S, K, E, score, coef, loss, counts, tokens, ws_ptr,
            ws_bytes)
    return out


def moe_balance_loss_backward(d_loss, logits, topk_idx, num_tokens_per_expert, num_tokens, coef, score=MOE_SCORE_SOFTMAX,
                              d_logits=None, stream=None):
    """The balance loss's gradient d_logits ([S, E] of the logits' type) of d_loss (fp32 [1]), with the forward's
    arguments and counts; or with the sums of both num_tokens_per_expert and num_tokens over several GPUs, for the loss over
    all their tokens."""
    dev, S, K, E, ptr, stride, kind, table = _router_args(logits, topk_idx)
    dl_ptr = _dense(d_loss, "d_loss", _fp32, (1,), dev)
    counts = _dense(num_tokens_per_expert, "num_tokens_per_expert", _int32, (E,), dev)
    tokens = _dense(num_tokens, "num_tokens", _int32, (1,), dev)
    if d_logits is None:
        d_logits = _out(S, E, logits.dtype, dev, stream)
        out_ptr = d_logits.data_ptr()
    else:
        out_ptr = _dense(d_logits, "d_logits", logits.dtype, (S, E), dev)
    _launch(dev, stream, _lib.moe_balance_loss_backward, dl_ptr, ptr, stride, kind, table, counts, tokens, S, K, E, score,
            coef, out_ptr)
    return d_logits


__all__ = [
    "MOE_OK", "MOE_ERR_ARG", "MOE_ERR_ALIGN", "MOE_ERR_WINDOW", "MOE_ERR_UNSUPPORTED",
    "MOE_ERR_HIP", "MOE_QUANT_NONE", "MOE_QUANT_FP8_E4M3_DYN", "MOE_QUANT_INT8_DYN", "MOE_LAYOUT_AUTO",
    "MOE_LAYOUT_MULTI", "MOE_LAYOUT_SINGLE", "MoeError", "Layout",
    "empty_layout", "moe_slot_bytes", "moe_window_bytes", "moe_slot_offsets", "moe_layout",
    "moe_dispatch", "moe_dispatch_workspace_bytes", "moe_dispatch_ws", "moe_dispatch_noalloc", "MOE_ERR_SCRATCH",
    "moe_layout_dispatch_workspace_bytes", "moe_layout_ws", "moe_dispatch_planned", "moe_layout_dispatch_ws",
    "MOE_NOALLOC_SCRATCH_BYTES", "moe_layout_dispatch", "moe_combine", "moe_combine_scatter", "moe_combine_staged", "moe_unpack", "Unpacked", "moe_unpack_padded", "PaddedUnpacked",
    "moe_dedup_window_bytes", "moe_rank_rows", "RankRows", "moe_dispatch_dedup", "moe_expand_dedup",
    "moe_status_string", "Plan", "plan_layout", "plan_dispatch_ws", "plan_layout_dispatch", "plan_combine",
    "plan_layout_ws", "plan_dispatch_planned",
    "MOE_PLAN_BYTES",
    "MOE_MX_E2M1", "MOE_MX_E4M3", "MOE_MX_PLAIN", "MOE_MX_GATED", "MxRows", "moe_combine_backward",
    "moe_combine_checkpoint", "moe_combine_backward_mx", "moe_dispatch_backward", "moe_mx_row_bytes",
    "moe_mx_quantize", "moe_mx_dequantize", "moe_mx_product",
    "MOE_BF16", "MOE_FP32", "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID", "ScaledRows", "moe_row_quantize", "moe_row_dequantize",
    "moe_scaled_product", "RmsNorm", "moe_rms_norm", "moe_rms_norm_backward", "moe_rms_norm_backward_workspace_bytes",
    "BalanceLoss", "moe_balance_loss", "moe_balance_loss_backward", "moe_balance_loss_workspace_bytes",
]
