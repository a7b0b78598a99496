"""Sparse MoE FFN layer forward on one B200: Python binding of libmoe_b200.so.

The binding only marshals arguments (torch tensors -> device pointers, the
current CUDA stream) into the C ABI declared in include/moe_b200.h; every step
of the layer runs in the library's CUDA kernels.  There is no CPU or PyTorch
fallback: if the shared library is missing, importing the entry points raises.

Entry points (same names as the C ABI): moe_workspace_size, moe_buffer_rows,
moe_workspace_init, moe_get_device_status, moe_route, moe_dispatch,
moe_expert_ffn, moe_combine, moe_balance_stats, moe_layer_forward,
moe_selftest_wait_timeout; for serving moe_layer_forward_few (at most 16
tokens in one kernel), moe_mxfp4_quantize, moe_mxfp4_dequantize,
moe_mxfp4_tile_scales and moe_mxfp4_matmul (shapes from make_mxfp4_shape).
`MoELayer` bundles a config, its workspace and its weights for the common
whole-layer calls.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_b200.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_CUDA = 3
MOE_ERR_BAD_ROUTING = 4
MOE_ERR_DEVICE_TIMEOUT = 5
MOE_DEV_BAD_ROUTING = 0x1
MOE_DEV_TIMEOUT = 0x2
MOE_F32, MOE_BF16, MOE_FP8_E4M3_BLOCK, MOE_MXFP4 = 0, 1, 2, 3
MOE_ACT_NONE, MOE_ACT_SILU = 0, 1
MOE_FEW_MAX_TOKENS = 16
MOE_BIAS_LOGITS, MOE_BIAS_SELECTION = 0, 1
MOE_PRIORITY_TOKEN, MOE_PRIORITY_SLOT = 0, 1
MOE_OVERFLOW_DROP, MOE_OVERFLOW_PASS = 0, 1

EXPORTED = (
    "moe_workspace_size", "moe_buffer_rows", "moe_workspace_init", "moe_get_device_status",
    "moe_last_cuda_error", "moe_status_string", "moe_route", "moe_dispatch", "moe_expert_ffn",
    "moe_combine", "moe_balance_stats", "moe_layer_forward", "moe_selftest_wait_timeout",
    "moe_dispatch_noalloc", "moe_kernel_launches", "moe_backward_workspace_size", "moe_layer_backward",
    "moe_expert_ffn_segments", "moe_few_workspace_size", "moe_few_workspace_init", "moe_layer_forward_few",
    "moe_mxfp4_quantize", "moe_mxfp4_dequantize", "moe_mxfp4_tile_scales", "moe_mxfp4_workspace_size",
    "moe_mxfp4_workspace_init", "moe_mxfp4_get_device_status", "moe_mxfp4_matmul",
)


class moe_config(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_routed", ctypes.c_int32),
        ("top_k", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("n_shared", ctypes.c_int32),
        ("d_ff_shared", ctypes.c_int32), ("capacity_factor", ctypes.c_float),
        ("alpha", ctypes.c_float), ("dtype", ctypes.c_int32), ("bias_mode", ctypes.c_int32),
        ("capacity_priority", ctypes.c_int32), ("overflow_mode", ctypes.c_int32),
    ]


class moe_mxfp4_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "n", "k", "n_mats", "n_seg", "activation", "out_dtype")]


class moe_backward_io(ctypes.Structure):
    """Pointers of moe_layer_backward, in the header's order."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "x", "W_r", "W1", "b1", "W2", "b2", "Ws1", "bs1", "Ws2", "bs2",
        "logits", "topk_idx", "gates", "counts", "offsets", "slot_row", "row_slot", "x_disp", "y",
        "dout",
        "dx", "dW_r", "d_logit_bias", "dW1", "db1", "dW2", "db2", "dWs1", "dbs1", "dWs2", "dbs2")]


BACKWARD_IO_FIELDS = tuple(n for n, _ in moe_backward_io._fields_)


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = lib().moe_status_string(status).decode()
        extra = ""
        if status == MOE_ERR_CUDA:
            extra = f" (cudaError {lib().moe_last_cuda_error()})"
        super().__init__(f"{where}: {name}{extra}")


_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded shared library.  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m sparse_mixture_experts_20_b200.build` (nvcc, sm_100a)")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        cfgp = ctypes.POINTER(moe_config)
        shp = ctypes.POINTER(moe_mxfp4_shape)
        I = ctypes.c_int
        i32, i64 = ctypes.c_int32, ctypes.c_int64
        sig = {
            "moe_workspace_size": [cfgp, ctypes.POINTER(ctypes.c_size_t)],
            "moe_buffer_rows": [cfgp] + [ctypes.POINTER(ctypes.c_int32)] * 4,
            "moe_workspace_init": [cfgp, P, P],
            "moe_get_device_status": [cfgp, P, P, ctypes.POINTER(ctypes.c_int32), ctypes.c_int32],
            "moe_last_cuda_error": [],
            "moe_status_string": [I],
            "moe_route": [cfgp, P, P, P, P, P, P, P, P],
            "moe_dispatch": [cfgp, P, P, P, P, P, P, P, P, P, P, P],
            "moe_expert_ffn": [cfgp] + [P] * 19,
            "moe_combine": [cfgp, P, P, P, P, P, P],
            "moe_balance_stats": [cfgp, P, P, P, P, P, P],
            "moe_layer_forward": [cfgp] + [P] * 24,
            "moe_selftest_wait_timeout": [cfgp, ctypes.c_int64, P, P],
            "moe_dispatch_noalloc": [cfgp, P, P, P, P, P, P, P, P, P, P],
            "moe_kernel_launches": [],
            "moe_backward_workspace_size": [cfgp, ctypes.POINTER(ctypes.c_size_t)],
            "moe_layer_backward": [cfgp, ctypes.c_float, ctypes.POINTER(moe_backward_io), P, P],
            "moe_expert_ffn_segments": [cfgp, P, P, P, P, ctypes.c_int32] + [P] * 9,
            "moe_few_workspace_size": [cfgp, ctypes.POINTER(ctypes.c_size_t)],
            "moe_few_workspace_init": [cfgp, P, P],
            "moe_layer_forward_few": [cfgp] + [P] * 24,
            "moe_mxfp4_quantize": [P, i32, i64, i32, P, P, P],
            "moe_mxfp4_dequantize": [P, P, i64, i32, P, i32, P],
            "moe_mxfp4_tile_scales": [P, i64, i32, i32, P, P],
            "moe_mxfp4_workspace_size": [shp, ctypes.POINTER(ctypes.c_size_t)],
            "moe_mxfp4_workspace_init": [shp, P, P],
            "moe_mxfp4_get_device_status": [shp, P, P, ctypes.POINTER(i32), i32],
            "moe_mxfp4_matmul": [shp] + [P] * 11,
        }
        restype = {"moe_status_string": ctypes.c_char_p, "moe_kernel_launches": ctypes.c_uint64}
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = restype.get(name, I)
        _LIB = L
    return _LIB


def make_config(shape=None, **kw) -> moe_config:
    """moe_config from any object with the fields T, d_model, n_routed, top_k,
    d_ff, n_shared, d_ff_shared, capacity_factor, alpha, dtype, bias_mode,
    capacity_priority, overflow_mode (keyword arguments override)."""
    fields = [f for f, _ in moe_config._fields_]
    vals = {f: getattr(shape, f) for f in fields if shape is not None and hasattr(shape, f)}
    vals.update(kw)
    vals.setdefault("n_shared", 0)
    vals.setdefault("d_ff_shared", 0)
    vals.setdefault("capacity_factor", 0.0)
    vals.setdefault("alpha", 0.01)
    vals.setdefault("dtype", MOE_BF16)
    vals.setdefault("bias_mode", MOE_BIAS_LOGITS)
    vals.setdefault("capacity_priority", MOE_PRIORITY_TOKEN)
    vals.setdefault("overflow_mode", MOE_OVERFLOW_DROP)
    return moe_config(**{f: vals[f] for f in fields})


def _p(t) -> Optional[int]:
    """Device pointer of a tensor (None for None)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        if torch.cuda.is_initialized():                        # the same handle, without building a Stream object
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _current(stream):
    """A context with `stream` (None, a torch stream or a raw handle) as the current one, for the memory that a launch
    on it writes: what the allocator hands out may still be in use by work queued on the stream it was asked on."""
    import torch
    if stream is not None and not hasattr(stream, "wait_stream"):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)                           # (None: no change)


def _on_current_device(t, what: str):
    """The library launches on the current device and its stream: a tensor of another one is refused."""
    import torch
    if t.is_cuda and t.device.index != torch._C._cuda_getDevice():
        raise ValueError(f"{what}: the tensors are on {t.device}, which is not the current device")


def _typed(t, name: str, what: str, *types):
    """Refuses a tensor that holds none of `types`; uint8 and int8 stand for the bytes of any."""
    import torch
    if t.dtype not in types and t.dtype is not torch.uint8 and t.dtype is not torch.int8:
        raise ValueError(f"{what}: {name} is {t.dtype}, not {types[0]}")


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoEError(status, where)


def moe_workspace_size(cfg: moe_config) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def moe_buffer_rows(cfg: moe_config):
    """(capacity or -1, R_cap, x_disp rows, y rows)."""
    vals = [ctypes.c_int32(0) for _ in range(4)]
    _check(lib().moe_buffer_rows(ctypes.byref(cfg), *[ctypes.byref(v) for v in vals]), "moe_buffer_rows")
    return tuple(v.value for v in vals)


def moe_workspace_init(cfg, ws, stream=None):
    _check(lib().moe_workspace_init(ctypes.byref(cfg), _p(ws), _stream(stream)), "moe_workspace_init")


def moe_get_device_status(cfg, ws, stream=None, clear: bool = False) -> int:
    st = ctypes.c_int32(0)
    _check(lib().moe_get_device_status(ctypes.byref(cfg), _p(ws), _stream(stream), ctypes.byref(st),
                                       1 if clear else 0), "moe_get_device_status")
    return st.value


def moe_kernel_launches() -> int:
    """Kernels the library has launched in this process since it was loaded."""
    return int(lib().moe_kernel_launches())


def moe_route(cfg, x, W_r, logit_bias, topk_idx, gates, logits_out, ws, stream=None):
    _check(lib().moe_route(ctypes.byref(cfg), _p(x), _p(W_r), _p(logit_bias), _p(topk_idx), _p(gates),
                           _p(logits_out), _p(ws), _stream(stream)), "moe_route")


def moe_dispatch(cfg, x, topk_idx, counts, kept, offsets, slot_row, row_slot, x_disp, x_disp_scales,
                 ws, stream=None):
    _check(lib().moe_dispatch(ctypes.byref(cfg), _p(x), _p(topk_idx), _p(counts), _p(kept), _p(offsets),
                              _p(slot_row), _p(row_slot), _p(x_disp), _p(x_disp_scales), _p(ws),
                              _stream(stream)), "moe_dispatch")


def moe_expert_ffn(cfg, x, x_disp, x_disp_scales, offsets, W1, W1_scales, b1, W2, W2_scales, b2,
                   Ws1, Ws1_scales, bs1, Ws2, Ws2_scales, bs2, y, ws, stream=None):
    _check(lib().moe_expert_ffn(ctypes.byref(cfg), _p(x), _p(x_disp), _p(x_disp_scales), _p(offsets),
                                _p(W1), _p(W1_scales), _p(b1), _p(W2), _p(W2_scales), _p(b2),
                                _p(Ws1), _p(Ws1_scales), _p(bs1), _p(Ws2), _p(Ws2_scales), _p(bs2),
                                _p(y), _p(ws), _stream(stream)), "moe_expert_ffn")


def moe_expert_ffn_segments(cfg, x_rows, x_rows_scales, seg_offsets, seg_expert, n_seg: int,
                            W1, W1_scales, b1, W2, W2_scales, b2, y, ws, stream=None):
    """The grouped expert FFN over caller-made segments: rows seg_offsets[i] ..
    seg_offsets[i+1]-1 of x_rows through expert seg_expert[i] (cfg: the held
    experts, top_k 1, T = rows, no shared experts, no capacity)."""
    _check(lib().moe_expert_ffn_segments(ctypes.byref(cfg), _p(x_rows), _p(x_rows_scales), _p(seg_offsets),
                                         _p(seg_expert), int(n_seg), _p(W1), _p(W1_scales), _p(b1), _p(W2),
                                         _p(W2_scales), _p(b2), _p(y), _p(ws), _stream(stream)),
           "moe_expert_ffn_segments")


def moe_combine(cfg, y, gates, slot_row, out, stream=None, x=None):
    """x (the layer input) is read only with overflow_mode = MOE_OVERFLOW_PASS."""
    _check(lib().moe_combine(ctypes.byref(cfg), _p(y), _p(gates), _p(slot_row), _p(x), _p(out),
                             _stream(stream)), "moe_combine")


def moe_balance_stats(cfg, counts, ws, f, P, loss, stream=None):
    _check(lib().moe_balance_stats(ctypes.byref(cfg), _p(counts), _p(ws), _p(f), _p(P), _p(loss),
                                   _stream(stream)), "moe_balance_stats")


def moe_layer_forward(cfg, x, W_r, logit_bias, W1, W1_scales, b1, W2, W2_scales, b2,
                      Ws1, Ws1_scales, bs1, Ws2, Ws2_scales, bs2, out, f, P, loss,
                      topk_idx, gates, counts, ws, stream=None):
    _check(lib().moe_layer_forward(ctypes.byref(cfg), _p(x), _p(W_r), _p(logit_bias), _p(W1), _p(W1_scales),
                                   _p(b1), _p(W2), _p(W2_scales), _p(b2), _p(Ws1), _p(Ws1_scales), _p(bs1),
                                   _p(Ws2), _p(Ws2_scales), _p(bs2), _p(out), _p(f), _p(P), _p(loss),
                                   _p(topk_idx), _p(gates), _p(counts), _p(ws), _stream(stream)),
           "moe_layer_forward")


def moe_selftest_wait_timeout(cfg, timeout_ns: int, ws, stream=None):
    _check(lib().moe_selftest_wait_timeout(ctypes.byref(cfg), int(timeout_ns), _p(ws), _stream(stream)),
           "moe_selftest_wait_timeout")


def moe_backward_workspace_size(cfg: moe_config) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_backward_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), "moe_backward_workspace_size")
    return n.value


def backward_io(tensors: dict) -> moe_backward_io:
    """moe_backward_io from a dict of tensors keyed by the header's field
    names (missing or None fields are NULL)."""
    unknown = set(tensors) - set(BACKWARD_IO_FIELDS)
    if unknown:
        raise KeyError(f"not moe_backward_io fields: {sorted(unknown)}")
    return moe_backward_io(**{n: _p(tensors.get(n)) for n in BACKWARD_IO_FIELDS})


def moe_layer_backward(cfg, lam: float, tensors: dict, bws, stream=None):
    """Gradients of <dout, out> + lam * L_balance (fp32, written into the dx,
    dW_r, ... tensors of `tensors`); bws: moe_backward_workspace_size() bytes."""
    io = backward_io(tensors)
    _check(lib().moe_layer_backward(ctypes.byref(cfg), ctypes.c_float(lam), ctypes.byref(io), _p(bws),
                                    _stream(stream)), "moe_layer_backward")


def moe_dispatch_noalloc(cfg, x, topk_idx, counts, kept, offsets, slot_row, row_slot, x_disp,
                         x_disp_scales, stream=None):
    """moe_dispatch with its scratch in the library's own 2 MiB device array
    instead of a workspace: for callers that cannot allocate device memory.
    Calls that overlap on the GPU race on that array."""
    _check(lib().moe_dispatch_noalloc(ctypes.byref(cfg), _p(x), _p(topk_idx), _p(counts), _p(kept),
                                      _p(offsets), _p(slot_row), _p(row_slot), _p(x_disp),
                                      _p(x_disp_scales), _stream(stream)), "moe_dispatch_noalloc")


def moe_few_workspace_size(cfg: moe_config) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_few_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), "moe_few_workspace_size")
    return n.value


def moe_few_workspace_init(cfg, ws, stream=None):
    _check(lib().moe_few_workspace_init(ctypes.byref(cfg), _p(ws), _stream(stream)), "moe_few_workspace_init")


def moe_layer_forward_few(cfg, x, W_r, logit_bias, W1, W1_scales, b1, W2, W2_scales, b2,
                          Ws1, Ws1_scales, bs1, Ws2, Ws2_scales, bs2, out, f, P, loss,
                          topk_idx, gates, counts, ws, stream=None):
    """moe_layer_forward for at most MOE_FEW_MAX_TOKENS tokens, in one kernel (bf16, FP8 or MXFP4 experts,
    the last with scales from moe_mxfp4_tile_scales); ws: moe_few_workspace_size() bytes after
    moe_few_workspace_init."""
    _check(lib().moe_layer_forward_few(ctypes.byref(cfg), _p(x), _p(W_r), _p(logit_bias), _p(W1), _p(W1_scales),
                                       _p(b1), _p(W2), _p(W2_scales), _p(b2), _p(Ws1), _p(Ws1_scales), _p(bs1),
                                       _p(Ws2), _p(Ws2_scales), _p(bs2), _p(out), _p(f), _p(P), _p(loss),
                                       _p(topk_idx), _p(gates), _p(counts), _p(ws), _stream(stream)),
           "moe_layer_forward_few")


def _mxfp4_args(dense, codes, scales, what: str, stream):
    """(dtype, rows, cols, stream handle) of a dense matrix and its MXFP4 form, checked against each other."""
    import torch
    dt = dense.dtype
    if dt is not torch.float32 and dt is not torch.bfloat16:
        raise ValueError(f"{what}: the dense matrix must be float32 or bfloat16")
    if dense.dim() < 1 or codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise ValueError(f"{what}: codes and scales are uint8 matrices")
    cols, n = dense.shape[-1], dense.numel()
    if cols < 1 or cols % 32:
        raise ValueError(f"{what}: the last dimension ({cols}) must be a multiple of 32")
    if codes.numel() * 2 != n or scales.numel() * 32 != n:
        raise ValueError(f"{what}: codes need (..., cols / 2) and scales (..., cols / 32) elements")
    dev = dense.get_device()                                   # -1: not on a GPU
    if dev != codes.get_device() or dev != scales.get_device():
        raise ValueError(f"{what}: all tensors must be on one device")
    if dev < 0:
        raise ValueError("tensor must live on a CUDA device")
    if not (dense.is_contiguous() and codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("tensor must be contiguous")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{what}: the tensors are on cuda:{dev}, which is not the current device")
    st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    return MOE_F32 if dt is torch.float32 else MOE_BF16, n // cols, cols, st


def moe_mxfp4_quantize(x, codes, scales, stream=None):
    """x (..., cols) float32 / bfloat16 into MXFP4: codes uint8 (..., cols / 2), scales uint8 (..., cols / 32)."""
    dtype, rows, cols, st = _mxfp4_args(x, codes, scales, "moe_mxfp4_quantize", stream)
    _check(lib().moe_mxfp4_quantize(x.data_ptr(), dtype, rows, cols, codes.data_ptr(), scales.data_ptr(), st),
           "moe_mxfp4_quantize")


def moe_mxfp4_dequantize(codes, scales, out, stream=None):
    """The values of an MXFP4 matrix into out (..., cols) float32 / bfloat16."""
    dtype, rows, cols, st = _mxfp4_args(out, codes, scales, "moe_mxfp4_dequantize", stream)
    _check(lib().moe_mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, out.data_ptr(), dtype, st),
           "moe_mxfp4_dequantize")


def moe_mxfp4_tile_scales(scales, stream=None):
    """The scales (n_mats, rows, cols / 32) uint8 of a stack of MXFP4 matrices, in the order that
    moe_layer_forward_few streams."""
    import torch
    if scales.dim() != 3 or scales.dtype != torch.uint8 or scales.shape[1] < 1 or scales.shape[2] < 1:
        raise ValueError("moe_mxfp4_tile_scales: scales are a uint8 stack (n_mats, rows, cols / 32)")
    _on_current_device(scales, "moe_mxfp4_tile_scales")
    n, rows, cols = scales.shape[0], scales.shape[1], scales.shape[2] * 32
    with _current(stream):
        tiled = torch.empty((n, (rows + 127) // 128, cols // 128, 512), dtype=torch.uint8, device=scales.device)
    _check(lib().moe_mxfp4_tile_scales(_p(scales), n, rows, cols, _p(tiled), _stream(stream)), "moe_mxfp4_tile_scales")
    return tiled


def make_mxfp4_shape(rows: int, n: int, k: int, n_mats: int = 1, n_seg: int = 1, activation: int = MOE_ACT_NONE,
                     out_dtype: int = MOE_BF16) -> moe_mxfp4_shape:
    return moe_mxfp4_shape(rows, n, k, n_mats, n_seg, activation, out_dtype)


def moe_mxfp4_workspace_size(shape: moe_mxfp4_shape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_mxfp4_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "moe_mxfp4_workspace_size")
    return n.value


def moe_mxfp4_workspace_init(shape, ws, stream=None):
    _check(lib().moe_mxfp4_workspace_init(ctypes.byref(shape), _p(ws), _stream(stream)), "moe_mxfp4_workspace_init")


def moe_mxfp4_get_device_status(shape, ws, stream=None, clear: bool = False) -> int:
    st = ctypes.c_int32(0)
    _check(lib().moe_mxfp4_get_device_status(ctypes.byref(shape), _p(ws), _stream(stream), ctypes.byref(st),
                                             1 if clear else 0), "moe_mxfp4_get_device_status")
    return st.value


_MXFP4_TYPES: list = []


def moe_mxfp4_matmul(shape, a, a_scales, seg_offsets, seg_mat, w, w_scales, bias, y, y_scales, ws, stream=None):
    """y[r] = act(W_e a[r] + bias_e) over segments of rows, both operands in MXFP4 (shape: make_mxfp4_shape);
    seg_offsets and seg_mat int32, bias float32, y as the shape's out_dtype says."""
    import torch
    rows, n, k, n_mats, n_seg, dtype = shape.rows, shape.n, shape.k, shape.n_mats, shape.n_seg, shape.out_dtype
    ak, yn, wb = rows * k, rows * n, n_mats * n * k
    if not _MXFP4_TYPES:                                       # what an operand may be; uint8 and int8 are bytes
        raw = (torch.uint8, torch.int8)
        _MXFP4_TYPES.extend(((*raw, torch.float4_e2m1fn_x2), (*raw, torch.float8_e8m0fnu), (torch.int32, *raw),
                             (torch.float32, *raw), (torch.bfloat16, *raw)))
    codes, scales, i32, f32, bf16 = _MXFP4_TYPES
    out, bits = ((f32, 32) if dtype == MOE_F32 else (bf16, 16) if dtype == MOE_BF16 else
                 (codes, 4 if dtype == MOE_MXFP4 else 0))
    ptrs, devices = [], set()
    for name, t, types, nbytes in (
            ("a", a, codes, ak // 2), ("a_scales", a_scales, scales, ak // 32),
            ("seg_offsets", seg_offsets, i32, 4 * (n_seg + 1)), ("seg_mat", seg_mat, i32, 4 * n_seg),
            ("w", w, codes, wb // 2), ("w_scales", w_scales, scales, wb // 32), ("bias", bias, f32, 4 * n_mats * n),
            ("y", y, out, yn * bits // 8), ("y_scales", y_scales, scales, yn // 32),
            ("ws", ws, codes, 256)):
        if t is None:
            ptrs.append(None)
            continue
        if t.dtype not in types:
            raise ValueError(f"moe_mxfp4_matmul: {name} is {t.dtype}, not one of {types}")
        if t.nbytes < nbytes:
            raise ValueError(f"moe_mxfp4_matmul: {name} is smaller than its shape says")
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        devices.add(t.get_device())                            # -1: not on a GPU
        ptrs.append(t.data_ptr())
    if -1 in devices:
        raise ValueError("tensor must live on a CUDA device")
    if devices and devices != {torch._C._cuda_getDevice()}:
        raise ValueError("moe_mxfp4_matmul: every tensor must be on the current device")
    _check(lib().moe_mxfp4_matmul(ctypes.byref(shape), *ptrs, _stream(stream)), "moe_mxfp4_matmul")


_FEW_WEIGHTS = ("W_r", "logit_bias", "W1", "W1_scales", "b1", "W2", "W2_scales", "b2",
                "Ws1", "Ws1_scales", "bs1", "Ws2", "Ws2_scales", "bs2")


class MoELayer:
    """A layer shape plus device-resident weights and workspace.

    weights: dict with W_r, logit_bias (or None), W1, W1_scales, b1, W2,
    W2_scales, b2, Ws1, Ws1_scales, bs1, Ws2, Ws2_scales, bs2 (CUDA tensors or
    None where not used).  forward(x) runs moe_layer_forward on the current
    stream and returns (out, f, P, loss); forward_few(x) is the same layer
    through moe_layer_forward_few, for at most MOE_FEW_MAX_TOKENS tokens.  A
    layer of MXFP4 experts has forward_few only; its weights are codes and
    scales as moe_mxfp4_quantize writes them, the scales tiled here once.  A
    layer is of cfg.T tokens; layers of other T over the same experts take this
    one's w, tiled scales included, and keep no second copy.
    Building clears the workspace (and tiles scales) on the current stream:
    calls on other streams are ordered behind it by the caller, except that the
    first of forward_few waits by itself.
    """

    def __init__(self, cfg: moe_config, weights: dict, device="cuda"):
        import torch
        self.cfg = cfg
        self.w = weights
        self.device = torch.device(device)
        if cfg.dtype == MOE_MXFP4:
            self.w = dict(weights)
            for k in ("W1_scales", "W2_scales", "Ws1_scales", "Ws2_scales"):
                if weights.get(k) is not None and weights[k].dim() != 4:       # (4: another layer's w has them tiled)
                    self.w[k] = moe_mxfp4_tile_scales(weights[k])
            self.ws = self._few_workspace()
        else:
            self.ws = torch.empty(moe_workspace_size(cfg), dtype=torch.uint8, device=self.device)
            moe_workspace_init(cfg, self.ws)
        self._few_ws = None
        self._cfg_ref = ctypes.byref(cfg)
        out_dt = torch.float32 if cfg.dtype == MOE_F32 else torch.bfloat16
        self.out = torch.empty((cfg.T, cfg.d_model), dtype=out_dt, device=self.device)
        self.f = torch.empty(cfg.n_routed, dtype=torch.float32, device=self.device)
        self.P = torch.empty(cfg.n_routed, dtype=torch.float32, device=self.device)
        self.loss = torch.empty(1, dtype=torch.float32, device=self.device)
        self.topk_idx = torch.empty((cfg.T, cfg.top_k), dtype=torch.int32, device=self.device)
        self.gates = torch.empty((cfg.T, cfg.top_k), dtype=torch.float32, device=self.device)
        self.counts = torch.empty(cfg.n_routed, dtype=torch.int32, device=self.device)

    def forward(self, x, stream=None):
        w = self.w
        g = lambda k: w.get(k)  # noqa: E731
        moe_layer_forward(self.cfg, x, g("W_r"), g("logit_bias"), g("W1"), g("W1_scales"), g("b1"),
                          g("W2"), g("W2_scales"), g("b2"), g("Ws1"), g("Ws1_scales"), g("bs1"),
                          g("Ws2"), g("Ws2_scales"), g("bs2"), self.out, self.f, self.P, self.loss,
                          self.topk_idx, self.gates, self.counts, self.ws, stream)
        return self.out, self.f, self.P, self.loss

    def _few_workspace(self):
        """The few-token layer's workspace; refuses weights of other types, smaller than the layer's shape says, or on
        another device than the current one.  (A stack's matrices are compared in shape as well: bytes alone would
        let eight-bit weights pass for twice as many in four.)"""
        import torch
        c = self.cfg
        size = moe_few_workspace_size(c)                       # refuses what no weights would make a layer of
        f32 = torch.float32
        weight, bits = {MOE_BF16: (torch.bfloat16, 16), MOE_FP8_E4M3_BLOCK: (torch.float8_e4m3fn, 8),
                        MOE_MXFP4: (torch.float4_e2m1fn_x2, 4)}[c.dtype]
        up = lambda n: (n + 127) // 128  # noqa: E731
        need = {"W_r": (f32, (c.n_routed, 4 * c.d_model)), "logit_bias": (f32, (4 * c.n_routed,))}
        for p, e, ff in (("W", c.n_routed, c.d_ff), ("Ws", c.n_shared, c.d_ff_shared)):
            for i, rows, cols in ((1, ff, c.d_model), (2, c.d_model, ff)):
                need[f"{p}{i}"] = weight, (e, rows, cols * bits // 8)
                need[f"{p.replace('W', 'b')}{i}"] = f32, (e, 4 * rows)
                if c.dtype == MOE_FP8_E4M3_BLOCK:
                    need[f"{p}{i}_scales"] = f32, (e, up(rows), 4 * up(cols))
                elif c.dtype == MOE_MXFP4:                     # tiled
                    need[f"{p}{i}_scales"] = torch.uint8, (e, up(rows), up(cols), 512)
        for name, (dtype, shape) in need.items():              # shape: the last dimension in bytes
            t = self.w.get(name)
            if t is None:
                continue
            _typed(t, name, "forward_few", dtype)
            if t.nbytes < math.prod(shape):
                raise ValueError(f"forward_few: {name} is smaller than its shape says")
            if len(shape) > 2 and t.dim() == len(shape) and (*t.shape[1:-1], t.shape[-1] * t.element_size()) != shape[1:]:
                raise ValueError(f"forward_few: {name} has matrices of another shape, {tuple(t.shape[1:])}")
            _on_current_device(t, "forward_few")
        ws = torch.empty(size, dtype=torch.uint8, device=self.device)
        moe_few_workspace_init(c, ws)
        return ws

    def _first_few(self, stream):
        """The workspace of the first call of forward_few, cleared on the stream that the call runs on, which waits
        for the current one (where the layer may just have been built)."""
        import torch
        here = torch.cuda.current_stream()
        captured = torch.cuda.is_current_stream_capturing()
        with _current(stream):
            captured = captured or torch.cuda.is_current_stream_capturing()
            if self.cfg.dtype == MOE_MXFP4 and captured:
                return self.ws                                  # cleared when the layer was built
            if captured:
                raise RuntimeError("forward_few: its first call clears the workspace: make it before capturing")
            torch.cuda.current_stream().wait_stream(here)
            self._few_ws = self.ws if self.cfg.dtype == MOE_MXFP4 else self._few_workspace()
        return self._few_ws

    def forward_few(self, x, stream=None):
        """forward(x) in one kernel, for T <= MOE_FEW_MAX_TOKENS.  The first call allocates and clears the
        workspace (bf16 and FP8 layers) and orders its stream behind the current one: make it before capturing calls
        into a graph.  Calls share the workspace and the outputs: those on different streams are yours to order."""
        ws = self._few_ws
        if ws is None:
            ws = self._first_few(stream)
        w = self.w
        tensors = [w.get(k) for k in _FEW_WEIGHTS]
        tensors += (self.out, self.f, self.P, self.loss, self.topk_idx, self.gates, self.counts, ws)
        if x.dtype != self.out.dtype or x.numel() != self.out.numel():
            raise ValueError("forward_few: x must be bfloat16 (T, d_model)")
        _on_current_device(x, "forward_few")
        _check(lib().moe_layer_forward_few(self._cfg_ref, _p(x), *map(_p, tensors), _stream(stream)), "moe_layer_forward_few")
        return self.out, self.f, self.P, self.loss

    def _forward_into(self, x, out, loss, stream=None):
        w = self.w
        g = lambda k: w.get(k)  # noqa: E731
        moe_layer_forward(self.cfg, x, g("W_r"), g("logit_bias"), g("W1"), g("W1_scales"), g("b1"),
                          g("W2"), g("W2_scales"), g("b2"), g("Ws1"), g("Ws1_scales"), g("bs1"),
                          g("Ws2"), g("Ws2_scales"), g("bs2"), out, self.f, self.P, loss,
                          self.topk_idx, self.gates, self.counts, self.ws, stream)

    def forward_host_batches(self, x_hosts, out_hosts, loss_hosts, between=None):
        """Runs the layer on consecutive batches that live in pinned host
        memory and writes each batch's output and loss back to host memory.

        Batch k's host->device copy runs on a copy-in stream and its
        device->host copies on a copy-out stream, so they overlap the compute
        of batches k-1 and k+1 (device inputs and outputs are double-buffered;
        events order the three streams).  `between`, if given, is called on
        the compute stream before each batch.  Returns the (start, end) CUDA
        events that bracket the whole run: the first input copy to the last
        output copy.  f, P, topk_idx, gates and counts hold the last batch's."""
        import torch
        dev = self.device
        n = len(x_hosts)
        assert len(out_hosts) == n and len(loss_hosts) == n
        cur = torch.cuda.current_stream(dev)
        s_in = torch.cuda.Stream(device=dev)
        s_out = torch.cuda.Stream(device=dev)
        x_dev = [torch.empty_like(x_hosts[0], device=dev) for _ in range(2)]
        out_dev = [torch.empty_like(self.out) for _ in range(2)]
        loss_dev = [torch.empty_like(self.loss) for _ in range(2)]
        ev = lambda: torch.cuda.Event()  # noqa: E731
        in_ready = [ev(), ev()]
        computed = [ev(), ev()]
        copied_out = [ev(), ev()]
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        s_in.wait_stream(cur)
        s_out.wait_stream(cur)
        start.record(s_in)
        for k in range(n):
            b = k & 1
            with torch.cuda.stream(s_in):
                if k >= 2:
                    s_in.wait_event(computed[b])            # x_dev[b] no longer read
                x_dev[b].copy_(x_hosts[k], non_blocking=True)
                in_ready[b].record(s_in)
            cur.wait_event(in_ready[b])
            if k >= 2:
                cur.wait_event(copied_out[b])               # out_dev[b] already copied back
            if between is not None:
                between()
            self._forward_into(x_dev[b], out_dev[b], loss_dev[b], stream=cur)
            computed[b].record(cur)
            with torch.cuda.stream(s_out):
                s_out.wait_event(computed[b])
                out_hosts[k].copy_(out_dev[b], non_blocking=True)
                loss_hosts[k].copy_(loss_dev[b], non_blocking=True)
                copied_out[b].record(s_out)
        end.record(s_out)
        cur.wait_stream(s_out)
        return start, end

    def device_status(self, clear: bool = False, stream=None) -> int:
        """The status bits of the layer's calls so far, forward_few's included, after synchronising `stream` (the
        current one by default)."""
        status = moe_get_device_status(self.cfg, self.ws, stream, clear)
        if self._few_ws is not None and self._few_ws is not self.ws:
            status |= moe_get_device_status(self.cfg, self._few_ws, stream, clear)
        return status
