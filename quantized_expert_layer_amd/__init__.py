"""Python binding of libmoe_wq.so, the MI355X (gfx950) weight-only-quantized MoE expert layer.

Argument marshalling only: every step of the layer runs in the library's HIP kernels.
PyTorch supplies device memory (tensors) and the stream; nothing here computes.  The
functions carry the names of the C entry points declared in include/moe_wq.h.

The library is loaded on first use and a missing or unloadable library raises
`MoELibraryError`: there is no fallback implementation.
"""
import contextlib
import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import numpy as np

__all__ = [
    "MOE_OK", "MOE_ERR_INVALID", "MOE_ERR_UNSUPPORTED", "MOE_ERR_WORKSPACE",
    "MOE_ERR_NO_DEVICE", "MOE_ERR_HIP",
    "GATE_TOPK", "GATE_ALL", "W_INT4", "W_INT8", "W_FP16", "ACT_NONE", "ACT_RELU",
    "ACT_SWIGLU", "PATH_AUTO", "PATH_STREAM", "PATH_TILE", "TILE_AUTO", "TILE_64x256",
    "TILE_64x128", "TILE_128x128", "TILE_48x256", "TILE_48x128", "I2F_TRICK", "I2F_NATIVE",
    "MOE_MAX_EXPERTS", "MOE_MAX_TOPK", "MOE_MAX_SPLIT_K",
    "MoEError", "MoELibraryError", "lib", "lib_path", "status_str", "version",
    "moe_route_topk", "moe_route_topk_active", "moe_permute", "moe_grouped_gemm_wq",
    "moe_grouped_gemm_wq_rows",
    "moe_unpermute_combine",
    "moe_dequant", "moe_pack_wq", "moe_packed_bytes", "moe_gemm_workspace_size",
    "moe_permute_workspace_size", "GemmOpts", "EXPORTED_SYMBOLS", "new_output",
    "moe_probe_read", "moe_probe_mfma", "moe_decode_layer", "moe_decode_workspace_size",
    "moe_decode_layer_noalloc", "MOE_DECODE_SCRATCH_BYTES", "moe_decode_layer_shared",
    "moe_decode_shared_workspace_size",
    "MOE_DECODE_MAX_TOKENS", "MOE_DECODE_MAX_ROWS", "moe_elb_accumulate", "moe_elb_top_m",
    "moe_bf16_recombine", "ACT_SILU", "ACT_GELU", "DT_FP16", "DT_BF16", "DT_FP32",
    "moe_linear", "moe_linear_workspace_size", "moe_linear_backward",
    "moe_linear_backward_workspace_size", "moe_balance_loss", "moe_balance_workspace_size",
    "moe_route_backward", "moe_combine_backward",
]

MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE = 0, -1, -2, -3
MOE_ERR_NO_DEVICE, MOE_ERR_HIP = -4, -5
GATE_TOPK, GATE_ALL = 0, 1
W_INT4, W_INT8, W_FP16 = 0, 1, 2
ACT_NONE, ACT_RELU, ACT_SWIGLU, ACT_SILU, ACT_GELU = 0, 1, 2, 3, 4
DT_FP16, DT_BF16, DT_FP32 = 0, 1, 2
PATH_AUTO, PATH_STREAM, PATH_TILE = 0, 1, 2
TILE_AUTO, TILE_64x256, TILE_64x128, TILE_128x128, TILE_48x256, TILE_48x128 = 0, 1, 2, 3, 4, 5
I2F_TRICK, I2F_NATIVE = 0, 1
I2FS = {"trick": I2F_TRICK, "native": I2F_NATIVE}
MOE_MAX_EXPERTS, MOE_MAX_TOPK, MOE_MAX_SPLIT_K = 256, 8, 8
MOE_DECODE_MAX_TOKENS, MOE_DECODE_MAX_ROWS = 64, 512
MOE_DECODE_SCRATCH_BYTES = 8 << 20

WTYPES = {"int4": W_INT4, "int8": W_INT8, "fp16": W_FP16}
ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "swiglu": ACT_SWIGLU}
LINEAR_ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU}
GATES = {"topk": GATE_TOPK, "all": GATE_ALL}

lib_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_wq.so")

# Every symbol include/moe_wq.h declares.
EXPORTED_SYMBOLS = (
    "moe_route_topk", "moe_permute", "moe_permute_workspace_size", "moe_grouped_gemm_wq",
    "moe_grouped_gemm_wq_rows", "moe_gemm_workspace_size", "moe_unpermute_combine", "moe_dequant", "moe_packed_bytes",
    "moe_pack_wq", "moe_status_str", "moe_version", "moe_probe_read", "moe_probe_mfma",
    "moe_decode_layer", "moe_decode_workspace_size", "moe_route_topk_active",
    "moe_decode_layer_noalloc", "moe_decode_layer_shared", "moe_decode_shared_workspace_size",
    "moe_elb_accumulate", "moe_elb_top_m", "moe_bf16_recombine",
    "moe_linear", "moe_linear_workspace_size", "moe_linear_backward",
    "moe_linear_backward_workspace_size", "moe_balance_loss", "moe_balance_workspace_size",
    "moe_route_backward", "moe_combine_backward",
)


class MoEError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {status_str(status)} ({status})")


class MoELibraryError(ImportError):
    pass


class GemmOpts(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("split_k", ctypes.c_int32),
                ("tile", ctypes.c_int32), ("i2f", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 4)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int32
_SZ = ctypes.c_size_t
_L = ctypes.c_int64
_F = ctypes.c_float


def lib():
    """The loaded library (loaded once; raises MoELibraryError when unavailable)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(lib_path):
        raise MoELibraryError(f"{lib_path} is missing: build it with "
                              "`python -m quantized_expert_layer_amd.build`")
    # torch ships its own HIP runtime under the same soname.  Load it first so that the
    # library binds to that copy: two HIP runtimes in one process do not share devices,
    # and the library would then find no usable device for torch's tensors.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    try:
        L = ctypes.CDLL(lib_path)
    except OSError as e:
        raise MoELibraryError(f"cannot load {lib_path}: {e}") from e
    sig = {
        "moe_route_topk": (_I, [_P, _I, _I, _I, _I, _P, _P, _P]),
        "moe_permute": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
        "moe_permute_workspace_size": (_SZ, [_I, _I, _I]),
        "moe_grouped_gemm_wq": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _I, _I, _I, _P, _P, _P,
                                     _P, _SZ, _P]),
        "moe_grouped_gemm_wq_rows": (_I, [_P, _I, _P, _I, _P, _I, _I, _I, _I, _P, _P, _I, _I,
                                          _I, _P, _P, _I, _P, _P, _P, _SZ, _P]),
        "moe_gemm_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _P]),
        "moe_unpermute_combine": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P]),
        "moe_dequant": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P]),
        "moe_packed_bytes": (_SZ, [_I, _I, _I, _I]),
        "moe_pack_wq": (_I, [_P, _I, _I, _I, _I, _P]),
        "moe_status_str": (ctypes.c_char_p, [_I]),
        "moe_version": (_I, []),
        "moe_probe_read": (_I, [_P, _SZ, _P, _I, _P]),
        "moe_probe_mfma": (_I, [_I, _P, _I, _P]),
        "moe_decode_layer": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _I,
                                  _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
        "moe_decode_layer_noalloc": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                                          _I, _I, _P, _P, _P, _P, _P, _P]),
        "moe_route_topk_active": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P]),
        "moe_elb_accumulate": (_I, [_P, _I, _I, _I, _I, _P, _P]),
        "moe_elb_top_m": (_I, [_P, _I, _I, _I, _P, _P, _P]),
        "moe_bf16_recombine": (_I, [_P, _P, _SZ, _P, _P]),
        "moe_decode_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
        "moe_decode_layer_shared": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                                         _I, _I, _P, _P, _I, _P, _P, _P, _P, _SZ, _P]),
        "moe_decode_shared_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
        "moe_linear": (_I, [_P, _L, _P, _L, _P, _P, _L, _I, _I, _I, _I, _I, _P, _L, _I, _P, _L, _P,
                            _SZ, _P]),
        "moe_linear_workspace_size": (_SZ, [_I, _I, _I, _L, _L]),
        "moe_linear_backward": (_I, [_P, _L, _I, _P, _L, _P, _L, _P, _L, _I, _I, _I, _I, _I, _P,
                                     _P, _P, _P, _SZ, _P]),
        "moe_linear_backward_workspace_size": (_SZ, [_I, _I, _I, _L, _L, _L, _I, _I]),
        "moe_balance_loss": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P, _SZ,
                                  _P]),
        "moe_balance_workspace_size": (_SZ, [_I, _I, _I]),
        "moe_route_backward": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _F, _P,
                                    _P, _P]),
        "moe_combine_backward": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def status_str(status: int) -> str:
    return lib().moe_status_str(int(status)).decode()


def version() -> int:
    return lib().moe_version()


def _check(fn, status):
    if status != MOE_OK:
        raise MoEError(fn, status)


# ---------------------------------------------------------------- tensor marshalling
# MOE_WQ_POISON=1: outputs (and layer workspaces) the binding allocates start as NaN (floating
# point) or 0 (integer) instead of whatever the allocator hands back, so an element a kernel
# failed to write cannot pass a test by holding a previous call's correct value.
_POISON = os.environ.get("MOE_WQ_POISON", "") not in ("", "0")


def new_output(shape, dtype, device):
    """torch.empty, pre-filled with the poison pattern when MOE_WQ_POISON is set."""
    torch = _torch()
    t = torch.empty(shape, dtype=dtype, device=device)
    if _POISON:
        t.fill_(float("nan") if t.is_floating_point() else 0)
    return t


def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t, dtype, name, numel=None):
    torch = _torch()
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name}: expected a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name}: needs at least {numel} elements, has {t.numel()}")


def _opts(path=PATH_AUTO, split_k=0, tile=TILE_AUTO, i2f=I2F_TRICK):
    if path == PATH_AUTO and split_k == 0 and tile == TILE_AUTO and i2f == I2F_TRICK:
        return None
    o = GemmOpts()
    o.path, o.split_k, o.tile, o.i2f = int(path), int(split_k), int(tile), int(i2f)
    return o


# ---------------------------------------------------------------- the five calls
def moe_route_topk(logits, k, gate_mode, topk_ids=None, topk_w=None, stream=None, active=None):
    """active (uint8 [T] device tensor or None): batch pruning, moe_route_topk_active."""
    torch = _torch()
    T, E = logits.shape
    gm = GATES.get(gate_mode, gate_mode)
    if topk_ids is None:
        topk_ids = new_output((T, k), torch.int32, logits.device)
    if topk_w is None:
        topk_w = new_output((T, k), torch.float32, logits.device)
    _need(logits, torch.float32, "logits")
    _need(topk_ids, torch.int32, "topk_ids", T * k)
    _need(topk_w, torch.float32, "topk_w", T * k)
    if active is None:
        _check("moe_route_topk", lib().moe_route_topk(_ptr(logits), T, E, k, gm, _ptr(topk_ids),
                                                      _ptr(topk_w), _stream(stream)))
    else:
        _need(active, torch.uint8, "active", T)
        _check("moe_route_topk_active", lib().moe_route_topk_active(
            _ptr(logits), _ptr(active), T, E, k, gm, _ptr(topk_ids), _ptr(topk_w),
            _stream(stream)))
    return topk_ids, topk_w


def moe_permute(topk_ids, topk_w, x, E, want_w_perm=True, out=None, stream=None,
                want_x_perm=True, ws=None):
    """Returns (perm, inv_perm, expert_offsets, x_perm or None, w_perm or None).
    want_x_perm=False skips the row copy (the first GEMM then reads x through perm).
    ws: uint8 device workspace of moe_permute_workspace_size bytes (allocated if None)."""
    torch = _torch()
    T, k = topk_ids.shape
    d = x.shape[1]
    R = T * k
    dev = x.device
    if out is None:
        out = (new_output(R, torch.int32, dev),
               new_output(R, torch.int32, dev),
               new_output(E + 1, torch.int32, dev),
               new_output((R, d), torch.float16, dev) if want_x_perm else None,
               new_output(R, torch.float32, dev)
               if (want_w_perm and topk_w is not None) else None)
    perm, inv_perm, offsets, x_perm, w_perm = out
    _need(topk_ids, torch.int32, "topk_ids")
    _need(topk_w, torch.float32, "topk_w")
    _need(x, torch.float16, "x")
    _need(perm, torch.int32, "perm", R)
    _need(inv_perm, torch.int32, "inv_perm", R)
    _need(offsets, torch.int32, "expert_offsets", E + 1)
    _need(x_perm, torch.float16, "x_perm", R * d)
    _need(w_perm, torch.float32, "w_perm", R)
    need = lib().moe_permute_workspace_size(T, k, E)
    if need and ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _need(ws, torch.uint8, "ws")
    _check("moe_permute", lib().moe_permute(
        _ptr(topk_ids), _ptr(topk_w), _ptr(x), T, k, E, d, _ptr(perm), _ptr(inv_perm),
        _ptr(offsets), _ptr(x_perm), _ptr(w_perm), _ptr(ws), 0 if ws is None else ws.numel(),
        _stream(stream)))
    return perm, inv_perm, offsets, x_perm, w_perm


def moe_gemm_workspace_size(R, E, K, N, wtype, act, path=PATH_AUTO, split_k=0):
    o = _opts(path, split_k)
    return lib().moe_gemm_workspace_size(R, E, K, N, WTYPES.get(wtype, wtype),
                                         ACTS.get(act, act), ctypes.byref(o) if o else None)


def moe_permute_workspace_size(T, k, E):
    return lib().moe_permute_workspace_size(T, k, E)


def moe_grouped_gemm_wq(a, expert_offsets, E, K, N, w_packed, scales, wtype, group_size, act,
                        row_scale=None, out=None, path=PATH_AUTO, split_k=0, ws=None,
                        stream=None, tile=TILE_AUTO, i2f=I2F_TRICK):
    torch = _torch()
    R = a.shape[0]
    wt = WTYPES.get(wtype, wtype)
    ac = ACTS.get(act, act)
    n_out = N // 2 if ac == ACT_SWIGLU else N
    if out is None:
        out = new_output((R, n_out), torch.float16, a.device)
    o = _opts(path, split_k, tile, I2FS.get(i2f, i2f))
    need_ws = lib().moe_gemm_workspace_size(R, E, K, N, wt, ac, ctypes.byref(o) if o else None)
    if need_ws and ws is None:
        ws = torch.empty(need_ws, dtype=torch.uint8, device=a.device)
    _need(a, torch.float16, "a", R * K)
    _need(expert_offsets, torch.int32, "expert_offsets", E + 1)
    _need(w_packed, torch.uint8, "w_packed")
    _need(scales, torch.float16, "scales")
    _need(row_scale, torch.float32, "row_scale", R)
    _need(out, torch.float16, "out", R * n_out)
    _need(ws, torch.uint8, "ws")
    _check("moe_grouped_gemm_wq", lib().moe_grouped_gemm_wq(
        _ptr(a), _ptr(expert_offsets), R, E, K, N, _ptr(w_packed), _ptr(scales), wt,
        int(group_size), ac, _ptr(row_scale), _ptr(out), ctypes.byref(o) if o else None,
        _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return out


def moe_grouped_gemm_wq_rows(a, a_rows, a_row_div, expert_offsets, R, E, K, N, w_packed, scales,
                             wtype, group_size, act, row_scale=None, out=None, out_rows=None,
                             path=PATH_AUTO, split_k=0, stream=None, tile=TILE_AUTO,
                             i2f=I2F_TRICK):
    """GEMM row p reads a[a_rows[p] // a_row_div] (a[p] if a_rows is None) and writes
    out[out_rows[p]] (out[p] if out_rows is None); R = number of GEMM rows."""
    torch = _torch()
    wt = WTYPES.get(wtype, wtype)
    ac = ACTS.get(act, act)
    n_out = N // 2 if ac == ACT_SWIGLU else N
    if out is None:
        out = new_output((R, n_out), torch.float16, a.device)
    o = _opts(path, split_k, tile, I2FS.get(i2f, i2f))
    a_nrows = a.shape[0]
    out_nrows = out.shape[0]
    _need(a, torch.float16, "a", a_nrows * K)
    _need(a_rows, torch.int32, "a_rows", R)
    _need(expert_offsets, torch.int32, "expert_offsets", E + 1)
    _need(w_packed, torch.uint8, "w_packed")
    _need(scales, torch.float16, "scales")
    _need(row_scale, torch.float32, "row_scale", R)
    _need(out, torch.float16, "out", out_nrows * n_out)
    _need(out_rows, torch.int32, "out_rows", R)
    _check("moe_grouped_gemm_wq_rows", lib().moe_grouped_gemm_wq_rows(
        _ptr(a), a_nrows, _ptr(a_rows), int(a_row_div), _ptr(expert_offsets), R, E, K, N,
        _ptr(w_packed), _ptr(scales), wt, int(group_size), ac, _ptr(row_scale), _ptr(out),
        out_nrows, _ptr(out_rows), ctypes.byref(o) if o else None, None, 0, _stream(stream)))
    return out


def moe_probe_read(src, blocks, sink=None, stream=None):
    """Attainable-read probe: reads all of `src` (a device tensor, bytes % 16 == 0) once;
    returns the per-block XOR sink (uint32 as int32 [blocks])."""
    torch = _torch()
    if sink is None:
        sink = torch.empty(blocks, dtype=torch.int32, device=src.device)
    _need(sink, torch.int32, "sink", blocks)
    if not src.is_contiguous():
        raise ValueError("src must be contiguous")
    _check("moe_probe_read", lib().moe_probe_read(_ptr(src), src.numel() * src.element_size(),
                                                  _ptr(sink), int(blocks), _stream(stream)))
    return sink


def moe_probe_mfma(iters, blocks, out=None, device="cuda", stream=None):
    """Attainable-MFMA probe: blocks x 4 waves x iters x 16 MFMA 16x16x32 fp16; returns the
    fp32 [blocks * 256] result (every element 512 * iters)."""
    torch = _torch()
    if out is None:
        out = torch.empty(blocks * 256, dtype=torch.float32, device=device)
    _need(out, torch.float32, "out", blocks * 256)
    _check("moe_probe_mfma", lib().moe_probe_mfma(int(iters), _ptr(out), int(blocks),
                                                  _stream(stream)))
    return out


def moe_decode_workspace_size(T, k, E, d, inter, wtype):
    return lib().moe_decode_workspace_size(T, k, E, d, inter, WTYPES.get(wtype, wtype))


def moe_decode_layer(logits, x, k, gate_mode, inter, act, w1, s1, w2, s2, wtype, group_size,
                     addend=None, topk_ids=None, topk_w=None, out=None, ws=None, stream=None,
                     active=None, addend_ready=None):
    """The routed layer for a decode / verify step (T <= MOE_DECODE_MAX_TOKENS tokens).
    Returns (out fp16 [T, d], topk_ids int32 [T, k], topk_w fp32 [T, k]).  addend_ready: a
    recorded torch.cuda.Event the call waits for before it first reads addend."""
    torch = _torch()
    T, E = logits.shape
    d = x.shape[1]
    wt = WTYPES.get(wtype, wtype)
    dev = x.device
    if out is None:
        out = new_output((T, d), torch.float16, dev)
    if topk_ids is None:
        topk_ids = new_output((T, k), torch.int32, dev)
    if topk_w is None:
        topk_w = new_output((T, k), torch.float32, dev)
    if ws is None:
        need = lib().moe_decode_workspace_size(T, k, E, d, inter, wt)
        ws = new_output(max(need, 16), torch.uint8, dev)
    _need(logits, torch.float32, "logits", T * E)
    _need(x, torch.float16, "x", T * d)
    _need(w1, torch.uint8, "w1")
    _need(s1, torch.float16, "s1")
    _need(w2, torch.uint8, "w2")
    _need(s2, torch.float16, "s2")
    _need(addend, torch.float16, "addend", T * d)
    _need(topk_ids, torch.int32, "topk_ids", T * k)
    _need(topk_w, torch.float32, "topk_w", T * k)
    _need(out, torch.float16, "out", T * d)
    _need(ws, torch.uint8, "ws")
    _need(active, torch.uint8, "active", T)
    _check("moe_decode_layer", lib().moe_decode_layer(
        _ptr(logits), _ptr(active), _ptr(x), T, E, k, GATES.get(gate_mode, gate_mode), d, int(inter),
        ACTS.get(act, act), _ptr(w1), _ptr(s1), _ptr(w2), _ptr(s2), wt, int(group_size),
        _ptr(addend), None if addend_ready is None else addend_ready.cuda_event,
        _ptr(topk_ids), _ptr(topk_w), _ptr(out), _ptr(ws),
        0 if ws is None else ws.numel(), _stream(stream)))
    return out, topk_ids, topk_w


def moe_decode_shared_workspace_size(T, k, E, d, inter, wtype, shared_inter):
    return lib().moe_decode_shared_workspace_size(T, k, E, d, inter, WTYPES.get(wtype, wtype),
                                                  shared_inter)


def moe_decode_layer_shared(logits, x, k, gate_mode, inter, act, w1, s1, w2, s2, wtype,
                            group_size, shared_w1, shared_w2, shared_inter, topk_ids=None,
                            topk_w=None, out=None, ws=None, stream=None, active=None):
    """moe_decode_layer with the shared experts (fp16, SwiGLU, packed for E = 1) computed in
    the same launches.  Returns (out fp16 [T, d], topk_ids int32 [T, k], topk_w fp32 [T, k])."""
    torch = _torch()
    T, E = logits.shape
    d = x.shape[1]
    wt = WTYPES.get(wtype, wtype)
    dev = x.device
    if out is None:
        out = new_output((T, d), torch.float16, dev)
    if topk_ids is None:
        topk_ids = new_output((T, k), torch.int32, dev)
    if topk_w is None:
        topk_w = new_output((T, k), torch.float32, dev)
    if ws is None:
        need = lib().moe_decode_shared_workspace_size(T, k, E, d, inter, wt, int(shared_inter))
        ws = new_output(max(need, 16), torch.uint8, dev)
    _need(logits, torch.float32, "logits", T * E)
    _need(x, torch.float16, "x", T * d)
    _need(w1, torch.uint8, "w1")
    _need(s1, torch.float16, "s1")
    _need(w2, torch.uint8, "w2")
    _need(s2, torch.float16, "s2")
    _need(shared_w1, torch.uint8, "shared_w1")
    _need(shared_w2, torch.uint8, "shared_w2")
    _need(topk_ids, torch.int32, "topk_ids", T * k)
    _need(topk_w, torch.float32, "topk_w", T * k)
    _need(out, torch.float16, "out", T * d)
    _need(ws, torch.uint8, "ws")
    _need(active, torch.uint8, "active", T)
    _check("moe_decode_layer_shared", lib().moe_decode_layer_shared(
        _ptr(logits), _ptr(active), _ptr(x), T, E, k, GATES.get(gate_mode, gate_mode), d,
        int(inter), ACTS.get(act, act), _ptr(w1), _ptr(s1), _ptr(w2), _ptr(s2), wt,
        int(group_size), _ptr(shared_w1), _ptr(shared_w2), int(shared_inter), _ptr(topk_ids),
        _ptr(topk_w), _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return out, topk_ids, topk_w


def moe_decode_layer_noalloc(logits, x, k, gate_mode, inter, act, w1, s1, w2, s2, wtype,
                             group_size, addend=None, topk_ids=None, topk_w=None, out=None,
                             stream=None, active=None, addend_ready=None):
    """moe_decode_layer on the library's own scratch array (no workspace argument; calls that
    overlap on one device race).  Returns (out, topk_ids, topk_w)."""
    torch = _torch()
    T, E = logits.shape
    d = x.shape[1]
    wt = WTYPES.get(wtype, wtype)
    dev = x.device
    if out is None:
        out = new_output((T, d), torch.float16, dev)
    if topk_ids is None:
        topk_ids = new_output((T, k), torch.int32, dev)
    if topk_w is None:
        topk_w = new_output((T, k), torch.float32, dev)
    _need(logits, torch.float32, "logits", T * E)
    _need(x, torch.float16, "x", T * d)
    _need(w1, torch.uint8, "w1")
    _need(s1, torch.float16, "s1")
    _need(w2, torch.uint8, "w2")
    _need(s2, torch.float16, "s2")
    _need(addend, torch.float16, "addend", T * d)
    _need(topk_ids, torch.int32, "topk_ids", T * k)
    _need(topk_w, torch.float32, "topk_w", T * k)
    _need(out, torch.float16, "out", T * d)
    _need(active, torch.uint8, "active", T)
    _check("moe_decode_layer_noalloc", lib().moe_decode_layer_noalloc(
        _ptr(logits), _ptr(active), _ptr(x), T, E, k, GATES.get(gate_mode, gate_mode), d,
        int(inter), ACTS.get(act, act), _ptr(w1), _ptr(s1), _ptr(w2), _ptr(s2), wt,
        int(group_size), _ptr(addend), None if addend_ready is None else addend_ready.cuda_event,
        _ptr(topk_ids), _ptr(topk_w), _ptr(out), _stream(stream)))
    return out, topk_ids, topk_w


def moe_elb_accumulate(ids, E, counts, stream=None):
    """One draft step: ids int32 [L, T, k] (device), counts int32 [L, E] updated in place."""
    torch = _torch()
    L, T, k = ids.shape
    _need(ids, torch.int32, "ids")
    _need(counts, torch.int32, "counts", L * E)
    _check("moe_elb_accumulate", lib().moe_elb_accumulate(_ptr(ids), L, T, k, E, _ptr(counts),
                                                          _stream(stream)))
    return counts


def moe_elb_top_m(counts, M, experts=None, top_counts=None, stream=None):
    """Per layer the M most-counted experts: returns (experts int32 [L, M], counts [L, M])."""
    torch = _torch()
    L, E = counts.shape
    if experts is None:
        experts = new_output((L, M), torch.int32, counts.device)
    if top_counts is None:
        top_counts = new_output((L, M), torch.int32, counts.device)
    _need(counts, torch.int32, "counts", L * E)
    _need(experts, torch.int32, "experts", L * M)
    _need(top_counts, torch.int32, "top_counts", L * M)
    _check("moe_elb_top_m", lib().moe_elb_top_m(_ptr(counts), L, E, int(M), _ptr(experts),
                                                _ptr(top_counts), _stream(stream)))
    return experts, top_counts


def moe_bf16_recombine(exponents, sign_mantissa, out=None, stream=None):
    """BF16 tensor [n] from uint8 exponent bytes [n] and sign-mantissa bytes [n] (device)."""
    torch = _torch()
    n = exponents.numel()
    if out is None:
        out = new_output(n, torch.bfloat16, exponents.device)
    _need(exponents, torch.uint8, "exponents", n)
    _need(sign_mantissa, torch.uint8, "sign_mantissa", n)
    _need(out, torch.bfloat16, "out", n)
    _check("moe_bf16_recombine", lib().moe_bf16_recombine(_ptr(exponents), _ptr(sign_mantissa),
                                                          n, _ptr(out), _stream(stream)))
    return out


def moe_unpermute_combine(y_perm, inv_perm, topk_w, addend, T, k, out=None, stream=None):
    torch = _torch()
    d = y_perm.shape[1]
    if out is None:
        out = new_output((T, d), torch.float16, y_perm.device)
    _need(y_perm, torch.float16, "y_perm")
    _need(inv_perm, torch.int32, "inv_perm", T * k)
    _need(topk_w, torch.float32, "topk_w", T * k)
    _need(addend, torch.float16, "addend", T * d)
    _need(out, torch.float16, "out", T * d)
    _check("moe_unpermute_combine", lib().moe_unpermute_combine(
        _ptr(y_perm), _ptr(inv_perm), _ptr(topk_w), _ptr(addend), T, k, d, _ptr(out),
        _stream(stream)))
    return out


def moe_dequant(w_packed, scales, wtype, group_size, E, K, N, out=None, stream=None):
    torch = _torch()
    if out is None:
        out = new_output((E, K, N), torch.float16, w_packed.device)
    _need(w_packed, torch.uint8, "w_packed")
    _need(scales, torch.float16, "scales")
    _need(out, torch.float16, "w_out", E * K * N)
    _check("moe_dequant", lib().moe_dequant(_ptr(w_packed), _ptr(scales), WTYPES.get(wtype, wtype),
                                            int(group_size), E, K, N, _ptr(out), _stream(stream)))
    return out


# ---------------------------------------------------------------- dense products, router gradients
_HERE = contextlib.nullcontext()


def _place(ref, stream):
    """The context in which a call on ref's device is made and its outputs and workspace are
    allocated: that device current, and `stream` (default: the device's current one) its current
    stream, so that the allocator orders the memory by the stream that uses it."""
    torch = _torch()
    dev = ref.device
    if not ref.is_cuda:
        raise TypeError("expected device tensors")
    if stream is None:
        return _HERE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    elif stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream)


def _here(dev):
    """Handle of dev's current stream (asked for without building a Stream object: that costs as
    much host time as the call itself)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream(dev).cuda_stream if raw is None else raw(dev.index)


def _sizes(*sizes):
    """Refuses what the C entry points' 32-bit sizes would cut off."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"sizes must be below 2^31, got {sizes}")


def _refuse(t, dtype, name, shape, dev):
    """Raises for the first thing that is wrong with t's type, device or shape."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name}: expected a tensor on {dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _dense(t, dtype, name, shape, dev):
    """Address of a dense device tensor of exactly this type, shape and device (None: None)."""
    if t is None:
        return None
    if not (getattr(t, "dtype", None) is dtype and t.shape == shape and t.device == dev):
        _refuse(t, dtype, name, shape, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _out(t, dtype, name, shape, dev):
    """(t, its address) of a dense output, allocated if None."""
    if t is None:
        t = new_output(shape, dtype, dev)
        return t, t.data_ptr()
    return t, _dense(t, dtype, name, shape, dev)


def _rows(t, dtype, name, shape, dev):
    """(address, row stride) of a device matrix of this type and shape whose rows are contiguous
    ((None, 0): None)."""
    if t is None:
        return None, 0
    if not (getattr(t, "dtype", None) is dtype and t.shape == shape and t.device == dev):
        _refuse(t, dtype, name, shape, dev)
    rows, cols = shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    if rows <= 1 or cols == 0:
        return t.data_ptr(), cols
    if ld < cols:
        raise ValueError(f"{name}: rows must not overlap")
    return t.data_ptr(), ld


def _dt(dtype, name):
    torch = _torch()
    if dtype == torch.float16:
        return DT_FP16
    if dtype == torch.bfloat16:
        return DT_BF16
    raise TypeError(f"{name}: expected torch.float16 or torch.bfloat16, got {dtype}")


def _linear_act(act):
    if act in LINEAR_ACTS:
        return LINEAR_ACTS[act]
    if act in LINEAR_ACTS.values():
        return act
    raise ValueError(f"act: expected one of {sorted(LINEAR_ACTS)}, got {act!r}")


def _workspace(need, ws, dev):
    """(ws, its address, its bytes), allocated if None."""
    if ws is None:
        if not need:
            return None, None, 0
        ws = _torch().empty(need, dtype=_torch().uint8, device=dev)
        return ws, ws.data_ptr(), need
    return ws, _dense(ws, _torch().uint8, "ws", (ws.numel(),), dev), ws.numel()


def moe_linear_workspace_size(M, N, K, lda=None, ldw=None):
    """Workspace bytes of moe_linear; row strides default to dense rows."""
    return lib().moe_linear_workspace_size(M, N, K, K if lda is None else lda,
                                           K if ldw is None else ldw)


def moe_linear(a, w, bias=None, act="none", residual=None, out=None, out_dtype=None, preact=None,
               ws=None, stream=None):
    """act(a @ w.T + bias) + residual for fp16 or bf16 a [M, K] and w [N, K] (rows may be strided).
    act: "none" | "relu" | "silu" | "gelu".  out_dtype: a's type (default) or torch.float32.
    preact ([M, N] of a's type): receives the activation's argument for moe_linear_backward.
    out may be `residual` itself."""
    torch = _torch()
    if a.dim() != 2 or w.dim() != 2:
        raise ValueError("a and w must have two dimensions")
    M, K = a.shape
    N = w.shape[0]
    _sizes(M, N, K)
    dev, dtype = a.device, a.dtype
    dt = _dt(dtype, "a")
    with _place(a, stream):
        if out is None:
            out = new_output((M, N), out_dtype or dtype, dev)
            po, ldo = out.data_ptr(), N
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
        else:
            po, ldo = _rows(out, out.dtype, "out", (M, N), dev)
        od = DT_FP32 if out.dtype == torch.float32 else _dt(out.dtype, "out")
        pa, lda = _rows(a, dtype, "a", (M, K), dev)
        pw, ldw = _rows(w, dtype, "w", (N, K), dev)
        pr, ldr = _rows(residual, dtype, "residual", (M, N), dev)
        pp, ldp = _rows(preact, dtype, "preact", (M, N), dev)
        pb = _dense(bias, dtype, "bias", (N,), dev)
        ac = _linear_act(act)
        L = lib()
        ws, pws, nws = _workspace(L.moe_linear_workspace_size(M, N, K, lda, ldw), ws, dev)
        _check("moe_linear", L.moe_linear(pa, lda, pw, ldw, pb, pr, ldr, M, N, K, dt, ac, po, ldo,
                                          od, pp, ldp, pws, nws, _here(dev)))
    return out


def moe_linear_backward_workspace_size(M, N, K, lda=None, ldw=None, ldg=None, grad_f32=False,
                                       act="none"):
    """Workspace bytes of moe_linear_backward; row strides default to dense rows."""
    return lib().moe_linear_backward_workspace_size(
        M, N, K, K if lda is None else lda, K if ldw is None else ldw, N if ldg is None else ldg,
        DT_FP32 if grad_f32 else DT_FP16, _linear_act(act))


def moe_linear_backward(grad_out, a, w, act="none", preact=None, need_a=True, need_w=True,
                        need_bias=True, grad_a=None, grad_w=None, grad_bias=None, ws=None,
                        stream=None):
    """Gradients (grad_a [M, K], grad_w [N, K], grad_bias [N], of a's type; None where not needed)
    of moe_linear.  grad_out [M, N] of a's type or float32; preact: what moe_linear stored."""
    torch = _torch()
    if a.dim() != 2 or w.dim() != 2:
        raise ValueError("a and w must have two dimensions")
    M, K = a.shape
    N = w.shape[0]
    _sizes(M, N, K)
    dev, dtype = a.device, a.dtype
    dt = _dt(dtype, "a")
    ac = _linear_act(act)
    with _place(a, stream):
        pga = pgw = pgb = None
        if grad_a is not None or need_a:
            grad_a, pga = _out(grad_a, dtype, "grad_a", (M, K), dev)
        if grad_w is not None or need_w:
            grad_w, pgw = _out(grad_w, dtype, "grad_w", (N, K), dev)
        if grad_bias is not None or need_bias:
            grad_bias, pgb = _out(grad_bias, dtype, "grad_bias", (N,), dev)
        gd = grad_out.dtype
        gdt = DT_FP32 if gd == torch.float32 else _dt(gd, "grad_out")
        pg, ldg = _rows(grad_out, gd, "grad_out", (M, N), dev)
        pa, lda = _rows(a, dtype, "a", (M, K), dev)
        pw, ldw = _rows(w, dtype, "w", (N, K), dev)
        pp, ldp = _rows(preact, dtype, "preact", (M, N), dev)
        L = lib()
        need = L.moe_linear_backward_workspace_size(M, N, K, lda, ldw, ldg, gdt, ac)
        ws, pws, nws = _workspace(need, ws, dev)
        _check("moe_linear_backward", L.moe_linear_backward(
            pg, ldg, gdt, pp, ldp, pa, lda, pw, ldw, M, N, K, dt, ac, pga, pgw, pgb, pws, nws,
            _here(dev)))
    return grad_a, grad_w, grad_bias


def moe_balance_workspace_size(T, E, S=1):
    return lib().moe_balance_workspace_size(T, E, S)


def _segments(seq_offsets, dev):
    """(number of segments, address) of seq_offsets (int32 [S + 1], or None: one segment)."""
    if seq_offsets is None:
        return 1, None
    S = seq_offsets.numel() - 1
    _sizes(S)
    ps = _dense(seq_offsets, _torch().int32, "seq_offsets", (S + 1,), dev)
    if S < 1:
        raise ValueError("seq_offsets needs at least two entries")
    return S, ps


def moe_balance_loss(logits, topk_ids, coef, active=None, seq_offsets=None, loss=None, counts=None,
                     probs=None, tokens=None, ws=None, stream=None):
    """Router balance loss of fp32 logits [T, E] and routed ids [T, k]: returns (loss fp32 [1],
    counts int32 [S, E], probs fp32 [S, E], tokens int32 [S]); S = 1 without seq_offsets."""
    torch = _torch()
    T, E = logits.shape
    k = topk_ids.shape[1]
    _sizes(T, E, k)
    dev = logits.device
    with _place(logits, stream):
        S, ps = _segments(seq_offsets, dev)
        f32, i32 = torch.float32, torch.int32
        loss, po = _out(loss, f32, "loss", (1,), dev)
        counts, pc = _out(counts, i32, "counts", (S, E), dev)
        probs, pp = _out(probs, f32, "probs", (S, E), dev)
        tokens, pt = _out(tokens, i32, "tokens", (S,), dev)
        pl = _dense(logits, f32, "logits", (T, E), dev)
        pi = _dense(topk_ids, i32, "topk_ids", (T, k), dev)
        pa = _dense(active, torch.uint8, "active", (T,), dev)
        L = lib()
        ws, pws, nws = _workspace(L.moe_balance_workspace_size(T, E, S), ws, dev)
        _check("moe_balance_loss", L.moe_balance_loss(
            pl, pi, pa, ps, S, T, E, k, float(coef), po, pc, pp, pt, pws, nws, _here(dev)))
    return loss, counts, probs, tokens


def moe_route_backward(logits, topk_ids, gate_mode="topk", topk_w=None, grad_w=None, active=None,
                       counts=None, tokens=None, coef=0.0, grad_loss=None, seq_offsets=None,
                       grad_logits=None, stream=None):
    """Gradient fp32 [T, E] of the router logits through the gate weights (topk_w with their
    gradient grad_w, both fp32 [T, k]), the balance loss (counts and tokens of moe_balance_loss,
    its coef and seq_offsets, grad_loss fp32 [1] or None for 1), or both."""
    torch = _torch()
    T, E = logits.shape
    k = topk_ids.shape[1]
    _sizes(T, E, k)
    dev = logits.device
    with _place(logits, stream):
        S, ps = _segments(seq_offsets, dev)
        f32, i32 = torch.float32, torch.int32
        grad_logits, po = _out(grad_logits, f32, "grad_logits", (T, E), dev)
        pl = _dense(logits, f32, "logits", (T, E), dev)
        pi = _dense(topk_ids, i32, "topk_ids", (T, k), dev)
        pw = _dense(topk_w, f32, "topk_w", (T, k), dev)
        pg = _dense(grad_w, f32, "grad_w", (T, k), dev)
        pa = _dense(active, torch.uint8, "active", (T,), dev)
        pc = _dense(counts, i32, "counts", (S, E), dev)
        pt = _dense(tokens, i32, "tokens", (S,), dev)
        pgl = _dense(grad_loss, f32, "grad_loss", (1,), dev)
        _check("moe_route_backward", lib().moe_route_backward(
            pl, pi, pw, pg, pa, ps, S, T, E, k, GATES.get(gate_mode, gate_mode), pc, pt,
            float(coef), pgl, po, _here(dev)))
    return grad_logits


def moe_combine_backward(grad_out, y_perm, inv_perm, topk_w, need_w=True, need_y=True, grad_w=None,
                         grad_y=None, stream=None):
    """Gradients (grad_w fp32 [T, k], grad_y fp16 like y_perm; None where not needed) of
    moe_unpermute_combine called with topk_w [T, k] on unscaled expert rows y_perm [R, d]."""
    torch = _torch()
    T, d = grad_out.shape
    k = topk_w.shape[1]
    R = y_perm.shape[0]
    _sizes(T, d, k)
    dev = grad_out.device
    with _place(grad_out, stream):
        pgw = pgy = None
        if grad_w is not None or need_w:
            grad_w, pgw = _out(grad_w, torch.float32, "grad_w", (T, k), dev)
        if grad_y is not None or need_y:
            grad_y, pgy = _out(grad_y, torch.float16, "grad_y", (R, d), dev)
        pg = _dense(grad_out, torch.float16, "grad_out", (T, d), dev)
        py = _dense(y_perm, torch.float16, "y_perm", (R, d), dev)
        if R < T * k:
            raise ValueError(f"y_perm: needs at least {T * k} rows, has {R}")
        pi = _dense(inv_perm, torch.int32, "inv_perm", (T * k,), dev)
        pw = _dense(topk_w, torch.float32, "topk_w", (T, k), dev)
        _check("moe_combine_backward", lib().moe_combine_backward(
            pg, py, pi, pw, T, k, d, pgw, pgy, _here(dev)))
    return grad_w, grad_y


# ---------------------------------------------------------------- host helpers
def moe_packed_bytes(wtype, E, K, N):
    return lib().moe_packed_bytes(WTYPES.get(wtype, wtype), E, K, N)


def moe_pack_wq(codes: np.ndarray, wtype) -> np.ndarray:
    """Pack host codes [E, K, N] (int8 codes, or float16 weights for "fp16") -> uint8 array."""
    wt = WTYPES.get(wtype, wtype)
    codes = np.ascontiguousarray(codes)
    if wt == W_FP16:
        if codes.dtype != np.float16:
            raise TypeError("fp16 weights must be float16")
    elif codes.dtype != np.int8:
        raise TypeError("integer codes must be int8")
    E, K, N = codes.shape
    nbytes = lib().moe_packed_bytes(wt, E, K, N)
    if nbytes == 0:
        raise MoEError("moe_pack_wq", MOE_ERR_UNSUPPORTED)
    out = np.empty(nbytes, dtype=np.uint8)
    _check("moe_pack_wq", lib().moe_pack_wq(codes.ctypes.data_as(_P), wt, E, K, N,
                                            out.ctypes.data_as(_P)))
    return out


from .layer import DeviceLayer, Workspace  # noqa: E402,F401
