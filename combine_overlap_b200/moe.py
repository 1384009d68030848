"""Thin ctypes binding over libmoe_b200.so (the C ABI in include/moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (PyTorch provides device memory and
streams); calls are issued on the current torch stream.  If the library is not
built this module raises at import -- there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_b200.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run combine_overlap_b200.build.build() "
                      "(nvcc, sm_100a) first")

_lib = ctypes.CDLL(LIB_PATH)

MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_TIMEOUT, MOE_ERR_WORKSPACE = range(6)
MODE_SEQUENTIAL, MODE_OVERLAPPED = 0, 1
DBG_SKIP_FLAG_BAND = 0x1
SCHED_NO_JOIN = 0x2
SCHED_ONE_CTA = 0x4
DBG_TIMESTAMPS = 0x8
SCHED_GATHER_A = 0x10
SCHED_CTA_PAIR = 0x20
SCHED_B_PER_ATOM = 0x40
SCHED_FULL_TILES = 0x80
SCHED_WIDE_CTA = 0x100
DBG_IDENTITY_EXPERTS = 0x200
SCHED_INTERLEAVE = 0x400
SCHED_EVICT_FIRST = 0x800
SCHED_SIDE_COMBINE = 0x1000
SCHED_EXP_SILU = 0x4000
SCHED_GATHER_LSU = 0x8000


SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = range(4)
DTYPE_BF16, DTYPE_F32 = 0, 1


class MoEError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        self.cuda_error = last_cuda_error() if code == MOE_ERR_CUDA else 0
        detail = f"; {cuda_error_string(self.cuda_error)} (cudaError {self.cuda_error})" \
            if self.cuda_error else ""
        super().__init__(f"{what}: {status_string(code)} (code {code}){detail}")


class LayerArgs(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int), ("d", ctypes.c_int), ("f", ctypes.c_int), ("E", ctypes.c_int),
        ("k", ctypes.c_int),
        ("x", ctypes.c_void_p), ("logits", ctypes.c_void_p),
        ("W1", ctypes.c_void_p), ("W3", ctypes.c_void_p), ("W2", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("topk_idx", ctypes.c_void_p), ("topk_gate", ctypes.c_void_p),
        ("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p),
        ("consumer_sms", ctypes.c_int), ("mgb", ctypes.c_int), ("flags", ctypes.c_uint),
        ("timeout_us", ctypes.c_int),
        ("ev_ffn_begin", ctypes.c_void_p), ("ev_ffn_end", ctypes.c_void_p),
    ]


MAX_EP_RANKS = 8


class EpOwnerArgs(ctypes.Structure):
    _fields_ = [
        ("W", ctypes.c_int), ("rank", ctypes.c_int), ("N", ctypes.c_int), ("d", ctypes.c_int),
        ("f", ctypes.c_int), ("El", ctypes.c_int), ("k", ctypes.c_int),
        ("x_recv", ctypes.c_void_p), ("slot_recv", ctypes.c_void_p), ("recv_counts", ctypes.c_void_p),
        ("W1", ctypes.c_void_p), ("W3", ctypes.c_void_p), ("W2", ctypes.c_void_p),
        ("recv_base", ctypes.c_int * MAX_EP_RANKS),
        ("home_y", ctypes.c_void_p * MAX_EP_RANKS),
        ("home_arrive", ctypes.c_void_p * MAX_EP_RANKS),
        ("consumer_sms", ctypes.c_int), ("mgb", ctypes.c_int), ("flags", ctypes.c_uint),
        ("timeout_us", ctypes.c_int),
    ]


class RouterArgs(ctypes.Structure):
    _fields_ = [
        ("score", ctypes.c_int), ("bias", ctypes.c_void_p),
        ("n_groups", ctypes.c_int), ("topk_groups", ctypes.c_int), ("group_score", ctypes.c_int),
        ("renorm", ctypes.c_int), ("scale", ctypes.c_float),
    ]


class LinearArgs(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int), ("K", ctypes.c_int), ("N", ctypes.c_int),
        ("x", ctypes.c_void_p), ("W", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("residual", ctypes.c_void_p), ("act", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("out", ctypes.c_void_p), ("pre", ctypes.c_void_p),
    ]


class LinearBwdArgs(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int), ("K", ctypes.c_int), ("N", ctypes.c_int),
        ("dout", ctypes.c_void_p), ("x", ctypes.c_void_p), ("W", ctypes.c_void_p),
        ("pre", ctypes.c_void_p), ("act", ctypes.c_int), ("dout_dtype", ctypes.c_int),
        ("dW_dtype", ctypes.c_int), ("dx", ctypes.c_void_p), ("dW", ctypes.c_void_p),
        ("dbias", ctypes.c_void_p),
    ]


class LinearDebug(ctypes.Structure):
    _fields_ = [("cg", ctypes.c_int), ("bn", ctypes.c_int), ("s", ctypes.c_int), ("sw", ctypes.c_int),
                ("timeout_us", ctypes.c_int), ("withhold", ctypes.c_int)]


_P, _I, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_lib.moe_workspace_size.argtypes = [_I, _I, _I, _I, _I]
_lib.moe_workspace_size.restype = _S
_lib.moe_route.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _S, _P]
_lib.moe_permute.argtypes = [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _S, _P]
_lib.moe_grouped_ffn.argtypes = [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, ctypes.c_uint,
                                 _P, _S, _P]
_lib.moe_combine.argtypes = [_P, _P, _P, _I, _I, _I, _P, _P]
_lib.moe_layer_forward.argtypes = [ctypes.POINTER(LayerArgs), _I, _P, _S, _P]
_lib.moe_get_status.argtypes = [_P, _P, ctypes.POINTER(_I), ctypes.POINTER(_I)]
_lib.moe_status_string.argtypes = [_I]
_lib.moe_status_string.restype = ctypes.c_char_p
_lib.moe_num_sms.restype = _I
_lib.moe_tile_variant.argtypes = [_I, _I, _I, _I, ctypes.c_uint]
_lib.moe_tile_variant.restype = _I
_lib.moe_last_cuda_error.restype = _I
_lib.moe_cuda_error_string.argtypes = [_I]
_lib.moe_cuda_error_string.restype = ctypes.c_char_p
_lib.moe_debug_stamps.argtypes = [_P, _P, _P, _I, ctypes.POINTER(_I)]
_lib.moe_debug_stamps.restype = _I
_lib.moe_debug_band_stamps.argtypes = [_P, _P, _P, _I]
_lib.moe_debug_band_stamps.restype = _I
_lib.moe_debug_tokens_combined.argtypes = [_P, _I, _I, _I, _I, _I, _P, ctypes.POINTER(_I)]
_lib.moe_debug_tokens_combined.restype = _I
_lib.moe_permute_noalloc.argtypes = [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]
_lib.moe_permute_noalloc.restype = _I
_lib.moe_permute_noalloc_scratch_bytes.restype = _S
_lib.moe_ep_owner_workspace_size.argtypes = [_I, _I, _I, _I, _I]
_lib.moe_ep_owner_workspace_size.restype = _S
_lib.moe_ep_owner_forward.argtypes = [ctypes.POINTER(EpOwnerArgs), _I, _P, _S, _P]
_lib.moe_ep_home_combine.argtypes = [_P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _P]
_lib.moe_ep_debug_plan.argtypes = [_P, _I, _I, _I, _I, _I, _P, _P, _I]
_lib.moe_ep_debug_plan.restype = _I
_lib.moe_route_scored.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _P, _S, _P]
_lib.moe_route_scored_backward.argtypes = [_P, _P, _P, _I, _I, _I, _P, _P, _P]
_lib.moe_layer_forward_scored.argtypes = [ctypes.POINTER(LayerArgs), ctypes.POINTER(RouterArgs), _I, _P,
                                          _S, _P]
_lib.moe_combine_backward.argtypes = [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P]
_lib.moe_linear_workspace_size.argtypes = [_I, _I, _I]
_lib.moe_linear_workspace_size.restype = _S
_lib.moe_linear_backward_workspace_size.argtypes = [_I, _I, _I]
_lib.moe_linear_backward_workspace_size.restype = _S
_lib.moe_linear.argtypes = [_P, _P, _S, _P]
_lib.moe_linear_backward.argtypes = [_P, _P, _S, _P]
_lib.moe_linear_debug_set.argtypes = [_P]
_lib.moe_linear_debug_set.restype = _I
_lib.moe_linear_timeouts.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32)]
_lib.moe_linear_timeouts.restype = _I
_lib.moe_linear_get_status.argtypes = [_P]
_lib.moe_linear_get_status.restype = _I
for _fn in ("moe_route_scored", "moe_route_scored_backward", "moe_layer_forward_scored",
            "moe_combine_backward", "moe_linear", "moe_linear_backward"):
    getattr(_lib, _fn).restype = _I
for _fn in ("moe_route", "moe_permute", "moe_grouped_ffn", "moe_combine", "moe_layer_forward",
            "moe_get_status", "moe_ep_owner_forward", "moe_ep_home_combine"):
    getattr(_lib, _fn).restype = _I


def declared_symbols() -> list[str]:
    """Function names declared in include/moe.h."""
    with open(HEADER) as fh:
        text = fh.read()
    return sorted(set(re.findall(r"^\s*(?:[\w\*]+\s+)+\**(moe_\w+)\s*\(", text, re.M)))


def status_string(code: int) -> str:
    return _lib.moe_status_string(int(code)).decode()


TILE_VARIANTS = {1: "128x256 per CTA", 2: "256x256 per CTA pair (cta_group::2)",
                 3: "256x256 per CTA (two 128-row MMAs)"}


def tile_variant(T: int, f: int, E: int, k: int, flags: int = 0) -> int:
    """The MMA tile variant the library picks for this shape and flags (1, 2, 3)."""
    return int(_lib.moe_tile_variant(T, f, E, k, int(flags)))


def last_cuda_error() -> int:
    """The cudaError_t value behind this thread's latest MOE_ERR_CUDA (0: none)."""
    return int(_lib.moe_last_cuda_error())


def cuda_error_string(code: int) -> str:
    return _lib.moe_cuda_error_string(int(code)).decode()


def _check(code: int, what: str):
    if code != MOE_OK:
        raise MoEError(code, what)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, dtype, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _shape(t: torch.Tensor, shape: tuple, name: str):
    """The library sees pointers only: a tensor of another shape would be read or
    written out of bounds on the device, so sizes are checked here."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _weights(W1, W3, W2, d=None):
    """Checks W1, W3 [E][d][f] and W2 [E][f][d]; returns (E, d, f)."""
    for n, w in (("W1", W1), ("W3", W3), ("W2", W2)):
        _need(w, torch.bfloat16, n)
        if w.dim() != 3:
            raise ValueError(f"{n} must be 3-D, got shape {tuple(w.shape)}")
    E, dw, f = W1.shape
    if d is not None and dw != d:
        raise ValueError(f"W1 is [E][{dw}][f] but the rows have d = {d}")
    _shape(W3, (E, dw, f), "W3")
    _shape(W2, (E, f, dw), "W2")
    return E, dw, f


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def workspace_size(T: int, d: int, f: int, E: int, k: int) -> int:
    return int(_lib.moe_workspace_size(T, d, f, E, k))


def num_sms() -> int:
    return int(_lib.moe_num_sms())


def alloc_workspace(T, d, f, E, k, device="cuda") -> torch.Tensor:
    n = workspace_size(T, d, f, E, k)
    if n == 0:
        raise MoEError(MOE_ERR_UNSUPPORTED, "moe_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def route(logits: torch.Tensor, k: int, ws: torch.Tensor, counts: bool = False):
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    gate = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    cnt = torch.empty(E, dtype=torch.int32, device=logits.device) if counts else None
    _check(_lib.moe_route(_ptr(logits), T, E, k, _ptr(idx), _ptr(gate), _ptr(cnt), _ptr(ws),
                          ws.numel(), _stream()), "moe_route")
    return (idx, gate, cnt) if counts else (idx, gate)


def permute(x: torch.Tensor, topk_idx: torch.Tensor, E: int, ws: torch.Tensor):
    _need(x, torch.bfloat16, "x")
    _need(topk_idx, torch.int32, "topk_idx")
    T, d = x.shape
    k = topk_idx.shape[1]
    _shape(topk_idx, (T, k), "topk_idx")
    dev = x.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(T * k, dtype=torch.int32, device=dev)
    row_of = torch.empty(T * k, dtype=torch.int32, device=dev)
    x_perm = torch.empty((T * k, d), dtype=torch.bfloat16, device=dev)
    _check(_lib.moe_permute(_ptr(x), T, d, E, k, _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                            _ptr(perm), _ptr(row_of), _ptr(x_perm), _ptr(ws), ws.numel(),
                            _stream()), "moe_permute")
    return counts, offsets, perm, row_of, x_perm


def permute_noalloc(x: torch.Tensor, topk_idx: torch.Tensor, E: int):
    """moe_permute without a workspace: the library's fixed scratch array is used
    instead (for callers that cannot allocate device memory; T <= 65536)."""
    _need(x, torch.bfloat16, "x")
    _need(topk_idx, torch.int32, "topk_idx")
    T, d = x.shape
    k = topk_idx.shape[1]
    _shape(topk_idx, (T, k), "topk_idx")
    dev = x.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(T * k, dtype=torch.int32, device=dev)
    row_of = torch.empty(T * k, dtype=torch.int32, device=dev)
    x_perm = torch.empty((T * k, d), dtype=torch.bfloat16, device=dev)
    _check(_lib.moe_permute_noalloc(_ptr(x), T, d, E, k, _ptr(topk_idx), _ptr(counts),
                                    _ptr(offsets), _ptr(perm), _ptr(row_of), _ptr(x_perm),
                                    _stream()), "moe_permute_noalloc")
    return counts, offsets, perm, row_of, x_perm


def grouped_ffn(x_perm: torch.Tensor, offsets: torch.Tensor, W1, W3, W2, T: int, k: int,
                ws: torch.Tensor, want_h: bool = True, flags: int = 0):
    """x_perm: [T*k][d] bf16 (rows past offsets[E] unused); flags: SCHED_ONE_CTA,
    SCHED_CTA_PAIR, SCHED_B_PER_ATOM, SCHED_FULL_TILES."""
    _need(x_perm, torch.bfloat16, "x_perm")
    _need(offsets, torch.int32, "offsets")
    E, d, f = _weights(W1, W3, W2, x_perm.shape[1])
    _shape(x_perm, (T * k, d), "x_perm")
    _shape(offsets, (E + 1,), "offsets")
    dev = x_perm.device
    y = torch.empty((T * k, d), dtype=torch.bfloat16, device=dev)
    h = torch.empty((T * k, f), dtype=torch.bfloat16, device=dev) if want_h else None
    _check(_lib.moe_grouped_ffn(_ptr(x_perm), _ptr(offsets), T, d, f, E, k, _ptr(W1), _ptr(W3),
                                _ptr(W2), _ptr(h), _ptr(y), int(flags), _ptr(ws), ws.numel(),
                                _stream()),
           "moe_grouped_ffn")
    return h, y


def combine(y: torch.Tensor, row_of: torch.Tensor, topk_gate: torch.Tensor, out=None):
    _need(y, torch.bfloat16, "y")
    _need(row_of, torch.int32, "row_of")
    _need(topk_gate, torch.float32, "topk_gate")
    T, k = topk_gate.shape
    d = y.shape[1]
    _shape(y, (T * k, d), "y")
    _shape(row_of, (T * k,), "row_of")
    if out is None:
        out = torch.empty((T, d), dtype=torch.bfloat16, device=y.device)
    _need(out, torch.bfloat16, "out")
    _shape(out, (T, d), "out")
    _check(_lib.moe_combine(_ptr(y), _ptr(row_of), _ptr(topk_gate), T, d, k, _ptr(out), _stream()),
           "moe_combine")
    return out


def make_args(x, logits, W1, W3, W2, k, out, topk_idx=None, topk_gate=None, counts=None,
              offsets=None, perm=None, consumer_sms=0, mgb=1, flags=0, timeout_us=0,
              ev_begin=None, ev_end=None, d_ff=None) -> LayerArgs:
    T, d = x.shape
    E = logits.shape[1]
    f = W1.shape[2] if W1 is not None else d_ff
    wp = [0 if w is None else w.data_ptr() for w in (W1, W3, W2)]
    return LayerArgs(T, d, f, E, k, x.data_ptr(), logits.data_ptr(), *wp, out.data_ptr(),
                     *(0 if t is None else t.data_ptr() for t in (topk_idx, topk_gate, counts, offsets, perm)),
                     consumer_sms, mgb, flags, timeout_us,
                     None if ev_begin is None else ev_begin.cuda_event,
                     None if ev_end is None else ev_end.cuda_event)


def layer_forward(x, logits, W1, W3, W2, k, ws, mode=MODE_OVERLAPPED, out=None, outputs=False,
                  consumer_sms=0, mgb=1, flags=0, timeout_us=0, stream=None, ev_begin=None,
                  ev_end=None, d_ff=None, router=None):
    """One MoE layer.  Returns out, or (out, dict of routing outputs) if outputs.
    router: a Router, for its routing (moe_layer_forward_scored) in the place of the
    softmax over the chosen logits.
    With flags DBG_IDENTITY_EXPERTS the weights may be None (then d_ff gives the
    FFN width the workspace was sized for)."""
    _need(x, torch.bfloat16, "x")
    _need(logits, torch.float32, "logits")
    T, d = x.shape
    if W1 is None and W3 is None and W2 is None and (flags & DBG_IDENTITY_EXPERTS):
        E, f = logits.shape[1], int(d_ff)
    else:
        E, _, f = _weights(W1, W3, W2, d)
    _shape(logits, (T, E), "logits")
    if ws.numel() < workspace_size(T, d, f, E, k):
        raise ValueError("workspace smaller than moe_workspace_size for this shape")
    dev = x.device
    if out is None:
        out = torch.empty((T, d), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, "out")
    _shape(out, (T, d), "out")
    extra = {}
    if outputs:
        extra = dict(topk_idx=torch.empty((T, k), dtype=torch.int32, device=dev),
                     topk_gate=torch.empty((T, k), dtype=torch.float32, device=dev),
                     counts=torch.empty(E, dtype=torch.int32, device=dev),
                     offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                     perm=torch.empty(T * k, dtype=torch.int32, device=dev))
    # torch creates an event lazily and only times events it has seen recorded:
    # record them here first (this also creates them); the library records them
    # again at the FFN boundaries, and the last record is the one timed.
    s = stream if stream is not None else torch.cuda.current_stream()
    for ev in (ev_begin, ev_end):
        if ev is not None:
            ev.record(s)
    args = make_args(x, logits, W1, W3, W2, k, out, consumer_sms=consumer_sms, mgb=mgb,
                     flags=flags, timeout_us=timeout_us, ev_begin=ev_begin, ev_end=ev_end,
                     d_ff=f, **extra)

    if router is not None:
        _check(_lib.moe_layer_forward_scored(ctypes.byref(args), ctypes.byref(router.args(E, dev)), int(mode),
                                             _ptr(ws), ws.numel(), _stream(stream)),
               "moe_layer_forward_scored")
    else:
        _check(_lib.moe_layer_forward(ctypes.byref(args), int(mode), _ptr(ws), ws.numel(),
                                      _stream(stream)), "moe_layer_forward")
    return (out, extra) if outputs else out


def get_status(ws: torch.Tensor, stream=None):
    """(status code, consumer SMs used, row bands) of the last call on ws; syncs."""
    c = ctypes.c_int(0)
    nb = ctypes.c_int(0)
    code = _lib.moe_get_status(_ptr(ws), _stream(stream), ctypes.byref(c), ctypes.byref(nb))
    return int(code), int(c.value), int(nb.value)


def debug_stamps(ws: torch.Tensor, stream=None):
    """Per-CTA stamps of the last persistent launch run with DBG_TIMESTAMPS: a
    uint64 array [n_ctas][8] (start, GEMM1 queue drained, producer done,
    consumer done -- globaltimer ns -- GEMM1 tiles, GEMM2 tiles, consumer bands,
    cluster rank)."""
    import numpy as np
    out = np.zeros((256, 8), dtype=np.uint64)
    n = ctypes.c_int(0)
    _check(_lib.moe_debug_stamps(_ptr(ws), _stream(stream), out.ctypes.data_as(ctypes.c_void_p), 256,
                                 ctypes.byref(n)), "moe_debug_stamps")
    return out[:n.value]


def debug_band_stamps(ws: torch.Tensor, n_bands: int, stream=None):
    """Per consumed row band of the last DBG_TIMESTAMPS launch: [n][4] uint64 (ready
    ns, combined ns, tokens completed, consuming CTA)."""
    import numpy as np
    n = max(1, min(int(n_bands), 2048))
    out = np.zeros((n, 4), dtype=np.uint64)
    _check(_lib.moe_debug_band_stamps(_ptr(ws), _stream(stream), out.ctypes.data_as(ctypes.c_void_p), n),
           "moe_debug_band_stamps")
    return out


def debug_tokens_combined(ws: torch.Tensor, T: int, d: int, f: int, E: int, k: int, stream=None) -> int:
    """Tokens of the last overlapped call on ws (this shape) that the persistent
    kernel combined itself; the combine pass after it did the rest."""
    n = ctypes.c_int(0)
    _check(_lib.moe_debug_tokens_combined(_ptr(ws), T, d, f, E, k, _stream(stream), ctypes.byref(n)),
           "moe_debug_tokens_combined")
    return int(n.value)


# ---- the linear layer, the scored router and their gradients ----------------
# These calls are short on the device, so their own time on the host counts: arguments go
# to the library as packed bytes, and a tensor's checks are one pass that falls back to
# _need for the error's words.
_LINEAR = struct.Struct("iiiPPPPiiPP")
_LINEAR_BWD = struct.Struct("iiiPPPPiiiPPP")
_ROUTER = struct.Struct("iPiiiif0P")
assert (_LINEAR.size, _LINEAR_BWD.size, _ROUTER.size) == tuple(
    ctypes.sizeof(c) for c in (LinearArgs, LinearBwdArgs, RouterArgs))
_BF16, _F32 = torch.bfloat16, torch.float32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = torch.cuda.current_device


def _same_device(*named):
    """Every given tensor on one device, the current one: the library launches there.
    Returns its current stream."""
    cur = _current_device()
    for t, name in named:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{cur}")
    return _raw_stream(cur)


def _dtype_code(dtype, name: str) -> int:
    if dtype is _BF16:
        return DTYPE_BF16
    if dtype is _F32:
        return DTYPE_F32
    raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {dtype}")


def _need2(t, dtype, name: str):
    """The shape of a contiguous 2-D CUDA tensor of dtype."""
    try:
        if t.dtype is dtype and t.is_cuda and t.is_contiguous():
            shape = t.shape
            if len(shape) == 2:
                return shape
    except AttributeError:
        pass
    _need(t, dtype, name)
    raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")


def _given(t, dtype, shape: tuple, name: str) -> int:
    """The address of a contiguous CUDA tensor of dtype and shape."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, dtype, name)
    _shape(t, shape, name)
    return t.data_ptr()


def _scratch(ws, need: int, like, what: str):
    """The caller's workspace, or one from torch's allocator (of the current stream)."""
    if need >= 1 << 62:
        raise MoEError(MOE_ERR_INVALID, what)
    if ws is None:
        return like.new_empty(need, dtype=torch.uint8) if need else None
    _need(ws, torch.uint8, "ws")
    if ws.numel() < need:
        raise ValueError(f"workspace smaller than {what} for this shape")
    return ws


def linear_workspace_size(M: int, K: int, N: int) -> int:
    return int(_lib.moe_linear_workspace_size(M, K, N))


def linear_backward_workspace_size(M: int, K: int, N: int) -> int:
    return int(_lib.moe_linear_backward_workspace_size(M, K, N))


def linear(x, W, bias=None, residual=None, act=ACT_NONE, out_dtype=torch.bfloat16, pre=False, out=None,
           ws=None, stream=None):
    """out = act(x W + bias) + residual (moe_linear): x [M][K], W [K][N] bf16, bias [N]
    fp32, residual and out [M][N] of out_dtype (bf16 or fp32; out may be residual).
    pre=True also returns x W + bias in bf16, which linear_backward wants with an
    activation.  ws: linear_workspace_size(M, K, N) bytes (None: allocated here)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear(x, W, bias, residual, act, out_dtype, pre, out, ws)
    M, K = _need2(x, _BF16, "x")
    Kw, N = _need2(W, _BF16, "W")
    if Kw != K:
        _shape(W, (K, N), "W")
    code = _dtype_code(out_dtype, "out_dtype")
    b_ptr = _given(bias, _F32, (N,), "bias") if bias is not None else 0
    r_ptr = _given(residual, out_dtype, (M, N), "residual") if residual is not None else 0
    if out is not None:
        _given(out, out_dtype, (M, N), "out")
    elif residual is not None:
        out = torch.empty_like(residual)
    else:
        out = x.new_empty((M, N), dtype=out_dtype)
    u = x.new_empty((M, N)) if pre else None
    ws = _scratch(ws, _lib.moe_linear_workspace_size(M, K, N), x, "moe_linear_workspace_size")
    st = _same_device((x, "x"), (W, "W"), (bias, "bias"), (residual, "residual"), (out, "out"), (ws, "ws"))
    a = _LINEAR.pack(M, K, N, x.data_ptr(), W.data_ptr(), b_ptr, r_ptr, act, code, out.data_ptr(),
                     u.data_ptr() if pre else 0)
    r = _lib.moe_linear(a, None, 0, st) if ws is None else _lib.moe_linear(a, ws.data_ptr(), ws.numel(), st)
    if r:
        _check(r, "moe_linear")
    return (out, u) if pre else out


def linear_backward(dout, x, W, pre=None, act=ACT_NONE, dW_dtype=torch.float32, want_dx=True, want_dW=True,
                    want_dbias=False, ws=None, stream=None):
    """The gradients of linear (moe_linear_backward): dout [M][N] bf16 or fp32 ->
    (dx [M][K] bf16, dW [K][N] of dW_dtype, dbias [N] fp32), None where not wanted.
    dW_dtype float32 also keeps 16 bits of the pre-activation's gradient for dx, bfloat16
    8.  The residual's gradient is dout itself.  pre: linear's second result, with an
    activation.  ws: linear_backward_workspace_size(M, K, N) bytes (None: allocated here)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_backward(dout, x, W, pre, act, dW_dtype, want_dx, want_dW, want_dbias, ws)
    M, K = _need2(x, _BF16, "x")
    Kw, N = _need2(W, _BF16, "W")
    if Kw != K:
        _shape(W, (K, N), "W")
    code, dW_code = _dtype_code(dout.dtype, "dout"), _dtype_code(dW_dtype, "dW_dtype")
    d_ptr = _given(dout, dout.dtype, (M, N), "dout")
    p_ptr = 0
    if act != ACT_NONE:
        if pre is None:
            raise ValueError("linear_backward needs pre (linear(..., pre=True)) with an activation")
        p_ptr = _given(pre, _BF16, (M, N), "pre")
    else:
        pre = None
    dx = torch.empty_like(x) if want_dx else None
    dW = torch.empty_like(W, dtype=dW_dtype) if want_dW else None
    db = x.new_empty(N, dtype=_F32) if want_dbias else None
    ws = _scratch(ws, _lib.moe_linear_backward_workspace_size(M, K, N), x, "moe_linear_backward_workspace_size")
    st = _same_device((x, "x"), (W, "W"), (dout, "dout"), (pre, "pre"), (ws, "ws"))
    a = _LINEAR_BWD.pack(M, K, N, d_ptr, x.data_ptr(), W.data_ptr(), p_ptr, act, code, dW_code,
                         dx.data_ptr() if want_dx else 0, dW.data_ptr() if want_dW else 0,
                         db.data_ptr() if want_dbias else 0)
    r = _lib.moe_linear_backward(a, *((None, 0) if ws is None else (ws.data_ptr(), ws.numel())), st)
    if r:
        _check(r, "moe_linear_backward")
    return dx, dW, db


_thread = threading.local()


@contextlib.contextmanager
def linear_debug(cg=0, bn=0, s=1, sw=1, timeout_us=0, withhold=False):
    """Within it, this thread's tensor-core products run with the given tile and splits
    (moe_linear_debug_set; cg = 0: the library's choice); MOE_ERR_UNSUPPORTED where a
    product of that size is never cut that way.  timeout_us bounds their device waits
    (0: 2 s); withhold makes those of the first tile run out."""
    d, before = LinearDebug(cg, bn, s, sw, timeout_us, int(withhold)), getattr(_thread, "linear_debug", None)
    _check(_lib.moe_linear_debug_set(ctypes.byref(d)), "moe_linear_debug_set")
    _thread.linear_debug = d
    try:
        yield
    finally:
        _thread.linear_debug = before
        _lib.moe_linear_debug_set(None if before is None else ctypes.byref(before))


def linear_get_status(stream=None) -> int:
    """Whether a bounded wait of linear or linear_backward ran out on the current device
    since this thread's last call of this (MOE_OK or MOE_ERR_TIMEOUT); syncs."""
    return int(_lib.moe_linear_get_status(_stream(stream)))


def linear_timeouts(stream=None) -> int:
    """How many thread blocks of linear and linear_backward have given up a bounded wait on
    the current device so far; syncs.  Callers that compare it with a count of their own
    do not depend on who else asks."""
    n = ctypes.c_uint32()
    _check(_lib.moe_linear_timeouts(_stream(stream), ctypes.byref(n)), "moe_linear_timeouts")
    return int(n.value)


def _router_args(E, device, score, bias, n_groups, topk_groups, group_score, renorm, scale) -> RouterArgs:
    if bias is not None:
        _given(bias, _F32, (E,), "bias")
        if bias.device != device:
            raise ValueError(f"bias is on {bias.device}, the logits on {device}")
    return RouterArgs(int(score), None if bias is None else bias.data_ptr(), int(n_groups), int(topk_groups),
                      int(group_score), 1 if renorm else 0, float(scale))


def route_scored(logits, k: int, score=SCORE_SOFTMAX, bias=None, n_groups=1, topk_groups=0,
                 group_score=GROUP_MAX, renorm=True, scale=1.0, counts=False, ws=None, stream=None):
    """The scored router (moe_route_scored): logits [T][E] fp32 -> (topk_idx [T][k] int32,
    topk_gate [T][k] fp32), and counts [E] int32 with counts=True (then ws, of
    alloc_workspace, is needed).  bias [E] fp32 steers the choice only."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return route_scored(logits, k, score, bias, n_groups, topk_groups, group_score, renorm, scale,
                                counts, ws)
    T, E = _need2(logits, _F32, "logits")
    b_ptr = _given(bias, _F32, (E,), "bias") if bias is not None else 0
    idx = logits.new_empty((T, k), dtype=torch.int32)
    gate = logits.new_empty((T, k))
    cnt = logits.new_empty(E, dtype=torch.int32) if counts else None
    st = _same_device((logits, "logits"), (bias, "bias"), (ws, "ws"))
    r = _lib.moe_route_scored(logits.data_ptr(), T, E, k,
                              _ROUTER.pack(score, b_ptr, n_groups, topk_groups, group_score, 1 if renorm else 0, scale),
                              idx.data_ptr(), gate.data_ptr(), cnt.data_ptr() if counts else None,
                              *((None, 0) if ws is None else (ws.data_ptr(), ws.numel())), st)
    if r:
        _check(r, "moe_route_scored")
    return (idx, gate, cnt) if counts else (idx, gate)


def route_scored_backward(dgate, logits, topk_idx, score=SCORE_SOFTMAX, renorm=True, scale=1.0,
                          dlogits=None, stream=None):
    """The gradient of route_scored's gates (moe_route_scored_backward): dgate [T][k]
    -> dlogits [T][E], all of it written."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return route_scored_backward(dgate, logits, topk_idx, score, renorm, scale, dlogits)
    T, E = _need2(logits, _F32, "logits")
    k = _need2(dgate, _F32, "dgate")[1]
    d_ptr = _given(dgate, _F32, (T, k), "dgate")
    i_ptr = _given(topk_idx, torch.int32, (T, k), "topk_idx")
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    else:
        _given(dlogits, _F32, (T, E), "dlogits")
    st = _same_device((logits, "logits"), (dgate, "dgate"), (topk_idx, "topk_idx"), (dlogits, "dlogits"))
    r = _lib.moe_route_scored_backward(d_ptr, logits.data_ptr(), i_ptr, T, E, k,
                                       _ROUTER.pack(score, 0, 1, 0, GROUP_MAX, 1 if renorm else 0, scale),
                                       dlogits.data_ptr(), st)
    if r:
        _check(r, "moe_route_scored_backward")
    return dlogits


def combine_backward(dout, y, row_of, topk_gate, want_dy=True, dy=None, stream=None):
    """The gradient of combine (moe_combine_backward): dout [T][d] bf16 -> (dy [T*k][d]
    bf16 or None, dgate [T][k] fp32).  A row_of of -1 is a dropped slot (dgate 0); rows of
    dy that no slot names are left as they were, and 0 in a dy that is made here."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return combine_backward(dout, y, row_of, topk_gate, want_dy, dy)
    T, k = _need2(topk_gate, _F32, "topk_gate")
    d = _need2(y, _BF16, "y")[1]
    y_ptr = _given(y, _BF16, (T * k, d), "y")
    o_ptr = _given(dout, _BF16, (T, d), "dout")
    r_ptr = _given(row_of, torch.int32, (T * k,), "row_of")
    if dy is not None:
        _given(dy, _BF16, (T * k, d), "dy")
    elif want_dy:
        dy = torch.zeros_like(y)
    dgate = torch.empty_like(topk_gate)
    st = _same_device((dout, "dout"), (y, "y"), (row_of, "row_of"), (topk_gate, "topk_gate"), (dy, "dy"))
    r = _lib.moe_combine_backward(o_ptr, y_ptr, r_ptr, topk_gate.data_ptr(), T, d, k,
                                  None if dy is None else dy.data_ptr(), dgate.data_ptr(), st)
    if r:
        _check(r, "moe_combine_backward")
    return dy, dgate


class Router:
    """A router's options, and with Wg [d][E] bf16 (and bg [E] fp32) its gate projection."""

    def __init__(self, Wg=None, bg=None, score=SCORE_SOFTMAX, bias=None, n_groups=1, topk_groups=0,
                 group_score=GROUP_MAX, renorm=True, scale=1.0):
        self.Wg, self.bg, self.score, self.bias = Wg, bg, score, bias
        self.n_groups, self.topk_groups, self.group_score = n_groups, topk_groups, group_score
        self.renorm, self.scale = renorm, scale

    def args(self, E: int, device) -> RouterArgs:
        return _router_args(E, device, self.score, self.bias, self.n_groups, self.topk_groups,
                            self.group_score, self.renorm, self.scale)

    def logits(self, x, stream=None):
        """The gate projection x Wg + bg in fp32."""
        if self.Wg is None:
            raise ValueError("this Router has no gate projection (Wg)")
        return linear(x, self.Wg, bias=self.bg, out_dtype=torch.float32, stream=stream)

    def route(self, logits, k: int, **kw):
        return route_scored(logits, k, self.score, self.bias, self.n_groups, self.topk_groups,
                            self.group_score, self.renorm, self.scale, **kw)

    def backward(self, dgate, logits, topk_idx, stream=None):
        return route_scored_backward(dgate, logits, topk_idx, self.score, self.renorm, self.scale,
                                     stream=stream)


class MoELayer:
    """Holds the weights and a workspace; forward() runs the layer.  With a Router that
    has a gate projection, forward(x) makes the logits too, and forward_train / backward
    train the router over the (frozen) experts."""

    def __init__(self, W1, W3, W2, k: int, max_tokens: int, router: Router | None = None):
        self.W1, self.W3, self.W2, self.k = W1, W3, W2, k
        self.E, self.d, self.f = W1.shape
        self.max_tokens = max_tokens
        self.router = router
        self.ws = alloc_workspace(max_tokens, self.d, self.f, self.E, k, W1.device)
        self._timeouts = 0
        if router is not None and not torch.cuda.is_current_stream_capturing():
            self._timeouts = self._linear_timeouts()

    def _linear_timeouts(self, stream=None) -> int:
        with torch.cuda.device(self.ws.device):
            return linear_timeouts(stream)

    def get_status(self, stream=None):
        """get_status of the layer's last call, and with a Router of its gate projection and
        gradients too: MOE_ERR_TIMEOUT if a bounded wait of the layer's last call, or since the
        last call of this of any linear or linear_backward on the device, ran out.  Syncs."""
        code, consumers, bands = get_status(self.ws, stream)
        if self.router is not None:
            before, self._timeouts = self._timeouts, self._linear_timeouts(stream)
            if code == MOE_OK and self._timeouts != before:
                code = MOE_ERR_TIMEOUT
        return code, consumers, bands

    def forward(self, x, logits=None, mode=MODE_OVERLAPPED, **kw):
        if x.shape[0] > self.max_tokens:
            raise ValueError("more tokens than the workspace was sized for")
        if logits is None:
            if self.router is None:
                raise ValueError("logits are needed without a Router")
            logits = self.router.logits(x, stream=kw.get("stream"))
        return layer_forward(x, logits, self.W1, self.W3, self.W2, self.k, self.ws, mode,
                             router=self.router, **kw)

    def forward_train(self, x):
        """The layer step by step: (out, saved), with what backward needs."""
        if x.shape[0] > self.max_tokens:
            raise ValueError("more tokens than the workspace was sized for")
        if self.router is None:
            raise ValueError("forward_train needs a Router")
        logits = self.router.logits(x)
        idx, gate = self.router.route(logits, self.k)
        _, offsets, _, row_of, x_perm = permute(x, idx, self.E, self.ws)
        _, y = grouped_ffn(x_perm, offsets, self.W1, self.W3, self.W2, x.shape[0], self.k, self.ws, want_h=False)
        return combine(y, row_of, gate), dict(x=x, logits=logits, idx=idx, gate=gate, row_of=row_of, y=y)

    def backward(self, dout, saved, want_dy=False):
        """Gradients of the router from dout [T][d] bf16 and forward_train's saved: a dict
        of dWg, dbg (fp32; dbg None without bg), dx (the gate projection's share, bf16),
        dlogits, and with want_dy dy [T*k][d], the gradient of the experts' outputs."""
        r = self.router
        # forward_train drops no slot, so every row of dy is written
        dy = torch.empty_like(saved["y"]) if want_dy else None
        dy, dgate = combine_backward(dout, saved["y"], saved["row_of"], saved["gate"], want_dy=want_dy, dy=dy)
        dlogits = r.backward(dgate, saved["logits"], saved["idx"])
        dx, dWg, dbg = linear_backward(dlogits, saved["x"], r.Wg, want_dbias=r.bg is not None)
        return dict(dWg=dWg, dbg=dbg, dx=dx, dlogits=dlogits, dy=dy)


# ---- expert parallelism: the fused return -----------------------------------
def ep_owner_workspace_size(N: int, d: int, f: int, El: int, W: int) -> int:
    return int(_lib.moe_ep_owner_workspace_size(N, d, f, El, W))


def ep_owner_forward(x_recv, slot_recv, recv_counts, W1, W3, W2, k: int, rank: int, recv_base,
                     home_y, home_arrive, ws, mode=MODE_OVERLAPPED, consumer_sms=0, mgb=1,
                     flags=0, timeout_us=0, stream=None):
    """The owner side of an expert-parallel layer (moe_ep_owner_forward): runs
    this rank's experts on the rows it received and returns every finished row
    band into its home rank's buffer (home_y[s], home_arrive[s], one per rank)."""
    _need(x_recv, torch.bfloat16, "x_recv")
    _need(slot_recv, torch.int32, "slot_recv")
    _need(recv_counts, torch.int32, "recv_counts")
    N, d = x_recv.shape
    El, _, f = _weights(W1, W3, W2, d)
    W = recv_counts.shape[0]
    _shape(recv_counts, (W, El), "recv_counts")
    _shape(slot_recv, (N,), "slot_recv")
    if not (1 <= W <= MAX_EP_RANKS) or len(home_y) != W or len(home_arrive) != W or len(recv_base) != W:
        raise ValueError("one home buffer, arrival array and receive base per rank")
    for s_, (y, a) in enumerate(zip(home_y, home_arrive)):
        _need(y, torch.bfloat16, f"home_y[{s_}]")
        _need(a, torch.int32, f"home_arrive[{s_}]")
        if y.shape[1] != d:
            raise ValueError(f"home_y[{s_}] rows must have d = {d}")
    if ws.numel() < ep_owner_workspace_size(N, d, f, El, W):
        raise ValueError("workspace smaller than moe_ep_owner_workspace_size")
    if N == 0:
        return   # nothing received: no band to compute or return
    a = EpOwnerArgs()
    a.W, a.rank, a.N, a.d, a.f, a.El, a.k = W, rank, N, d, f, El, k
    a.x_recv, a.slot_recv, a.recv_counts = x_recv.data_ptr(), slot_recv.data_ptr(), recv_counts.data_ptr()
    a.W1, a.W3, a.W2 = W1.data_ptr(), W3.data_ptr(), W2.data_ptr()
    for s_ in range(W):
        a.recv_base[s_] = int(recv_base[s_])
        a.home_y[s_] = home_y[s_].data_ptr()
        a.home_arrive[s_] = home_arrive[s_].data_ptr()
    a.consumer_sms, a.mgb, a.flags, a.timeout_us = consumer_sms, mgb, flags, timeout_us
    _check(_lib.moe_ep_owner_forward(ctypes.byref(a), int(mode), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_ep_owner_forward")


def ep_home_combine(home_y, arrive, row_of, topk_gate, out=None, status=None, timeout_us=0,
                    stream=None):
    """The home side (moe_ep_home_combine): waits for each token's k returned
    rows, combines them and zeroes the arrival words.  Returns (out, status) with
    status a one-element int32 device tensor (0, or MOE_ERR_TIMEOUT)."""
    _need(home_y, torch.bfloat16, "home_y")
    _need(arrive, torch.int32, "arrive")
    _need(row_of, torch.int32, "row_of")
    _need(topk_gate, torch.float32, "topk_gate")
    T, k = topk_gate.shape
    d = home_y.shape[1]
    _shape(home_y, (T * k, d), "home_y")
    _shape(arrive, (T,), "arrive")
    _shape(row_of, (T * k,), "row_of")
    if out is None:
        out = torch.empty((T, d), dtype=torch.bfloat16, device=home_y.device)
    _shape(out, (T, d), "out")
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=home_y.device)
    _check(_lib.moe_ep_home_combine(_ptr(home_y), _ptr(arrive), _ptr(row_of), _ptr(topk_gate), T, d, k,
                                    _ptr(out), _ptr(status), int(timeout_us), _stream(stream)),
           "moe_ep_home_combine")
    return out, status


def ep_band_dest(ws, N: int, d: int, f: int, El: int, W: int, n_bands: int, stream=None):
    """The combine plan of the last owner call on ws: [n_bands][2] int32 (home
    rank, home row of the band's first row), bands in schedule order."""
    import numpy as np
    out = np.zeros((max(1, n_bands), 2), dtype=np.int32)
    _check(_lib.moe_ep_debug_plan(_ptr(ws), N, d, f, El, W, _stream(stream),
                                  out.ctypes.data_as(ctypes.c_void_p), max(1, n_bands)),
           "moe_ep_debug_plan")
    return out[:n_bands]
