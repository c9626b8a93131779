"""Thin ctypes binding of libdv (include/dv.h).

Each ``dv_*`` function here has the name of the C entry point it calls and
only marshals arguments: it takes torch CUDA tensors (PyTorch is used for
device memory and streams), derives sizes from their shapes, passes raw
pointers and the stream handle, and raises ``DvError`` on a non-OK status.
All computation happens in the library's CUDA kernels.  There is no
fallback: if libdv.so cannot be built or loaded, every call raises.
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Sequence

import torch

from . import build as _build

DV_F32, DV_F16, DV_BF16 = 0, 1, 2
DV_TOPK, DV_THRESHOLD = 0, 1

STATUS = {
    0: "DV_OK", 1: "DV_ERR_INVALID_ARG", 2: "DV_ERR_DTYPE", 3: "DV_ERR_WORKSPACE",
    4: "DV_ERR_CUDA", 5: "DV_ERR_INDEX_RANGE", 6: "DV_ERR_TIMEOUT", 7: "DV_ERR_UNSUPPORTED",
    8: "DV_ERR_CAPACITY", 9: "DV_ERR_POSITION",
}

_DT = {torch.float32: DV_F32, torch.float16: DV_F16, torch.bfloat16: DV_BF16}

# every entry point declared in include/dv.h
EXPORTS = (
    "dv_status_str", "dv_last_cuda_error", "dv_version", "dv_workspace_init", "dv_check",
    "dv_predict_workspace_size", "dv_predict", "dv_lookahead", "dv_predict_static",
    "dv_sparse_mlp_workspace_size", "dv_sparse_mlp",
    "dv_sparse_attn_workspace_size", "dv_sparse_attn", "dv_kv_repair",
    "dv_layernorm", "dv_positions_advance", "dv_set_launch_overlap", "dv_set_wait_limit_ns",
    "dv_kernel_launches", "dv_label_workspace_size", "dv_label_neurons", "dv_label_heads",
    "dv_select_scores", "dv_tree_attn_workspace_size", "dv_tree_attn", "dv_kv_compact", "dv_kv_reorder",
    "dv_beam_select_workspace_size", "dv_beam_select",
)


class DvError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} {detail}".rstrip())


class dv_predictor(ctypes.Structure):
    _fields_ = [("P1t", ctypes.c_void_p), ("P2t", ctypes.c_void_p), ("r", ctypes.c_int),
                ("N", ctypes.c_int), ("mode", ctypes.c_int), ("k", ctypes.c_int),
                ("t", ctypes.c_float), ("idx", ctypes.c_void_p), ("cap", ctypes.c_int),
                ("count", ctypes.c_void_p), ("scores", ctypes.c_void_p)]


class dv_kv(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("X", ctypes.c_void_p),
                ("valid", ctypes.c_void_p), ("n_max", ctypes.c_int)]


_lib = None
_lock = threading.Lock()

_c_int, _c_float, _vp, _sz = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
_SIGS = {
    "dv_status_str": ([_c_int], ctypes.c_char_p),
    "dv_last_cuda_error": ([], _c_int),
    "dv_version": ([], _c_int),
    "dv_workspace_init": ([_vp, _sz, _vp], _c_int),
    "dv_check": ([_vp, _vp, ctypes.POINTER(_c_int)], _c_int),
    "dv_predict_workspace_size": ([_c_int, _c_int, _c_int, _c_int, ctypes.POINTER(_sz)], _c_int),
    "dv_predict": ([_vp, _c_int, _c_int, _c_int, ctypes.POINTER(dv_predictor), _c_int, _vp, _sz, _vp],
                   _c_int),
    "dv_lookahead": ([_vp, _c_int, _c_int, _c_int, ctypes.POINTER(dv_predictor), _c_int, _vp, _sz,
                      _vp, _vp, _vp], _c_int),
    "dv_predict_static": ([_vp, _c_int, _c_int, _c_int, ctypes.POINTER(dv_predictor), _c_int, _vp],
                          _c_int),
    "dv_sparse_mlp_workspace_size": ([_c_int, _c_int, _c_int, _c_int, ctypes.POINTER(_sz)], _c_int),
    "dv_sparse_mlp": ([_vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _c_int, _vp, _c_int, _vp, _c_int,
                       _vp, _sz, _vp], _c_int),
    "dv_sparse_attn_workspace_size": ([_c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                       ctypes.POINTER(_sz)], _c_int),
    "dv_sparse_attn": ([_vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, ctypes.POINTER(dv_kv), _vp,
                        _vp, _c_int, _vp, _c_float, _c_int, _vp, _c_int, _vp, _sz, _vp], _c_int),
    "dv_kv_repair": ([ctypes.POINTER(dv_kv), _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _c_int,
                      _vp, _c_int, _vp, _sz, _vp], _c_int),
    "dv_layernorm": ([_vp, _c_int, _c_int, _c_float, _vp, _c_int, _vp], _c_int),
    "dv_positions_advance": ([_vp, _c_int, _c_int, _c_int, _vp], _c_int),
    "dv_set_launch_overlap": ([_c_int], _c_int),
    "dv_set_wait_limit_ns": ([ctypes.c_longlong], ctypes.c_longlong),
    "dv_kernel_launches": ([], ctypes.c_longlong),
    "dv_label_workspace_size": ([_c_int, _c_int, _c_int, _c_int, _c_int, ctypes.POINTER(_sz)], _c_int),
    "dv_label_neurons": ([_vp, _c_int, _c_int, _c_int, _vp, _c_int, _vp, _vp, _sz, _vp], _c_int),
    "dv_label_heads": ([_vp, _c_int, _c_int, _c_int, _c_int, _vp, _c_float, _c_int, _vp, _vp, _sz, _vp],
                       _c_int),
    "dv_select_scores": ([_vp, _c_int, _c_int, _c_int, _c_int, _c_float, _vp, _c_int, _vp, _vp, _sz, _vp],
                         _c_int),
    "dv_tree_attn_workspace_size": ([_c_int, _c_int, _c_int, _c_int, _c_int, ctypes.POINTER(_sz)], _c_int),
    "dv_tree_attn": ([_vp, _c_int, _c_int, _c_int, _c_int, _c_int, ctypes.POINTER(dv_kv), _vp, _vp, _vp, _c_int,
                      _vp, _c_int, _vp, _c_float, _c_int, _vp, _vp, _sz, _vp], _c_int),
    "dv_kv_compact": ([ctypes.POINTER(dv_kv), _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _c_int, _vp,
                       _c_int, _vp, _vp, _sz, _vp], _c_int),
    "dv_kv_reorder": ([ctypes.POINTER(dv_kv), _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp,
                       _c_int, _vp, _sz, _vp], _c_int),
    "dv_beam_select_workspace_size": ([_c_int, _c_int, _c_int, _c_int, ctypes.POINTER(_sz)], _c_int),
    "dv_beam_select": ([_vp, _c_int, _c_int, _c_int, ctypes.c_longlong, _c_int, _vp, _vp, _c_int, _c_int, _vp,
                        _vp, _vp, _vp, _sz, _vp], _c_int),
}


def lib_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libdv.so (building it in-tree first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            L = ctypes.CDLL(path)
            for name, (args, res) in _SIGS.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = res
            _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object around it (a third of the
# host's time of a small call); torch.cuda.current_stream() otherwise
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None and _current_device is not None and torch.cuda.is_initialized():
            return _raw_stream(_current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _event(ev) -> ctypes.c_void_p:
    if ev is None:
        return ctypes.c_void_p(0)
    h = ev.cuda_event if hasattr(ev, "cuda_event") else int(ev)
    if not h:
        raise ValueError("CUDA event not created yet: use make_event()")
    return ctypes.c_void_p(h)


def make_event(stream=None) -> torch.cuda.Event:
    """A torch CUDA event whose underlying cudaEvent_t already exists (torch
    creates it lazily on the first record)."""
    ev = torch.cuda.Event()
    ev.record(stream if stream is not None else torch.cuda.current_stream())
    return ev


def _dt(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise DvError(2, "dtype", str(t.dtype))


def _ok(st: int, where: str):
    if st != 0:
        detail = ""
        if st == 4:
            detail = f"(cudaError {lib().dv_last_cuda_error()})"
        raise DvError(st, where, detail)


# --------------------------------------------------------------------- utility

def dv_version() -> int:
    return lib().dv_version()


def dv_kernel_launches() -> int:
    """Kernels the library has enqueued in this process so far (captured
    launches included)."""
    return int(lib().dv_kernel_launches())


def dv_status_str(st: int) -> str:
    return lib().dv_status_str(st).decode()


def dv_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _ok(lib().dv_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
        "dv_workspace_init")


def workspace(nbytes: int, device="cuda", stream=None) -> torch.Tensor:
    """Allocate (through torch) and zero-fill a workspace of ``nbytes``."""
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    dv_workspace_init(ws, stream)
    return ws


def dv_check(ws: torch.Tensor, stream=None):
    """Synchronise and return (status, info) of the workspace's error word."""
    info = ctypes.c_int(0)
    st = lib().dv_check(_ptr(ws), _stream(stream), ctypes.byref(info))
    return st, info.value


# --------------------------------------------------------------------- predictor

class Predictor:
    """Arguments of one predictor (see dv_predictor in dv.h)."""

    def __init__(self, P1t, P2t, idx, count, mode=DV_TOPK, k=0, t=0.5, scores=None):
        self.P1t, self.P2t, self.idx, self.count, self.scores = P1t, P2t, idx, count, scores
        self.mode, self.k, self.t = int(mode), int(k), float(t)

    def c(self) -> dv_predictor:
        return dv_predictor(self.P1t.data_ptr(), self.P2t.data_ptr(), self.P1t.shape[0],
                            self.P2t.shape[0], self.mode, self.k, self.t, self.idx.data_ptr(),
                            self.idx.shape[-1], self.count.data_ptr(),
                            self.scores.data_ptr() if self.scores is not None else None)


def dv_predict_workspace_size(B: int, n_preds: int, r_max: int, N_max: int) -> int:
    n = ctypes.c_size_t(0)
    _ok(lib().dv_predict_workspace_size(B, n_preds, r_max, N_max, ctypes.byref(n)),
        "dv_predict_workspace_size")
    return n.value


def _preds(preds: Sequence[Predictor]):
    arr = (dv_predictor * len(preds))(*[p.c() for p in preds])
    return arr, len(preds)


def dv_predict(y: torch.Tensor, preds: Sequence[Predictor], ws: torch.Tensor, stream=None):
    arr, n = _preds(preds)
    B, d = y.shape
    _ok(lib().dv_predict(_ptr(y), B, d, _dt(y), arr, n, _ptr(ws), ws.numel(), _stream(stream)),
        "dv_predict")


def dv_predict_static(y: torch.Tensor, preds: Sequence[Predictor], stream=None):
    """dv_predict without a workspace: the library's fixed scratch array is
    used instead (for callers that cannot allocate; see dv.h for limits)."""
    arr, n = _preds(preds)
    B, d = y.shape
    _ok(lib().dv_predict_static(_ptr(y), B, d, _dt(y), arr, n, _stream(stream)),
        "dv_predict_static")


def dv_lookahead(y: torch.Tensor, preds: Sequence[Predictor], ws: torch.Tensor,
                 input_ready, side, done):
    arr, n = _preds(preds)
    B, d = y.shape
    _ok(lib().dv_lookahead(_ptr(y), B, d, _dt(y), arr, n, _ptr(ws), ws.numel(), _event(input_ready),
                           _stream(side), _event(done)), "dv_lookahead")


# --------------------------------------------------------------------- sparse MLP

def dv_sparse_mlp_workspace_size(B: int, d: int, N: int, cap: int) -> int:
    n = ctypes.c_size_t(0)
    _ok(lib().dv_sparse_mlp_workspace_size(B, d, N, cap, ctypes.byref(n)),
        "dv_sparse_mlp_workspace_size")
    return n.value


def dv_sparse_mlp(y, W1n, W2n, idx, count, out, ws, accumulate=False, stream=None):
    B, d = y.shape
    N = W1n.shape[0]
    _ok(lib().dv_sparse_mlp(_ptr(y), B, d, N, _ptr(W1n), _ptr(W2n), _ptr(idx), idx.shape[-1],
                            _ptr(count), _dt(y), _ptr(out), int(bool(accumulate)), _ptr(ws),
                            ws.numel(), _stream(stream)), "dv_sparse_mlp")


# --------------------------------------------------------------------- attention

class KV:
    """A batch's per-layer KV cache: K, V [B][h][n_max][d_h], X [B][n_max][d],
    valid [B][h][n_max] (uint8).  dv_tree_attn reads K and V alone: X and
    valid may be None there."""

    def __init__(self, K, V, X, valid):
        self.K, self.V, self.X, self.valid = K, V, X, valid
        self.n_max = K.shape[2]

    @classmethod
    def empty(cls, B, h, n_max, d_h, d, dtype, device="cuda"):
        return cls(torch.zeros(B, h, n_max, d_h, dtype=dtype, device=device),
                   torch.zeros(B, h, n_max, d_h, dtype=dtype, device=device),
                   torch.zeros(B, n_max, d, dtype=dtype, device=device),
                   torch.zeros(B, h, n_max, dtype=torch.uint8, device=device))

    def c(self) -> dv_kv:
        return dv_kv(self.K.data_ptr(), self.V.data_ptr(),
                     None if self.X is None else self.X.data_ptr(),
                     None if self.valid is None else self.valid.data_ptr(), self.n_max)


class KVLayers:
    """The caches of a decoder's layers, all of one shape, as one argument of
    dv_kv_compact and dv_kv_reorder (the descriptors are built once)."""

    def __init__(self, kvs: Sequence[KV]):
        self.kvs = list(kvs)
        kv = self.kvs[0]
        self.B, self.h, self.n_max, self.d_h = kv.K.shape
        self.d, self.dt = kv.X.shape[2], _dt(kv.K)
        for c in self.kvs:
            for t, shape in ((c.K, kv.K.shape), (c.V, kv.K.shape), (c.X, (self.B, self.n_max, self.d))):
                _laid_out(t, shape, kv.K.dtype, "KVLayers")
            _laid_out(c.valid, kv.K.shape[:3], torch.uint8, "KVLayers")
        self.n = len(self.kvs)
        self.array = (dv_kv * self.n)(*[c.c() for c in self.kvs])


def _counted(where: str, n: int, *tensors, dtype=torch.int32) -> None:
    """Contiguous tensors of n elements: the library reads or writes that many."""
    for t in tensors:
        if t is not None and (t.dtype != dtype or t.numel() != n or not t.is_contiguous()):
            raise DvError(1, where, f"contiguous tensors of {n} elements of {dtype} are wanted")


def _laid_out(t: torch.Tensor, shape, dtype, where: str) -> None:
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise DvError(1, where, f"a contiguous {tuple(shape)} tensor of {dtype} is wanted")


def dv_sparse_attn_workspace_size(B, d, h, d_h, cap, n_max) -> int:
    n = ctypes.c_size_t(0)
    _ok(lib().dv_sparse_attn_workspace_size(B, d, h, d_h, cap, n_max, ctypes.byref(n)),
        "dv_sparse_attn_workspace_size")
    return n.value


def dv_sparse_attn(y, Wqkv, Wo, kv: KV, pos, head_idx, head_count, scale, out, ws,
                   accumulate=False, stream=None):
    B, d = y.shape
    h, _, d_h, _ = Wqkv.shape
    c = kv.c()
    _ok(lib().dv_sparse_attn(_ptr(y), B, d, h, d_h, _ptr(Wqkv), _ptr(Wo), ctypes.byref(c), _ptr(pos),
                             _ptr(head_idx), head_idx.shape[-1], _ptr(head_count), float(scale),
                             _dt(y), _ptr(out), int(bool(accumulate)), _ptr(ws), ws.numel(),
                             _stream(stream)), "dv_sparse_attn")


def dv_kv_repair(kv: KV, Wqkv, pos, head_idx, head_count, ws, stream=None):
    B = kv.K.shape[0]
    h, _, d_h, d = Wqkv.shape
    c = kv.c()
    _ok(lib().dv_kv_repair(ctypes.byref(c), B, d, h, d_h, _ptr(Wqkv), _ptr(pos), _ptr(head_idx),
                           head_idx.shape[-1], _ptr(head_count), _dt(Wqkv), _ptr(ws), ws.numel(),
                           _stream(stream)), "dv_kv_repair")


# --------------------------------------------------------------------- several candidates per sequence

def dv_tree_attn_workspace_size(B: int, T: int, h: int, group: int, d_h: int) -> int:
    n = ctypes.c_size_t(0)
    _ok(lib().dv_tree_attn_workspace_size(B, T, h, group, d_h, ctypes.byref(n)), "dv_tree_attn_workspace_size")
    return n.value


def dv_tree_attn(q, kv: KV, pos, scale, out, ws, mask=None, nodes=None, head_idx=None, head_count=None, stream=None):
    """q, out [B][T][h g][d_h]; mask [T][T] or [B][T][T], bool or uint8 (None:
    a linear draft); see dv_tree_attn in dv.h."""
    where = "dv_tree_attn"
    K, V = kv.K, kv.V
    shape, cache, dtype = q.shape, K.shape, K.dtype
    B, T, hq, d_h = shape
    h = cache[1]
    _laid_out(q, shape, dtype, where)
    _laid_out(out, shape, dtype, where)
    _laid_out(K, (B, h, kv.n_max, d_h), dtype, where)
    _laid_out(V, cache, dtype, where)
    if hq % h:
        raise DvError(1, where, f"{hq} query heads on {h} K/V heads")
    batched = 0
    if mask is not None:
        batched = int(mask.dim() == 3)
        _laid_out(mask, (B, T, T) if batched else (T, T), torch.bool if mask.dtype == torch.bool else torch.uint8, where)
    _counted(where, B, pos, nodes, head_count)
    if head_idx is not None:
        _counted(where, B * head_idx.shape[-1], head_idx)
    st = (_lib or lib()).dv_tree_attn(
        q.data_ptr(), B, T, h, hq // h, d_h, dv_kv(K.data_ptr(), V.data_ptr(), None, None, kv.n_max), pos.data_ptr(),
        _ptr(nodes), _ptr(mask), batched, _ptr(head_idx), 0 if head_idx is None else head_idx.shape[-1],
        _ptr(head_count), scale, _DT[dtype] if dtype in _DT else _dt(q), out.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream(stream))
    if st:
        _ok(st, where)


def dv_kv_compact(layers: KVLayers, pos, idx, count, ws, new_pos=None, stream=None):
    """Keep nodes idx[b][:count[b]] of each tree (see dv_kv_compact in dv.h)."""
    _counted("dv_kv_compact", layers.B, pos, count, new_pos)
    _counted("dv_kv_compact", layers.B * idx.shape[-1], idx)
    st = (_lib or lib()).dv_kv_compact(
        layers.array, layers.n, layers.B, layers.d, layers.h, layers.d_h, pos.data_ptr(), idx.data_ptr(),
        idx.shape[-1], count.data_ptr(), layers.dt, None if new_pos is None else new_pos.data_ptr(), ws.data_ptr(),
        ws.numel(), _stream(stream))
    if st:
        _ok(st, "dv_kv_compact")


def dv_kv_reorder(layers: KVLayers, pos, parent, ws, start=None, stream=None):
    """Beam w of sequence s (cache row s * width + w) continues beam
    parent[s][w] (see dv_kv_reorder in dv.h)."""
    n_seq, width = parent.shape
    if n_seq * width != layers.B:
        raise DvError(1, "dv_kv_reorder", f"{n_seq} x {width} beams on {layers.B} cache rows")
    _counted("dv_kv_reorder", layers.B, pos, parent)
    if start is not None:
        _counted("dv_kv_reorder", n_seq, start)
    st = (_lib or lib()).dv_kv_reorder(
        layers.array, layers.n, n_seq, width, layers.d, layers.h, layers.d_h, pos.data_ptr(),
        None if start is None else start.data_ptr(), parent.data_ptr(), layers.dt, ws.data_ptr(), ws.numel(),
        _stream(stream))
    if st:
        _ok(st, "dv_kv_reorder")


def dv_beam_select_workspace_size(n_seq: int, width: int, V: int, K: int) -> int:
    n = ctypes.c_size_t(0)
    _ok(lib().dv_beam_select_workspace_size(n_seq, width, V, K, ctypes.byref(n)), "dv_beam_select_workspace_size")
    return n.value


def dv_beam_select(logits, cum, score, token, beam, ws, done=None, end_token=0, stream=None):
    """logits [n_seq][width][V] (rows evenly spaced, tokens adjacent), cum
    [n_seq][width]; score, token, beam [n_seq][K] (see dv_beam_select in dv.h)."""
    S, W, V = logits.shape
    K = score.shape[1]
    s0, s1, s2 = logits.stride()
    if W == 1:
        s1 = s0 if S > 1 else V
    if (V > 1 and s2 != 1) or (S > 1 and s0 != W * s1):
        raise DvError(1, "dv_beam_select", "rows of logits evenly spaced, tokens adjacent")
    _counted("dv_beam_select", S * W, cum, dtype=torch.float32)
    _counted("dv_beam_select", S * K, score, dtype=torch.float32)
    _counted("dv_beam_select", S * K, token, beam)
    if done is not None:
        _counted("dv_beam_select", S * W, done, dtype=torch.bool if done.dtype == torch.bool else torch.uint8)
    st = (_lib or lib()).dv_beam_select(
        logits.data_ptr(), S, W, V, s1, _dt(logits), cum.data_ptr(), None if done is None else done.data_ptr(),
        int(end_token), K, score.data_ptr(), token.data_ptr(), beam.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream(stream))
    if st:
        _ok(st, "dv_beam_select")


# --------------------------------------------------------------------- labels

def dv_label_workspace_size(T: int, d: int, N: int, h: int, d_h: int) -> int:
    n = ctypes.c_size_t(0)
    _ok(lib().dv_label_workspace_size(T, d, N, h, d_h, ctypes.byref(n)), "dv_label_workspace_size")
    return n.value


def dv_label_neurons(X, W1n, norms, ws, stream=None):
    T, d = X.shape
    _ok(lib().dv_label_neurons(_ptr(X), T, d, W1n.shape[0], _ptr(W1n), _dt(X), _ptr(norms), _ptr(ws),
                               ws.numel(), _stream(stream)), "dv_label_neurons")


def dv_label_heads(X, Wqkv, scale, norms, ws, stream=None):
    T, d = X.shape
    h, _, d_h, _ = Wqkv.shape
    _ok(lib().dv_label_heads(_ptr(X), T, d, h, d_h, _ptr(Wqkv), float(scale), _dt(X), _ptr(norms), _ptr(ws),
                             ws.numel(), _stream(stream)), "dv_label_heads")


def dv_select_scores(scores, mode, k, t, idx, count, ws, stream=None):
    B, N = scores.shape
    _ok(lib().dv_select_scores(_ptr(scores), B, N, int(mode), int(k), float(t), _ptr(idx), idx.shape[-1],
                               _ptr(count), _ptr(ws), ws.numel(), _stream(stream)), "dv_select_scores")


# --------------------------------------------------------------------- helpers

def dv_layernorm(x: torch.Tensor, y: torch.Tensor, eps: float = 1e-5, stream=None):
    B, d = x.shape
    _ok(lib().dv_layernorm(_ptr(x), B, d, float(eps), _ptr(y), _dt(y), _stream(stream)),
        "dv_layernorm")


def dv_positions_advance(pos: torch.Tensor, lo: int, hi: int, stream=None):
    _ok(lib().dv_positions_advance(_ptr(pos), pos.numel(), int(lo), int(hi), _stream(stream)),
        "dv_positions_advance")


def dv_set_launch_overlap(level: int) -> int:
    """Process-wide launch policy (see dv_set_launch_overlap in dv.h);
    returns the previous level."""
    return int(lib().dv_set_launch_overlap(int(level)))


def dv_set_wait_limit_ns(ns: int) -> int:
    """Process-wide bound of the device-side waits in nanoseconds (see
    dv_set_wait_limit_ns in dv.h; ns <= 0 restores one second); returns the
    previous bound."""
    return int(lib().dv_set_wait_limit_ns(int(ns)))
