"""Thin Python binding over libmita.so (ctypes).

Names match the C ABI in include/mita.h.  This module only marshals torch
tensors to pointers and picks the bf16 or `_f32` entry point; every step of the
computation runs in the library's CUDA kernels.  There is no fallback: if
libmita.so is missing, every call raises.

Tensors must be contiguous; Q/K/V/out are [B, H, N, d].  Calls run on the
current torch CUDA stream unless `stream` is given.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libmita.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "mita.h")

_lock = threading.Lock()
_lib = None

MITA_OK = 0
MITA_ERR_DEVICE_CHECK = 5


class MitaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[{status}] {message}")
        self.status = status


def load() -> ctypes.CDLL:
    """Load libmita.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m sparse_top_landmark_gb300.build` (there is no CPU fallback)")
            lib = ctypes.CDLL(LIB_PATH)
            P, I = ctypes.c_void_p, ctypes.c_int
            sigs = {
                "mita_pool": [P, I, I, I, I, I, I, I, P, P],
                "mita_landmark_topk_shared": [P, P, P, I, I, I, I, I, I, P, P, P],
                "mita_route": [P, P, P, I, I, I, I, I, I, P, P, P, P],
                "mita_expert_attn": [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P],
                "mita_forward": [P, P, P, I, I, I, I, I, I, I, I, I, P, P],
                "mita_forward_host": [P, P, P, I, I, I, I, I, I, I, I, I, P, P],
                "mita_forward_ex": [P, P, P, I, I, I, I, I, I, I, I, I, P, P, P],
                "mita_pool_grid": [P, I, I, I, I, I, I, I, I, P, P],
                "mita_dense_attn": [P, P, P, I, I, I, I, P, P],
                "mita_backward": [P, P, P, P, I, I, I, I, I, I, I, I, I, P, P, P, P, P],
            }
            I64, U64, F = ctypes.c_int64, ctypes.c_uint64, ctypes.c_float
            sigs.update({
                "mita_qk_norm_rope": [P] * 5 + [I64, P] + [I] * 7 + [F] + [P] * 7,
                "mita_qk_norm_rope_backward": [P] * 7 + [I64, P] + [I] * 7 + [F] + [P] * 7 + [U64]
                                              + [P] * 5,
                "mita_cache_append": [P] * 9 + [I] * 10 + [F] + [P] * 8,
                "mita_paged_attn": [P] * 6 + [I] * 7 + [P, F, F, I, P, U64] + [P] * 3,
            })
            for name, at in sigs.items():
                for suffix in ("", "_f32"):
                    f = getattr(lib, name + suffix)
                    f.argtypes = at
                    f.restype = I
            lib.mita_bucket.argtypes = [P, I, I, I, I, I, P, P, P]
            lib.mita_bucket.restype = I
            lib.mita_bucket_noalloc.argtypes = [P, I, I, I, I, I, P, P, P]
            lib.mita_bucket_noalloc.restype = I
            lib.mita_forward_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I]
            lib.mita_forward_workspace_bytes.restype = ctypes.c_uint64
            lib.mita_qk_norm_rope_backward_workspace_bytes.argtypes = [I]
            lib.mita_qk_norm_rope_backward_workspace_bytes.restype = U64
            lib.mita_paged_attn_workspace_bytes.argtypes = [I] * 7
            lib.mita_paged_attn_workspace_bytes.restype = U64
            lib.mita_status_string.argtypes = [I]
            lib.mita_status_string.restype = ctypes.c_char_p
            lib.mita_last_error_message.argtypes = []
            lib.mita_last_error_message.restype = ctypes.c_char_p
            lib.mita_get_last_device_error.argtypes = [P, ctypes.POINTER(I)]
            lib.mita_get_last_device_error.restype = I
            lib.mita_workspace_release.argtypes = []
            lib.mita_workspace_release.restype = I
            lib.mita_workspace_set_limit.argtypes = [ctypes.c_uint64]
            lib.mita_workspace_set_limit.restype = ctypes.c_uint64
            lib.mita_kernel_launches.argtypes = []
            lib.mita_kernel_launches.restype = ctypes.c_uint64
            lib.mita_check_bounded_wait.argtypes = [P, P]
            lib.mita_check_bounded_wait.restype = I
            _lib = lib
    return _lib


def declared_functions() -> list:
    """Names of every function include/mita.h declares."""
    import re
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(mita_[a-z0-9_]+)\s*\(", text)))


# ---------------------------------------------------------------------------
def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int):
    if rc != MITA_OK:
        lib = load()
        raise MitaError(rc, f"{lib.mita_status_string(rc).decode()}: "
                            f"{lib.mita_last_error_message().decode()}")


def _fn(name: str, dtype: torch.dtype):
    lib = load()
    if dtype == torch.bfloat16:
        return getattr(lib, name)
    if dtype == torch.float32:
        return getattr(lib, name + "_f32")
    raise TypeError(f"unsupported dtype {dtype}: use bfloat16 or float32")


def _need(t: torch.Tensor, name: str, dtype=None, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


class MitaOptions(ctypes.Structure):
    """mita_options of the C header."""
    _fields_ = [("shared_temperature", ctypes.c_int), ("landmark_grid_h", ctypes.c_int),
                ("landmark_grid_w", ctypes.c_int), ("branches", ctypes.c_int)]


SHARED_TEMPERATURES = {"sqrt_d": 0, "d": 1}
BRANCHES = {"both": 0, "routed": 1}


# ---------------------------------------------------------------------------
def mita_pool_grid(q, grid_h: int, grid_w: int, landmark_grid_h: int, landmark_grid_w: int,
                   q_tilde=None, stream=None):
    """Pooling onto an explicit landmark_grid_h x landmark_grid_w landmark grid."""
    _need(q, "q")
    B, H, N, d = q.shape
    m = landmark_grid_h * landmark_grid_w
    if q_tilde is None:
        q_tilde = torch.empty((B, H, m, d), dtype=q.dtype, device=q.device)
    _need(q_tilde, "q_tilde", q.dtype, q.device)
    _check(_fn("mita_pool_grid", q.dtype)(_ptr(q), B, H, N, d, grid_h, grid_w, landmark_grid_h,
                                          landmark_grid_w, _ptr(q_tilde),
                                          _stream(stream, q.device)))
    return q_tilde


def mita_forward_ex(q, k, v, grid_h: int, grid_w: int, m: int, topk: int, s: int = 1,
                    shared_temperature: str = "sqrt_d", landmark_grid=None,
                    branches: str = "both", out=None, stream=None):
    """mita_forward on device tensors with options: the shared logits' temperature
    ("sqrt_d": q.q~/sqrt(d), "d": q.q~/d), an explicit (rows, cols) landmark grid, and
    the branches ("both", or "routed": the routing-only ablation without shared pairs)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, q.device)
    B, H, N, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.dtype, q.device)
    opt = _options(shared_temperature, landmark_grid, branches)
    _check(_fn("mita_forward_ex", q.dtype)(_ptr(q), _ptr(k), _ptr(v), B, H, N, d, grid_h, grid_w,
                                           m, topk, s, ctypes.byref(opt), _ptr(out),
                                           _stream(stream, q.device)))
    return out


def _options(shared_temperature, landmark_grid, branches):
    lh, lw = landmark_grid if landmark_grid is not None else (0, 0)
    return MitaOptions(SHARED_TEMPERATURES[shared_temperature], lh, lw, BRANCHES[branches])


def mita_backward(q, k, v, dout, grid_h: int, grid_w: int, m: int, topk: int, s: int = 1,
                  shared_temperature: str = "sqrt_d", landmark_grid=None, branches: str = "both",
                  stream=None):
    """(dq, dk, dv), fp32, of mita_forward_ex's output for the upstream gradient ``dout``,
    with the forward's selections held constant."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _need(t, n, q.dtype, q.device)
    B, H, N, d = q.shape
    grads = [torch.empty(q.shape, dtype=torch.float32, device=q.device) for _ in range(3)]
    opt = _options(shared_temperature, landmark_grid, branches)
    _check(_fn("mita_backward", q.dtype)(
        _ptr(q), _ptr(k), _ptr(v), _ptr(dout), B, H, N, d, grid_h, grid_w, m, topk, s,
        ctypes.byref(opt), _ptr(grads[0]), _ptr(grads[1]), _ptr(grads[2]),
        _stream(stream, q.device)))
    return tuple(grads)


class MiTAFunction(torch.autograd.Function):
    """MiTA attention as an autograd function: forward through mita_forward_ex, backward
    through mita_backward (selections held constant; gradients cast to the input dtype)."""

    @staticmethod
    def forward(ctx, q, k, v, grid_h, grid_w, m, topk, s=1, shared_temperature="sqrt_d",
                landmark_grid=None, branches="both"):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        ctx.save_for_backward(q, k, v)
        ctx.cfg = (grid_h, grid_w, m, topk, s, shared_temperature, landmark_grid, branches)
        return mita_forward_ex(q, k, v, grid_h, grid_w, m, topk, s, shared_temperature,
                               landmark_grid, branches)

    @staticmethod
    def backward(ctx, dout):
        q, k, v = ctx.saved_tensors
        gh, gw, m, topk, s, temp, lg, br = ctx.cfg
        dq, dk, dv = mita_backward(q, k, v, dout.contiguous().to(q.dtype), gh, gw, m, topk, s,
                                   temp, lg, br)
        return (dq.to(q.dtype), dk.to(k.dtype), dv.to(v.dtype)) + (None,) * 8


# ---------------------------------------------------------------------------
# queries and keys on their way into attention; the paged cache
#
# These calls run on the tensors' device, whatever the current one is, and on `stream` (the
# device's current stream by default).  What they allocate (outputs, workspaces) belongs to that
# stream; the caller orders the stream with the ones its inputs come from.
# ---------------------------------------------------------------------------
class _Launch:
    """The device and stream of one call, as the current ones while it allocates and launches."""

    __slots__ = ("_outer", "handle")

    def __init__(self, stream, device: torch.device):
        self._outer = []
        if device.index != torch.cuda.current_device():
            self._outer.append(torch.cuda.device(device))
        if stream is None:
            self.handle = torch.cuda.current_stream(device).cuda_stream
        else:
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
            self.handle = stream.cuda_stream
            self._outer.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self._outer:
            c.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for c in reversed(self._outer):
            c.__exit__(*exc)


def _need_rows(t: torch.Tensor, name: str, dim: int, dtype=None, device=None, out: bool = False):
    """A CUDA tensor of contiguous rows (its other dimensions may have any strides)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {tuple(t.shape)}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if out and any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride())):
        raise ValueError(f"{name}: an output cannot be a broadcast view")
    return t


def _need_shape(t: torch.Tensor, name: str, shape):
    if t.shape != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _strides(t: torch.Tensor):
    s = t.stride()
    return (ctypes.c_int64 * (len(s) - 1))(*s[:-1])


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need_rope(inv_freq, weights, d: int, device):
    """Checks the frequencies and norm weights; returns the rotated width."""
    for w, name in weights:
        if w is not None:
            _need_shape(_need(w, name, torch.float32, device), name, (d,))
    if inv_freq is None:
        return 0
    _need(inv_freq, "inv_freq", torch.float64, device)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must have one dimension")
    return 2 * inv_freq.shape[0]


def _need_positions(positions, B: int, N: int, device):
    """(address, elements between batches) of positions [N] or [B, N]."""
    if positions is None:
        return None, 0
    if not positions.is_cuda or positions.dtype != torch.int32 or positions.device != device:
        raise TypeError(f"positions must be an int32 tensor on {device}")
    if positions.shape not in ((N,), (B, N)):
        raise ValueError(f"positions must be {(N,)} or {(B, N)}, got {tuple(positions.shape)}")
    if N > 1 and positions.stride(-1) != 1:
        raise ValueError("positions: the last dimension must be contiguous")
    return positions.data_ptr(), positions.stride(0) if positions.dim() == 2 and B > 1 else 0


def _like_rows(x: torch.Tensor) -> torch.Tensor:
    """An empty gradient for x [B, H, N, d]: dense like a dense x, else token-major (the heads of
    a token side by side, as in the projection's output that x is a view of)."""
    if x.is_contiguous():
        return torch.empty_like(x)
    B, H, N, d = x.shape
    return torch.empty((B, N, H, d), dtype=x.dtype, device=x.device).transpose(1, 2)


def mita_qk_norm_rope(q, k=None, inv_freq=None, q_weight=None, k_weight=None, positions=None,
                      eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None,
                      stream=None):
    """RMS norm of every head row of q [B,Hq,N,d] and k [B,Hkv,N,d], then rotation by position, in
    one pass; returns (q_out, k_out), dense [B,H,N,d] unless given (k_out None without k).

    q and k may be strided views, e.g. of one projection's [B,N,Hq+2Hkv,d] output transposed.
    inv_freq: float64 [rot/2], radians per position (None: no rotation; rot a multiple of 8, at
    most d).  q_weight, k_weight: float32 [d] (None: not normalised).  positions: int32 [N] or
    [B,N] (None: 0..N-1).  interleaved: pairs (2i, 2i+1) instead of (i, i + rot/2).
    q_out may be q and k_out may be k."""
    _need_rows(q, "q", 4)
    dev, dt = q.device, q.dtype
    fn = _fn("mita_qk_norm_rope", dt)
    B, Hq, N, d = q.shape
    Hkv = 0
    if k is not None:
        Hkv = _need_rows(k, "k", 4, dt, dev).shape[1]
        _need_shape(k, "k", (B, Hkv, N, d))
    rot = _need_rope(inv_freq, ((q_weight, "q_weight"), (k_weight, "k_weight")), d, dev)
    pos, pos_b = _need_positions(positions, B, N, dev)
    with _Launch(stream, dev) as st:
        if q_out is None:
            q_out = torch.empty((B, Hq, N, d), dtype=dt, device=dev)
        else:
            _need_shape(_need_rows(q_out, "q_out", 4, dt, dev, out=True), "q_out", q.shape)
        if k is None:
            k_out = None
        elif k_out is None:
            k_out = torch.empty((B, Hkv, N, d), dtype=dt, device=dev)
        else:
            _need_shape(_need_rows(k_out, "k_out", 4, dt, dev, out=True), "k_out", k.shape)
        _check(fn(_addr(q), _addr(k), _addr(q_weight), _addr(k_weight), pos, pos_b,
                  _addr(inv_freq), B, Hq, Hkv, N, d, rot, int(interleaved), eps, _strides(q),
                  None if k is None else _strides(k), _strides(q_out),
                  None if k is None else _strides(k_out), _addr(q_out), _addr(k_out), st))
    return q_out, k_out


def mita_qk_norm_rope_backward(q, k, dq_out, dk_out, inv_freq=None, q_weight=None, k_weight=None,
                               positions=None, eps: float = 1e-6, interleaved: bool = False,
                               dq=None, dk=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of mita_qk_norm_rope for the gradients dq_out, dk_out of its
    outputs.  dq and dk have the inputs' type, and unless given are dense where q is and token-major
    ([B,N,H,d] in memory) where it is a view; the weights' gradients are float32 (None
    without the weight).  k and dk_out may both be None.  dq may be dq_out, dk may be dk_out."""
    _need_rows(q, "q", 4)
    dev, dt = q.device, q.dtype
    fn = _fn("mita_qk_norm_rope_backward", dt)
    B, Hq, N, d = q.shape
    _need_shape(_need_rows(dq_out, "dq_out", 4, dt, dev), "dq_out", q.shape)
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out: both or neither")
    Hkv = 0
    if k is not None:
        Hkv = _need_rows(k, "k", 4, dt, dev).shape[1]
        _need_shape(k, "k", (B, Hkv, N, d))
        _need_shape(_need_rows(dk_out, "dk_out", 4, dt, dev), "dk_out", k.shape)
    else:
        k_weight = None
    rot = _need_rope(inv_freq, ((q_weight, "q_weight"), (k_weight, "k_weight")), d, dev)
    pos, pos_b = _need_positions(positions, B, N, dev)
    with _Launch(stream, dev) as st:
        if dq is None:
            dq = _like_rows(q)
        else:
            _need_shape(_need_rows(dq, "dq", 4, dt, dev, out=True), "dq", q.shape)
        if k is None:
            dk = None
        elif dk is None:
            dk = _like_rows(k)
        else:
            _need_shape(_need_rows(dk, "dk", 4, dt, dev, out=True), "dk", k.shape)
        dwq, dwk = (None if w is None else torch.empty(d, dtype=torch.float32, device=dev)
                    for w in (q_weight, k_weight))
        ws, nbytes = None, 0
        if dwq is not None or dwk is not None:
            nbytes = load().mita_qk_norm_rope_backward_workspace_bytes(d)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _check(fn(_addr(q), _addr(k), _addr(dq_out), _addr(dk_out), _addr(q_weight),
                  _addr(k_weight), pos, pos_b, _addr(inv_freq), B, Hq, Hkv, N, d, rot,
                  int(interleaved), eps, _strides(q), None if k is None else _strides(k),
                  _strides(dq_out), None if k is None else _strides(dk_out), _strides(dq),
                  None if k is None else _strides(dk), _addr(ws), nbytes, _addr(dq), _addr(dk),
                  _addr(dwq), _addr(dwk), st))
    return dq, dk, dwq, dwk


class QKNormRopeFunction(torch.autograd.Function):
    """mita_qk_norm_rope as an autograd function: gradients of q, k and the norm weights.
    To capture its backward into a CUDA graph, make the leaves and run forward and
    backward inside the capture (or call mita_qk_norm_rope_backward): a backward captured while an
    eager graph of the same leaves is alive accumulates on the eager graph's stream."""

    @staticmethod
    def forward(ctx, q, k, inv_freq=None, q_weight=None, k_weight=None, positions=None, eps=1e-6,
                interleaved=False):
        ctx.save_for_backward(q, k, inv_freq, q_weight, k_weight, positions)
        ctx.cfg = (eps, interleaved)
        return mita_qk_norm_rope(q, k, inv_freq, q_weight, k_weight, positions, eps, interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, inv_freq, q_weight, k_weight, positions = ctx.saved_tensors
        eps, interleaved = ctx.cfg
        dq, dk, dwq, dwk = mita_qk_norm_rope_backward(
            q, k, _rows_of(dq_out), None if k is None else _rows_of(dk_out), inv_freq, q_weight,
            k_weight, positions, eps, interleaved)
        return dq, dk, None, dwq, dwk, None, None, None


def _rows_of(t: torch.Tensor) -> torch.Tensor:
    """t itself where its rows can be read as they lie, else a dense copy (broadcast gradients)."""
    step = 16 // t.element_size()
    ok = t.stride(-1) == 1 and all(n == 1 or s % step == 0
                                   for n, s in zip(t.shape[:-1], t.stride()[:-1]))
    return t if ok and t.data_ptr() % 16 == 0 else t.contiguous()


def _need_cache(k_cache, v_cache, page_table, lengths, dtype, device):
    """(S, num_pages, Hkv, page_size, d, table width) of a paged cache."""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, name, dtype, device)
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must be [num_pages, Hkv, page_size, d]")
    _need(page_table, "page_table", torch.int32, device)
    _need(lengths, "lengths", torch.int32, device)
    if page_table.dim() != 2 or lengths.shape != (page_table.shape[0],):
        raise ValueError("page_table must be [S, width] and lengths [S]")
    pages, Hkv, page, d = k_cache.shape
    return page_table.shape[0], pages, Hkv, page, d, page_table.shape[1]


def mita_cache_append(k, v, k_cache, v_cache, page_table, lengths, seq_start=None, q=None,
                      inv_freq=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                      interleaved: bool = False, q_out=None, stream=None):
    """New tokens into a paged cache: k [T,Hkv,d] normalised and rotated (as by
    mita_qk_norm_rope, at its position in its sequence) and v [T,Hkv,d] to their rows of
    k_cache, v_cache [num_pages,Hkv,page_size,d]; returns q [T,Hq,d] normalised and rotated (None
    without q; in q_out where given).  k, v, q and q_out may be strided views.

    page_table: int32 [S,width]; lengths: int32 [S], tokens of each sequence with the new
    ones (0: an idle slot, nothing is written for it); seq_start: int32 [S+1], the rows of each
    sequence's new tokens (None: row s is sequence s's only one).  Rows that belong to no sequence
    or to an idle slot leave q_out as it is."""
    _need_rows(k, "k", 3)
    dev, dt = k.device, k.dtype
    fn = _fn("mita_cache_append", dt)
    S, pages, Hkv, page, d, width = _need_cache(k_cache, v_cache, page_table, lengths, dt, dev)
    T = k.shape[0]
    _need_shape(k, "k", (T, Hkv, d))
    _need_shape(_need_rows(v, "v", 3, dt, dev), "v", (T, Hkv, d))
    if seq_start is not None:
        _need_shape(_need(seq_start, "seq_start", torch.int32, dev), "seq_start", (S + 1,))
    Hq = 0
    if q is not None:
        Hq = _need_rows(q, "q", 3, dt, dev).shape[1]
        _need_shape(q, "q", (T, Hq, d))
    rot = _need_rope(inv_freq, ((q_weight, "q_weight"), (k_weight, "k_weight")), d, dev)
    with _Launch(stream, dev) as st:
        if q is None:
            q_out = None
        elif q_out is None:
            q_out = torch.empty((T, Hq, d), dtype=dt, device=dev)
        else:
            _need_shape(_need_rows(q_out, "q_out", 3, dt, dev, out=True), "q_out", q.shape)
        _check(fn(_addr(q), _addr(k), _addr(v), _addr(q_weight), _addr(k_weight), _addr(inv_freq),
                  _addr(page_table), _addr(lengths), _addr(seq_start), T, S, Hq, Hkv, d, pages,
                  page, width, rot, int(interleaved), eps, None if q is None else _strides(q),
                  _strides(k), _strides(v), None if q is None else _strides(q_out), _addr(q_out),
                  _addr(k_cache), _addr(v_cache), st))
    return q_out


def mita_paged_attn(q, k_cache, v_cache, page_table, lengths, scale: Optional[float] = None,
                    softcap: float = 0.0, window: int = 0, alibi_slopes=None,
                    return_lse: bool = False, out=None, stream=None):
    """Attention of one new token per sequence over the paged cache (layout and lengths as for
    mita_cache_append, the new token's key included): q [S,Hq,d], may be a strided view; returns
    out [S,Hq,d], with return_lse (out, lse [S,Hq] float32).

    scale: of the scores (None: d^-1/2).  softcap > 0: scores capped to softcap*tanh(z/softcap).
    alibi_slopes: float32 [Hq], adds slope*(key position - own position).  window > 0: only the
    last `window` keys.  Idle slots (length 0) get zeros and lse -inf."""
    _need_rows(q, "q", 3)
    dev, dt = q.device, q.dtype
    fn = _fn("mita_paged_attn", dt)
    S, pages, Hkv, page, d, width = _need_cache(k_cache, v_cache, page_table, lengths, dt, dev)
    Hq = q.shape[1]
    _need_shape(q, "q", (S, Hq, d))
    if alibi_slopes is not None:
        _need_shape(_need(alibi_slopes, "alibi_slopes", torch.float32, dev), "alibi_slopes", (Hq,))
    with _Launch(stream, dev) as st:
        if out is None:
            out = torch.empty((S, Hq, d), dtype=dt, device=dev)
        else:
            _need_shape(_need(out, "out", dt, dev), "out", q.shape)
        lse = torch.empty((S, Hq), dtype=torch.float32, device=dev) if return_lse else None
        nbytes = load().mita_paged_attn_workspace_bytes(S, Hq, Hkv, d, page, width,
                                                        int(dt == torch.float32))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _check(fn(_addr(q), _addr(k_cache), _addr(v_cache), _addr(page_table), _addr(lengths),
                  _addr(alibi_slopes), S, Hq, Hkv, d, pages, page, width, _strides(q),
                  d ** -0.5 if scale is None else scale, softcap, window, _addr(ws), nbytes,
                  _addr(out), _addr(lse), st))
    return (out, lse) if return_lse else out


def mita_dense_attn(q, k, v, out=None, stream=None):
    """Dense softmax attention over all N keys of each head (the comparison baseline)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, q.device)
    B, H, N, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.dtype, q.device)
    _check(_fn("mita_dense_attn", q.dtype)(_ptr(q), _ptr(k), _ptr(v), B, H, N, d, _ptr(out),
                                           _stream(stream, q.device)))
    return out


def mita_pool(q, grid_h: int, grid_w: int, m: int, q_tilde=None, stream=None):
    _need(q, "q")
    B, H, N, d = q.shape
    if q_tilde is None:
        q_tilde = torch.empty((B, H, m, d), dtype=q.dtype, device=q.device)
    _need(q_tilde, "q_tilde", q.dtype, q.device)
    _check(_fn("mita_pool", q.dtype)(_ptr(q), B, H, N, d, grid_h, grid_w, m, _ptr(q_tilde),
                                     _stream(stream, q.device)))
    return q_tilde


def mita_landmark_topk_shared(q_tilde, k, v, topk: int, topk_idx=None, v_tilde=None,
                              stream=None):
    for t, n in ((q_tilde, "q_tilde"), (k, "k"), (v, "v")):
        _need(t, n, k.dtype, k.device)
    B, H, N, d = k.shape
    m = q_tilde.shape[2]
    if topk_idx is None:
        topk_idx = torch.empty((B, H, m, topk), dtype=torch.int32, device=k.device)
    if v_tilde is None:
        v_tilde = torch.empty((B, H, m, d), dtype=torch.float32, device=k.device)
    _need(topk_idx, "topk_idx", torch.int32, k.device)
    _need(v_tilde, "v_tilde", torch.float32, k.device)
    _check(_fn("mita_landmark_topk_shared", k.dtype)(
        _ptr(q_tilde), _ptr(k), _ptr(v), B, H, N, d, m, topk, _ptr(topk_idx), _ptr(v_tilde),
        _stream(stream, k.device)))
    return topk_idx, v_tilde


def mita_route(q, q_tilde, v_tilde=None, s: int = 1, route_idx=None, shared: bool = False,
               stream=None):
    _need(q, "q")
    _need(q_tilde, "q_tilde", q.dtype, q.device)
    B, H, N, d = q.shape
    m = q_tilde.shape[2]
    if route_idx is None:
        route_idx = torch.empty((B, H, N, s), dtype=torch.int32, device=q.device)
    _need(route_idx, "route_idx", torch.int32, q.device)
    lse = o = None
    if shared:
        _need(v_tilde, "v_tilde", torch.float32, q.device)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
        o = torch.empty((B, H, N, d), dtype=torch.float32, device=q.device)
    _check(_fn("mita_route", q.dtype)(
        _ptr(q), _ptr(q_tilde), _ptr(v_tilde), B, H, N, d, m, s, _ptr(route_idx), _ptr(lse),
        _ptr(o), _stream(stream, q.device)))
    return (route_idx, lse, o) if shared else route_idx


def mita_bucket(route_idx, m: int, bucket_off=None, bucket_qidx=None, stream=None):
    _need(route_idx, "route_idx", torch.int32)
    B, H, N, s = route_idx.shape
    if bucket_off is None:
        bucket_off = torch.empty((B, H, m + 1), dtype=torch.int32, device=route_idx.device)
    if bucket_qidx is None:
        bucket_qidx = torch.empty((B, H, N * s), dtype=torch.int32, device=route_idx.device)
    _need(bucket_off, "bucket_off", torch.int32, route_idx.device)
    _need(bucket_qidx, "bucket_qidx", torch.int32, route_idx.device)
    _check(load().mita_bucket(_ptr(route_idx), B, H, N, m, s, _ptr(bucket_off),
                              _ptr(bucket_qidx), _stream(stream, route_idx.device)))
    return bucket_off, bucket_qidx


def mita_bucket_noalloc(route_idx, m: int, bucket_off, bucket_qidx, stream=None):
    """mita_bucket for callers that cannot allocate device memory: the caller
    passes both outputs, and the library uses its fixed 4 MiB device scratch
    instead of its workspace cache (limit B*H*(ceil(N*s/4096)+1)*m <= 1048576).
    Calls that overlap on the GPU race on that scratch; order them."""
    _need(route_idx, "route_idx", torch.int32)
    B, H, N, s = route_idx.shape
    _need(bucket_off, "bucket_off", torch.int32, route_idx.device)
    _need(bucket_qidx, "bucket_qidx", torch.int32, route_idx.device)
    _check(load().mita_bucket_noalloc(_ptr(route_idx), B, H, N, m, s, _ptr(bucket_off),
                                      _ptr(bucket_qidx), _stream(stream, route_idx.device)))
    return bucket_off, bucket_qidx


def mita_expert_attn(q, k, v, q_tilde, v_tilde, topk_idx, bucket_off, bucket_qidx,
                     shared_lse=None, shared_o=None, s: int = 1, out=None, stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, q.device)
    B, H, N, d = q.shape
    m, topk = topk_idx.shape[-2], topk_idx.shape[-1]
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.dtype, q.device)
    for t, n in ((topk_idx, "topk_idx"), (bucket_off, "bucket_off"), (bucket_qidx, "bucket_qidx")):
        _need(t, n, torch.int32, q.device)
    if bucket_qidx.numel() != B * H * N * s:
        raise ValueError(f"bucket_qidx holds {bucket_qidx.numel()} entries, expected B*H*N*s = "
                         f"{B * H * N * s}")
    if q_tilde is not None:
        _need(q_tilde, "q_tilde", q.dtype, q.device)
    if v_tilde is not None:
        _need(v_tilde, "v_tilde", torch.float32, q.device)
    _check(_fn("mita_expert_attn", q.dtype)(
        _ptr(q), _ptr(k), _ptr(v), _ptr(q_tilde), _ptr(v_tilde), _ptr(topk_idx),
        _ptr(bucket_off), _ptr(bucket_qidx), _ptr(shared_lse), _ptr(shared_o), B, H, N, d, m,
        topk, s, _ptr(out), _stream(stream, q.device)))
    return out


def mita_forward(q, k, v, grid_h: int, grid_w: int, m: int, topk: int, s: int = 1, out=None,
                 stream=None, device=None):
    """The whole forward pass.

    Device tensors: runs on the GPU and returns the device output.  Host
    tensors (ideally pinned) go through the library's host entry point, which
    copies Q, K, V to `device` (default cuda:0), runs, copies the output back
    into `out` (or a new pinned tensor) and synchronises before returning.
    """
    if not q.is_cuda:
        # host buffers: the library copies in, runs and copies out (one C call)
        dev = torch.device(device if device is not None else "cuda:0")
        for t, n in ((q, "q"), (k, "k"), (v, "v")):
            if t.is_cuda or t.dtype != q.dtype or t.shape != q.shape or not t.is_contiguous():
                raise ValueError(f"{n}: expected a contiguous host tensor like q")
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
        if out.is_cuda or out.dtype != q.dtype or out.shape != q.shape or not out.is_contiguous():
            raise ValueError("out: expected a contiguous host tensor like q")
        B, H, N, d = q.shape
        with torch.cuda.device(dev):
            _check(_fn("mita_forward_host", q.dtype)(
                _ptr(q), _ptr(k), _ptr(v), B, H, N, d, grid_h, grid_w, m, topk, s, _ptr(out),
                _stream(stream, dev)))
        return out
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, q.device)
    B, H, N, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.dtype, q.device)
    _check(_fn("mita_forward", q.dtype)(_ptr(q), _ptr(k), _ptr(v), B, H, N, d, grid_h, grid_w,
                                        m, topk, s, _ptr(out), _stream(stream, q.device)))
    return out


def forward_workspace_bytes(B, H, N, d, m, topk, dtype=torch.bfloat16, s: int = 1) -> int:
    return int(load().mita_forward_workspace_bytes(B, H, N, d, m, topk, s,
                                                    1 if dtype == torch.float32 else 0))


def get_last_device_error(stream=None, device=None) -> int:
    """Synchronise and return (and clear) the device status bits (0 = clean)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    bits = ctypes.c_int(0)
    rc = load().mita_get_last_device_error(_stream(stream, dev), ctypes.byref(bits))
    if rc not in (MITA_OK, MITA_ERR_DEVICE_CHECK):
        _check(rc)
    return bits.value


def workspace_release() -> None:
    _check(load().mita_workspace_release())


def workspace_set_limit(nbytes: int) -> int:
    """Cap the growth of each cached buffer (0: no cap); returns the previous cap.  Growth past
    it raises MitaError(MITA_ERR_OOM) before any allocation."""
    return int(load().mita_workspace_set_limit(int(nbytes)))


def kernel_launches() -> int:
    """Kernel launches this library has issued in this process so far."""
    return int(load().mita_kernel_launches())


def check_bounded_wait(stream=None, device=None) -> torch.Tensor:
    """Runs the library's wait-timeout probe (mita_check_bounded_wait): a kernel whose
    two bounded waits on a never-arrived mbarrier must give up after about a second.
    Returns the device int32[2] gave-up flags (1 = that wait gave up)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    gave_up = torch.full((2,), -1, dtype=torch.int32, device=dev)
    _check(load().mita_check_bounded_wait(_ptr(gave_up), _stream(stream, dev)))
    return gave_up
