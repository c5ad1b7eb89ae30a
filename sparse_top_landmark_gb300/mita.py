"""Thin Python binding over libmita.so (ctypes).

Names match the C ABI in include/mita.h.  This module only marshals torch
tensors to pointers and picks the bf16 or `_f32` entry point; every step of the
computation runs in the library's CUDA kernels.  There is no fallback: if
libmita.so is missing, every call raises.

Tensors must be contiguous; Q/K/V/out are [B, H, N, d].  (The norm and rotation of
queries and keys and the paged cache take strided views and packed tokens: their
docstrings say which.)  Calls run on the current torch CUDA stream unless `stream`
is given.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import struct
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
            # arguments in a struct, packed by the caller
            U64 = ctypes.c_uint64
            for name in ("mita_qk_norm_rope", "mita_qk_norm_rope_backward",
                         "mita_qk_norm_rope_axes", "mita_qk_norm_rope_axes_backward",
                         "mita_cache_append", "mita_paged_attn", "mita_cache_append_q4",
                         "mita_paged_attn_q4"):
                sigs[name] = [ctypes.c_char_p, P]
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
            for name in ("mita_paged_attn_workspace_bytes", "mita_paged_attn_q4_workspace_bytes"):
                getattr(lib, name).argtypes = [I] * 7
                getattr(lib, name).restype = U64
            lib.mita_cache_plan.argtypes = [ctypes.c_char_p, P]
            lib.mita_cache_plan.restype = I
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
# stream; the caller orders the stream with the ones its inputs come from and its outputs go to.
#
# A step of a decoder makes a few of these calls for microseconds of GPU work, so the binding's
# own time counts: arguments go to C as one packed struct (the layouts below are the
# header's *_params), and tensors are checked with as few attribute reads as it takes.
# ---------------------------------------------------------------------------
_NORM_ROPE = struct.Struct("8P13q7if")
_NORM_ROPE_BACKWARD = struct.Struct("13PQ19q7if")
_CACHE_APPEND = struct.Struct("12P8q10if4x")
_PAGED_ATTN = struct.Struct("9PQ2q8i2f")
_NORM_ROPE_AXES = struct.Struct("9P14q8if4x")
_NORM_ROPE_AXES_BACKWARD = struct.Struct("14PQ20q8if4x")
_CACHE_PLAN = struct.Struct("11P5i4x")
_CACHE_APPEND_Q4 = struct.Struct("7P8q5i4x")
_NO_STRIDES = (0, 0, 0)

_typed = {}


def _typed_fn(name: str, dtype: torch.dtype):
    fn = _typed.get((name, dtype))
    if fn is None:
        fn = _typed[name, dtype] = _fn(name, dtype)
    return fn


class _on:
    """`device` and `stream` (or its current stream) as the current ones; the tensors that a given
    stream's call uses stay allocated until that stream is done with them."""

    def __init__(self, stream, device: int, *tensors):
        if stream is not None and stream.device_index != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{device}")
        self._stack = contextlib.ExitStack()
        self._enter = (torch.cuda.device(device), torch.cuda.stream(stream))
        self._stream, self._tensors = stream, tensors

    def __enter__(self):
        for c in self._enter:
            self._stack.enter_context(c)

    def __exit__(self, *exc):
        if self._stream is not None and not torch.cuda.is_current_stream_capturing():
            for t in self._tensors:
                if t is not None and t.is_cuda:
                    t.record_stream(self._stream)
        return self._stack.__exit__(*exc)


def _device_of(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _refuse(t: torch.Tensor, name: str, shape, dtype, device: int, layout: str):
    """Raises what is wrong with a tensor that _rows or _dense does not take."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: {layout}")


def _rows(t: torch.Tensor, name: str, shape, dtype, device: int):
    """Checks a strided input of contiguous rows; returns the strides of its other dimensions."""
    s = t.stride()
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or s[-1] != 1:
        _refuse(t, name, shape, dtype, device, "the last dimension must be contiguous")
    return s[:-1]


def _out_rows(t: torch.Tensor, name: str, shape, dtype, device: int):
    """_rows of an output that the caller gave."""
    s = _rows(t, name, shape, dtype, device)
    if 0 in s and any(n > 1 and step == 0 for n, step in zip(shape, s)):
        raise ValueError(f"{name}: an output cannot be a broadcast view")
    return s


def _dense_strides(H: int, N: int, d: int):
    return (H * N * d, N * d, d)


def _dense(t: torch.Tensor, name: str, shape, dtype, device: int):
    """Checks a contiguous tensor; returns its address."""
    if (t.dtype is not dtype or t.get_device() != device or t.shape != shape
            or not t.is_contiguous()):
        _refuse(t, name, shape, dtype, device, "must be contiguous")
    return t.data_ptr()


def _rope_of(inv_freq, device: int):
    """(address, rotated width) of the frequencies."""
    if inv_freq is None:
        return 0, 0
    n = inv_freq.numel()
    return _dense(inv_freq, "inv_freq", (n,), torch.float64, device), 2 * n


def _weight(w, name: str, d: int, device: int):
    return 0 if w is None else _dense(w, name, (d,), torch.float32, device)


def _positions_of(positions, B: int, N: int, device: int):
    """(address, elements between batches) of positions [N] or [B, N]."""
    if positions is None:
        return 0, 0
    if positions.dim() == 2:
        step, = _rows(positions, "positions", (B, N), torch.int32, device)
        return positions.data_ptr(), step if B > 1 else 0
    return _dense(positions, "positions", (N,), torch.int32, device), 0


def _axes_of(positions, freq_axis, rot: int, B: int, N: int, device: int):
    """(addresses of positions [axes, N] or [axes, B, N] and of freq_axis, elements between batches
    and between axes, axes)."""
    A = positions.shape[0]
    if positions.dim() == 3:
        a, b = _rows(positions, "positions", (A, B, N), torch.int32, device)
    else:
        a, = _rows(positions, "positions", (A, N), torch.int32, device)
        b = 0
    faxis = 0 if rot == 0 else _dense(freq_axis, "freq_axis", (rot // 2,), torch.int32, device)
    return positions.data_ptr(), faxis, b if B > 1 else 0, a if A > 1 else 0, A


def _like_rows(x: torch.Tensor, shape):
    """An empty gradient for x [B, H, N, d] and its strides: dense like a dense x, else token-major
    (the heads of a token side by side, as in the projection's output that x is a view of)."""
    B, H, N, d = shape
    s = _dense_strides(H, N, d) if x.is_contiguous() else (N * H * d, d, H * d)
    return torch.empty_strided(shape, s + (1,), dtype=x.dtype, device=x.device), s


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
    return _norm_rope(q, k, inv_freq, None, q_weight, k_weight, positions, eps, interleaved, q_out,
                      k_out, stream)


def mita_qk_norm_rope_axes(q, k, inv_freq, freq_axis, positions, q_weight=None, k_weight=None,
                           eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None,
                           stream=None):
    """mita_qk_norm_rope for tokens that stand somewhere on several axes (rows and columns of an image;
    time, rows and columns of a video): frequency i turns its pair by the angle
    positions[freq_axis[i]] * inv_freq[i].

    positions: int32 [axes,N] or [axes,B,N].  freq_axis: int32 [rot/2], the axis of each frequency, in
    any order (sections, or dealt in turn).  k may be None.  The rest as for mita_qk_norm_rope."""
    if positions is None or (freq_axis is None and inv_freq is not None):
        raise ValueError("positions and freq_axis are needed: the axes that the frequencies turn with")
    return _norm_rope(q, k, inv_freq, (freq_axis,), q_weight, k_weight, positions, eps, interleaved,
                      q_out, k_out, stream)


def _norm_rope(q, k, inv_freq, axes, q_weight, k_weight, positions, eps, interleaved, q_out, k_out,
               stream):
    """Both forms; axes: None, or (freq_axis,) for positions of several axes."""
    dev = _device_of(q, "q")
    if stream is not None or dev != torch.cuda.current_device():
        with _on(stream, dev, q, k, inv_freq, q_weight, k_weight, positions, q_out, k_out,
                 *(axes or ())):
            return _norm_rope(q, k, inv_freq, axes, q_weight, k_weight, positions, eps, interleaved,
                              q_out, k_out, None)
    dt = q.dtype
    fn = _typed_fn("mita_qk_norm_rope" if axes is None else "mita_qk_norm_rope_axes", dt)
    shape = B, Hq, N, d = q.shape
    qs = _rows(q, "q", shape, dt, dev)
    freq, rot = _rope_of(inv_freq, dev)
    if axes is None:
        pos, pos_b = _positions_of(positions, B, N, dev)
    else:
        pos, faxis, pos_b, pos_a, A = _axes_of(positions, axes[0], rot, B, N, dev)
    qw, kw = _weight(q_weight, "q_weight", d, dev), _weight(k_weight, "k_weight", d, dev)
    if q_out is None:
        q_out = torch.empty(shape, dtype=dt, device=q.device)
        qos = _dense_strides(Hq, N, d)
    else:
        qos = _out_rows(q_out, "q_out", shape, dt, dev)
    Hkv = kp = kop = 0
    ks = kos = _NO_STRIDES
    if k is None:
        k_out = None
    else:
        Hkv = k.shape[1]
        kshape = (B, Hkv, N, d)
        ks = _rows(k, "k", kshape, dt, dev)
        if k_out is None:
            k_out = torch.empty(kshape, dtype=dt, device=q.device)
            kos = _dense_strides(Hkv, N, d)
        else:
            kos = _out_rows(k_out, "k_out", kshape, dt, dev)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    if axes is None:
        args = _NORM_ROPE.pack(q.data_ptr(), kp, qw, kw, pos, freq, q_out.data_ptr(), kop, *qs, *ks,
                               *qos, *kos, pos_b, B, Hq, Hkv, N, d, rot, interleaved, eps)
    else:
        args = _NORM_ROPE_AXES.pack(q.data_ptr(), kp, qw, kw, pos, faxis, freq, q_out.data_ptr(), kop,
                                    *qs, *ks, *qos, *kos, pos_b, pos_a, B, Hq, Hkv, N, d, rot,
                                    interleaved, A, eps)
    rc = fn(args, _raw_stream(dev))
    if rc:
        _check(rc)
    return q_out, k_out


def mita_qk_norm_rope_backward(q, k, dq_out, dk_out, inv_freq=None, q_weight=None, k_weight=None,
                               positions=None, eps: float = 1e-6, interleaved: bool = False,
                               dq=None, dk=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of mita_qk_norm_rope for the gradients dq_out, dk_out of its
    outputs.  dq and dk have the inputs' type, and unless given are dense where q is and token-major
    ([B,N,H,d] in memory) where it is a view; the weights' gradients are float32 (None
    without the weight).  k and dk_out may both be None.  dq may be dq_out, dk may be dk_out."""
    return _norm_rope_backward(q, k, dq_out, dk_out, inv_freq, None, q_weight, k_weight, positions,
                               eps, interleaved, dq, dk, stream)


def mita_qk_norm_rope_axes_backward(q, k, dq_out, dk_out, inv_freq, freq_axis, positions,
                                    q_weight=None, k_weight=None, eps: float = 1e-6,
                                    interleaved: bool = False, dq=None, dk=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of mita_qk_norm_rope_axes, as mita_qk_norm_rope_backward gives
    them for mita_qk_norm_rope."""
    if positions is None or (freq_axis is None and inv_freq is not None):
        raise ValueError("positions and freq_axis are needed: the axes that the frequencies turn with")
    return _norm_rope_backward(q, k, dq_out, dk_out, inv_freq, (freq_axis,), q_weight, k_weight,
                               positions, eps, interleaved, dq, dk, stream)


def _norm_rope_backward(q, k, dq_out, dk_out, inv_freq, axes, q_weight, k_weight, positions, eps,
                        interleaved, dq, dk, stream):
    """Both forms; axes: None, or (freq_axis,) for positions of several axes."""
    dev = _device_of(q, "q")
    if stream is not None or dev != torch.cuda.current_device():
        with _on(stream, dev, q, k, dq_out, dk_out, inv_freq, q_weight, k_weight, positions, dq,
                 dk, *(axes or ())):
            return _norm_rope_backward(q, k, dq_out, dk_out, inv_freq, axes, q_weight, k_weight,
                                       positions, eps, interleaved, dq, dk, None)
    dt = q.dtype
    fn = _typed_fn("mita_qk_norm_rope_backward" if axes is None
                   else "mita_qk_norm_rope_axes_backward", dt)
    shape = B, Hq, N, d = q.shape
    qs = _rows(q, "q", shape, dt, dev)
    dqos = _rows(dq_out, "dq_out", shape, dt, dev)
    freq, rot = _rope_of(inv_freq, dev)
    if axes is None:
        pos, pos_b = _positions_of(positions, B, N, dev)
    else:
        pos, faxis, pos_b, pos_a, A = _axes_of(positions, axes[0], rot, B, N, dev)
    if dq is None:
        dq, dqs = _like_rows(q, shape)
    else:
        dqs = _out_rows(dq, "dq", shape, dt, dev)
    Hkv = kp = dkop = dkp = 0
    ks = dkos = dks = _NO_STRIDES
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out: both or neither")
    if k is None:
        dk = k_weight = None
    else:
        Hkv = k.shape[1]
        kshape = (B, Hkv, N, d)
        ks = _rows(k, "k", kshape, dt, dev)
        dkos = _rows(dk_out, "dk_out", kshape, dt, dev)
        if dk is None:
            dk, dks = _like_rows(k, kshape)
        else:
            dks = _out_rows(dk, "dk", kshape, dt, dev)
        kp, dkop, dkp = k.data_ptr(), dk_out.data_ptr(), dk.data_ptr()
    qw, kw = _weight(q_weight, "q_weight", d, dev), _weight(k_weight, "k_weight", d, dev)
    dwq = dwk = ws = None
    nbytes = 0
    if qw or kw:
        # for this call alone: it launches twice, and another thread's call on the same stream may
        # come in between (one kept for each thread and stream took 1.5 us less of 42 and outlived its
        # thread's and stream's use)
        nbytes = _norm_rope_backward_bytes(d, dev)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        dwq = torch.empty(d, dtype=torch.float32, device=q.device) if qw else None
        dwk = torch.empty(d, dtype=torch.float32, device=q.device) if kw else None
    grads = (dq.data_ptr(), dkp, dwq.data_ptr() if qw else 0, dwk.data_ptr() if kw else 0,
             ws.data_ptr() if nbytes else 0, nbytes)
    strides = (*qs, *ks, *dqos, *dkos, *dqs, *dks, pos_b)
    if axes is None:
        args = _NORM_ROPE_BACKWARD.pack(q.data_ptr(), kp, dq_out.data_ptr(), dkop, qw, kw, pos, freq,
                                        *grads, *strides, B, Hq, Hkv, N, d, rot, interleaved, eps)
    else:
        args = _NORM_ROPE_AXES_BACKWARD.pack(q.data_ptr(), kp, dq_out.data_ptr(), dkop, qw, kw, pos,
                                             faxis, freq, *grads, *strides, pos_a, B, Hq, Hkv, N, d,
                                             rot, interleaved, A, eps)
    rc = fn(args, _raw_stream(dev))
    if rc:
        _check(rc)
    return dq, dk, dwq, dwk


@functools.lru_cache(maxsize=None)
def _norm_rope_backward_bytes(d: int, device: int) -> int:
    return load().mita_qk_norm_rope_backward_workspace_bytes(d)


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
            q, k, _aligned_rows(dq_out), None if k is None else _aligned_rows(dk_out), inv_freq,
            q_weight, k_weight, positions, eps, interleaved)
        return dq, dk, None, dwq, dwk, None, None, None


class QKNormRopeAxesFunction(torch.autograd.Function):
    """mita_qk_norm_rope_axes as an autograd function: gradients of q, k and the norm weights.  For
    capture into a CUDA graph as QKNormRopeFunction."""

    @staticmethod
    def forward(ctx, q, k, inv_freq, freq_axis, positions, q_weight=None, k_weight=None, eps=1e-6,
                interleaved=False):
        ctx.save_for_backward(q, k, inv_freq, freq_axis, positions, q_weight, k_weight)
        ctx.cfg = (eps, interleaved)
        return mita_qk_norm_rope_axes(q, k, inv_freq, freq_axis, positions, q_weight, k_weight, eps,
                                      interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, inv_freq, freq_axis, positions, q_weight, k_weight = ctx.saved_tensors
        dq, dk, dwq, dwk = mita_qk_norm_rope_axes_backward(
            q, k, _aligned_rows(dq_out), None if k is None else _aligned_rows(dk_out), inv_freq,
            freq_axis, positions, q_weight, k_weight, *ctx.cfg)
        return dq, dk, None, None, None, dwq, dwk, None, None


def _aligned_rows(t: torch.Tensor) -> torch.Tensor:
    """t itself where its rows can be read as they lie, else a dense copy."""
    step = 16 // t.element_size()
    ok = t.stride(-1) == 1 and all(n == 1 or s % step == 0
                                   for n, s in zip(t.shape[:-1], t.stride()[:-1]))
    if ok and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)   # contiguous() may return t itself


def _cache_of(k_cache, v_cache, page_table, lengths, dtype, device: int):
    """(addresses), (S, num_pages, Hkv, page_size, d, table width) of a paged cache."""
    shape = k_cache.shape
    if len(shape) != 4 or page_table.dim() != 2:
        raise ValueError("k_cache must be [num_pages, Hkv, page_size, d] and page_table [S, width]")
    S, width = tshape = page_table.shape
    return ((_dense(k_cache, "k_cache", shape, dtype, device),
             _dense(v_cache, "v_cache", shape, dtype, device),
             _dense(page_table, "page_table", tshape, torch.int32, device),
             _dense(lengths, "lengths", (S,), torch.int32, device)), (S, *shape, width))


def mita_cache_append(k, v, k_cache, v_cache, page_table, lengths, seq_start=None, q=None,
                      inv_freq=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                      interleaved: bool = False, q_out=None, stream=None, granted=None):
    """New tokens into a paged cache: k [T,Hkv,d] normalised and rotated (as by
    mita_qk_norm_rope, at its position in its sequence) and v [T,Hkv,d] to their rows of
    k_cache, v_cache [num_pages,Hkv,page_size,d]; returns q [T,Hq,d] normalised and rotated (None
    without q; in q_out where given).  k, v, q and q_out may be strided views.

    page_table: int32 [S,width]; lengths: int32 [S], tokens of each sequence with the new
    ones (0: an idle slot, nothing is written for it); seq_start: int32 [S+1], the rows of each
    sequence's new tokens (None: row s is sequence s's only one); granted: int32 [S], as
    mita_cache_plan gives it: a sequence with 0 is an idle slot, whatever its length (for a step some of
    whose sequences got no page; a captured one too).  Rows that belong to no sequence or to an
    idle slot leave q_out as it is."""
    dev = _device_of(k, "k")
    if stream is not None or dev != torch.cuda.current_device():
        with _on(stream, dev, k, v, k_cache, v_cache, page_table, lengths, seq_start, q, inv_freq,
                 q_weight, k_weight, q_out, granted):
            return mita_cache_append(k, v, k_cache, v_cache, page_table, lengths, seq_start, q,
                                     inv_freq, q_weight, k_weight, eps, interleaved, q_out,
                                     granted=granted)
    dt = k.dtype
    fn = _typed_fn("mita_cache_append", dt)
    (kc, vc, table, n), (S, pages, Hkv, page, d, width) = _cache_of(k_cache, v_cache, page_table,
                                                                    lengths, dt, dev)
    if granted is not None:
        _dense(granted, "granted", (S,), torch.int32, dev)
        lengths = torch.where(granted > 0, lengths, 0)
        n = lengths.data_ptr()
    T = k.shape[0]
    ks, vs = _rows(k, "k", (T, Hkv, d), dt, dev), _rows(v, "v", (T, Hkv, d), dt, dev)
    start = 0 if seq_start is None else _dense(seq_start, "seq_start", (S + 1,), torch.int32, dev)
    freq, rot = _rope_of(inv_freq, dev)
    qw, kw = _weight(q_weight, "q_weight", d, dev), _weight(k_weight, "k_weight", d, dev)
    Hq = qp = qop = 0
    qs = qos = (0, 0)
    if q is None:
        q_out = None
    else:
        Hq = q.shape[1]
        qs = _rows(q, "q", (T, Hq, d), dt, dev)
        if q_out is None:
            q_out = torch.empty((T, Hq, d), dtype=dt, device=q.device)
            qos = (Hq * d, d)
        else:
            qos = _out_rows(q_out, "q_out", (T, Hq, d), dt, dev)
        qp, qop = q.data_ptr(), q_out.data_ptr()
    rc = fn(_CACHE_APPEND.pack(qp, k.data_ptr(), v.data_ptr(), qw, kw, freq, table, n, start, qop,
                               kc, vc, *qs, *ks, *vs, *qos, T, S, Hq, Hkv, d, pages, page, width,
                               rot, interleaved, eps), _raw_stream(dev))
    if rc:
        _check(rc)
    return q_out


def mita_cache_plan(new_tokens, lengths, page_table, free_pages, free_count, tokens: int,
                    page_size: int, new_lengths=None, new_free_count=None, seq_start=None,
                    positions=None, slots=None, granted=None, stream=None):
    """A serving step's pages, dealt out on the device; returns (seq_start, positions, slots, granted).

    new_tokens: int32 [S], each sequence's new tokens, -1 for one that is done (its pages go back to
    the pool).  lengths: int32 [S], tokens before the step; page_table: int32 [S,width]; free_pages:
    int32 [num_pages], a stack whose first free_count (int32 [1]) entries are the free pages.  These
    are brought up to date in place (lengths and free_count in new_lengths and new_free_count where
    given).  tokens: rows of the step's packed (and padded) tokens.

    seq_start: int32 [S+1], the rows of each sequence.  positions: int32 [tokens], in the
    sequence.  slots: int64 [tokens], page*page_size + row in the page, -1 for rows that belong to nobody
    or to a sequence that was not granted.  granted: int32 [S], new_tokens, or 0 where its tokens fit
    neither the pool (first come, first served), the table nor the rows: such a sequence stays
    as it is.  mita_cache_append_q4 goes by slots and passes its rows over; mita_cache_append goes by
    lengths and is given `granted`, or it would write them over the sequence's last tokens."""
    dev = _device_of(new_tokens, "new_tokens")
    if stream is not None or dev != torch.cuda.current_device():
        with _on(stream, dev, new_tokens, lengths, page_table, free_pages, free_count, new_lengths,
                 new_free_count, seq_start, positions, slots, granted):
            return mita_cache_plan(new_tokens, lengths, page_table, free_pages, free_count, tokens,
                                   page_size, new_lengths, new_free_count, seq_start, positions,
                                   slots, granted)
    if page_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("page_table must be [S, width] and free_pages [num_pages]")
    i32 = torch.int32
    (S, width), pages = page_table.shape, free_pages.shape[0]
    # what is not given is made here and needs no checks (four allocations: three of them as parts of one
    # took 4 us more)
    empty, where = torch.empty, new_tokens.device
    if seq_start is None:
        seq_start = empty(S + 1, dtype=i32, device=where)
        start_at = seq_start.data_ptr()
    else:
        start_at = _dense(seq_start, "seq_start", (S + 1,), i32, dev)
    if positions is None:
        positions = empty(tokens, dtype=i32, device=where)
        position_at = positions.data_ptr()
    else:
        position_at = _dense(positions, "positions", (tokens,), i32, dev)
    if slots is None:
        slots = empty(tokens, dtype=torch.int64, device=where)
        slot_at = slots.data_ptr()
    else:
        slot_at = _dense(slots, "slots", (tokens,), torch.int64, dev)
    if granted is None:
        granted = empty(S, dtype=i32, device=where)
        granted_at = granted.data_ptr()
    else:
        granted_at = _dense(granted, "granted", (S,), i32, dev)
    n = _dense(lengths, "lengths", (S,), i32, dev)
    count = _dense(free_count, "free_count", (1,), i32, dev)
    rc = _plan_fn()(_CACHE_PLAN.pack(
        _dense(new_tokens, "new_tokens", (S,), i32, dev), n,
        n if new_lengths is None else _dense(new_lengths, "new_lengths", (S,), i32, dev),
        _dense(page_table, "page_table", (S, width), i32, dev),
        _dense(free_pages, "free_pages", (pages,), i32, dev), count,
        count if new_free_count is None else _dense(new_free_count, "new_free_count", (1,), i32, dev),
        start_at, position_at, slot_at, granted_at, S, tokens, pages, page_size, width), _raw_stream(dev))
    if rc:
        _check(rc)
    return seq_start, positions, slots, granted


@functools.lru_cache(maxsize=None)
def _plan_fn():
    return load().mita_cache_plan


def cache_q4_shape(num_pages: int, Hkv: int, page_size: int, d: int):
    """The shape of a 4-bit cache's k_cache and v_cache (uint8; zero or empty to begin with)."""
    return num_pages, Hkv, page_size * (17 * d // 32)


def _cache_q4_of(k_cache, v_cache, d: int, device: int):
    """(addresses), (num_pages, Hkv, page_size) of a 4-bit cache for heads of d."""
    shape = k_cache.shape
    if len(shape) != 3 or d < 32 or shape[2] % (17 * d // 32) != 0:
        raise ValueError(f"k_cache must be uint8 [num_pages, Hkv, page_size * {17 * d // 32}] for heads "
                         f"of {d}, got {tuple(shape)}")
    return ((_dense(k_cache, "k_cache", shape, torch.uint8, device),
             _dense(v_cache, "v_cache", shape, torch.uint8, device)),
            (shape[0], shape[1], shape[2] // (17 * d // 32)))


def mita_cache_append_q4(k, v, k_cache, v_cache, slots, k_out=None, v_out=None, stream=None):
    """New tokens' keys (normalised and rotated already: mita_qk_norm_rope) and values, k, v [T,Hkv,d],
    into a paged cache of 4-bit codes with a scale for every 32 values (cache_q4_shape).

    slots: int64 [T], each token's page*page_size + row, as mita_cache_plan gives them; -1: passed over.
    k_out, v_out [T,Hkv,d]: where given, the values that the cache now holds for each token (a row
    passed over stays as it is); they may be k and v.  All four may be strided views."""
    dev = _device_of(k, "k")
    if stream is not None or dev != torch.cuda.current_device():
        with _on(stream, dev, k, v, k_cache, v_cache, slots, k_out, v_out):
            return mita_cache_append_q4(k, v, k_cache, v_cache, slots, k_out, v_out)
    dt = k.dtype
    fn = _typed_fn("mita_cache_append_q4", dt)
    shape = T, Hkv, d = k.shape
    (kc, vc), (pages, heads, page) = _cache_q4_of(k_cache, v_cache, d, dev)
    if heads != Hkv:
        raise ValueError(f"k has {Hkv} heads, k_cache {heads}")
    ks, vs = _rows(k, "k", shape, dt, dev), _rows(v, "v", shape, dt, dev)
    kos = vos = (0, 0)
    if k_out is not None:
        kos = _out_rows(k_out, "k_out", shape, dt, dev)
    if v_out is not None:
        vos = _out_rows(v_out, "v_out", shape, dt, dev)
    rc = fn(_CACHE_APPEND_Q4.pack(
        k.data_ptr(), v.data_ptr(), _dense(slots, "slots", (T,), torch.int64, dev), kc, vc,
        0 if k_out is None else k_out.data_ptr(), 0 if v_out is None else v_out.data_ptr(), *ks, *vs,
        *kos, *vos, T, Hkv, d, pages, page), _raw_stream(dev))
    if rc:
        _check(rc)


def mita_paged_attn(q, k_cache, v_cache, page_table, lengths, scale: Optional[float] = None,
                    softcap: float = 0.0, window: int = 0, alibi_slopes=None,
                    return_lse: bool = False, out=None, stream=None):
    """Attention of one new token per sequence over the paged cache (layout and lengths as for
    mita_cache_append, the new token's key included): q [S,Hq,d], may be a strided view; returns
    out [S,Hq,d], with return_lse (out, lse [S,Hq] float32).

    scale: of the scores (None: d^-1/2).  softcap > 0: scores capped to softcap*tanh(z/softcap).
    alibi_slopes: float32 [Hq], adds slope*(key position - own position).  window > 0: only the
    last `window` keys.  Idle slots (length 0) get zeros and lse -inf."""
    return _paged_attn(False, q, k_cache, v_cache, page_table, lengths, scale, softcap, window,
                       alibi_slopes, return_lse, out, stream)


def mita_paged_attn_q4(q, k_cache, v_cache, page_table, lengths, scale: Optional[float] = None,
                       softcap: float = 0.0, window: int = 0, alibi_slopes=None,
                       return_lse: bool = False, out=None, stream=None):
    """mita_paged_attn over a paged cache of 4-bit codes (mita_cache_append_q4's; uint8
    [num_pages,Hkv,page_size*17*d/32]); q and out are bf16 or fp32."""
    return _paged_attn(True, q, k_cache, v_cache, page_table, lengths, scale, softcap, window,
                       alibi_slopes, return_lse, out, stream)


def _paged_attn(q4, q, k_cache, v_cache, page_table, lengths, scale, softcap, window, alibi_slopes,
                return_lse, out, stream):
    dev = _device_of(q, "q")
    if stream is not None or dev != torch.cuda.current_device():
        with _on(stream, dev, q, k_cache, v_cache, page_table, lengths, alibi_slopes, out):
            return _paged_attn(q4, q, k_cache, v_cache, page_table, lengths, scale, softcap, window,
                               alibi_slopes, return_lse, out, None)
    dt = q.dtype
    fn = _typed_fn("mita_paged_attn_q4" if q4 else "mita_paged_attn", dt)
    if q4:
        Hq, d = q.shape[1:]
        (kc, vc), (pages, Hkv, page) = _cache_q4_of(k_cache, v_cache, d, dev)
        S, width = tshape = page_table.shape
        table = _dense(page_table, "page_table", tshape, torch.int32, dev)
        n = _dense(lengths, "lengths", (S,), torch.int32, dev)
    else:
        (kc, vc, table, n), (S, pages, Hkv, page, d, width) = _cache_of(k_cache, v_cache, page_table,
                                                                        lengths, dt, dev)
        Hq = q.shape[1]
    shape = (S, Hq, d)
    qs = _rows(q, "q", shape, dt, dev)
    window = min(window, 0x7fffffff)
    slopes = 0
    if alibi_slopes is not None:
        slopes = _dense(alibi_slopes, "alibi_slopes", (Hq,), torch.float32, dev)
    if out is None:
        out = (torch.empty_like(q) if q.is_contiguous()
               else torch.empty(shape, dtype=dt, device=q.device))
        op = out.data_ptr()
    else:
        op = _dense(out, "out", shape, dt, dev)
    lse = torch.empty((S, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    nbytes = _paged_attn_bytes(S, Hq, Hkv, d, page, width, dt is torch.float32, dev, q4)
    stream = _raw_stream(dev)
    ws = _paged_workspace(nbytes, dev, stream)
    rc = fn(_PAGED_ATTN.pack(q.data_ptr(), kc, vc, table, n, slopes, ws.data_ptr(), op,
                             lse.data_ptr() if return_lse else 0, nbytes, *qs, S, Hq, Hkv, d,
                             pages, page, width, window, d ** -0.5 if scale is None else scale,
                             softcap), stream)
    if rc:
        _check(rc)
    return (out, lse) if return_lse else out


_paged_workspaces = {}     # (device, stream) -> uint8 tensor
_PAGED_COUNTERS = 2048     # its first bytes: zero between calls (the header's MITA_PAGED_COUNTERS)


def _paged_workspace(nbytes: int, device: int, stream: int) -> torch.Tensor:
    """mita_paged_attn's workspace: one for each stream, whose calls (one launch each) follow one
    another, its counters zeroed when it is made or grows.  A captured call has one of its
    graph's own."""
    capturing = torch.cuda.is_current_stream_capturing()
    ws = None if capturing else _paged_workspaces.get((device, stream))
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", device))
        ws[:_PAGED_COUNTERS].zero_()
        if not capturing:
            _paged_workspaces[device, stream] = ws
    return ws


@functools.lru_cache(maxsize=1024)
def _paged_attn_bytes(S, Hq, Hkv, d, page, width, f32, device: int, q4: bool = False) -> int:
    lib = load()
    f = lib.mita_paged_attn_q4_workspace_bytes if q4 else lib.mita_paged_attn_workspace_bytes
    return f(S, Hq, Hkv, d, page, width, f32)


# the handle of torch.cuda.current_stream(device), without making a Stream object of it (1.1 us);
# a torch without CUDA, on which this module can still be imported, has no such function
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


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
    """Frees the cached workspaces, the library's and the binding's."""
    _paged_workspaces.clear()
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
