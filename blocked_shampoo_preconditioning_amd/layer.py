"""The feed-forward half of a decoder layer, forward and backward, on the
library's own kernels: the gated feed-forward block, the norms before and
after a block with gate, dropout and residual scale, and counter-based dropout
(the C ABI in include/shampoo_layer.h).

Weights are [in, out] matrices as `shampoo.Shampoo` registers them, and the
weight gradients go to its `step` as they are. Tensors are 2-D CUDA tensors of
float32 or bfloat16 with contiguous rows (any row stride); a call's tensors
share one dtype. Every call runs on torch's current stream, returns before it
has run, and takes its scratch memory from torch's allocator on that stream.
Results are deterministic.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import shampoo as _s
from .shampoo import HEADER_PATH as _CORE_HEADER
from .shampoo import SHAMPOO_BF16, SHAMPOO_F32

LAYER_HEADER_PATH = os.path.join(os.path.dirname(_CORE_HEADER), "shampoo_layer.h")
ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}
NORMS = {"none": 0, None: 0, "rms": 1, "layer": 2}
MAX_NORM_WIDTH = 8192

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
_U32, _U64 = ctypes.c_uint32, ctypes.c_uint64
_F, _D = ctypes.c_float, ctypes.c_double


class FFNArgs(ctypes.Structure):
    _fields_ = [("tokens", _I64), ("d_model", _I64), ("d_hidden", _I64), ("dtype", _I32), ("activation", _I32),
                ("x", _P), ("w_gate", _P), ("w_up", _P), ("w_down", _P),
                ("ld_x", _I64), ("ld_gate", _I64), ("ld_up", _I64), ("ld_down", _I64),
                ("y", _P), ("ld_y", _I64), ("saved", _P),
                ("dy", _P), ("ld_dy", _I64), ("dx", _P), ("dw_gate", _P), ("dw_up", _P), ("dw_down", _P),
                ("ld_dx", _I64), ("ld_dw_gate", _I64), ("ld_dw_up", _I64), ("ld_dw_down", _I64)]


class NormArgs(ctypes.Structure):
    _fields_ = [("rows", _I64), ("width", _I64), ("dtype", _I32), ("post_kind", _I32), ("next_kind", _I32),
                ("eps", _F), ("residual_scale", _F), ("dropout", _D), ("seed", _U64), ("offset", _U32),
                ("rows_per_gate", _I64),
                ("z", _P), ("x", _P), ("ld_z", _I64), ("ld_x", _I64), ("r", _P), ("n", _P), ("ld_r", _I64), ("ld_n", _I64),
                ("post_weight", _P), ("post_bias", _P), ("gate", _P), ("next_weight", _P), ("next_bias", _P),
                ("ld_gate", _I64), ("stats", _P),
                ("dr", _P), ("dn", _P), ("ld_dr", _I64), ("ld_dn", _I64), ("dx", _P), ("dz", _P), ("ld_dx", _I64), ("ld_dz", _I64),
                ("d_post_weight", _P), ("d_post_bias", _P), ("d_gate", _P), ("d_next_weight", _P), ("d_next_bias", _P),
                ("ld_d_gate", _I64)]


class DropoutArgs(ctypes.Structure):
    _fields_ = [("rows", _I64), ("cols", _I64), ("dtype", _I32), ("offset", _U32), ("dropout", _D), ("seed", _U64),
                ("x", _P), ("y", _P), ("ld_x", _I64), ("ld_y", _I64)]


_SIZE = ctypes.POINTER(ctypes.c_size_t)
_FFN, _NORM, _DROP = (ctypes.POINTER(t) for t in (FFNArgs, NormArgs, DropoutArgs))
_SIGNATURES = {
    "shampoo_ffn_saved_size": [_FFN, _SIZE],
    "shampoo_ffn_workspace_size": [_FFN, _I32, _SIZE],
    "shampoo_ffn_forward": [_FFN, _P, ctypes.c_size_t, _P],
    "shampoo_ffn_backward": [_FFN, _P, ctypes.c_size_t, _P],
    "shampoo_norm_workspace_size": [_NORM, _SIZE],
    "shampoo_norm_forward": [_NORM, _P],
    "shampoo_norm_backward": [_NORM, _P, ctypes.c_size_t, _P],
    "shampoo_dropout": [_DROP, _P],
}
_lib = None


def load_library():
    """The HIP library with the layer operators' signatures set (once)."""
    global _lib
    if _lib is None:
        lib = _s.load_library()
        for name, argtypes in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = argtypes, ctypes.c_int
        _lib = lib
    return _lib


def _check(code):
    if code:
        _s._check(code)


_DTYPES = {torch.bfloat16: SHAMPOO_BF16, torch.float32: SHAMPOO_F32}


def _matrix(name, t, rows, cols, like=None):
    """(pointer, leading dimension) of a 2-D tensor of that shape."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected ({rows}, {cols})")
    if like is not None:
        _same(name, t, like)
    row, col = t.stride()
    if col != 1 and cols > 1:
        raise ValueError(f"{name}: rows must be contiguous (stride {t.stride()})")
    if rows <= 1:
        row = cols
    elif row < cols:
        raise ValueError(f"{name}: rows overlap (stride {t.stride()})")
    # an empty tensor has a NULL pointer, which would mean "not given"; it is never read
    return t.data_ptr() or 256, row


def _vector(name, t, n, like):
    """Pointer of a 1-D tensor of n elements (None: NULL)."""
    if t is None:
        return None
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} elements, got shape {tuple(t.shape)}")
    _same(name, t, like)
    return t.data_ptr()


def _same(name, t, like):
    if t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {like.dtype} on {like.device}")


def _dtype(name, t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} is {t.dtype}: float32 and bfloat16 are supported")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D (tokens, width), got shape {tuple(t.shape)}")
    return _DTYPES[t.dtype]


def _stream(t):
    return torch.cuda.current_stream(t.device).cuda_stream


def _workspace(nbytes, like):
    return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


# ------------------------------------------------------ gated feed-forward block
def _ffn_args(x, w_gate, w_up, w_down, activation):
    dt = _dtype("x", x)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is not one of {sorted(ACTIVATIONS)}")
    n, d = x.shape
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate must be 2-D, got shape {tuple(w_gate.shape)}")
    f = w_gate.shape[1]
    px, lx = _matrix("x", x, n, d)
    pg, lg = _matrix("w_gate", w_gate, d, f, x)
    pu, lu = _matrix("w_up", w_up, d, f, x)
    pd, ld = _matrix("w_down", w_down, f, d, x)
    return FFNArgs(n, d, f, dt, ACTIVATIONS[activation], px, pg, pu, pd, lx, lg, lu, ld)


def _ffn_call(a, backward, like):
    lib, size = load_library(), ctypes.c_size_t()
    ref = ctypes.byref(a)
    with torch.cuda.device(like.device):
        _check(lib.shampoo_ffn_workspace_size(ref, backward, ctypes.byref(size)))
        ws = _workspace(size.value, like) if size.value else None
        fn = lib.shampoo_ffn_backward if backward else lib.shampoo_ffn_forward
        _check(fn(ref, ws.data_ptr() if ws is not None else None, size.value, _stream(like)))


def ffn_forward(x, w_gate, w_up, w_down, activation="silu", save=False):
    """y = (act(x w_gate) * (x w_up)) w_down for x [tokens, d], w_gate and w_up
    [d, f], w_down [f, d]. With `save` returns (y, saved), `saved` being what
    `ffn_backward` needs (an opaque tensor of three f-wide rows a token).
    activation: "silu", "gelu" (tanh form) or "relu"."""
    a = _ffn_args(x, w_gate, w_up, w_down, activation)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    a.y, a.ld_y = y.data_ptr(), x.shape[1]
    saved = None
    if save:
        size = ctypes.c_size_t()
        _check(load_library().shampoo_ffn_saved_size(ctypes.byref(a), ctypes.byref(size)))
        saved = torch.empty(size.value, dtype=torch.uint8, device=x.device)
        a.saved = saved.data_ptr()
    _ffn_call(a, 0, x)
    return (y, saved) if save else y


def ffn_backward(dy, x, w_gate, w_up, w_down, saved, activation="silu", need_dx=True, need_dw=True):
    """(dx, dw_gate, dw_up, dw_down) from dy, the forward pass's inputs and what
    it saved. need_dx / need_dw: None is returned for what is not needed."""
    a = _ffn_args(x, w_gate, w_up, w_down, activation)
    n, d, f = a.tokens, a.d_model, a.d_hidden
    a.dy, a.ld_dy = _matrix("dy", dy, n, d, x)
    size = ctypes.c_size_t()
    _check(load_library().shampoo_ffn_saved_size(ctypes.byref(a), ctypes.byref(size)))
    if saved.dtype != torch.uint8 or saved.numel() != size.value or saved.device != x.device:
        raise ValueError("saved is not what ffn_forward kept for these sizes")
    a.saved = saved.data_ptr()

    def new(rows, cols):
        return torch.empty((rows, cols), dtype=x.dtype, device=x.device)
    dx = dwg = dwu = dwd = None
    if need_dx:
        dx = new(n, d)
        a.dx, a.ld_dx = dx.data_ptr(), d
    if need_dw:
        dwg, dwu, dwd = new(d, f), new(d, f), new(f, d)
        a.dw_gate, a.dw_up, a.dw_down = dwg.data_ptr(), dwu.data_ptr(), dwd.data_ptr()
        a.ld_dw_gate, a.ld_dw_up, a.ld_dw_down = f, f, d
    if need_dx or need_dw:
        _ffn_call(a, 1, x)
    return dx, dwg, dwu, dwd


# ------------------------------------------------------- norms around a block
def _norm_args(x, z, post, post_weight, post_bias, gate, rows_per_gate, residual_scale, dropout, seed, offset, next,
               next_weight, next_bias, eps):
    dt = _dtype("x", x)
    n, d = x.shape
    if post not in NORMS or next not in NORMS:
        raise ValueError("post and next are one of 'none', 'rms', 'layer'")
    a = NormArgs(n, d, dt, NORMS[post], NORMS[next], eps, residual_scale, dropout, seed & 0xFFFFFFFFFFFFFFFF,
                 offset & 0xFFFFFFFF, 1)
    a.x, a.ld_x = _matrix("x", x, n, d)
    if z is not None:
        a.z, a.ld_z = _matrix("z", z, n, d, x)
    if gate is not None:
        a.rows_per_gate = max(n, 1) if rows_per_gate is None else rows_per_gate
        if a.rows_per_gate < 1:
            raise ValueError("rows_per_gate must be at least 1")
        a.gate, a.ld_gate = _matrix("gate", gate, -(-n // a.rows_per_gate), d, x)
    a.post_weight = _vector("post_weight", post_weight, d, x)
    a.post_bias = _vector("post_bias", post_bias, d, x)
    a.next_weight = _vector("next_weight", next_weight, d, x)
    a.next_bias = _vector("next_bias", next_bias, d, x)
    return a


def _norm_forward(a, x, r, stats):
    n = torch.empty(x.shape, dtype=x.dtype, device=x.device) if a.next_kind else None
    if n is not None:
        a.n, a.ld_n = n.data_ptr(), x.shape[1]
    if r is not None:
        a.r, a.ld_r = r.data_ptr(), x.shape[1]
    if stats:
        stats = torch.empty((x.shape[0], 4), dtype=torch.float32, device=x.device)
        a.stats = stats.data_ptr()
    with torch.cuda.device(x.device):
        _check(load_library().shampoo_norm_forward(ctypes.byref(a), _stream(x)))
    return n, stats


def residual_forward(x, z, *, post="rms", post_weight=None, post_bias=None, gate=None, rows_per_gate=None,
                     residual_scale=1.0, dropout=0.0, seed=0, offset=0, next="rms", next_weight=None, next_bias=None,
                     eps=1e-6):
    """The end of one block and the start of the next in one pass over the data:
        p = post-norm(z),  r = residual_scale * x + dropout(gate * p),  n = next-norm(r)
    for the block's output z and the residual stream x, [rows, width] (width up
    to 8192). Norms are "rms", "layer" or "none"; weights and biases are vectors
    or None. gate: [rows / rows_per_gate rounded up, width], row i // rows_per_gate
    for row i (rows_per_gate None: one row for all). dropout: probability, under
    the 64-bit `seed` and 32-bit `offset`. Returns (r, n, stats); n is None for
    next="none"; stats go to `residual_backward`."""
    a = _norm_args(x, z, post, post_weight, post_bias, gate, rows_per_gate, residual_scale, dropout, seed, offset, next,
                   next_weight, next_bias, eps)
    if z is None:
        raise ValueError("z is None: norm_forward is the norm alone")
    r = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    n, stats = _norm_forward(a, x, r, True)
    return r, n, stats


def norm_forward(x, kind="rms", weight=None, bias=None, eps=1e-6):
    """n = norm(x), [rows, width]; returns (n, stats for `norm_backward`)."""
    if kind in ("none", None):
        raise ValueError("kind must be 'rms' or 'layer'")
    a = _norm_args(x, None, "none", None, None, None, None, 1.0, 0.0, 0, 0, kind, weight, bias, eps)
    return _norm_forward(a, x, None, True)


def _norm_backward(a, x, z, dr, dn, stats):
    n, d = x.shape
    if stats.shape != (n, 4) or stats.dtype != torch.float32 or not stats.is_contiguous() or stats.device != x.device:
        raise ValueError("stats is not what the forward pass returned for these sizes")
    a.stats = stats.data_ptr()
    if dr is not None:
        a.dr, a.ld_dr = _matrix("dr", dr, n, d, x)
    if a.next_kind:
        if dn is None:
            raise ValueError("dn is None: the next norm's gradient is needed")
        a.dn, a.ld_dn = _matrix("dn", dn, n, d, x)

    def new(*shape):
        return torch.empty(shape, dtype=x.dtype, device=x.device)
    g = dict.fromkeys(("x", "z", "post_weight", "post_bias", "gate", "next_weight", "next_bias"))
    g["x"] = new(n, d)
    a.dx, a.ld_dx = g["x"].data_ptr(), d
    if z is not None:
        g["z"] = new(n, d)
        a.dz, a.ld_dz = g["z"].data_ptr(), d
    for name in ("post_weight", "post_bias", "next_weight", "next_bias"):
        if getattr(a, name):
            g[name] = new(d)
            setattr(a, "d_" + name, g[name].data_ptr())
    if a.gate:
        g["gate"] = new(-(-n // a.rows_per_gate), d)
        a.d_gate, a.ld_d_gate = g["gate"].data_ptr(), d
    lib, size = load_library(), ctypes.c_size_t()
    with torch.cuda.device(x.device):
        _check(lib.shampoo_norm_workspace_size(ctypes.byref(a), ctypes.byref(size)))
        ws = _workspace(size.value, x) if size.value else None
        _check(lib.shampoo_norm_backward(ctypes.byref(a), ws.data_ptr() if ws is not None else None, size.value, _stream(x)))
    return g


def residual_backward(dr, dn, r, z, stats, *, post="rms", post_weight=None, post_bias=None, gate=None, rows_per_gate=None,
                      residual_scale=1.0, dropout=0.0, seed=0, offset=0, next="rms", next_weight=None, next_bias=None,
                      eps=1e-6):
    """Gradients of `residual_forward` from those of r and n (dr None: zero),
    its r, z and stats, with the same settings: a dict with "x", "z",
    "post_weight", "post_bias", "gate", "next_weight", "next_bias" (None for
    what was not given)."""
    a = _norm_args(r, z, post, post_weight, post_bias, gate, rows_per_gate, residual_scale, dropout, seed, offset, next,
                   next_weight, next_bias, eps)
    a.r, a.ld_r = a.x, a.ld_x
    return _norm_backward(a, r, z, dr, dn, stats)


def norm_backward(dn, x, stats, dr=None, kind="rms", weight=None, bias=None, eps=1e-6):
    """Gradients of `norm_forward`, with a gradient dr that reaches x by another
    way (the residual stream) added: a dict with "x", "weight", "bias"."""
    if kind in ("none", None):
        raise ValueError("kind must be 'rms' or 'layer'")
    a = _norm_args(x, None, "none", None, None, None, None, 1.0, 0.0, 0, 0, kind, weight, bias, eps)
    g = _norm_backward(a, x, None, dr, dn, stats)
    return {"x": g["x"], "weight": g["next_weight"], "bias": g["next_bias"]}


# -------------------------------------------------------------------- dropout
def dropout(x, p, seed, offset=0, out=None):
    """x with elements dropped with probability p (a multiple of 2^-16) and the
    others scaled to keep the expectation. Which ones goes by (row, column,
    seed, offset) alone, so the gradient is the same call on the gradient.
    out: a tensor to write to (may be x)."""
    dt = _dtype("x", x)
    n, d = x.shape
    px, lx = _matrix("x", x, n, d)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device) if out is None else out
    py, ly = _matrix("out", y, n, d, x)
    a = DropoutArgs(n, d, dt, offset & 0xFFFFFFFF, p, seed & 0xFFFFFFFFFFFFFFFF, px, py, lx, ly)
    with torch.cuda.device(x.device):
        _check(load_library().shampoo_dropout(ctypes.byref(a), _stream(x)))
    return y
