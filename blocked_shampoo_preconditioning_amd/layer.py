"""The feed-forward half of a decoder layer, forward and backward, on the
library's own kernels: the gated feed-forward block, the norms before and
after a block with gate, dropout and residual scale, and counter-based dropout
(the C ABI in include/shampoo_layer.h).

Weights are [in, out] matrices as `shampoo.Shampoo` registers them, and the
weight gradients go to its `step` as they are. Tensors are 2-D CUDA tensors of
float32 or bfloat16 with contiguous rows (any row stride); a call's tensors
share one dtype. Every call runs on torch's current stream, returns before it
has run, and takes its scratch memory from torch's allocator on that stream.
Results are deterministic. The calls record no autograd graph, also where an
input requires a gradient: a program calls the backward functions itself.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import shampoo as _s
from .shampoo import HEADER_PATH as _CORE_HEADER
from .shampoo import SHAMPOO_BF16, SHAMPOO_F32

LAYER_HEADER_PATH = os.path.join(os.path.dirname(_CORE_HEADER), "shampoo_layer.h")
ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}
NORMS = {"none": 0, None: 0, "rms": 1, "layer": 2}
MAX_NORM_WIDTH = 8192

# The C argument structs, field by field (native sizes and alignment); packing
# one takes a fraction of the time of filling a ctypes structure, which counts
# where a call is a few microseconds. "P" is a pointer, 0 for NULL.
_FFN = struct.Struct("@qqq ii PPPP qqqq P q P P q PPPP qqqq")
_NORM = struct.Struct("@qq iii f f d Q I q PP qq PP qq PPPPP q P PP qq PP qq PPPPP q")
_DROP = struct.Struct("@qq i I d Q PP qq")

_A, _SIZE = ctypes.c_char_p, ctypes.POINTER(ctypes.c_size_t)
_SIGNATURES = {
    "shampoo_ffn_saved_size": [_A, _SIZE],
    "shampoo_ffn_workspace_size": [_A, ctypes.c_int32, _SIZE],
    "shampoo_ffn_forward": [_A, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
    "shampoo_ffn_backward": [_A, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
    "shampoo_ffn_normed_workspace_size": [_A, _A, _SIZE],
    "shampoo_ffn_forward_normed": [_A, _A, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
    "shampoo_norm_workspace_size": [_A, _SIZE],
    "shampoo_norm_forward": [_A, ctypes.c_void_p],
    "shampoo_norm_backward": [_A, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
    "shampoo_dropout": [_A, ctypes.c_void_p],
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


_DTYPES = {torch.bfloat16: SHAMPOO_BF16, torch.float32: SHAMPOO_F32}
_U64, _U32 = 0xFFFFFFFFFFFFFFFF, 0xFFFFFFFF


# The current stream's handle: torch.cuda.current_stream builds a Stream object for it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _call(name, args, dev, *more):
    """Runs an entry point on device `dev` and torch's current stream there."""
    fn = getattr(_lib or load_library(), name)
    if dev == torch.cuda.current_device():
        code = fn(args, *more, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            code = fn(args, *more, _raw_stream(dev))
    if code:
        _s._check(code)


def _size(name, args, *more):
    out = ctypes.c_size_t()
    code = getattr(_lib or load_library(), name)(args, *more, ctypes.byref(out))
    if code:
        _s._check(code)
    return out.value


def _first(name, t):
    """dtype code, rows and columns of the tensor that sets a call's dtype and device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} is {t.dtype}: float32 and bfloat16 are supported")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D (tokens, width), got shape {tuple(t.shape)}")
    rows, cols = t.shape
    return code, rows, cols


def _unlike(name, t, like):
    return ValueError(f"{name} is {t.dtype} on {t.device}, expected {like.dtype} on {like.device}")


def _matrix(name, t, rows, cols, like):
    """(pointer, leading dimension) of a 2-D tensor of that shape, dtype and device."""
    if t.dtype is not like.dtype or t.get_device() != like.get_device():
        raise _unlike(name, t, like)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({rows}, {cols})")
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
    """Pointer of a 1-D tensor of n elements (None: 0)."""
    if t is None:
        return 0
    if t.dtype is not like.dtype or t.get_device() != like.get_device():
        raise _unlike(name, t, like)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} elements, got shape {tuple(t.shape)}")
    return t.data_ptr()


def _new(like, rows, cols):
    return like.new_empty((rows, cols))


def _new_like(t):
    """A contiguous tensor of t's shape, dtype and device."""
    return torch.empty_like(t, memory_format=_CONTIGUOUS)


_CONTIGUOUS = torch.contiguous_format


def _workspace(nbytes, like):
    """(pointer, tensor that owns it)."""
    if not nbytes:
        return 0, None
    ws = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    return ws.data_ptr(), ws


_sizes = {}  # what a call's byte count goes by -> the count
_MAX_SIZES = 4096


def _known_size(key, name, args, *more):
    """A byte count of the library, asked once for each key; the table is emptied when it is full."""
    size = _sizes.get(key)
    if size is None:
        size = _size(name, args, *more)
        if len(_sizes) >= _MAX_SIZES:
            _sizes.clear()
        _sizes[key] = size
    return size


# ------------------------------------------------------ gated feed-forward block
def _ffn_inputs(x, w_gate, w_up, w_down, activation):
    """The leading fields of the C struct, tokens to ld_down."""
    dt, n, d = _first("x", x)
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation {activation!r} is not one of {sorted(ACTIVATIONS)}")
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate must be 2-D, got shape {tuple(w_gate.shape)}")
    f = w_gate.shape[1]
    px, lx = _matrix("x", x, n, d, x)
    pg, lg = _matrix("w_gate", w_gate, d, f, x)
    pu, lu = _matrix("w_up", w_up, d, f, x)
    pd, ld = _matrix("w_down", w_down, f, d, x)
    return n, d, f, dt, act, px, pg, pu, pd, lx, lg, lu, ld


def _ffn_workspace(fields, args, backward, more, norm=None):
    """Workspace bytes of a call, which go by sizes, direction, leading dimensions and alignments."""
    key = (fields[:4], backward, fields[9:], fields[5] & 15, fields[6] & 15, fields[7] & 15, fields[8] & 15, more)
    if norm:
        return _known_size(key, "shampoo_ffn_normed_workspace_size", args, norm)
    return _known_size(key, "shampoo_ffn_workspace_size", args, backward)


_NO_GRADIENTS = (0,) * 10


def ffn_forward(x, w_gate, w_up, w_down, activation="silu", save=False):
    """y = (act(x w_gate) * (x w_up)) w_down for x [tokens, d], w_gate and w_up
    [d, f], w_down [f, d]. With `save` returns (y, saved), `saved` being what
    `ffn_backward` needs (an opaque tensor: g, u and h of every token).
    activation: "silu", "gelu" (tanh form) or "relu". Where bf16 x is the result
    of `norm_forward` itself, a saved ReLU block takes g and u from it as it was
    before its rounding, which would move g over 0 in one element of 2000 (an
    element of x that was changed since is taken as it is)."""
    fields = _ffn_inputs(x, w_gate, w_up, w_down, activation)
    n, d, f = fields[:3]
    y = _new_like(x)
    saved = None
    if save:
        saved = torch.empty(_saved_size(fields), dtype=torch.uint8, device=x.device)
    args = _FFN.pack(*fields, y.data_ptr() or 256, d, saved.data_ptr() if save else 0, *_NO_GRADIENTS)
    norm = _norm_of(x) if save and activation == "relu" and fields[3] == SHAMPOO_BF16 else None
    if norm:
        size = _ffn_workspace(fields, args, 0, "normed", norm)
        ws, keep = _workspace(size, x)
        _call("shampoo_ffn_forward_normed", args, x.get_device(), norm, ws, size)
        return y, saved
    size = _ffn_workspace(fields, args, 0, save)
    ws, keep = _workspace(size, x)
    _call("shampoo_ffn_forward", args, x.get_device(), ws, size)
    return (y, saved) if save else y


def _norm_of(x):
    """The C struct of the `norm_forward` call that returned x; None if no such call did, or its tensors are others by now."""
    made = getattr(x, "_norm_call", None)
    if made is None:
        return None
    head, source, weight, bias, stats = made
    n, d = head[:2]
    try:
        px, lx = _matrix("n", x, n, d, x)
        ps, ls = _matrix("x", source, n, d, x)
        pw, pb = _vector("weight", weight, d, x), _vector("bias", bias, d, x)
        _matrix("stats", stats, n, 4, stats)
    except ValueError:
        return None
    return _NORM.pack(*head, 0, ps, 0, ls, 0, px, 0, lx, 0, 0, 0, pw, pb, 0, stats.data_ptr(), *_NO_NORM_GRADIENTS)


def _saved_size(fields):
    return _sizes.get(fields[:4]) or _known_size(fields[:4], "shampoo_ffn_saved_size", _FFN.pack(*fields, *(0,) * 13))


def ffn_backward(dy, x, w_gate, w_up, w_down, saved, activation="silu", need_dx=True, need_dw=True):
    """(dx, dw_gate, dw_up, dw_down) from dy, the forward pass's inputs and what
    it saved. need_dx / need_dw: None is returned for what is not needed."""
    fields = _ffn_inputs(x, w_gate, w_up, w_down, activation)
    n, d, f = fields[:3]
    pdy, ldy = _matrix("dy", dy, n, d, x)
    if saved.dtype is not torch.uint8 or saved.numel() != _saved_size(fields) or saved.get_device() != x.get_device():
        raise ValueError("saved is not what ffn_forward kept for these sizes")
    dx = _new_like(x) if need_dx else None
    dwg = dwu = dwd = None
    pointers = (dx.data_ptr() or 256 if need_dx else 0, 0, 0, 0)
    if need_dw:
        dwg, dwu, dwd = _new_like(w_gate), _new_like(w_up), _new_like(w_down)
        pointers = (pointers[0], dwg.data_ptr(), dwu.data_ptr(), dwd.data_ptr())
    if need_dx or need_dw:
        args = _FFN.pack(*fields, 0, 0, saved.data_ptr(), pdy, ldy, *pointers, d, f, f, d)
        size = _ffn_workspace(fields, args, 1, (need_dx, need_dw, ldy, pdy & 15))
        ws, keep = _workspace(size, x)
        _call("shampoo_ffn_backward", args, x.get_device(), ws, size)
    return dx, dwg, dwu, dwd


# ------------------------------------------------------- norms around a block
def _norm_head(dt, n, d, post, next, eps, residual_scale, dropout, seed, offset, rows_per_gate):
    kp, kn = NORMS.get(post), NORMS.get(next)
    if kp is None or kn is None:
        raise ValueError("post and next are one of 'none', 'rms', 'layer'")
    if rows_per_gate is None:
        rows_per_gate = n or 1
    elif rows_per_gate < 1:
        raise ValueError("rows_per_gate must be at least 1")
    return n, d, dt, kp, kn, eps, residual_scale, dropout, seed & _U64, offset & _U32, rows_per_gate


def _norm_vectors(like, n, d, post_weight, post_bias, gate, rows_per_gate, next_weight, next_bias):
    """Pointers of weights, biases and gate, and the gate's leading dimension."""
    pg, lg = _matrix("gate", gate, -(-n // rows_per_gate), d, like) if gate is not None else (0, 0)
    return (_vector("post_weight", post_weight, d, like), _vector("post_bias", post_bias, d, like), pg,
            _vector("next_weight", next_weight, d, like), _vector("next_bias", next_bias, d, like), lg)


_NO_NORM_GRADIENTS = (0,) * 14


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
    dt, n, d = _first("x", x)
    if z is None:
        raise ValueError("z is None: norm_forward is the norm alone")
    head = _norm_head(dt, n, d, post, next, eps, residual_scale, dropout, seed, offset, rows_per_gate)
    px, lx = _matrix("x", x, n, d, x)
    pz, lz = _matrix("z", z, n, d, x)
    vectors = _norm_vectors(x, n, d, post_weight, post_bias, gate, head[-1], next_weight, next_bias)
    r = _new_like(x)
    out = _new_like(x) if head[4] else None
    stats = torch.empty((n, 4), dtype=torch.float32, device=x.device)
    args = _NORM.pack(*head, pz, px, lz, lx, r.data_ptr(), out.data_ptr() if out is not None else 0, d, d, *vectors,
                      stats.data_ptr(), *_NO_NORM_GRADIENTS)
    _call("shampoo_norm_forward", args, x.get_device())
    return r, out, stats


def norm_forward(x, kind="rms", weight=None, bias=None, eps=1e-6):
    """n = norm(x), [rows, width]; returns (n, stats for `norm_backward`). bf16 n
    knows this call's inputs (and keeps them in memory as long as it is there), for
    a ReLU block that takes it: see `ffn_forward`."""
    if kind in ("none", None):
        raise ValueError("kind must be 'rms' or 'layer'")
    dt, n, d = _first("x", x)
    head = _norm_head(dt, n, d, "none", kind, eps, 1.0, 0.0, 0, 0, None)
    px, lx = _matrix("x", x, n, d, x)
    vectors = _norm_vectors(x, n, d, None, None, None, 1, weight, bias)
    out = _new_like(x)
    stats = torch.empty((n, 4), dtype=torch.float32, device=x.device)
    args = _NORM.pack(*head, 0, px, 0, lx, 0, out.data_ptr(), d, d, *vectors, stats.data_ptr(), *_NO_NORM_GRADIENTS)
    _call("shampoo_norm_forward", args, x.get_device())
    if dt == SHAMPOO_BF16:
        out._norm_call = (head, x, weight, bias, stats)
    return out, stats


def _norm_workspace(head, args):
    """Workspace bytes of a backward call, which go by rows, width and dtype alone."""
    return _known_size(head[:3], "shampoo_norm_workspace_size", args)


def _norm_backward(head, x, z, px, lx, vectors, dr, dn, stats):
    """x: the forward pass's r (or its input, where there is no z)."""
    n, d = head[:2]
    if stats.shape != (n, 4) or stats.dtype is not torch.float32 or not stats.is_contiguous() or \
            stats.get_device() != x.get_device():
        raise ValueError("stats is not what the forward pass returned for these sizes")
    pz, lz = _matrix("z", z, n, d, x) if z is not None else (0, 0)
    pdr, ldr = _matrix("dr", dr, n, d, x) if dr is not None else (0, 0)
    pdn, ldn = 0, 0
    if head[4]:
        if dn is None:
            raise ValueError("dn is None: the next norm's gradient is needed")
        pdn, ldn = _matrix("dn", dn, n, d, x)
    dx = _new_like(x)
    dz = _new_like(x) if z is not None else None
    # the vectors' gradients, in the struct's order: post weight, post bias, gate, next weight, next bias;
    # those of one row come from one allocation
    gate_rows = -(-n // head[10]) if vectors[2] else 0
    rows = [gate_rows if i == 2 else 1 if v else 0 for i, v in enumerate(vectors[:5])]
    one = sum(r == 1 for r in rows)
    shared = iter(()) if not one else iter(x.new_empty((one, d)).unbind(0))
    grads = [None if r == 0 else next(shared) if r == 1 else _new(x, r, d) for r in rows]
    if vectors[2] and rows[2] < 2:
        grads[2] = grads[2].view(1, d) if rows[2] else _new(x, 0, d)
    pointers = [g.data_ptr() if g is not None else 0 for g in grads]  # an empty one: 0, nothing to write
    args = _NORM.pack(*head, pz, px, lz, lx, px if z is not None else 0, 0, lx, 0, *vectors, stats.data_ptr(), pdr, pdn, ldr,
                      ldn, dx.data_ptr(), dz.data_ptr() if z is not None else 0, d, d, *pointers, d)
    size = _norm_workspace(head, args)
    ws, keep = _workspace(size, x)
    _call("shampoo_norm_backward", args, x.get_device(), ws, size)
    return dx, dz, grads


def residual_backward(dr, dn, r, z, stats, *, post="rms", post_weight=None, post_bias=None, gate=None, rows_per_gate=None,
                      residual_scale=1.0, dropout=0.0, seed=0, offset=0, next="rms", next_weight=None, next_bias=None,
                      eps=1e-6):
    """Gradients of `residual_forward` from those of r and n (dr None: zero),
    its r, z and stats, with the same settings: a dict with "x", "z",
    "post_weight", "post_bias", "gate", "next_weight", "next_bias" (None for
    what was not given)."""
    dt, n, d = _first("r", r)
    head = _norm_head(dt, n, d, post, next, eps, residual_scale, dropout, seed, offset, rows_per_gate)
    px, lx = _matrix("r", r, n, d, r)
    vectors = _norm_vectors(r, n, d, post_weight, post_bias, gate, head[-1], next_weight, next_bias)
    dx, dz, g = _norm_backward(head, r, z, px, lx, vectors, dr, dn, stats)
    return {"x": dx, "z": dz, "post_weight": g[0], "post_bias": g[1], "gate": g[2], "next_weight": g[3], "next_bias": g[4]}


def norm_backward(dn, x, stats, dr=None, kind="rms", weight=None, bias=None, eps=1e-6):
    """Gradients of `norm_forward`, with a gradient dr that reaches x by another
    way (the residual stream) added: a dict with "x", "weight", "bias"."""
    if kind in ("none", None):
        raise ValueError("kind must be 'rms' or 'layer'")
    dt, n, d = _first("x", x)
    head = _norm_head(dt, n, d, "none", kind, eps, 1.0, 0.0, 0, 0, None)
    px, lx = _matrix("x", x, n, d, x)
    vectors = _norm_vectors(x, n, d, None, None, None, 1, weight, bias)
    dx, _, g = _norm_backward(head, x, None, px, lx, vectors, dr, dn, stats)
    return {"x": dx, "weight": g[3], "bias": g[4]}


# -------------------------------------------------------------------- dropout
def dropout(x, p, seed, offset=0, out=None):
    """x with elements dropped with probability p (a multiple of 2^-16) and the
    others scaled to keep the expectation. Which ones goes by (row, column,
    seed, offset) alone, so the gradient is the same call on the gradient.
    out: a tensor to write to (may be x)."""
    dt, n, d = _first("x", x)
    px, lx = _matrix("x", x, n, d, x)
    if out is None:
        out, ly = _new_like(x), d
        py = out.data_ptr()
    else:
        py, ly = _matrix("out", out, n, d, x)
    args = _DROP.pack(n, d, dt, offset & _U32, p, seed & _U64, px, py, lx, ly)
    _call("shampoo_dropout", args, x.get_device())
    return out
