"""The experts' path of a feed-forward block, forward and backward, on the
library's own kernels: tokens sorted by expert and back, with weights applied
(the C ABI in include/shampoo_experts.h).

    plan = experts.sort_tokens(ids, n_experts)       # ids [tokens, slots]: each token's experts
    xs = experts.dispatch(x, plan)                   # rows by expert
    ...                                              # each expert's matrices on its rows of xs: ys
    y = experts.combine(ys, plan, weights)           # back, with the router's weights

Tensors are as `layer` takes them: 2-D CUDA tensors of float32 or bfloat16 with
contiguous rows (any row stride). Every call runs on torch's current stream,
returns before it has run (nothing waits for the GPU: how many rows an expert
has stays on it), and takes its scratch memory from torch's allocator on that
stream. Results are deterministic. The calls record no autograd graph: a
program calls the backward functions itself.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple

import torch

from . import layer as _layer
from . import shampoo as _s
from .layer import _first, _matrix, _raw_stream, _unlike, _workspace
from .shampoo import HEADER_PATH as _CORE_HEADER

EXPERTS_HEADER_PATH = os.path.join(os.path.dirname(_CORE_HEADER), "shampoo_experts.h")
MAX_EXPERTS = 1024

# The C argument structs, field by field (native sizes and alignment), as in `layer`.
_SORT = struct.Struct("@q iii P q PPP")
_ROUTE = struct.Struct("@qq ii PP PP qq PP qq P")

_A, _SIZE = ctypes.c_char_p, ctypes.POINTER(ctypes.c_size_t)
_SIGNATURES = {
    "shampoo_sort_workspace_size": [_A, _SIZE],
    "shampoo_sort_tokens": [_A, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
    "shampoo_dispatch": [_A, ctypes.c_void_p],
    "shampoo_combine": [_A, ctypes.c_void_p],
    "shampoo_combine_backward": [_A, ctypes.c_void_p],
}
_lib = None


def load_library():
    """The HIP library with the experts' signatures set (once)."""
    global _lib
    if _lib is None:
        lib = _s.load_library()
        for name, argtypes in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = argtypes, ctypes.c_int
        _lib = lib
    return _lib


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


_sizes = {}  # what a call's byte count goes by -> the count
_MAX_SIZES = 4096


def _known_size(key, name, args, *more):
    """A byte count of the library, asked once for each key; the table is emptied when it is full."""
    size = _sizes.get(key)
    if size is None:
        out = ctypes.c_size_t()
        code = getattr(_lib or load_library(), name)(args, *more, ctypes.byref(out))
        if code:
            _s._check(code)
        size = out.value
        if len(_sizes) >= _MAX_SIZES:
            _sizes.clear()
        _sizes[key] = size
    return size


# ----------------------------------------------------------- tokens by expert
class Plan(NamedTuple):
    """Where the slots of a batch go, as `sort_tokens` returns it (int32 CUDA tensors).
    offsets [experts + 1]: expert e has rows offsets[e] to offsets[e + 1].
    rows [tokens, slots]: a slot's row; ~row (negative) for a slot left out.
    source [tokens * slots]: a row's slot number t * slots + j; its ~ for a slot left out."""
    offsets: torch.Tensor
    rows: torch.Tensor
    source: torch.Tensor


_INT_BYTES = {torch.int32: 4, torch.int64: 8}


def sort_tokens(ids, n_experts):
    """The `Plan` that sorts slots by expert: ids [tokens, slots], int32 or int64,
    the expert of each slot of each token (contiguous rows, any row stride). Slots
    of one expert keep their order; an id outside 0 .. n_experts - 1 leaves its
    slot out (its row comes behind all experts'). Up to 1024 experts and slots."""
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda:
        raise ValueError("ids must be a CUDA tensor")
    size = _INT_BYTES.get(ids.dtype)
    if size is None:
        raise ValueError(f"ids is {ids.dtype}: int32 and int64 are supported")
    if ids.dim() != 2:
        raise ValueError(f"ids must be 2-D (tokens, slots), got shape {tuple(ids.shape)}")
    if not 1 <= n_experts <= MAX_EXPERTS:
        raise ValueError(f"n_experts must be in [1, {MAX_EXPERTS}], got {n_experts}")
    tokens, slots = ids.shape
    ptr, ld = _matrix("ids", ids, tokens, slots, ids)
    offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=ids.device)
    rows = torch.empty((tokens, slots), dtype=torch.int32, device=ids.device)
    source = torch.empty(tokens * slots, dtype=torch.int32, device=ids.device)
    args = _SORT.pack(tokens, slots, n_experts, size, ptr, ld, offsets.data_ptr(), rows.data_ptr(), source.data_ptr())
    need = _known_size(("sort", tokens, slots, n_experts), "shampoo_sort_workspace_size", args)
    ws, keep = _workspace(need, ids)
    _call("shampoo_sort_tokens", args, ids.get_device(), ws, need)
    return Plan(offsets, rows, source)


def _plan_rows(plan, like):
    """(pointer, tokens, slots) of a plan's rows."""
    rows = plan.rows
    if rows.dtype is not torch.int32 or rows.get_device() != like.get_device() or rows.dim() != 2 or not rows.is_contiguous():
        raise ValueError("plan.rows must be a contiguous 2-D int32 tensor on the call's device")
    return rows.data_ptr(), rows.shape[0], rows.shape[1]


def _weights(name, weights, tokens, slots, like):
    if weights.dtype is not torch.float32 or weights.get_device() != like.get_device():
        raise ValueError(f"{name} is {weights.dtype} on {weights.device}, expected torch.float32 on {like.device}")
    if weights.shape != (tokens, slots) or not weights.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape ({tokens}, {slots}), got {tuple(weights.shape)}")
    return weights.data_ptr()


def dispatch(x, plan):
    """xs [tokens * slots, width]: row plan.rows[t, j] is x[t], for x [tokens,
    width]; rows of slots left out are 0."""
    dt, n, d = _first("x", x)
    rows, tokens, slots = _plan_rows(plan, x)
    px, lx = _matrix("x", x, tokens, d, x)
    xs = x.new_empty((tokens * slots, d))
    _call("shampoo_dispatch", _ROUTE.pack(tokens, d, slots, dt, rows, 0, px, 0, lx, 0, 0, xs.data_ptr(), 0, d, 0), x.get_device())
    return xs


def combine(ys, plan, weights=None):
    """y [tokens, width]: y[t] = sum over j of weights[t, j] * ys[plan.rows[t, j]],
    for ys [tokens * slots, width]; slots left out add nothing, and what their rows
    and weights hold is not read. weights: float32 [tokens, slots], or None for 1."""
    dt, n, d = _first("ys", ys)
    rows, tokens, slots = _plan_rows(plan, ys)
    py, ly = _matrix("ys", ys, tokens * slots, d, ys)
    pw = _weights("weights", weights, tokens, slots, ys) if weights is not None else 0
    y = ys.new_empty((tokens, d))
    _call("shampoo_combine", _ROUTE.pack(tokens, d, slots, dt, rows, pw, 0, py, 0, ly, y.data_ptr(), 0, d, 0, 0), ys.get_device())
    return y


def dispatch_backward(dxs, plan):
    """Gradient of `dispatch`: dx [tokens, width], the sum of a token's rows of dxs."""
    return combine(dxs, plan)


def combine_backward(dy, ys, plan, weights=None):
    """Gradients of `combine` from dy [tokens, width]: (dys, dweights). dys rows of
    slots left out are 0, and so are their dweights (float32; None without weights)."""
    if weights is None:
        return dispatch(dy, plan), None
    dt, n, d = _first("dy", dy)
    rows, tokens, slots = _plan_rows(plan, dy)
    pdy, ldy = _matrix("dy", dy, tokens, d, dy)
    pys, lys = _matrix("ys", ys, tokens * slots, d, dy)
    pw = _weights("weights", weights, tokens, slots, dy)
    dys = dy.new_empty((tokens * slots, d))
    dweights = torch.empty((tokens, slots), dtype=torch.float32, device=dy.device)
    _call("shampoo_combine_backward", _ROUTE.pack(tokens, d, slots, dt, rows, pw, pdy, pys, ldy, lys, 0, dys.data_ptr(), 0, d, dweights.data_ptr()),
          dy.get_device())
    return dys, dweights
