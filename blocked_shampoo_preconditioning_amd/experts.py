"""The experts' path of a feed-forward block, forward and backward, on the
library's own kernels: tokens sorted by expert and back, with weights applied,
and matrix products in 8-bit floating point with a scale for each block of 128,
dense or one matrix an expert (the C ABI in include/shampoo_experts.h).

    w8 = experts.quantize_weight(w)                                # w [n_experts, in, out], once
    plan = experts.sort_tokens(ids, n_experts)                     # ids [tokens, slots]: each token's experts
    ys = experts.product8_forward(x, w8, plan, gather=True)        # each expert's matrix on its tokens
    y = experts.combine(ys, plan, weights)                         # back, with the router's weights

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

from . import shampoo as _s
from .layer import _first, _matrix, _raw_stream, _workspace
from .shampoo import HEADER_PATH as _CORE_HEADER

EXPERTS_HEADER_PATH = os.path.join(os.path.dirname(_CORE_HEADER), "shampoo_experts.h")
MAX_EXPERTS = 1024

# The C argument structs, field by field (native sizes and alignment), as in `layer`.
_SORT = struct.Struct("@q iii P q PPP")
_ROUTE = struct.Struct("@qq ii PP PP qq PP qq P")
_WEIGHT = struct.Struct("@qq ii P qq PPPP")
_PRODUCT = struct.Struct("@qqq ii PP q i P PPPP P q P q P P q P q P qq")

_A, _SIZE = ctypes.c_char_p, ctypes.POINTER(ctypes.c_size_t)
_SIGNATURES = {
    "shampoo_sort_workspace_size": [_A, _SIZE],
    "shampoo_sort_tokens": [_A, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
    "shampoo_dispatch": [_A, ctypes.c_void_p],
    "shampoo_combine": [_A, ctypes.c_void_p],
    "shampoo_combine_backward": [_A, ctypes.c_void_p],
    "shampoo_quantize_weight": [_A, ctypes.c_void_p],
    "shampoo_product8_saved_size": [_A, _SIZE],
    "shampoo_product8_workspace_size": [_A, ctypes.c_int32, _SIZE],
    "shampoo_product8_forward": [_A, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
    "shampoo_product8_backward": [_A, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
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
    rows = torch.empty_like(ids, dtype=torch.int32, memory_format=torch.contiguous_format)
    offsets, source = rows.new_empty(n_experts + 1), rows.new_empty(tokens * slots)
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


# --------------------------------------------------------- products in 8 bits
class Weight8(NamedTuple):
    """8-bit weights of one [n_in, n_out] matrix, or of one for each expert (a leading dimension more), as
    `quantize_weight` returns them; a program may make them itself from values and scales that it has.
    values float8_e4m3fn [n_out, n_in rounded up to 128]: the transposed matrix over its scales, 0 behind n_in.
    scales float8_e8m0fnu [n_out / 128, n_in / 128], both rounded up, then the latter up to a multiple of 4: a
    power of two (2^-126 .. 2^127) for each block of 128 x 128.
    back_values, back_scales: the same with in and out exchanged, for `product8_backward`'s dx (or None)."""
    values: torch.Tensor
    scales: torch.Tensor
    n_in: int
    n_out: int
    back_values: torch.Tensor | None = None
    back_scales: torch.Tensor | None = None


_MAX_DIM = 1 << 21


def _blocks(n):
    return (n + 127) // 128


def _weight_shapes(lead, n_in, n_out):
    return (*lead, n_out, _blocks(n_in) * 128), (*lead, _blocks(n_out), (_blocks(n_in) + 3) // 4 * 4)


def quantize_weight(w, backward=False):
    """`Weight8` of w [in, out], or [n_experts, in, out] (contiguous rows, any distance apart; matrices one behind the
    other, or side by side as in a transposed view of [in, n_experts, out], any distance apart):
    every block of 128 x 128 over the smallest power of two that brings it to 448 at most, rounded to e4m3.
    backward: also as dx needs it."""
    if not isinstance(w, torch.Tensor) or not w.is_cuda:
        raise ValueError("w must be a CUDA tensor")
    if w.dim() not in (2, 3):
        raise ValueError(f"w must be [in, out] or [experts, in, out], got shape {tuple(w.shape)}")
    flat = w if w.dim() == 3 else w[None]
    n_experts, n_in, n_out = flat.shape
    if not (1 <= n_experts <= MAX_EXPERTS and 1 <= n_in <= _MAX_DIM and 1 <= n_out <= _MAX_DIM):
        raise ValueError(f"w has shape {tuple(w.shape)}: up to {MAX_EXPERTS} matrices of 1 to 2^21 rows and columns are supported")
    dt, _, _ = _first("w", flat[0])
    ptr, ld = _matrix("w", flat[0], n_in, n_out, w)
    stride = flat.stride(0) if n_experts > 1 else n_in * ld
    lead = w.shape[:-2]
    made = []
    for rows, cols in ((n_in, n_out), (n_out, n_in)) if backward else ((n_in, n_out),):
        values, scales = _weight_shapes(lead, rows, cols)
        made.append(torch.empty(values, dtype=torch.float8_e4m3fn, device=w.device))
        made.append(torch.empty(scales, dtype=torch.float8_e8m0fnu, device=w.device))
    pointers = [t.data_ptr() for t in made] + [0, 0] * (not backward)
    _call("shampoo_quantize_weight", _WEIGHT.pack(n_in, n_out, n_experts, dt, ptr, ld, stride, *pointers), w.get_device())
    return Weight8(made[0], made[1], n_in, n_out, *made[2:])


_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _weight_pointers(name, values, scales, lead, n_in, n_out, like):
    """Pointers of 8-bit weights of these sizes, leading dimensions and device."""
    dev = like.get_device()
    shape, scale_shape = _weight_shapes(lead, n_in, n_out)
    if values.dtype is _E4M3 and scales.dtype is _E8M0 and values.get_device() == dev and scales.get_device() == dev and \
            values.shape == shape and scales.shape == scale_shape and values.is_contiguous() and scales.is_contiguous():
        return values.data_ptr(), scales.data_ptr()
    for t, dtype, want, what in ((values, _E4M3, shape, "values"), (scales, _E8M0, scale_shape, "scales")):
        if t.dtype is not dtype or t.get_device() != dev:
            raise ValueError(f"{name}{what} must be a {dtype} tensor on {like.device}, got {t.dtype} on {t.device}")
        if t.shape != want or not t.is_contiguous():
            raise ValueError(f"{name}{what} must be contiguous with shape {tuple(want)}, got {tuple(t.shape)}")


def _offsets(plan, n_experts, like):
    """Pointer of a plan's offsets."""
    offsets = plan.offsets
    if offsets.dtype is not torch.int32 or offsets.get_device() != like.get_device() or not offsets.is_contiguous():
        raise ValueError("plan.offsets must be a contiguous int32 tensor on the call's device")
    if offsets.shape != (n_experts + 1,):
        raise ValueError(f"plan.offsets has shape {tuple(offsets.shape)}, expected ({n_experts + 1},)")
    return offsets.data_ptr()


def _lead(w8, plan):
    """Leading dimensions of the weights (none, or experts) and how many matrices they are."""
    lead = w8.values.shape[:-2]
    if len(lead) > 1:
        raise ValueError(f"w8.values has shape {tuple(w8.values.shape)}: one matrix, or one for each expert")
    if plan is None:
        if lead:
            raise ValueError("plan is None: with a matrix for each expert it says which rows are whose")
        return lead, 1
    return lead, lead[0] if lead else 1


def product8_forward(x, w8, plan=None, gather=False, save=False):
    """y = Q(x) W for x [rows, in] and the 8-bit weights W of `w8`, where Q rounds every 128 columns of a row to
    e4m3 over their own power of two. With a plan, rows are those of `dispatch` and meet their expert's
    matrix; with `gather` x has a row for each token, and the product takes them by plan.source itself. y [rows,
    out]; rows behind the last expert's are 0. With `save` returns (y, saved), saved being what
    `product8_backward` needs for dw (an opaque tensor: x in 8 bits by 128 rows of a column)."""
    n_in, n_out = w8.n_in, w8.n_out
    dt, x_rows, _ = _first("x", x)
    lead, n_experts = _lead(w8, plan)
    rows, offsets, source, slots, slot_rows = x_rows, 0, 0, 1, 0
    if plan is not None:
        offsets = _offsets(plan, n_experts, x)
        slot_rows, tokens, slots = _plan_rows(plan, x)
        rows = tokens * slots
        if gather:
            x_rows, src = tokens, plan.source
            if src.dtype is not torch.int32 or src.get_device() != x.get_device() or src.shape != (rows,) or not src.is_contiguous():
                raise ValueError(f"plan.source must be a contiguous int32 tensor of {rows} elements on the call's device")
            source = src.data_ptr() or 256
        else:
            x_rows = rows
    elif gather:
        raise ValueError("gather needs a plan")
    px, lx = _matrix("x", x, x_rows, n_in, x)
    values, scales = _weight_pointers("w8.", w8.values, w8.scales, lead, n_in, n_out, x)
    y = x.new_empty((rows, n_out))
    head = (rows, n_in, n_out, n_experts, dt, offsets, source, x_rows, slots or 1, slot_rows)
    key = (rows, n_in, n_out, n_experts, dt, plan is None)
    saved = None
    if save:
        size = _known_size(("saved", key), "shampoo_product8_saved_size", _PRODUCT.pack(*head, *_NO_PRODUCT))
        saved = torch.empty(size, dtype=torch.uint8, device=x.device)
    args = _PRODUCT.pack(*head, values, scales, 0, 0, px, lx, y.data_ptr(), n_out, saved.data_ptr() if save else 0, 0, 0, 0, 0, 0, 0, 0)
    if rows <= _FEW_ROWS and not save:
        size = ws = 0
    else:
        size = _known_size(("forward", key, save), "shampoo_product8_workspace_size", args, 0)
        ws, keep = _workspace(size, x)
    _call("shampoo_product8_forward", args, x.get_device(), ws, size)
    return (y, saved) if save else y


_FEW_ROWS = 64  # up to here a call that saves nothing needs no workspace
_NO_PRODUCT = (0,) * 16


def product8_backward(dy, w8, saved, plan=None, need_dx=True, need_dw=True):
    """(dx, dw) from dy [rows, out], the forward pass's w8 and plan and what it saved: dx = Q(dy) W^T by rows, [rows,
    in] (with a plan in sorted order: `dispatch_backward` takes it to the tokens), and dw = Q(x)^T Q(dy) with both by
    128 rows of a column, in w's shape and dy's dtype. The roundings of x, W and dy themselves have gradient 1.
    need_dx (needs w8.back_values) / need_dw (needs saved): None is returned for what is not needed."""
    n_in, n_out = w8.n_in, w8.n_out
    dt, rows, _ = _first("dy", dy)
    lead, n_experts = _lead(w8, plan)
    offsets = 0
    if plan is not None:
        offsets = _offsets(plan, n_experts, dy)
        _, tokens, slots = _plan_rows(plan, dy)
        rows = tokens * slots
    pdy, ldy = _matrix("dy", dy, rows, n_out, dy)
    back = (0, 0)
    if need_dx:
        if w8.back_values is None:
            raise ValueError("w8 has no backward values: quantize_weight(w, backward=True)")
        back = _weight_pointers("w8.back_", w8.back_values, w8.back_scales, lead, n_out, n_in, dy)
    head = (rows, n_in, n_out, n_experts, dt, offsets, 0, rows, 1, 0)
    key = (rows, n_in, n_out, n_experts, dt, plan is None)
    dx = dw = None
    if need_dx:
        dx = dy.new_empty((rows, n_in))
    psaved = 0
    if need_dw:
        size = _known_size(("saved", key), "shampoo_product8_saved_size", _PRODUCT.pack(*head, *_NO_PRODUCT))
        if not isinstance(saved, torch.Tensor) or saved.dtype is not torch.uint8 or saved.numel() != size or saved.get_device() != dy.get_device() or not saved.is_contiguous():
            raise ValueError("saved is not what product8_forward kept for these sizes")
        psaved = saved.data_ptr()
        dw = dy.new_empty((*lead, n_in, n_out))
    if need_dx or need_dw:
        args = _PRODUCT.pack(*head, 0, 0, *back, 0, 0, 0, 0, psaved, pdy, ldy, (dx.data_ptr() or 256) if need_dx else 0, n_in,
                             dw.data_ptr() if need_dw else 0, n_out, n_in * n_out)
        size = _known_size(("backward", key, need_dx, need_dw), "shampoo_product8_workspace_size", args, 1)
        ws, keep = _workspace(size, dy)
        _call("shampoo_product8_backward", args, dy.get_device(), ws, size)
    return dx, dw
