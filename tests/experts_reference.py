"""Plain 64-bit forms of the experts' path, for the tests (CPU, numpy and torch)."""
import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # largest relative error of one rounding


def plan(ids, experts):
    """(offsets, rows, source) of a [tokens, slots] array of ids, by going through the slots one expert at a time."""
    flat = np.asarray(ids, dtype=np.int64).reshape(-1)
    lists = [np.flatnonzero(flat == e) for e in range(experts)] + [np.flatnonzero((flat < 0) | (flat >= experts))]
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in lists[:experts]])])
    slots = np.concatenate(lists) if flat.size else np.zeros(0, np.int64)
    rows = np.empty(flat.size, np.int64)
    rows[slots] = np.arange(flat.size)
    out = (flat < 0) | (flat >= experts)
    return offsets, np.where(out, ~rows, rows).reshape(np.shape(ids)), np.where(out[slots], ~slots, slots)


def kept_pairs(rows):
    """(token, slot, row) arrays of the slots that take part."""
    t, j = np.nonzero(rows >= 0)
    return torch.from_numpy(t), torch.from_numpy(j), torch.from_numpy(rows[t, j])


def dispatch(x, rows):
    t, _, r = kept_pairs(rows)
    xs = torch.zeros(rows.size, x.shape[1], dtype=torch.float64)
    xs[r] = x.double()[t]
    return xs


def combine(ys, rows, weights=None):
    """(y, sum of the terms' magnitudes)."""
    t, j, r = kept_pairs(rows)
    w = weights.double()[t, j][:, None] if weights is not None else 1.0
    terms = ys.double()[r] * w
    y = torch.zeros(rows.shape[0], ys.shape[1], dtype=torch.float64)
    return y.index_add(0, t, terms), y.index_add(0, t, terms.abs())


def combine_backward(dy, ys, rows, weights):
    """(dys, dweights, sum of the magnitudes of dweights' terms)."""
    t, j, r = kept_pairs(rows)
    dys = torch.zeros(rows.size, dy.shape[1], dtype=torch.float64)
    dys[r] = dy.double()[t] * weights.double()[t, j][:, None]
    terms = dy.double()[t] * ys.double()[r]
    dw, size = torch.zeros(rows.shape, dtype=torch.float64), torch.zeros(rows.shape, dtype=torch.float64)
    dw[t, j], size[t, j] = terms.sum(1), terms.abs().sum(1)
    return dys, dw, size
