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


# ------------------------------------------------------------ products in 8 bits
def quantized(x, dims):
    """(values, exponents) of x by blocks of 128 along `dims` together: values in float64 over 2^exponent, from the format's
    definition (e4m3: three bits behind the leading one, exponents from -6, to nearest even), NaN where x is not finite."""
    x = x.double()
    dims = [d % x.dim() for d in dims]
    split, inner, pads = [], [], []
    for i, m in enumerate(x.shape):
        pads.append(-m % 128 if i in dims else 0)
        split += [(m + pads[i]) // 128, 128] if i in dims else [m]
        if i in dims:
            inner.append(len(split) - 1)
    p = torch.zeros([m + q for m, q in zip(x.shape, pads)], dtype=torch.float64)
    p[tuple(slice(0, m) for m in x.shape)] = x
    p = p.reshape(split)
    amax = torch.where(torch.isfinite(p), p.abs(), 0.0).amax(inner, keepdim=True)
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [1/2, 1); 448 = 7/8 2^9
    e = torch.where(amax > 0, torch.where(m > 0.875, e - 8, e - 9), -126).clamp(min=-126)
    v = torch.ldexp(p, -e.to(torch.float64))
    _, top = torch.frexp(v)
    step = torch.exp2((top - 1).clamp(min=-6).double() - 3)
    q = torch.where(torch.isfinite(v), torch.round(v / step) * step, float("nan"))
    e = e.expand_as(p).reshape([m + t for m, t in zip(x.shape, pads)])[tuple(slice(0, m) for m in x.shape)]
    return q.reshape([m + t for m, t in zip(x.shape, pads)])[tuple(slice(0, m) for m in x.shape)], e


def rounded(x, dims):
    """x in 8 bits, as the float64 values that these stand for."""
    q, e = quantized(x, dims)
    return torch.ldexp(q, e.double())


def expert_rows(offsets, rows):
    """(expert, slice) of each expert's rows; one of all rows without offsets."""
    if offsets is None:
        return [(0, slice(0, rows))]
    return [(e, slice(int(offsets[e]), int(offsets[e + 1]))) for e in range(len(offsets) - 1)]


def product(x, w, offsets=None):
    """(y, root sum of squares of each result's terms, sum of their magnitudes) for w [experts, in, out]."""
    y = torch.zeros(3, x.shape[0], w.shape[2], dtype=torch.float64)
    w = rounded(w, (-2, -1))
    for e, part in expert_rows(offsets, x.shape[0]):
        q = rounded(x[part], (1,))
        y[0, part], y[1, part], y[2, part] = q @ w[e], (q.square() @ w[e].square()).sqrt(), q.abs() @ w[e].abs()
    return y


def product_dw(x, dy, offsets, experts):
    """The same three of dw [experts, in, out]."""
    dw = torch.zeros(3, experts, x.shape[1], dy.shape[1], dtype=torch.float64)
    for e, part in expert_rows(offsets, x.shape[0]):
        q, g = rounded(x[part], (0,)).t(), rounded(dy[part], (0,))
        dw[0, e], dw[1, e], dw[2, e] = q @ g, (q.square() @ g.square()).sqrt(), q.abs() @ g.abs()
    return dw


def largest_of_groups(a, b):
    """Sum over groups of eight k of the largest |a[m][k] b[k][n]| of each: what the 8-bit matrix instruction's loss goes by."""
    total = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float64)
    for k in range(0, a.shape[1], 8):
        total += (a[:, k:k + 8, None].abs() * b[None, k:k + 8].abs()).amax(1)
    return total
