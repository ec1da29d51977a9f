"""Plain 64-bit forms of the layer operators, for the tests: definitions in
torch.float64 on the CPU, gradients from the formulas, and dropout's words from
a pure-integer Philox4x32-10."""
from __future__ import annotations

import math

import numpy as np
import torch

BF16_STEP = 2.0 ** -9   # largest relative error of one rounding to bf16
F32_STEP = 2.0 ** -24   # and to fp32


def rel(a, b, terms=None):
    """2-norm of a - b over that of b (of a where b is zero), or over that of
    `terms`, the root sum of squares of the terms that b's elements are sums
    of, where it is larger: terms that cancel keep their own roundings."""
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    nb = float(torch.linalg.vector_norm(b))
    if terms is not None:
        nb = max(nb, float(torch.linalg.vector_norm(terms)))
    return float(torch.linalg.vector_norm(a - b)) / (nb if nb > 0 else 1.0)


def act(g, name):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        k, c = math.sqrt(2 / math.pi), 0.044715
        t = torch.tanh(k * (g + c * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * c * g * g)
    return torch.relu(g), (g > 0).double()


def ffn(x, wg, wu, wd, name, dy=None):
    """y, and with dy also (dx, dwg, dwu, dwd) and the root sums of squares of the five results' terms."""
    x, wg, wu, wd = (t.detach().double().cpu() for t in (x, wg, wu, wd))
    g, u = x @ wg, x @ wu
    a, da = act(g, name)
    h = a * u
    y = h @ wd
    if dy is None:
        return y
    dy = dy.detach().double().cpu()
    dh = dy @ wd.T
    dg, du = dh * u * da, dh * a
    x2, g2, u2, h2, y2 = (t.square() for t in (x, dg, du, h, dy))
    terms = (h2 @ wd.square(), g2 @ wg.square().T + u2 @ wu.square().T, x2.T @ g2, x2.T @ u2, h2.T @ y2)
    return y, (dg @ wg.T + du @ wu.T, x.T @ dg, x.T @ du, h.T @ dy), [t.sqrt() for t in terms]


def philox(counter, key):
    """Philox4x32-10 of one counter (four words) under a two-word key, in Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def drop_factors(rows, cols, p, seed, offset):
    """0 or 1 / (1 - p) for each element, p rounded to a multiple of 2^-16."""
    t = min(65535, round(p * 65536))
    out = np.zeros((rows, -(-cols // 8) * 8))
    for r in range(rows):
        for c in range(out.shape[1] // 8):
            w = philox((c, r & 0xFFFFFFFF, r >> 32, offset), (seed & 0xFFFFFFFF, seed >> 32))
            out[r, 8 * c:8 * c + 8] = [h >= t for x in w for h in (x & 0xFFFF, x >> 16)]
    return torch.from_numpy(out[:, :cols] * (65536 / (65536 - t)))


def norm(v, kind, w, b, eps):
    """norm(v), v^ and 1 / deviation."""
    if kind == "none":
        return v, v, None
    c = v - v.mean(1, keepdim=True) if kind == "layer" else v
    rstd = (c.square().mean(1, keepdim=True) + eps).rsqrt()
    hat = c * rstd
    return (hat * w if w is not None else hat) + (b if b is not None else 0), hat, rstd


def norm_grad(dn, hat, rstd, kind, w):
    if kind == "none":
        return dn
    c = dn * w if w is not None else dn
    dv = c - hat * (c * hat).mean(1, keepdim=True)
    return rstd * (dv - c.mean(1, keepdim=True) if kind == "layer" else dv)


def residual(x, z, s, mask=None, dr=None, dn=None):
    """r, n and, with gradients coming in, a dict of gradients and the terms' size of those that can cancel. s: settings as
    layer.residual_forward takes them."""
    def f(t):
        return t.detach().double().cpu() if t is not None else None
    x, z = f(x), f(z)
    wp, bp, wn, bn, gate = (f(s.get(k)) for k in ("post_weight", "post_bias", "next_weight", "next_bias", "gate"))
    n, d = x.shape
    post, nxt, eps, alpha = s.get("post", "rms"), s.get("next", "rms"), s.get("eps", 1e-6), s.get("residual_scale", 1.0)
    rpg = s.get("rows_per_gate") or max(n, 1)
    rows = torch.arange(n) // rpg
    g = gate[rows] if gate is not None else torch.ones(n, d, dtype=torch.float64)
    m = mask if mask is not None else torch.ones(n, d, dtype=torch.float64)
    p, zh, zr = norm(z, post, wp, bp, eps)
    r = alpha * x + g * p * m
    out, rh, rr = norm(r, nxt, wn, bn, eps)
    if dr is None and dn is None:
        return r, (None if nxt == "none" else out), None, None
    dr = f(dr) if dr is not None else torch.zeros(n, d, dtype=torch.float64)
    grads = {}
    if nxt != "none":
        dn = f(dn)
        grads["next_weight"], grads["next_bias"] = (dn * rh).sum(0), dn.sum(0)
        dr = dr + norm_grad(dn, rh, rr, nxt, wn)
    db = dr * m
    dp = db * g
    grads["x"] = alpha * dr
    sizes = {"x": alpha * dn * (wn if wn is not None else 1) * rr} if nxt != "none" else {}
    if post != "none":
        sizes["z"] = dp * (wp if wp is not None else 1) * zr
    grads["z"] = norm_grad(dp, zh, zr, post, wp)
    grads["post_weight"], grads["post_bias"] = (dp * zh).sum(0), dp.sum(0)
    if gate is not None:
        grads["gate"] = torch.zeros(gate.shape, dtype=torch.float64).index_add_(0, rows, db * p)
    return r, (None if nxt == "none" else out), grads, sizes
