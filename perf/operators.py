"""The measured cases of the feed-forward half of a decoder layer, forward and backward: the gated feed-forward block, the norms
before and after a block with gate, dropout and residual scale, and counter-based dropout.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once at the end), or, where `own` is
true, by the framework's entry points in `blocked_shampoo_preconditioning_amd.layer`."""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MASK32 = 0xFFFFFFFF


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a 1B-class decoder while it is sampled from: every weight is read for one row
        {"name": "ffn_one_token_bf16", "op": "ffn", "train": False, "tokens": 1, "d": 2048, "f": 8192, "act": "silu", "dtype": "bf16"},
        # a few tokens (a small batch of requests), fp32 weights, GPT-small width
        {"name": "ffn_few_tokens_f32", "op": "ffn", "train": False, "tokens": 13, "d": 768, "f": 2048, "act": "gelu", "dtype": "f32"},
        # the training step of one layer of the 1B-class set on four sequences of 2048
        {"name": "ffn_train_1b_bf16", "op": "ffn", "train": True, "tokens": 8192, "d": 2048, "f": 8192, "act": "silu", "dtype": "bf16"},
        # the same at GPT-small width on one sequence of 1024: too few tiles to fill the card
        {"name": "ffn_train_small_bf16", "op": "ffn", "train": True, "tokens": 1024, "d": 768, "f": 2048, "act": "gelu", "dtype": "bf16"},
        # fp32 training at GPT-small width
        {"name": "ffn_train_f32", "op": "ffn", "train": True, "tokens": 4096, "d": 768, "f": 2048, "act": "silu", "dtype": "f32"},
        # packed sequences of uneven length and widths that are no multiple of 8
        {"name": "ffn_train_ragged_bf16", "op": "ffn", "train": True, "tokens": 1537, "d": 1001, "f": 2730, "act": "relu", "dtype": "bf16"},
        # the norms around a block for one token
        {"name": "norm_one_token_bf16", "op": "norm", "train": False, "tokens": 1, "d": 2048, "kind": "rms", "gate": "channel",
         "alpha": 1.0, "p": 0.0, "dtype": "bf16"},
        # the norms around a block in training at the 1B-class width, with dropout and a learned gate for each channel
        {"name": "norm_train_1b_bf16", "op": "norm", "train": True, "tokens": 16384, "d": 2048, "kind": "rms", "gate": "channel",
         "alpha": 1.0, "p": 0.1, "dtype": "bf16"},
        # fp32 layer norms of odd width, a gate for each sequence, a scaled residual
        {"name": "norm_train_ragged_f32", "op": "norm", "train": True, "tokens": 3001, "d": 777, "kind": "layer", "gate": "sequence",
         "alpha": 0.75, "p": 0.2, "dtype": "f32"},
        # dropout of hidden activations of one layer, both directions
        {"name": "dropout_hidden_bf16", "op": "dropout", "tokens": 8192, "d": 8192, "p": 0.1, "dtype": "bf16"},
        # dropout of a small odd array: latency
        {"name": "dropout_small_f32", "op": "dropout", "tokens": 257, "d": 1001, "p": 0.5, "dtype": "f32"},
        # the whole feed-forward half of a layer in training: norm, block, dropout, gate, norm, residual, next norm, and all gradients
        {"name": "half_layer_train_bf16", "op": "half", "train": True, "tokens": 4096, "d": 768, "f": 2048, "act": "silu", "kind": "rms",
         "gate": "channel", "alpha": 1.0, "p": 0.1, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width over its logarithm: mostly a multiple of 64, some of 8, some of nothing."""
    n = _log(rng, lo, hi)
    step = rng.choice((64, 64, 64, 8, 1))
    return min(hi, max(step, n // step * step))


def draw(rng):
    op = rng.choice(("ffn_serve", "ffn", "ffn", "norm_serve", "norm", "dropout", "half"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    act, kind = rng.choice(("silu", "gelu", "relu")), rng.choice(("rms", "layer"))
    gate, alpha = rng.choice(("none", "channel", "sequence")), rng.choice((1.0, 0.75))
    p = rng.choice((0.0, 0.1, 0.3))
    if op == "ffn_serve":
        return {"op": "ffn", "train": False, "tokens": _log(rng, 1, 64), "d": _width(rng, 256, 2048), "f": _width(rng, 512, 8192),
                "act": act, "dtype": dtype}
    if op == "ffn":
        return {"op": "ffn", "train": True, "tokens": _log(rng, 1, 8192), "d": _width(rng, 64, 2048), "f": _width(rng, 128, 8192),
                "act": act, "dtype": dtype}
    if op == "norm_serve":
        return {"op": "norm", "train": False, "tokens": _log(rng, 1, 64), "d": _width(rng, 64, 8192), "kind": kind, "gate": gate,
                "alpha": alpha, "p": 0.0, "dtype": dtype}
    if op == "norm":
        return {"op": "norm", "train": True, "tokens": _log(rng, 1, 16384), "d": _width(rng, 64, 2048), "kind": kind, "gate": gate,
                "alpha": alpha, "p": p, "dtype": dtype}
    if op == "dropout":
        return {"op": "dropout", "tokens": _log(rng, 1, 8192), "d": _log(rng, 64, 8192), "p": rng.choice((0.05, 0.1, 0.5)), "dtype": dtype}
    return {"op": "half", "train": True, "tokens": _log(rng, 16, 4096), "d": _width(rng, 64, 768), "f": _width(rng, 128, 2048),
            "act": act, "kind": kind, "gate": gate, "alpha": alpha, "p": p, "dtype": dtype}


def _rows_per_gate(case):
    """Tokens that share a row of the gate: all for a gate per channel, a sequence's for a gate per sequence."""
    return max(1, case["tokens"]) if case["gate"] != "sequence" else max(1, -(-case["tokens"] // 4))


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    n, d, op = case["tokens"], case["d"], case["op"]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dt)

    s = {"case": case, "seed": (seed * 2654435761 + 12345) & 0xFFFFFFFFFFFF, "offset": seed % 1000}
    if op == "dropout":
        s["x"], s["dy"] = normal(n, d), normal(n, d, std=1e-2)
        return s
    s["x"] = normal(n, d)
    if op in ("ffn", "half"):  # weights as they are at the start of training
        f = case["f"]
        s["w_gate"], s["w_up"], s["w_down"] = normal(d, f, std=d ** -0.5), normal(d, f, std=d ** -0.5), normal(f, d, std=f ** -0.5)
        if op == "ffn" and case["train"]:
            s["dy"] = normal(n, d, std=1e-2)
    if op in ("norm", "half"):
        layer = case["kind"] == "layer"
        for name in ("post", "next") + (("pre",) if op == "half" else ()):
            s[name + "_weight"] = normal(d, std=0.1, mean=1.0)
            s[name + "_bias"] = normal(d, std=0.1) if layer else None
        rows = -(-n // _rows_per_gate(case))
        s["gate"] = normal(rows, d, std=0.3, mean=0.5) if case["gate"] != "none" else None
        if op == "norm":
            s["z"] = normal(n, d, std=0.5, mean=0.1)
        if case["train"]:
            s["dr"], s["dn"] = normal(n, d, std=1e-2), normal(n, d, std=1e-2)
    return s


def _kwargs(s):
    """The settings of the norms around a block, as the framework's calls take them."""
    c = s["case"]
    return dict(post=c["kind"], post_weight=s["post_weight"], post_bias=s["post_bias"], gate=s["gate"], rows_per_gate=_rows_per_gate(c),
                residual_scale=c["alpha"], dropout=c["p"], seed=s["seed"], offset=s["offset"], next=c["kind"],
                next_weight=s["next_weight"], next_bias=s["next_bias"], eps=1e-6)


# ----------------------------------------------------------------------- run
def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    out = {"dropout": _plain_dropout, "ffn": _plain_ffn, "norm": _plain_norm, "half": _plain_half}[case["op"]](s)
    return {k: v.to(dt) for k, v in out.items() if v is not None}


def _run_own(s):
    from blocked_shampoo_preconditioning_amd import layer
    c = s["case"]
    if c["op"] == "dropout":
        return {"y": layer.dropout(s["x"], c["p"], s["seed"], s["offset"]),
                "dx": layer.dropout(s["dy"], c["p"], s["seed"], s["offset"])}
    if c["op"] == "ffn":
        if not c["train"]:
            return {"y": layer.ffn_forward(s["x"], s["w_gate"], s["w_up"], s["w_down"], activation=c["act"])}
        y, saved = layer.ffn_forward(s["x"], s["w_gate"], s["w_up"], s["w_down"], activation=c["act"], save=True)
        dx, dwg, dwu, dwd = layer.ffn_backward(s["dy"], s["x"], s["w_gate"], s["w_up"], s["w_down"], saved, activation=c["act"])
        return {"y": y, "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}
    kw = _kwargs(s)
    if c["op"] == "norm":
        r, n, stats = layer.residual_forward(s["x"], s["z"], **kw)
        if not c["train"]:
            return {"r": r, "n": n}
        g = layer.residual_backward(s["dr"], s["dn"], r, s["z"], stats, **kw)
        return {k: v for k, v in {"r": r, "n": n, **{"d" + k: v for k, v in g.items()}}.items() if v is not None}
    pre = dict(kind=c["kind"], weight=s["pre_weight"], bias=s["pre_bias"], eps=1e-6)
    a, pre_stats = layer.norm_forward(s["x"], **pre)
    w = (s["w_gate"], s["w_up"], s["w_down"])
    z, saved = layer.ffn_forward(a, *w, activation=c["act"], save=True)
    r, n, stats = layer.residual_forward(s["x"], z, **kw)
    g = layer.residual_backward(s["dr"], s["dn"], r, z, stats, **kw)
    da, dwg, dwu, dwd = layer.ffn_backward(g["z"], a, *w, saved, activation=c["act"])
    h = layer.norm_backward(da, s["x"], pre_stats, dr=g["x"], **pre)
    out = {"r": r, "n": n, "dx": h["x"], "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd, "dpre_weight": h["weight"], "dpre_bias": h["bias"],
           "dgate": g["gate"]}
    out.update({"d" + k: g[k] for k in ("post_weight", "post_bias", "next_weight", "next_bias")})
    return {k: v for k, v in out.items() if v is not None}


# --------------------------------------------------------------- plain forms
def _mul_hi_lo(a, m):
    """High and low 32 bits of a * m for 32-bit values held in 64, by 16-bit limbs (no product passes 2^48)."""
    low = (a & 0xFFFF) * m
    up = (a >> 16) * m + (low >> 16)
    return up >> 16, ((up & 0xFFFF) << 16) | (low & 0xFFFF)


def _plain_mask(rows, cols, p, seed, offset, device):
    """Dropout factors (0 or 1 / (1 - p)) of a rows x cols array: 16 bits each of Philox4x32-10 on (column group, row, offset)."""
    drop = min(65535, int(round(p * 65536)))
    groups = -(-cols // 8)
    row = torch.arange(rows, device=device, dtype=torch.int64)[:, None]
    c = [torch.arange(groups, device=device, dtype=torch.int64)[None, :].expand(rows, groups), (row & MASK32).expand(rows, groups),
         (row >> 32).expand(rows, groups), torch.full((rows, groups), offset, device=device, dtype=torch.int64)]
    k0, k1 = seed & MASK32, (seed >> 32) & MASK32
    for _ in range(10):
        h0, l0 = _mul_hi_lo(c[0], 0xD2511F53)
        h1, l1 = _mul_hi_lo(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    halves = torch.stack([v for w in c for v in (w & 0xFFFF, w >> 16)], dim=-1).reshape(rows, groups * 8)[:, :cols]
    return (halves >= drop).float() * (65536.0 / (65536 - drop))


def _plain_dropout(s):
    c = s["case"]
    m = _plain_mask(c["tokens"], c["d"], c["p"], s["seed"], s["offset"], s["x"].device)
    return {"y": s["x"].float() * m, "dx": s["dy"].float() * m}


def _act(g, name):
    """The activation and its derivative."""
    if name == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return g * sg, sg * (1 + g * (1 - sg))
    if name == "gelu":  # the tanh form
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)
    on = (g > 0).float()
    return g * on, on


def _plain_ffn_forward(x, wg, wu, wd, act):
    g, u = x @ wg, x @ wu
    a, da = _act(g, act)
    h = a * u
    return h @ wd, (u, a, da, h)


def _plain_ffn_backward(dy, x, wg, wu, wd, kept):
    u, a, da, h = kept
    dh = dy @ wd.t()
    dg, du = dh * u * da, dh * a
    return dg @ wg.t() + du @ wu.t(), x.t() @ dg, x.t() @ du, h.t() @ dy


def _plain_ffn(s):
    w = [s[k].float() for k in ("w_gate", "w_up", "w_down")]
    x = s["x"].float()
    y, kept = _plain_ffn_forward(x, *w, s["case"]["act"])
    if not s["case"]["train"]:
        return {"y": y}
    dx, dwg, dwu, dwd = _plain_ffn_backward(s["dy"].float(), x, *w, kept)
    return {"y": y, "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}


def _plain_normed(v, kind, w, b, eps=1e-6):
    """(normalised, reciprocal deviation, weighted)."""
    c = v - v.mean(1, keepdim=True) if kind == "layer" else v
    rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    hat = c * rstd
    return hat, rstd, hat * w + b if b is not None else hat * w


def _plain_norm_backward(dn, hat, rstd, kind, w):
    c = dn * w
    dv = c - hat * (c * hat).mean(1, keepdim=True)
    return (dv - c.mean(1, keepdim=True) if kind == "layer" else dv) * rstd


def _f(t):
    return t.float() if t is not None else None


def _plain_residual(s, x, z):
    """Forward of the norms around a block, and what its gradient needs."""
    c = s["case"]
    n, d = x.shape
    zh, zr, p = _plain_normed(z, c["kind"], _f(s["post_weight"]), _f(s["post_bias"]))
    gate = _f(s["gate"]).repeat_interleave(_rows_per_gate(c), 0)[:n] if s["gate"] is not None else torch.ones(1, 1, device=x.device)
    m = _plain_mask(n, d, c["p"], s["seed"], s["offset"], x.device) if c["p"] > 0 else torch.ones(1, 1, device=x.device)
    r = c["alpha"] * x + gate * p * m
    rh, rr, nx = _plain_normed(r, c["kind"], _f(s["next_weight"]), _f(s["next_bias"]))
    return r, nx, (zh, zr, p, gate, m, rh, rr)


def _plain_residual_backward(s, kept):
    c = s["case"]
    zh, zr, p, gate, m, rh, rr = kept
    dn = s["dn"].float()
    dr = s["dr"].float() + _plain_norm_backward(dn, rh, rr, c["kind"], _f(s["next_weight"]))
    db = dr * m
    dp = db * gate
    out = {"x": c["alpha"] * dr, "z": _plain_norm_backward(dp, zh, zr, c["kind"], _f(s["post_weight"])),
           "post_weight": (dp * zh).sum(0), "next_weight": (dn * rh).sum(0)}
    if c["kind"] == "layer":
        out["post_bias"], out["next_bias"] = dp.sum(0), dn.sum(0)
    if s["gate"] is not None:
        rows = torch.arange(dn.shape[0], device=dn.device) // _rows_per_gate(c)
        out["gate"] = torch.zeros(s["gate"].shape, device=dn.device).index_add_(0, rows, db * p)
    return out


def _plain_norm(s):
    r, n, kept = _plain_residual(s, s["x"].float(), s["z"].float())
    if not s["case"]["train"]:
        return {"r": r, "n": n}
    return {"r": r, "n": n, **{"d" + k: v for k, v in _plain_residual_backward(s, kept).items()}}


def _plain_half(s):
    c = s["case"]
    x = s["x"].float()
    w = [s[k].float() for k in ("w_gate", "w_up", "w_down")]
    hat, rstd, a = _plain_normed(x, c["kind"], _f(s["pre_weight"]), _f(s["pre_bias"]))
    z, kept_f = _plain_ffn_forward(a, *w, c["act"])
    r, n, kept = _plain_residual(s, x, z)
    g = _plain_residual_backward(s, kept)
    da, dwg, dwu, dwd = _plain_ffn_backward(g.pop("z"), a, *w, kept_f)
    dx = g.pop("x") + _plain_norm_backward(da, hat, rstd, c["kind"], _f(s["pre_weight"]))
    out = {"r": r, "n": n, "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd, "dpre_weight": (da * hat).sum(0)}
    if c["kind"] == "layer":
        out["dpre_bias"] = da.sum(0)
    return {**out, **{"d" + k: v for k, v in g.items()}}


# --------------------------------------------------------------------- exact
def _exact_mask(rows, cols, p, seed, offset):
    """The dropout factors once more, with 64-bit unsigned numpy words."""
    u = np.uint64
    low, sh = u(MASK32), u(32)
    groups = (cols + 7) // 8
    a = np.broadcast_to(np.arange(groups, dtype=u), (rows, groups))
    i = np.arange(rows, dtype=u)[:, None]
    b, c, d = i & low, i >> sh, u(offset)
    k = [seed & MASK32, seed >> 32 & MASK32]
    for _ in range(10):
        x, y = a * u(0xD2511F53), c * u(0xCD9E8D57)
        a, b, c, d = (y >> sh) ^ b ^ u(k[0]), y & low, (x >> sh) ^ d ^ u(k[1]), x & low
        k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
    words = np.stack(np.broadcast_arrays(a, b, c, d), axis=-1).astype("<u4")
    drop = min(65535, round(p * 65536))
    keep = words.view("<u2").reshape(rows, groups * 8)[:, :cols] >= drop
    return torch.from_numpy(keep).cuda().double() * (65536 / (65536 - drop))


def exact(case, seed):
    """The operators from their definitions in 64 bits, gradients by differentiating the definition."""
    s = prepare(case, seed)
    op, n, d = case["op"], case["tokens"], case["d"]
    v = {k: t.double().requires_grad_() for k, t in s.items() if torch.is_tensor(t) and k not in ("dy", "dr", "dn")}
    mask = _exact_mask(n, d, case["p"], s["seed"], s["offset"]) if case.get("p") else 1.0
    if op == "dropout":
        return {"y": (v["x"] * mask).detach(), "dx": s["dy"].double() * mask}

    def ffn(x):
        act = {"silu": torch.nn.functional.silu, "relu": torch.nn.functional.relu,
               "gelu": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[case["act"]]
        return (act(x @ v["w_gate"]) * (x @ v["w_up"])) @ v["w_down"]

    def norm(x, name):
        if case["kind"] == "layer":
            return torch.nn.functional.layer_norm(x, (d,), v[name + "_weight"], v[name + "_bias"], 1e-6)
        return x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * v[name + "_weight"]

    def around(x, z):
        b = norm(z, "post")
        if "gate" in v:
            b = b * v["gate"][torch.arange(n, device="cuda") // _rows_per_gate(case)]
        r = case["alpha"] * x + b * mask
        return r, norm(r, "next")

    if op == "ffn":
        out = {"y": ffn(v["x"])}
    else:
        out = dict(zip(("r", "n"), around(v["x"], v["z"] if op == "norm" else ffn(norm(v["x"], "pre")))))
    grads = {}
    if case["train"]:
        names = list(v)
        got = torch.autograd.grad(list(out.values()), [v[k] for k in names], [s[k].double() for k in (("dy",) if op == "ffn" else ("dr", "dn"))])
        grads = {"d" + k: t for k, t in zip(names, got)}
    return {**{k: t.detach() for k, t in out.items()}, **grads}


# ---------------------------------------------------------------------- work
def work(case):
    """What a pass cannot do without: inputs read once, outputs written once, the products' operations."""
    e = 2 if case["dtype"] == "bf16" else 4
    n, d, op = case["tokens"], case["d"], case["op"]
    if op == "dropout":
        return {"bytes": 4 * n * d * e, "flops": 2 * n * d}
    train = case["train"]
    weights = 3 * d * case["f"] if "f" in case else 0
    flops = (6 if train else 2) * n * weights
    vectors = 0
    if op != "ffn":
        vectors = {"norm": 2, "half": 3}[op] * d * (2 if case["kind"] == "layer" else 1)
        vectors += -(-n // _rows_per_gate(case)) * d if case["gate"] != "none" else 0
        flops += (60 if train else 20) * n * d
    # activations: ffn x -> y (and dy -> dx); norm x, z -> r, n (and dr, dn -> dx, dz); half x -> r, n (and dr, dn -> dx)
    acts = {"ffn": 4 if train else 2, "norm": 8 if train else 4, "half": 6 if train else 3}[op] * n * d
    return {"bytes": (acts + (weights + vectors) * (2 if train else 1)) * e, "flops": flops}
