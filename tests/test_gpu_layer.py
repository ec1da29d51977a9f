"""The feed-forward half of a decoder layer on the GPU against plain 64-bit
forms (tests/layer_reference.py): gated feed-forward block, norms around a
block, dropout; forward and backward; and the block together with the Shampoo
step.

Tolerances (2-norm of the error over that of the result, or of its terms' root
sum of squares where that is larger), set before the first run. One rounding to bf16 is off by at most 2^-9 = BF16_STEP of the value.
 - y: h and y are rounded: 2 BF16_STEP, and as much again for the activation's
   argument.  dw_down: h and the result.
 - dx, dw_gate, dw_up: the kept g and u (each up to twice through act'), dg or
   du, and the result: 6 BF16_STEP.
 - norms: each result is rounded once; n's and the gradients' r^ comes from the
   rounded r: 3 BF16_STEP.
fp32: the kept fp32 accumulation over K terms of random sign is off by about
sqrt(K) F32_STEP of their root sum of squares, the chain of two products by
twice that, and the operands' split by 2^-24 a product: 8 (4 + sqrt(K))
F32_STEP with K the longest sum."""
import math

import pytest
import torch

from blocked_shampoo_preconditioning_amd import layer
from blocked_shampoo_preconditioning_amd.shampoo import Shampoo, ShampooError
from tests import layer_reference as ref
from tests.gpu_common import log
from tests.layer_reference import BF16_STEP, F32_STEP, rel

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f32_tol(k):
    return 8 * (4 + math.sqrt(k)) * F32_STEP


def normal(gen, *shape, std=1.0, mean=0.0, dtype="bf16", ld=None):
    t = (torch.randn(*shape, generator=gen) * std + mean).to(DT[dtype])
    if ld is None:
        return t.cuda()
    wide = torch.full((shape[0], ld), float("nan"), dtype=DT[dtype])  # what lies between rows must not enter
    wide[:, :shape[1]] = t
    return wide.cuda()[:, :shape[1]]


def ffn_case(seed, n, d, f, dtype, pad=0):
    g = torch.Generator().manual_seed(seed)
    up = lambda c: c + pad if pad else None  # noqa: E731
    x = normal(g, n, d, dtype=dtype, ld=up(d))
    wg = normal(g, d, f, std=d ** -0.5, dtype=dtype, ld=up(f))
    wu = normal(g, d, f, std=d ** -0.5, dtype=dtype, ld=up(f))
    wd = normal(g, f, d, std=f ** -0.5, dtype=dtype, ld=up(d))
    dy = normal(g, n, d, std=1e-2, dtype=dtype, ld=up(d))
    return x, wg, wu, wd, dy


def check_ffn(n, d, f, act, dtype, pad=0, seed=0):
    x, wg, wu, wd, dy = ffn_case(seed, n, d, f, dtype, pad)
    log(f"ffn {n} x {d} x {f} {act} {dtype} pad {pad}")
    y, saved = layer.ffn_forward(x, wg, wu, wd, activation=act, save=True)
    got = layer.ffn_backward(dy, x, wg, wu, wd, saved, activation=act)
    y2 = layer.ffn_forward(x, wg, wu, wd, activation=act)
    want_y, want, terms = ref.ffn(x, wg, wu, wd, act, dy)
    tol_y, tol_g, tol_d = (4 * BF16_STEP, 6 * BF16_STEP, 3 * BF16_STEP) if dtype == "bf16" else (f32_tol(max(n, d, f)),) * 3
    errs = [rel(a, b, t) for a, b, t in zip((y, *got), (want_y, *want), terms)]
    log("   errors " + " ".join(f"{e:.2e}" for e in errs))
    assert rel(y2, want_y, terms[0]) <= tol_y
    for e, t in zip(errs, (tol_y, tol_g, tol_g, tol_g, tol_d)):
        assert e <= t


FFN_SIZES = [
    (1, 64, 128), (2, 8, 8), (3, 1, 1), (17, 40, 24), (33, 100, 70), (128, 128, 128), (130, 257, 391), (256, 256, 512),
    (257, 264, 520), (300, 512, 1024), (700, 129, 65), (1024, 768, 512), (5, 2048, 4096), (64, 1000, 1003)]


@pytest.mark.parametrize("n,d,f", FFN_SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_sizes(n, d, f, dtype):
    check_ffn(n, d, f, "silu", dtype)


@pytest.mark.parametrize("act", ["gelu", "relu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_activations(act, dtype):
    check_ffn(200, 192, 320, act, dtype, seed=3)


@pytest.mark.parametrize("pad", [8, 3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_strided(pad, dtype):
    check_ffn(150, 136, 264, "silu", dtype, pad=pad, seed=4)


@pytest.mark.parametrize("n", [13, 16, 17, 32, 33, 63, 64, 65])
@pytest.mark.parametrize("d,f", [(66, 70), (768, 513), (258, 2048)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_few_tokens(n, d, f, dtype):
    """Around every token count where another kernel takes over; last columns that make half a pair."""
    check_ffn(n, d, f, "gelu", dtype, seed=6)


@pytest.mark.parametrize("pad", [1, 2, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_few_tokens_strided(pad, dtype):
    check_ffn(9, 131, 77, "silu", dtype, pad=pad, seed=7)


def test_ffn_256_tiles():
    """Enough rows and columns that the largest tiles run, ragged at every edge."""
    check_ffn(4000, 520, 3000, "silu", "bf16", seed=5)


@pytest.mark.parametrize("n,d,f", [(4612, 72, 843), (5383, 1491, 72), (757, 975, 3156), (500, 588, 4184), (1537, 520, 900),
                                   (4097, 40, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_tiles(n, d, f, dtype):
    """The first sizes at which each product takes each tile: one set of waves or two (with an odd number of K steps), K whole or
    in up to 32 parts."""
    check_ffn(n, d, f, "gelu", dtype, seed=8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropout_alone(dtype):
    g = torch.Generator().manual_seed(1)
    for rows, cols, p, seed, offset in [(1, 1, 0.5, 1, 0), (5, 7, 0.3, 2 ** 63 + 11, 4), (33, 257, 0.1, 77, 2 ** 32 - 1),
                                        (64, 64, 0.0, 5, 0), (3, 2100, 0.999, 6, 1)]:
        x = normal(g, rows, cols, dtype=dtype)
        m = ref.drop_factors(rows, cols, p, seed, offset)
        y = layer.dropout(x, p, seed, offset)
        want = (x.double().cpu() * m).to(DT[dtype])
        # one product of fp32 values and one rounding: at most a step apart
        assert torch.equal((y.cpu() == 0) & (x.cpu() != 0), (m == 0) & (x.cpu() != 0))
        assert rel(y, want.double()) <= (BF16_STEP if dtype == "bf16" else 2 * F32_STEP)
        z = x.clone()
        assert torch.equal(layer.dropout(z, p, seed, offset, out=z), y) and torch.equal(z, y)
        wide = torch.zeros(rows, cols + 3, dtype=DT[dtype], device="cuda")
        wide[:, :cols] = x
        assert torch.equal(layer.dropout(wide[:, :cols], p, seed, offset), y)


def norm_case(seed, n, d, dtype, kind, gate, pad=0):
    g = torch.Generator().manual_seed(seed)
    up = d + pad if pad else None
    t = {k: normal(g, n, d, std=s, mean=m, dtype=dtype, ld=up) for k, s, m in
         (("x", 1.0, 0.0), ("z", 0.5, 0.3), ("dr", 1e-2, 0.0), ("dn", 1e-2, 0.0))}
    s = dict(post=kind[0], next=kind[1], eps=1e-5)
    for name, k in (("post", kind[0]), ("next", kind[1])):
        if k != "none":
            s[name + "_weight"] = normal(g, d, std=0.1, mean=1.0, dtype=dtype)
        if k == "layer":
            s[name + "_bias"] = normal(g, d, std=0.1, dtype=dtype)
    if gate:
        s["rows_per_gate"] = gate
        s["gate"] = normal(g, -(-n // gate), d, std=0.3, mean=0.5, dtype=dtype)
    return t, s


def check_norm(n, d, dtype, kind=("rms", "rms"), gate=None, alpha=1.0, p=0.0, pad=0, seed=0):
    t, s = norm_case(seed, n, d, dtype, kind, gate, pad)
    s.update(residual_scale=alpha, dropout=p, seed=1234567 + (seed << 40), offset=seed)
    log(f"norm {n} x {d} {dtype} {kind} gate {gate} alpha {alpha} p {p} pad {pad}")
    mask = ref.drop_factors(n, d, p, s["seed"], s["offset"]) if p else None
    r, nn, stats = layer.residual_forward(t["x"], t["z"], **s)
    g = layer.residual_backward(t["dr"], t["dn"] if kind[1] != "none" else None, r, t["z"], stats, **s)
    wr, wn, wg, sizes = ref.residual(t["x"], t["z"], s, mask, t["dr"], t["dn"])
    tol = 3 * BF16_STEP if dtype == "bf16" else f32_tol(max(n, d))
    assert rel(r, wr) <= tol
    if kind[1] != "none":
        assert rel(nn, wn) <= tol
    else:
        assert nn is None
    for k, v in g.items():
        if v is None:
            assert k in ("gate", "post_weight", "post_bias", "next_weight", "next_bias") and s.get(k) is None
            continue
        e = rel(v, wg[k], sizes.get(k))
        log(f"   {k} {e:.2e}")
        assert e <= tol, k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(1, 1), (1, 2048), (3, 7), (64, 64), (65, 511), (130, 513), (37, 1025), (1500, 96), (20, 2050),
                                 (9, 5000), (6, 8192)])
def test_norm_sizes(n, d, dtype):
    check_norm(n, d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", [("layer", "layer"), ("rms", "layer"), ("none", "rms"), ("layer", "none"), ("none", "none")])
def test_norm_kinds(kind, dtype):
    check_norm(70, 200, dtype, kind, gate=70, alpha=0.75, p=0.25, seed=2)


@pytest.mark.parametrize("n,gate", [(1, 1), (100, 1), (100, 7), (3000, 3000), (3000, 1499), (3000, 2), (2500, 3), (5000, 40)])
def test_norm_gates(n, gate):
    check_norm(n, 72, "f32", gate=gate, alpha=0.5, p=0.1, seed=3)


def test_norm_strided_and_dropped():
    check_norm(50, 333, "bf16", ("layer", "rms"), gate=50, p=0.5, pad=5, seed=4)
    check_norm(50, 333, "f32", ("rms", "layer"), gate=11, p=0.5, pad=2, seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_alone(kind, dtype):
    g = torch.Generator().manual_seed(8)
    x, dn, dr = (normal(g, 77, 300, dtype=dtype) for _ in range(3))
    w = normal(g, 300, std=0.1, mean=1.0, dtype=dtype)
    b = normal(g, 300, dtype=dtype) if kind == "layer" else None
    n, stats = layer.norm_forward(x, kind, w, b, eps=1e-5)
    got = layer.norm_backward(dn, x, stats, dr=dr, kind=kind, weight=w, bias=b, eps=1e-5)
    d64 = [t.double().cpu() if t is not None else None for t in (x, w, b)]
    want, hat, rstd = ref.norm(d64[0], kind, d64[1], d64[2], 1e-5)
    tol = 3 * BF16_STEP if dtype == "bf16" else f32_tol(300)
    dn64 = dn.double().cpu()
    assert rel(n, want) <= tol
    assert rel(got["x"], dr.double().cpu() + ref.norm_grad(dn64, hat, rstd, kind, d64[1])) <= tol
    assert rel(got["weight"], (dn64 * hat).sum(0)) <= tol
    assert (got["bias"] is None) == (b is None)
    if b is not None:
        assert rel(got["bias"], dn64.sum(0)) <= tol
    only = layer.norm_backward(dn, x, stats, kind=kind, weight=w, bias=b, eps=1e-5)
    assert rel(only["x"], ref.norm_grad(dn64, hat, rstd, kind, d64[1])) <= tol


def test_norm_large_mean_and_zero_rows():
    """A layer norm of rows far from zero keeps its digits; rows of zeros give 0 (RMS) without a NaN."""
    g = torch.Generator().manual_seed(9)
    x = normal(g, 8, 400, std=1.0, mean=1000.0, dtype="f32")
    n, _ = layer.norm_forward(x, "layer", eps=1e-6)
    assert rel(n, ref.norm(x.double().cpu(), "layer", None, None, 1e-6)[0]) <= 1000 * 4 * F32_STEP
    x[3] = 0
    z = torch.zeros_like(x)
    for kind in ("rms", "layer"):
        r, n, st = layer.residual_forward(x, z, post=kind, next=kind)
        g2 = layer.residual_backward(x, x, r, z, st, post=kind, next=kind)
        assert torch.equal(r, x) and torch.all(n[3] == 0)
        assert all(torch.isfinite(v).all() for v in (n, g2["x"], g2["z"]))


def test_empty():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w, v = torch.randn(64, 32, device="cuda").bfloat16(), torch.randn(32, 64, device="cuda").bfloat16()
    y, saved = layer.ffn_forward(e, w, w, v, save=True)
    dx, a, b, c = layer.ffn_backward(e, e, w, w, v, saved)
    assert y.shape == dx.shape == (0, 64) and not a.any() and not b.any() and not c.any()
    s = dict(post_weight=w[:, 0].contiguous(), next_weight=w[:, 1].contiguous())
    r, n, st = layer.residual_forward(e, e, **s)
    g = layer.residual_backward(e, e, r, e, st, **s)
    assert r.shape == n.shape == (0, 64) and not g["post_weight"].any() and not g["next_weight"].any()
    assert layer.dropout(e, 0.5, 1).shape == (0, 64)


def test_rows_do_not_mix():
    """A row that is not finite leaves every other row's results as they are."""
    x, wg, wu, wd, dy = ffn_case(11, 200, 128, 256, "bf16")
    y, s = layer.ffn_forward(x, wg, wu, wd, save=True)
    dx = layer.ffn_backward(dy, x, wg, wu, wd, s, need_dw=False)[0]
    x2 = x.clone()
    x2[77] = float("nan")
    y2, s2 = layer.ffn_forward(x2, wg, wu, wd, save=True)
    dx2 = layer.ffn_backward(dy, x2, wg, wu, wd, s2, need_dw=False)[0]
    keep = torch.arange(200, device="cuda") != 77
    assert torch.equal(y[keep], y2[keep]) and torch.equal(dx[keep], dx2[keep])
    assert torch.isnan(y2[77]).all()
    t, st = norm_case(12, 40, 100, "f32", ("rms", "layer"), 40)
    r, n, _ = layer.residual_forward(t["x"], t["z"], **st)
    z2 = t["z"].clone()
    z2[5] = float("inf")
    r2, n2, _ = layer.residual_forward(t["x"], z2, **st)
    keep = torch.arange(40, device="cuda") != 5
    assert torch.equal(r[keep], r2[keep]) and torch.equal(n[keep], n2[keep])


def test_deterministic_and_on_another_stream():
    x, wg, wu, wd, dy = ffn_case(13, 333, 256, 512, "bf16")
    y, s = layer.ffn_forward(x, wg, wu, wd, save=True)
    first = layer.ffn_backward(dy, x, wg, wu, wd, s)
    t, st = norm_case(14, 3000, 256, "bf16", ("rms", "rms"), 3000)
    rn = layer.residual_forward(t["x"], t["z"], **st)
    gn = layer.residual_backward(t["dr"], t["dn"], rn[0], t["z"], rn[2], **st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, s2 = layer.ffn_forward(x, wg, wu, wd, save=True)
        again = layer.ffn_backward(dy, x, wg, wu, wd, s2)
        rn2 = layer.residual_forward(t["x"], t["z"], **st)
        gn2 = layer.residual_backward(t["dr"], t["dn"], rn2[0], t["z"], rn2[2], **st)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(first, again))
    assert torch.equal(rn[1], rn2[1]) and all(torch.equal(v, gn2[k]) for k, v in gn.items() if v is not None)


def test_gradients_against_differences():
    """Directional differences of the fp32 forward passes: the loss sum(y c) moved by +-t along a random direction of every input.
    The difference's own error: t^2 from the third derivative and F32 rounding over t; t = 2^-6 keeps both below 2e-3."""
    g = torch.Generator().manual_seed(21)
    x, wg, wu, wd, dy = ffn_case(15, 48, 64, 96, "f32")
    _, s = layer.ffn_forward(x, wg, wu, wd, activation="gelu", save=True)
    grads = layer.ffn_backward(dy, x, wg, wu, wd, s, activation="gelu")
    for k, (t, gr) in enumerate(zip((x, wg, wu, wd), grads)):
        v = torch.randn(t.shape, generator=g).cuda() * t.std()
        side = []
        for sign in (1, -1):
            args = [x, wg, wu, wd]
            args[k] = t + sign * 2.0 ** -6 * v
            side.append((layer.ffn_forward(*args, activation="gelu").double() * dy.double()).sum())
        diff = float((side[0] - side[1]) / 2.0 ** -5)
        size = float(torch.linalg.vector_norm(gr.double()) * torch.linalg.vector_norm(v.double()))
        assert abs(diff - float((gr.double() * v.double()).sum())) <= 2e-3 * size
    t, st = norm_case(16, 30, 80, "f32", ("layer", "rms"), 30)
    st.update(dropout=0.25, seed=9, residual_scale=0.7)
    r, _, stats = layer.residual_forward(t["x"], t["z"], **st)
    grads = layer.residual_backward(t["dr"], t["dn"], r, t["z"], stats, **st)
    for name, gr in grads.items():
        if gr is None:
            continue
        base = t[name] if name in t else st[name]
        v = torch.randn(base.shape, generator=g).cuda() * 0.5
        side = []
        for sign in (1, -1):
            tt, ss = dict(t), dict(st)
            (tt if name in t else ss)[name] = base + sign * 2.0 ** -6 * v
            r2, n2, _ = layer.residual_forward(tt["x"], tt["z"], **ss)
            side.append((r2.double() * t["dr"].double()).sum() + (n2.double() * t["dn"].double()).sum())
        diff = float((side[0] - side[1]) / 2.0 ** -5)
        size = float(torch.linalg.vector_norm(gr.double()) * torch.linalg.vector_norm(v.double()))
        assert abs(diff - float((gr.double() * v.double()).sum())) <= 2e-3 * size, name


def test_saved_free_inference_equals_training_forward():
    x, wg, wu, wd, _ = ffn_case(17, 65, 128, 200, "bf16")
    y, _ = layer.ffn_forward(x, wg, wu, wd, save=True)
    assert torch.equal(y, layer.ffn_forward(x, wg, wu, wd))


def test_weight_gradients_feed_the_shampoo_step():
    """The block's weight gradients go to the optimizer as they are, and the loss falls."""
    g = torch.Generator().manual_seed(31)
    x, wg, wu, wd, _ = ffn_case(18, 256, 128, 256, "f32")
    goal = torch.randn(256, 128, generator=g).cuda() * 0.3
    ws = [wg, wu, wd]
    opt = Shampoo([tuple(w.shape) for w in ws], 128, 128, lr=2e-2, root_every=2)
    losses = []
    for _ in range(12):
        y, s = layer.ffn_forward(x, *ws, save=True)
        losses.append(float((y - goal).square().mean()))
        _, *grads = layer.ffn_backward((y - goal) * (2.0 / goal.numel()), x, *ws, s, need_dx=False)
        opt.step(ws, grads)
    log(f"  losses {losses[0]:.4f} -> {losses[-1]:.4f}")
    opt.close()
    assert losses[-1] < 0.8 * losses[0]


def test_refusals():
    x, wg, wu, wd, dy = ffn_case(41, 8, 16, 24, "bf16")
    cases = [
        (lambda: layer.ffn_forward(x, wg, wu, wd, activation="tanh"), "activation"),
        (lambda: layer.ffn_forward(x, wg, wu[:, :8], wd), "w_up has shape"),
        (lambda: layer.ffn_forward(x.float(), wg, wu, wd), "w_gate is"),
        (lambda: layer.ffn_forward(x.half(), wg, wu, wd), "float32 and bfloat16"),
        (lambda: layer.ffn_forward(x[0], wg, wu, wd), "2-D"),
        (lambda: layer.ffn_forward(x, wd.t(), wu, wd), "contiguous"),
        (lambda: layer.ffn_forward(x[:1].expand(8, 16), wg, wu, wd), "overlap"),
        (lambda: layer.ffn_backward(dy, x, wg, wu, wd, torch.empty(8, dtype=torch.uint8, device="cuda")), "saved"),
        (lambda: layer.residual_forward(x, x, next="batch"), "one of"),
        (lambda: layer.residual_forward(x, None), "norm_forward"),
        (lambda: layer.residual_forward(x, x, post_weight=wg[:, 0]), "contiguous vector"),
        (lambda: layer.residual_forward(x, x, gate=x, rows_per_gate=4), "gate has shape"),
        (lambda: layer.residual_forward(x, x, gate=x, rows_per_gate=0), "rows_per_gate"),
        (lambda: layer.norm_forward(x, kind="none"), "kind"),
        (lambda: layer.residual_backward(x, None, x, x, torch.zeros(8, 4, device="cuda")), "dn"),
        (lambda: layer.residual_backward(x, x, x, x, torch.zeros(8, 3, device="cuda")), "stats"),
        (lambda: layer.dropout(x, 0.1, 1, out=x[:, :8]), "out has shape"),
    ]
    for call, text in cases:
        with pytest.raises(ValueError, match=text):
            call()
    wide = torch.zeros(2, 8200, device="cuda")
    for call, code in ((lambda: layer.norm_forward(wide), 2), (lambda: layer.dropout(x, 1.0, 1), 1), (lambda: layer.norm_forward(x, eps=0.0), 1),
                       (lambda: layer.residual_forward(x, x, dropout=-1.0), 1)):
        with pytest.raises(ShampooError) as e:
            call()
        assert e.value.code == code


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    """Rows of a few columns far apart: the last ones lie over 2^32 elements from the first. Results are those of a compact copy."""
    g = torch.Generator().manual_seed(42)
    n, d, ld = 2200, 64, 1 << 21
    big = torch.empty(n * ld, dtype=DT[dtype], device="cuda")
    far = big.as_strided((n, d), (ld, 1))
    x = normal(g, n, d, dtype=dtype)
    far.copy_(x)
    assert (n - 1) * ld > 2 ** 32
    log(f"ffn, norm and dropout {n} x {d} {dtype}, rows {ld} elements apart")
    wg, wu = normal(g, d, 128, std=0.1, dtype=dtype), normal(g, d, 128, std=0.1, dtype=dtype)
    wd = normal(g, 128, d, std=0.1, dtype=dtype)
    y, s = layer.ffn_forward(x, wg, wu, wd, save=True)
    y2, s2 = layer.ffn_forward(far, wg, wu, wd, save=True)
    assert torch.equal(y, y2)
    for a, b in zip(layer.ffn_backward(x, x, wg, wu, wd, s), layer.ffn_backward(far, far, wg, wu, wd, s2)):
        assert torch.equal(a, b)
    r, nn, st = layer.residual_forward(x, x, dropout=0.2, seed=3)
    r2, nn2, st2 = layer.residual_forward(far, far, dropout=0.2, seed=3)
    assert torch.equal(r, r2) and torch.equal(nn, nn2)
    a = layer.residual_backward(x, x, r, x, st, dropout=0.2, seed=3)
    b = layer.residual_backward(far, far, r2, far, st2, dropout=0.2, seed=3)
    assert torch.equal(a["x"], b["x"]) and torch.equal(a["z"], b["z"])
    assert torch.equal(layer.dropout(x, 0.3, 5), layer.dropout(far, 0.3, 5, out=far))


def test_captured_graph_replays():
    """Forward and backward in a captured graph: every replay, between eager work, gives the eager result."""
    x, wg, wu, wd, dy = ffn_case(43, 300, 256, 512, "f32")
    t, st = norm_case(44, 300, 256, "f32", ("rms", "layer"), 300)
    st.update(dropout=0.2, seed=8)

    def run():
        y, s = layer.ffn_forward(x, wg, wu, wd, save=True)
        r, n, stats = layer.residual_forward(x, y, **st)
        g = layer.residual_backward(dy, t["dn"], r, y, stats, **st)
        return [y, r, n, *layer.ffn_backward(g["z"], x, wg, wu, wd, s)] + [v for v in g.values() if v is not None]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for k in range(4):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(k)).cuda())
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k


@pytest.mark.parametrize("n", [5, 200])
def test_rows_do_not_mix_fp32(n):
    """fp32 operands share one scale: a row that is not finite leaves it, and the other rows, as they are."""
    x, wg, wu, wd, dy = ffn_case(45, n, 128, 256, "f32")
    y, s = layer.ffn_forward(x, wg, wu, wd, save=True)
    dx = layer.ffn_backward(dy, x, wg, wu, wd, s, need_dw=False)[0]
    keep = torch.arange(n, device="cuda") != 3
    for bad in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[3, 7] = bad
        y2, s2 = layer.ffn_forward(x2, wg, wu, wd, save=True)
        dx2 = layer.ffn_backward(dy, x2, wg, wu, wd, s2, need_dw=False)[0]
        assert not torch.isfinite(y2[3]).all()
        # finite rows: the scale goes by the largest finite value, which the bad element may have been
        assert rel(y2[keep], y[keep]) <= 4 * F32_STEP and rel(dx2[keep], dx[keep]) <= 16 * F32_STEP


def test_fp32_range():
    """fp32 operands of very large and very small size: the planes' scale follows them."""
    for scale in (1e-18, 1e12):
        x, wg, wu, wd, dy = ffn_case(46, 130, 64, 96, "f32")
        wd = wd * scale
        dy = dy / scale
        y, s = layer.ffn_forward(x, wg, wu, wd, activation="relu", save=True)
        got = layer.ffn_backward(dy, x, wg, wu, wd, s, activation="relu")
        want_y, want, terms = ref.ffn(x, wg, wu, wd, "relu", dy)
        for a, b, t in zip((y, *got), (want_y, *want), terms):
            assert rel(a, b, t) <= f32_tol(130)


def test_dropped_elements_are_zero():
    """A dropped element is 0 also where the value was not finite; a kept one stays what it was."""
    x = torch.full((16, 64), float("inf"), device="cuda")
    m = ref.drop_factors(16, 64, 0.5, 7, 0)
    y = layer.dropout(x, 0.5, 7).cpu()
    assert torch.equal(y == 0, m == 0) and torch.isinf(y[m != 0]).all()


def test_training_example():
    from blocked_shampoo_preconditioning_amd import train_ffn
    for dtype in ("f32", "bf16"):
        losses = train_ffn.train(layers=2, d=256, f=512, tokens=512, steps=16, block=256, dtype=dtype, log=log)
        assert all(math.isfinite(v) for v in losses) and losses[-1] < 0.9 * losses[0]
