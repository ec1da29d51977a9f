"""The layer operators' kernels on the paths that small sizes do not take: several rows of a workgroup at every width, widths over
4096 with every option, every tile and split of the block's products, pointers that are not 16-byte aligned, results over their
inputs. Tolerances are those of tests/test_gpu_layer.py."""
import math

import numpy as np
import pytest
import torch

from blocked_shampoo_preconditioning_amd import layer
from tests import layer_reference as ref
from tests import test_gpu_layer as base
from tests.gpu_common import log
from tests.layer_reference import BF16_STEP, rel

pytestmark = pytest.mark.gpu

DT = base.DT


def drop_factors(rows, cols, p, seed, offset):
    """ref.drop_factors for all rows and columns at once."""
    t = min(65535, round(p * 65536))
    u, low, sh = np.uint64, np.uint64(0xFFFFFFFF), np.uint64(32)
    groups = -(-cols // 8)
    row = np.arange(rows, dtype=u)[:, None]
    c = [np.broadcast_to(v, (rows, groups)) for v in (np.arange(groups, dtype=u)[None], row & low, row >> sh, np.full((1, 1), offset, dtype=u))]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p0, p1 = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(p1 >> sh) ^ c[1] ^ u(k[0]), p1 & low, (p0 >> sh) ^ c[3] ^ u(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.stack(c, axis=-1).astype("<u4").view("<u2").reshape(rows, groups * 8)[:, :cols]
    return torch.from_numpy((words >= t) * (65536 / (65536 - t)))


def test_fast_dropout_reference():
    for case in ((5, 33, 0.3, 2 ** 63 + 11, 4), (3, 8, 0.999, 7, 2 ** 32 - 1)):
        assert torch.equal(drop_factors(*case), ref.drop_factors(*case))


# rows over 512 give workgroups of several rows; 64, 128, 256, 512 and 512 lanes with two chunks each
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,kind,gate,alpha,p", [
    (1100, 100, ("layer", "layer"), 50, 0.75, 0.1), (1100, 777, ("layer", "layer"), 300, 1.0, 0.1), (1100, 1024, ("rms", "rms"), 1100, 1.0, 0.1),
    (1100, 1025, ("rms", "layer"), None, 1.0, 0.0), (1100, 2048, ("rms", "rms"), 1100, 0.5, 0.1), (1100, 2048, ("layer", "layer"), 7, 1.0, 0.0),
    (1100, 2050, ("layer", "rms"), 64, 1.0, 0.2), (1100, 4096, ("rms", "rms"), 1100, 1.0, 0.0), (1100, 4104, ("rms", "rms"), 7, 1.0, 0.1),
    (1100, 4104, ("none", "rms"), 1100, 1.0, 0.1), (600, 5001, ("layer", "layer"), 100, 0.75, 0.1), (600, 8192, ("layer", "layer"), 600, 1.0, 0.1),
    (3, 8191, ("layer", "layer"), None, 1.0, 0.0), (5, 8192, ("rms", "layer"), 2, 1.0, 0.5), (7, 4097, ("layer", "none"), 3, 1.0, 0.1)])
def test_norm_paths(n, d, kind, gate, alpha, p, dtype, monkeypatch):
    monkeypatch.setattr(ref, "drop_factors", drop_factors)
    base.check_norm(n, d, dtype, kind, gate=gate, alpha=alpha, p=p, seed=6)


def reference(x, wg, wu, wd, act, dy):
    """ref.ffn with its products on the GPU in 64 bits."""
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    g, u = x @ wg, x @ wu
    a, da = ref.act(g, act)
    h, dh = a * u, dy @ wd.t()
    dg, du = dh * u * da, dh * a
    x2, g2, u2, h2, y2 = (t.square() for t in (x, dg, du, h, dy))
    terms = (h2 @ wd.square(), g2 @ wg.square().t() + u2 @ wu.square().t(), x2.t() @ g2, x2.t() @ u2, h2.t() @ y2)
    return (h @ wd, dg @ wg.t() + du @ wu.t(), x.t() @ dg, x.t() @ du, h.t() @ dy), [t.sqrt().cpu() for t in terms]


def check_tiles(n, d, f, dtype):
    """Forward and backward pass against `reference`."""
    x, wg, wu, wd, dy = base.ffn_case(9, n, d, f, dtype)
    log(f"ffn {n} x {d} x {f} gelu {dtype}")
    y, saved = layer.ffn_forward(x, wg, wu, wd, activation="gelu", save=True)
    got = (y, *layer.ffn_backward(dy, x, wg, wu, wd, saved, activation="gelu"))
    want, terms = reference(x, wg, wu, wd, "gelu", dy)
    tols = (4 * BF16_STEP, *(6 * BF16_STEP,) * 3, 3 * BF16_STEP) if dtype == "bf16" else (base.f32_tol(max(n, d, f)),) * 5
    errs = [rel(a, b, t) for a, b, t in zip(got, want, terms)]
    log("   errors " + " ".join(f"{e:.2e}" for e in errs))
    assert all(e <= t for e, t in zip(errs, tols))


# sizes whose plan has a tile, or a tile with K whole or in parts, that no size of tests/test_gpu_layer.py has
@pytest.mark.parametrize("n,d,f,dtype", [
    # fp32, 128 x 256 tiles: y whole; the last three products with the weights' gradients in parts, with dx in parts too; dh and y in
    # parts; all whole
    (4682, 866, 40, "f32"), (7794, 150, 151, "f32"), (4389, 141, 485, "f32"), (1071, 1817, 1216, "f32"), (2209, 1766, 743, "f32"),
    # bf16: the last three products on two-set tiles with dx, with the weights' gradients in parts; on one-set tiles with both; dh on
    # two-set tiles in parts; the last three on 256 tiles with both, with the weights' gradients, with none in parts; y on 256 tiles in parts
    (34, 43, 674, "bf16"), (1330, 57, 73, "bf16"), (2208, 40, 428, "bf16"), (44, 1885, 6005, "bf16"), (6363, 129, 4329, "bf16"),
    (7718, 670, 1156, "bf16"), (3511, 1337, 1832, "bf16"), (6938, 542, 4164, "bf16")])
def test_ffn_tiles_and_splits(n, d, f, dtype):
    check_tiles(n, d, f, dtype)


def moved(t, offset, pad=0):
    """t's values in rows `pad` longer that start `offset` elements into an allocation; what lies around them is NaN."""
    rows, cols = t.shape if t.dim() == 2 else (1, t.numel())
    ld = cols + pad
    flat = torch.full((rows * ld + offset + 8,), float("nan"), dtype=t.dtype, device="cuda")
    out = flat.as_strided(t.shape, (ld, 1) if t.dim() == 2 else (1,), offset)
    out.copy_(t)
    assert out.data_ptr() % 16 == offset * t.element_size() % 16
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,f", [(9, 130, 78), (9, 131, 77), (40, 64, 72), (150, 136, 264), (300, 100, 70)])
def test_ffn_unaligned_pointers(n, d, f, dtype):
    """Each operand off the 16-byte (and 4-byte) alignment, alone and together: the results' bits are those of aligned operands."""
    names = ("x", "w_gate", "w_up", "w_down", "dy")
    t = dict(zip(names, base.ffn_case(10, n, d, f, dtype)))

    def run(v):
        x, wg, wu, wd, dy = (v[k] for k in names)
        y, s = layer.ffn_forward(x, wg, wu, wd, save=True)
        return [y, layer.ffn_forward(x, wg, wu, wd), *layer.ffn_backward(dy, x, wg, wu, wd, s)]
    want = run(t)
    for offset, pad in ((1, 0), (2, 0), (3, 5), (4, 8)):
        for moving in (*((k,) for k in names), names):
            log(f"ffn {n} x {d} x {f} {dtype}, {' '.join(moving)} {offset} elements on, pad {pad}")
            got = run({k: moved(v, offset, pad) if k in moving else v for k, v in t.items()})
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [9, 150])
def test_ffn_weights_of_different_strides(n, dtype):
    """w_gate and w_up with leading dimensions of their own are read as one pair of operands."""
    x, wg, wu, wd, dy = base.ffn_case(11, n, 136, 264, dtype)
    y, s = layer.ffn_forward(x, wg, wu, wd, save=True)
    want = [y, *layer.ffn_backward(dy, x, wg, wu, wd, s)]
    for pads in ((8, 0), (0, 16), (8, 24), (1, 2)):
        g, u = moved(wg, 0, pads[0]), moved(wu, 0, pads[1])
        y, s = layer.ffn_forward(x, g, u, wd, save=True)
        assert all(torch.equal(a, b) for a, b in zip([y, *layer.ffn_backward(dy, x, g, u, wd, s)], want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,kind", [(9, 64, ("rms", "rms")), (600, 333, ("layer", "layer")), (40, 4100, ("layer", "rms"))])
def test_norm_unaligned_pointers(n, d, kind, dtype):
    t, s = base.norm_case(12, n, d, dtype, kind, 7)
    s.update(dropout=0.2, seed=5, residual_scale=0.75)
    tensors = {**t, **{k: v for k, v in s.items() if torch.is_tensor(v)}}

    def run(v):
        kw = {**s, **{k: v[k] for k in v if k not in t}}
        r, nn, st = layer.residual_forward(v["x"], v["z"], **kw)
        g = layer.residual_backward(v["dr"], v["dn"], r, v["z"], st, **kw)
        return [r, nn, layer.dropout(v["x"], 0.3, 9), *(q for q in g.values() if q is not None)]
    want = run(tensors)
    for offset, pad in ((1, 0), (2, 0), (3, 5)):
        log(f"norm {n} x {d} {dtype}, {offset} elements on, pad {pad}")
        got = run({k: moved(v, offset, pad) for k, v in tensors.items()})
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(5, 64), (1100, 777), (600, 4104)])
def test_norm_results_over_their_inputs(n, d, dtype):
    """The C calls may write r over x or z, and dx and dz over dr or dn: the bits are those of separate results."""
    t, s = base.norm_case(13, n, d, dtype, ("layer", "rms"), 7)
    kw = dict(post=s["post"], next=s["next"], eps=s["eps"], residual_scale=0.75, dropout=0.2, seed=5, offset=3, rows_per_gate=7)
    vec = {k: s.get(k) for k in ("post_weight", "post_bias", "gate", "next_weight", "next_bias")}
    r, nn, st = layer.residual_forward(t["x"], t["z"], **kw, **vec)
    g = layer.residual_backward(t["dr"], t["dn"], r, t["z"], st, **kw, **vec)
    head = layer._norm_head(layer._DTYPES[DT[dtype]], n, d, kw["post"], kw["next"], kw["eps"], 0.75, 0.2, 5, 3, 7)
    vectors = layer._norm_vectors(r, n, d, vec["post_weight"], vec["post_bias"], vec["gate"], 7, vec["next_weight"], vec["next_bias"])

    def forward(x, z, out):
        n2, st2 = torch.empty_like(r), torch.empty_like(st)
        layer._call("shampoo_norm_forward", layer._NORM.pack(*head, z.data_ptr(), x.data_ptr(), d, d, out.data_ptr(), n2.data_ptr(), d, d,
                                                             *vectors, st2.data_ptr(), *layer._NO_NORM_GRADIENTS), r.get_device())
        return n2, st2
    for over in ("x", "z"):
        v = {k: t[k].clone() for k in ("x", "z")}
        n2, st2 = forward(v["x"], v["z"], v[over])
        assert torch.equal(v[over], r) and torch.equal(n2, nn) and torch.equal(st2, st)
    for dx, dz in (("dr", None), ("dn", None), (None, "dr"), (None, "dn"), ("dr", "dn"), ("dn", "dr")):
        log(f"norm {n} x {d} {dtype}: dx over {dx}, dz over {dz}")
        v = {k: t[k].clone() for k in ("dr", "dn")}
        out = [v[k] if k else torch.empty_like(r) for k in (dx, dz)]
        args = layer._NORM.pack(*head, t["z"].data_ptr(), 0, d, d, r.data_ptr(), 0, d, 0, *vectors, st.data_ptr(), v["dr"].data_ptr(),
                                v["dn"].data_ptr(), d, d, out[0].data_ptr(), out[1].data_ptr(), d, d, 0, 0, 0, 0, 0, d)
        size = layer._norm_workspace(head, args)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        layer._call("shampoo_norm_backward", args, r.get_device(), ws.data_ptr(), size)
        assert torch.equal(out[0], g["x"]) and torch.equal(out[1], g["z"])
