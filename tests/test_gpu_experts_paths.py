"""The experts' path on the GPU at calls and sizes that tests/test_gpu_experts_product.py and test_gpu_experts_route.py do not
reach. Bounds are those files'. The cases name the kernels that they are there for; tests/test_experts_launches.py checks
without a GPU that they launch these, and that no kernel is without a case."""
import numpy as np
import pytest
import torch

from blocked_shampoo_preconditioning_amd import experts
from tests import experts_reference as ref
from tests import test_gpu_experts_route as routes
from tests.gpu_common import log
from tests.test_gpu_experts_product import check_product, check_weight, close
from tests.test_gpu_experts_route import DT, check_plan, make_ids, padded

pytestmark = pytest.mark.gpu


def few(f32, columns, kept=0):
    """Up to 64 rows: tiles of 16 or 32 columns, x kept over a workgroup's tiles (so many K blocks a wave) or not."""
    return f"few_kernel<{'true' if f32 else 'false'}, {columns // 16}, 8, {kept}>"


def tile(f32, side, steps):
    """The product of more rows: tiles of 128 or 256, two or four steps in LDS."""
    operands = side // 32
    waves = 1 if side == 256 or steps == 4 else 2
    return f"product_kernel<Tile<{operands}, {operands}, 2, 2, {steps}, {'true' if f32 else 'false'}, {waves}> >"


@pytest.mark.parametrize("n_experts,n_in,n_out", [(3, 130, 200), (2, 257, 8), (5, 1, 40), (8, 64, 1), (1, 40, 40)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_side_by_side(n_experts, n_in, n_out, dtype):
    """Matrices whose rows lie side by side: a transposed view of [in, n_experts, out], also with columns behind."""
    log(f"side by side {n_experts} of {n_in} x {n_out} {dtype}")
    g = torch.Generator().manual_seed(n_in)
    w = torch.randn(n_experts, n_in, n_out, generator=g).to(DT[dtype])
    for behind in (0, 3):
        wide = torch.full((n_in, n_experts * n_out + behind), float("nan"), dtype=w.dtype)
        wide[:, :n_experts * n_out] = w.transpose(0, 1).reshape(n_in, -1)
        view = wide.cuda()[:, :n_experts * n_out].unflatten(1, (n_experts, n_out)).transpose(0, 1)
        assert torch.equal(view.cpu(), w)
        check_weight(experts.quantize_weight(view, backward=True), w)


@pytest.mark.parametrize("rows,n_in,n_out,n_experts", [(70, 140, 100, 0), (40, 200, 130, 0), (200, 140, 100, 3), (300, 130, 90, 5)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_small_whole_numbers(rows, n_in, n_out, n_experts, dtype):
    """Operands of -1, 0 and 1: 8 bits hold them, products are 0 or of one size, and no sum is over 256, which bf16 holds as well. So
    y is linear in x and in w without any rounding, the central difference of <dy, y> is <dx, u> and <dw, v> exactly, and every
    element of the gradients is the formula's. Each difference is another number than 0, so a gradient of 0 or of the other sign fails."""
    g = torch.Generator().manual_seed(rows + n_out)
    dt = DT[dtype]

    def signs(*shape):
        return torch.randint(-1, 2, shape, generator=g).double()
    lead = (n_experts,) if n_experts else ()
    x, u, dy = signs(rows, n_in), signs(rows, n_in), signs(rows, n_out)
    w, v = signs(*lead, n_in, n_out), signs(*lead, n_in, n_out)
    plan, parts = None, [slice(0, rows)]
    if n_experts:
        ids = torch.randint(0, n_experts, (rows, 1), generator=g)
        plan = experts.sort_tokens(ids.cuda(), n_experts)
        offsets = [0] + torch.bincount(ids.flatten(), minlength=n_experts).cumsum(0).tolist()
        parts = [slice(a, b) for a, b in zip(offsets, offsets[1:])]

    def matrix(w, e):
        return w[e] if n_experts else w

    def product(x, w):
        want = torch.cat([x[p] @ matrix(w, e) for e, p in enumerate(parts)])
        assert want.abs().max() <= 256
        y = experts.product8_forward(x.to(dt).cuda(), experts.quantize_weight(w.to(dt).cuda()), plan)
        assert torch.equal(y.double().cpu(), want)
        return y.double().cpu()
    w8 = experts.quantize_weight(w.to(dt).cuda(), backward=True)
    y, saved = experts.product8_forward(x.to(dt).cuda(), w8, plan, save=True)
    dx, dw = (t.double().cpu() for t in experts.product8_backward(dy.to(dt).cuda(), w8, saved, plan))
    assert torch.equal(y.double().cpu(), product(x, w))
    for got, d, plus, minus in ((dx, u, (x + u, w), (x - u, w)), (dw, v, (x, w + v), (x, w - v))):
        want = ((product(*plus) - product(*minus)) * dy).sum() / 2
        assert want != 0 and (got * d).sum() == want
    assert torch.equal(dx, torch.cat([dy[p] @ matrix(w, e).t() for e, p in enumerate(parts)]))
    assert torch.equal(dw, torch.stack([x[p].t() @ dy[p] for p in parts]).view(w.shape))


# ------------------------------------------------------- up to 64 rows, wide matrices
# (type, experts, rows of the experts that have some, slots left out, in, out, the kernel of y, the kernel of dx)
FEW = [
    # one token and a few through a wide matrix: a tile of 32 columns a workgroup
    ("bf16", 0, {0: 1}, 0, 2048, 8192, few(False, 32), few(False, 16)),
    ("f32", 0, {0: 1}, 0, 2048, 8192, few(True, 32), few(True, 16)),
    ("bf16", 0, {0: 17}, 0, 300, 8200, few(False, 32), few(False, 16)),
    ("f32", 0, {0: 17}, 0, 300, 8200, few(True, 32), few(True, 16)),
    ("bf16", 0, {0: 64}, 0, 1000, 8192, few(False, 32), few(False, 16)),
    ("f32", 0, {0: 64}, 0, 1000, 8199, few(True, 32), few(True, 16)),
    ("bf16", 0, {0: 33}, 0, 16384, 130, few(False, 16), few(False, 32)),
    ("bf16", 8, {0: 1, 3: 20, 7: 9}, 2, 520, 1030, few(False, 32), few(False, 16)),
    ("f32", 8, {1: 1, 3: 20, 6: 9}, 2, 1033, 520, few(True, 16), few(True, 32)),
    # more than two tiles a CU, x kept over them; the last columns of a matrix end inside a tile
    ("bf16", 0, {0: 1}, 0, 200, 16416, few(False, 32, 4), few(False, 16)),
    ("f32", 0, {0: 1}, 0, 200, 16415, few(True, 32, 2), few(True, 16)),
    ("bf16", 0, {0: 40}, 0, 130, 16900, few(False, 32, 4), few(False, 16)),
    ("f32", 0, {0: 64}, 0, 130, 16900, few(True, 32, 2), few(True, 16)),
    ("bf16", 8, {0: 3, 2: 17, 5: 1, 7: 33}, 4, 300, 2100, few(False, 32, 4), few(False, 16)),
    ("f32", 8, {1: 3, 2: 17, 5: 1, 6: 33}, 4, 300, 2101, few(True, 32, 2), few(True, 16)),
    ("bf16", 8, {4: 64}, 0, 1000, 2100, few(False, 32, 4), few(False, 16)),
    ("bf16", 8, {0: 9, 6: 5}, 0, 1300, 2059, few(False, 32, 4), few(False, 32)),  # eleven K blocks on eight waves
    ("f32", 8, {0: 9, 6: 5}, 2, 1300, 2059, few(True, 32, 2), few(True, 32)),
    ("bf16", 8, {3: 18, 5: 2}, 0, 4096, 2080, few(False, 32, 4), few(False, 32, 4)),  # the most that is kept
    ("f32", 8, {3: 18, 5: 2}, 0, 2048, 2080, few(True, 32, 2), few(True, 32)),
    ("bf16", 8, {2: 30, 5: 8}, 2, 2200, 1000, few(False, 16), few(False, 32, 4)),
    ("f32", 8, {2: 30, 5: 8}, 2, 2200, 1000, few(True, 16), few(True, 32, 2)),
    ("bf16", 64, {e: 2 + e % 3 for e in range(0, 64, 5)}, 6, 520, 420, few(False, 32, 4), few(False, 32, 4)),
    ("f32", 64, {e: 2 + e % 3 for e in range(0, 64, 5)}, 6, 520, 420, few(True, 32, 2), few(True, 32, 2)),
    # as many tiles, but a K block more than is kept
    ("bf16", 8, {3: 18, 5: 2}, 0, 4097, 2100, few(False, 32), few(False, 32, 4)),
    ("f32", 8, {3: 18, 5: 2}, 0, 2049, 2060, few(True, 32), few(True, 32)),
]


def ids_of(counts, left, slots, seed=0):
    """ids [tokens, slots] with so many slots of each expert and so many left out, in no order."""
    ids = np.repeat(list(counts) + [-1], list(counts.values()) + [left])
    return np.random.default_rng(seed).permutation(ids).reshape(-1, slots)


@pytest.mark.parametrize("dtype,n_experts,counts,left,n_in,n_out,kernel,back_kernel", FEW)
def test_few_rows(dtype, n_experts, counts, left, n_in, n_out, kernel, back_kernel):
    rows = sum(counts.values()) + left
    slots = 2 if rows % 2 == 0 else 1
    log(f"few rows {rows} x {n_in} x {n_out} {dtype} experts {n_experts} {kernel} {back_kernel}")
    g = torch.Generator(device="cuda").manual_seed(rows + n_in)
    dt = DT[dtype]
    x, dy = (torch.randn(rows, n, generator=g, device="cuda").to(dt) for n in (n_in, n_out))
    w = (torch.randn(max(1, n_experts), n_in, n_out, generator=g, device="cuda") * n_in ** -0.5).to(dt)
    w8 = experts.quantize_weight(w if n_experts else w[0], backward=True)
    plan, kept, offsets = None, rows, [0, rows]
    if n_experts:
        ids = ids_of(counts, left, slots)
        plan = experts.sort_tokens(torch.from_numpy(ids).cuda(), n_experts)
        offsets, _, source = ref.plan(ids, n_experts)
        kept = int(offsets[-1])
        x[kept:] = float("nan")  # not read
        dy[kept:] = float("nan")
    y = experts.product8_forward(padded(x.cpu(), 3), w8, plan)
    dx, _ = experts.product8_backward(padded(dy.cpu(), 5), w8, None, plan, need_dw=False)
    want_y, want_dx = (torch.zeros(3, rows, n, dtype=torch.float64) for n in (n_out, n_in))
    for e in counts:
        part = slice(int(offsets[e]), int(offsets[e + 1]))
        we = w[e].cpu()[None]
        want_y[:, part] = ref.product(x[part].cpu(), we)
        want_dx[:, part] = ref.product(dy[part].cpu(), we.transpose(1, 2))
    close("y", y, want_y, n_in)
    close("dx", dx, want_dx, n_out)
    assert torch.equal(experts.product8_forward(x, w8, plan), y)
    if n_experts:  # the same rows taken from the tokens
        tokens = torch.randn(rows // slots, n_in, generator=g, device="cuda").to(dt)
        xs = tokens[torch.from_numpy(np.where(source < 0, ~source, source) // slots).cuda()]
        assert torch.equal(experts.product8_forward(tokens, w8, plan, gather=True), experts.product8_forward(xs, w8, plan))


# ----------------------------------------------------------------- more rows
UNEVEN = {0: 700, 1: 1500, 3: 300, 4: 450}  # expert 2 has none; sums of dW are longer than those of dx for some, not for all
# (type, experts, rows of the experts or of all, slots left out, in, out, the kernel of y, the kernel of dx with dW)
MORE = [
    ("f32", 0, 2100, 0, 300, 2200, tile(True, 128, 2), tile(True, 128, 2)),
    ("f32", 0, 1100, 0, 1500, 2200, tile(True, 128, 2), tile(True, 128, 2)),
    ("f32", 5, {0: 211, 1: 640, 2: 129, 3: 1, 4: 479}, 77, 1001, 2730, tile(True, 128, 2), tile(True, 128, 2)),
    ("f32", 5, UNEVEN, 50, 1500, 390, tile(True, 128, 2), tile(True, 128, 2)),
    ("bf16", 5, UNEVEN, 50, 2048, 512, tile(False, 128, 4), tile(False, 256, 2)),
    ("bf16", 5, UNEVEN, 50, 1300, 999, tile(False, 128, 4), tile(False, 256, 2)),
    ("bf16", 5, UNEVEN, 50, 1301, 1200, tile(False, 128, 2), tile(False, 256, 2)),
]


@pytest.mark.parametrize("dtype,n_experts,counts,left,n_in,n_out,kernel,back_kernel", MORE)
def test_more_rows(dtype, n_experts, counts, left, n_in, n_out, kernel, back_kernel):
    log(f"more rows {kernel} {back_kernel}")
    if not n_experts:
        return check_product(counts, n_in, n_out, dtype, pad=3)
    rows = sum(counts.values()) + left
    slots = 2 if rows % 2 == 0 else 1
    check_product(rows, n_in, n_out, dtype, n_experts, ids_of(counts, left, slots), slots, True, pad=3)


SCATTER = [(40, 9), (30, 16), (30, 17)]  # tokens and slots: up to 16 slots tokens are quantized once for all of theirs


@pytest.mark.parametrize("tokens,slots", SCATTER)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_slots(tokens, slots, dtype):
    ids = np.random.default_rng(slots).integers(-1, 20, size=(tokens, slots))
    check_product(tokens * slots, 200, 136, dtype, 20, ids, slots, True, pad=3)


def test_more_experts_than_are_put_in_order():
    """Over 256 experts dW's tiles go in the experts' order. Of the 300, some are compared, and that those without rows are 0."""
    n_experts, rows, n_in, n_out = 300, 900, 512, 500
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = np.random.default_rng(1).integers(-1, 200, size=(rows, 1))
    ids[:300] = 137
    plan = experts.sort_tokens(torch.from_numpy(ids).cuda(), n_experts)
    offsets, _, source = ref.plan(ids, n_experts)
    x, dy = (torch.randn(rows, n, generator=g, device="cuda").bfloat16() for n in (n_in, n_out))
    w = (torch.randn(n_experts, n_in, n_out, generator=g, device="cuda") * n_in ** -0.5).bfloat16()
    w8 = experts.quantize_weight(w, backward=True)
    y, saved = experts.product8_forward(x, w8, plan, gather=True, save=True)
    dx, dw = experts.product8_backward(dy, w8, saved, plan)
    xs = x.cpu()[torch.from_numpy(np.where(source < 0, ~source, source))]
    for e in (0, 1, 7, 8, 64, 136, 137, 138, 199):
        part = slice(int(offsets[e]), int(offsets[e + 1]))
        close("y", y[part], ref.product(xs[part], w[e].cpu()[None]), n_in)
        close("dx", dx[part], ref.product(dy[part].cpu(), w[e].cpu()[None].transpose(1, 2)), n_out)
        close("dw", dw[e][None], ref.product_dw(xs[part], dy[part].cpu(), None, 1), rows)
    assert not dw[200:].any() and not y[offsets[-1]:].any() and not dx[offsets[-1]:].any()


# -------------------------------------------------------------------- routes
ROUTES = [(6000, 1, 2048, "f32", 0), (4400, 2, 1999, "f32", 3), (1100, 2, 300, "bf16", 0), (1030, 3, 512, "f32", 0)]


@pytest.mark.parametrize("tokens,slots,width,dtype,pad", ROUTES)
@pytest.mark.parametrize("left_out", [0.0, 0.25])
def test_more_routes(tokens, slots, width, dtype, pad, left_out):
    """Four groups of columns a wave in fp32, and one wave a token for narrow rows of many tokens."""
    routes.test_routes(tokens, slots, width, dtype, pad, left_out)


SORT = [(150000, 8, 64), (1060000, 1, 1024)]


@pytest.mark.parametrize("tokens,slots,n_experts", SORT)
def test_sort_of_a_million_slots(tokens, slots, n_experts):
    """Over 4096 slots a workgroup: ids are read twice."""
    ids, dev = make_ids(slots, tokens, slots, n_experts, 0.02, torch.int32)
    check_plan(experts.sort_tokens(dev, n_experts), ids, n_experts)


# -------------------------------------------------------------- largest sizes
def signs(g, *shape, dtype=torch.bfloat16):
    return torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


@pytest.mark.parametrize("rows,n_in,n_out", [(3, 5, 1 << 21), (3, 1 << 21, 5), (90, 5, 1 << 21), (90, 1 << 21, 5)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_widest_matrices(rows, n_in, n_out, dtype):
    """Operands of -1, 0 and 1: every sum is a whole number under 2^24, so results are those numbers, rounded once."""
    log(f"widest {rows} x {n_in} x {n_out} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(rows)
    dt = DT[dtype]
    x, w, dy = signs(g, rows, n_in, dtype=dt), signs(g, n_in, n_out, dtype=dt), signs(g, rows, n_out, dtype=dt)
    w8 = experts.quantize_weight(w, backward=True)
    y, saved = experts.product8_forward(x, w8, save=True)
    want_y, want_dx = x.double() @ w.double(), dy.double() @ w.double().t()
    assert torch.equal(y, want_y.to(dt)) and torch.equal(experts.product8_forward(x, w8), y)
    dx, dw = experts.product8_backward(dy, w8, saved)
    assert torch.equal(dx, want_dx.to(dt)) and torch.equal(dw, (x.double().t() @ dy.double()).to(dt))
    assert torch.equal(experts.product8_backward(dy, w8, None, need_dw=False)[0], dx)


def test_most_rows_that_are_saved():
    """2^23 - 2^18 rows, of one matrix and of three experts, with sums over all of them; and one row more is refused."""
    rows, n_in, n_out = 2 ** 23 - 2 ** 18, 300, 260
    log(f"most rows {rows} x {n_in} x {n_out}")
    g = torch.Generator(device="cuda").manual_seed(7)
    x, dy = signs(g, rows, n_in), signs(g, rows, n_out)
    for n_experts in (0, 3):
        w = signs(g, *((n_experts,) if n_experts else ()), n_in, n_out)
        plan, bounds = None, [0, rows]
        if n_experts:
            ids = torch.randint(0, n_experts, (rows, 1), generator=g, device="cuda", dtype=torch.int32)
            ids[:2 ** 22] = 1
            plan = experts.sort_tokens(ids, n_experts)
            bounds = plan.offsets.tolist()
        w8 = experts.quantize_weight(w, backward=True)
        y, saved = experts.product8_forward(x, w8, plan, save=True)
        dx, dw = experts.product8_backward(dy, w8, saved, plan)
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            we = w[e].float() if n_experts else w.float()
            want = torch.zeros(n_in, n_out, dtype=torch.float64, device="cuda")
            for a in range(lo, hi, 1 << 20):
                part = slice(a, min(hi, a + (1 << 20)))
                want += (x[part].float().t() @ dy[part].float()).double()
                assert torch.equal(y[part], (x[part].float() @ we).bfloat16()) and torch.equal(dx[part], (dy[part].float() @ we.t()).bfloat16())
            assert torch.equal(dw[e] if n_experts else dw, want.bfloat16())
        del y, dx, saved
    with pytest.raises(Exception, match="2\\^23 - 2\\^18"):
        experts.product8_forward(torch.zeros(rows + 1, 8, device="cuda").bfloat16(), experts.quantize_weight(torch.zeros(8, 8, device="cuda").bfloat16()), save=True)


def test_more_rows_than_are_saved():
    rows, n_in, n_out = 20_000_003, 40, 24
    log(f"more rows {rows} x {n_in} x {n_out}")
    g = torch.Generator(device="cuda").manual_seed(8)
    x, w = signs(g, rows, n_in), signs(g, n_in, n_out)
    y = experts.product8_forward(x, experts.quantize_weight(w))
    for a in range(0, rows, 1 << 22):
        assert torch.equal(y[a:a + (1 << 22)], (x[a:a + (1 << 22)].float() @ w.float()).bfloat16())
