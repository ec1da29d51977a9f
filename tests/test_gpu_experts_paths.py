"""The experts' path on the GPU at calls and sizes that tests/test_gpu_experts_product.py does not reach. Bounds are that file's."""
import pytest
import torch

from blocked_shampoo_preconditioning_amd import experts
from tests.gpu_common import log
from tests.test_gpu_experts_product import check_weight
from tests.test_gpu_experts_route import DT

pytestmark = pytest.mark.gpu


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
