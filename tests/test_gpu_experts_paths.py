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
