"""Calls at the edge of what the layer operators accept, on the GPU against plain 64-bit forms (tests/layer_reference.py)."""
import math

import pytest
import torch

from blocked_shampoo_preconditioning_amd import layer
from tests import layer_reference as ref
from tests.gpu_common import log
from tests.layer_reference import BF16_STEP, F32_STEP, rel

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f32_tol(k):
    """The fp32 results' tolerance for sums of k terms (their root sum of squares times this)."""
    return 8 * (4 + math.sqrt(k)) * F32_STEP


def normal(gen, *shape, std=1.0, mean=0.0, dtype="f32"):
    return (torch.randn(*shape, generator=gen) * std + mean).to(DT[dtype]).cuda()


# 2^63 - 1 - 2500: the number of gate rows, rounded up by an addition, would come out as -1
@pytest.mark.parametrize("rows_per_gate", [2 ** 63 - 1, 2 ** 63 - 1 - 2500, 2 ** 40])
def test_one_gate_row_for_any_number_of_rows(rows_per_gate):
    """rows_per_gate far over the rows is one row for all: the same bits as rows_per_gate = rows, every vector's gradient written."""
    g = torch.Generator().manual_seed(1)
    n, d = 3000, 72
    x, z, dr, dn = (normal(g, n, d) for _ in range(4))
    s = dict(gate=normal(g, 1, d, std=0.3, mean=0.5), post_weight=normal(g, d, std=0.1, mean=1.0), next_weight=normal(g, d, std=0.1, mean=1.0))
    log(f"norm {n} x {d}, rows_per_gate {rows_per_gate}")

    def run(rows):
        r, nn, st = layer.residual_forward(x, z, rows_per_gate=rows, **s)
        return [r, nn, *layer.residual_backward(dr, dn, r, z, st, rows_per_gate=rows, **s).values()]
    want = [t.clone() if t is not None else None for t in run(n)]
    # what the allocator hands out next holds NaN
    held = [torch.full(t.shape, float("nan"), device="cuda") for t in want if t is not None for _ in range(4)]
    del held
    for a, b in zip(run(rows_per_gate), want):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
