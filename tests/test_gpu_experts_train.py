"""The training example with experts: it runs, and its block's gradients are those of the block without roundings to 8 bits
within what these allow. One rounding is off by 2^-4 of a value at most, evenly spread, so by 2^-4 / sqrt(3) in the mean square;
up to eight of them, of independent values, enter a gradient (x, dz, three matrices, h, and g and u in the activation)."""
import math

import pytest
import torch

from blocked_shampoo_preconditioning_amd import experts, train_ffn
from tests.gpu_common import log

pytestmark = pytest.mark.gpu

TOLERANCE = 2.0 ** -4 / math.sqrt(3) * math.sqrt(8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_with_experts_runs(dtype):
    losses = train_ffn.train(layers=2, d=128, f=192, tokens=300, steps=4, block=128, dtype=dtype, n_experts=4, top=2, log=log)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_gradients(dtype):
    d, f, tokens, n_experts, top = 128, 256, 600, 4, 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    half = train_ffn.ExpertsHalfLayer(d, f, gen, dtype, n_experts, top, dropout=0.0)
    a = torch.randn(tokens, d, generator=gen, device="cuda").to(dtype)
    dz = torch.randn(tokens, d, generator=gen, device="cuda").to(dtype)
    z, saved = half.block_forward(a)
    da, matrices = half.block_backward(dz, a, saved)
    ids = saved[0]
    x, r = a.double().requires_grad_(), half.router.double().requires_grad_()
    w = [m.double().requires_grad_() for m in half.stacked]
    weights = (x @ r).gather(1, ids).softmax(1)
    want = torch.zeros_like(x)
    for e in range(n_experts):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        xe = x[t]
        ye = (torch.nn.functional.silu(xe @ w[0][e]) * (xe @ w[1][e])) @ w[2][e]
        want = want.index_add(0, t, ye * weights[t, j][:, None])
    grads = torch.autograd.grad(want, [x, r, *w], dz.double())
    got = {"z": (z, want.detach()), "da": (da, grads[0]), "router": (matrices[0], grads[1])}
    for k, name in enumerate(("gate", "up", "down")):
        got[name] = (torch.stack(matrices[1 + k * n_experts:1 + (k + 1) * n_experts]), grads[2 + k])
    for name, (value, exact) in got.items():
        off = ((value.double() - exact).norm() / exact.norm()).item()
        log(f"{name}: {off:.4f}")
        assert off <= TOLERANCE, name


def test_refusals():
    x = torch.zeros(4, 128, device="cuda")
    w8 = experts.quantize_weight(torch.zeros(128, 64, device="cuda"))
    several = experts.quantize_weight(torch.zeros(2, 128, 64, device="cuda"))
    plan = experts.sort_tokens(torch.zeros(4, 1, dtype=torch.int32, device="cuda"), 2)
    y, saved = experts.product8_forward(x, w8, save=True)
    calls = [
        (lambda: experts.sort_tokens(torch.zeros(4, dtype=torch.int64, device="cuda"), 2), "2-D"),
        (lambda: experts.sort_tokens(torch.zeros(4, 1, device="cuda"), 2), "int32 and int64"),
        (lambda: experts.sort_tokens(torch.zeros(4, 1, dtype=torch.int64, device="cuda"), 0), "n_experts"),
        (lambda: experts.sort_tokens(torch.zeros(4, 1, dtype=torch.int64, device="cuda"), 1025), "n_experts"),
        (lambda: experts.dispatch(x[:3], plan), "shape"),
        (lambda: experts.dispatch(x.half(), plan), "float32 and bfloat16"),
        (lambda: experts.dispatch(x.t(), plan), "shape"),
        (lambda: experts.combine(x[:3], plan), "shape"),
        (lambda: experts.combine(x, plan, torch.ones(4, 2, device="cuda")), "weights"),
        (lambda: experts.combine(x, plan, torch.ones(4, 1, device="cuda").bfloat16()), "weights"),
        (lambda: experts.combine(x, plan, torch.ones(4, 1)), "weights"),
        (lambda: experts.combine_backward(x, x.bfloat16(), plan, torch.ones(4, 1, device="cuda")), "ys"),
        (lambda: experts.combine(x, plan._replace(rows=plan.rows.long())), "plan.rows"),
        (lambda: experts.quantize_weight(torch.zeros(3, device="cuda")), r"\[in, out\]"),
        (lambda: experts.quantize_weight(torch.zeros(0, 3, device="cuda")), "shape"),
        (lambda: experts.quantize_weight(torch.zeros(4, 4, dtype=torch.float64, device="cuda")), "float64"),
        (lambda: experts.quantize_weight(torch.zeros(4, 4, device="cuda").t()[:, :2]), "contiguous"),
        (lambda: experts.product8_forward(x[:, :100], w8), "shape"),
        (lambda: experts.product8_forward(x, several), "plan is None"),
        (lambda: experts.product8_forward(x, w8, gather=True), "gather needs a plan"),
        (lambda: experts.product8_forward(x, several, plan._replace(offsets=plan.offsets[:2])), "plan.offsets"),
        (lambda: experts.product8_forward(x, several, plan._replace(source=plan.source[:3]), gather=True), "plan.source"),
        (lambda: experts.product8_forward(x[:3], several, plan), "shape"),
        (lambda: experts.product8_forward(x, w8._replace(values=w8.values[:, :64])), "w8.values"),
        (lambda: experts.product8_forward(x, w8._replace(scales=w8.scales.view(torch.uint8))), "w8.scales"),
        (lambda: experts.product8_forward(x, w8._replace(n_out=65)), "w8.values"),
        (lambda: experts.product8_backward(y, w8, saved), "no backward values"),
        (lambda: experts.product8_backward(y, w8, saved[:-1], need_dx=False), "saved"),
        (lambda: experts.product8_backward(y, w8, None, need_dx=False), "saved"),
        (lambda: experts.product8_backward(y[:, :10], w8, saved, need_dx=False), "shape"),
    ]
    for call, message in calls:
        with pytest.raises(ValueError, match=message):
            call()


def test_empty_batches():
    """No rows, and no columns where an operator allows them."""
    plan = experts.sort_tokens(torch.zeros(0, 2, dtype=torch.int64, device="cuda"), 3)
    assert plan.offsets.tolist() == [0, 0, 0, 0] and plan.rows.shape == (0, 2) and plan.source.shape == (0,)
    x = torch.zeros(0, 130, device="cuda").bfloat16()
    w8 = experts.quantize_weight(torch.ones(3, 130, 40, device="cuda").bfloat16(), backward=True)
    for gather in (False, True):
        y, saved = experts.product8_forward(x, w8, plan, gather=gather, save=True)
        dx, dw = experts.product8_backward(y, w8, saved, plan)
        assert y.shape == (0, 40) and dx.shape == (0, 130) and dw.shape == (3, 130, 40) and not dw.any()
    one = experts.quantize_weight(torch.ones(130, 40, device="cuda").bfloat16(), backward=True)
    y, saved = experts.product8_forward(x, one, save=True)
    dx, dw = experts.product8_backward(y, one, saved)
    assert y.shape == (0, 40) and dx.shape == (0, 130) and dw.shape == (130, 40) and not dw.any()
    assert experts.product8_forward(x, one).shape == (0, 40)
    ids = torch.zeros(5, 2, dtype=torch.int64, device="cuda")
    plan = experts.sort_tokens(ids, 3)
    none = torch.zeros(5, 0, device="cuda")
    xs = experts.dispatch(none, plan)
    assert xs.shape == (10, 0) and experts.combine(xs, plan, torch.ones(5, 2, device="cuda")).shape == (5, 0)
    dys, dweights = experts.combine_backward(none, xs, plan, torch.ones(5, 2, device="cuda"))
    assert dys.shape == (10, 0) and not dweights.any()


def test_no_gradient_of_a_plan_enters_autograd():
    """The calls record no graph, also for leaves that require a gradient, eager or captured."""
    x = torch.randn(64, 128, device="cuda", requires_grad=True)
    w = torch.randn(128, 96, device="cuda", requires_grad=True)
    y, saved = experts.product8_forward(x, experts.quantize_weight(w, backward=True), save=True)
    assert not y.requires_grad and y.grad_fn is None
    eager = (x * 2).sum()  # a graph of the same leaves that lives over the capture
    w8 = experts.quantize_weight(w.detach(), backward=True)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dx, dw = experts.product8_backward(y, w8, saved)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = experts.product8_backward(y, w8, saved)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    eager.backward()
    assert torch.equal(x.grad, torch.full_like(x, 2))


def test_calls_at_once_on_two_streams():
    """Each call's scratch memory is its own."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = [torch.randn(700, 256, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    w8 = experts.quantize_weight(torch.randn(4, 256, 384, generator=gen, device="cuda").bfloat16())
    ids = [torch.randint(0, 4, (700, 2), generator=gen, device="cuda") for _ in range(2)]

    def run(k):
        plan = experts.sort_tokens(ids[k], 4)
        return experts.combine(experts.product8_forward(x[k], w8, plan, gather=True), plan)
    want = [run(0), run(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(run(k))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[k]) for k in range(2) for t in got[k])
