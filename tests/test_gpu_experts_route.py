"""Tokens sorted by expert and back on the GPU against plain 64-bit forms (tests/experts_reference.py).

Plans and copies are exact. Tolerances, set before the first run, for each element: one rounding to the result's type
(HALF_STEP of the value), and for sums of k products in fp32 (k + 1) * 2^-24 of the sum of the terms' magnitudes, whatever
the order they are added in; results under 2^-126 absolute are not compared further."""
import numpy as np
import pytest
import torch

from blocked_shampoo_preconditioning_amd import experts
from tests import experts_reference as ref
from tests.experts_reference import HALF_STEP
from tests.gpu_common import log

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make_ids(seed, tokens, slots, n_experts, left_out=0.0, dtype=torch.int64, pad=0):
    g = np.random.default_rng(seed)
    ids = g.integers(0, n_experts, size=(tokens, slots))  # an expert may come twice in a token
    outside = g.choice([-1, n_experts, -(2 ** 31), 2 ** 31 - 1], size=ids.shape)
    ids = np.where(g.random(ids.shape) < left_out, outside, ids)
    wide = torch.zeros(tokens, slots + pad, dtype=dtype)
    wide[:, :slots] = torch.from_numpy(ids).to(dtype)
    return ids, wide.cuda()[:, :slots]


def padded(t, pad):
    """t on the GPU with `pad` elements of NaN behind every row."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype)
    wide[:, :t.shape[1]] = t
    return wide.cuda()[:, :t.shape[1]]


def close(name, got, want, dtype, size=None, terms=0):
    want = want.cuda()
    bound = want.abs() * HALF_STEP[dtype] * (1 + 2.0 ** -20) + 2.0 ** -126
    if size is not None:
        bound = bound + (terms + 1) * 2.0 ** -24 * size.cuda()
    worst = ((got.double() - want).abs() / bound).max().item() if want.numel() else 0.0
    assert worst <= 1.0, (name, worst)


def check_plan(plan, ids, n_experts):
    offsets, rows, source = ref.plan(ids, n_experts)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.rows.cpu().numpy(), rows)
    assert np.array_equal(plan.source.cpu().numpy(), source)
    return rows


@pytest.mark.parametrize("tokens,slots,n_experts,left_out", [
    (0, 2, 4, 0.0), (1, 1, 1, 0.0), (1, 2, 8, 0.0), (1, 8, 8, 1.0), (63, 1, 2, 0.1), (64, 3, 5, 0.0), (65, 2, 7, 0.3),
    (257, 8, 64, 0.05), (1000, 4, 13, 0.0), (4096, 1, 8, 0.0), (4097, 1, 8, 0.2), (700, 6, 1024, 0.1), (5000, 3, 1024, 0.0),
    (20000, 8, 64, 0.02), (300, 1024, 1023, 0.01), (33000, 2, 1, 0.5)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(tokens, slots, n_experts, left_out, dtype):
    log(f"sort {tokens} x {slots} of {n_experts} left out {left_out} {dtype}")
    ids, dev = make_ids(tokens + slots, tokens, slots, n_experts, left_out, dtype, pad=3)
    check_plan(experts.sort_tokens(dev, n_experts), ids, n_experts)


def test_sort_one_expert_takes_all():
    for value in (0, 5, -1):
        ids = np.full((9000, 2), value)
        check_plan(experts.sort_tokens(torch.from_numpy(ids).cuda(), 6), ids, 6)


@pytest.mark.parametrize("tokens,slots,width,dtype,pad", [
    (1, 2, 2048, "bf16", 0), (1, 1, 1, "f32", 0), (3, 2, 7, "bf16", 5), (64, 3, 8, "f32", 0), (65, 5, 777, "f32", 3),
    (100, 4, 1001, "bf16", 1), (257, 2, 2048, "f32", 0), (300, 3, 2056, "bf16", 8), (130, 2, 5000, "f32", 4),
    (70, 9, 8193, "bf16", 7), (33, 2, 16500, "f32", 0), (5000, 2, 600, "bf16", 0), (4500, 3, 2048, "bf16", 2),
    (4200, 2, 1536, "f32", 0), (9000, 2, 520, "f32", 0), (0, 2, 64, "bf16", 0)])
@pytest.mark.parametrize("left_out", [0.0, 0.25, 1.0])
def test_routes(tokens, slots, width, dtype, pad, left_out):
    log(f"routes {tokens} x {slots} x {width} {dtype} pad {pad} left out {left_out}")
    n_experts, dt = 6, DT[dtype]
    ids, dev = make_ids(tokens + width, tokens, slots, n_experts, left_out)
    plan = experts.sort_tokens(dev, n_experts)
    rows = check_plan(plan, ids, n_experts)
    g = torch.Generator().manual_seed(width)
    x, dy = (torch.randn(tokens, width, generator=g).to(dt) for _ in range(2))
    ys, dxs = (torch.randn(tokens * slots, width, generator=g).to(dt) for _ in range(2))
    weights = torch.rand(tokens, slots, generator=g)
    out = torch.from_numpy(rows < 0)
    weights[out] = float("nan")  # what left-out slots hold is not read
    behind = torch.from_numpy(~rows[rows < 0])
    ys[behind] = float("nan")
    dxs[behind] = float("inf")
    dx_, dys_ = padded(x, pad), padded(ys, pad)

    xs = experts.dispatch(dx_, plan)
    assert xs.shape == (tokens * slots, width) and torch.equal(xs.cpu().double(), ref.dispatch(x, rows))
    want, size = ref.combine(ys, rows, weights)
    close("y", experts.combine(dys_, plan, weights.cuda()), want, dt, size, slots)
    want, size = ref.combine(dxs, rows)
    close("dx", experts.dispatch_backward(padded(dxs, pad), plan), want, dt, size, slots)
    dys, dweights = experts.combine_backward(padded(dy, pad), dys_, plan, weights.cuda())
    want, dw, size = ref.combine_backward(dy, ys, rows, weights)
    close("dys", dys, want, dt, want.abs())  # the product's own rounding to fp32
    assert dweights.dtype == torch.float32
    close("dweights", dweights, dw, torch.float32, size, width)
    plain, none = experts.combine_backward(padded(dy, pad), dys_, plan)
    assert none is None and torch.equal(plain.cpu().double(), ref.dispatch(dy, rows))
    # the same bits again
    again = experts.combine_backward(padded(dy, pad), dys_, plan, weights.cuda())
    assert torch.equal(again[0], dys) and torch.equal(again[1], dweights)


def test_gradients_against_differences():
    """Of the whole way there and back, L = <dy, combine(dispatch(x) * s, weights)>: linear in x and in weights, so that a
    difference over a step is exact but for the roundings (fp32: 2^-24 of each of some 10^3 terms of the sums)."""
    tokens, slots, width = 40, 3, 96
    ids, dev = make_ids(5, tokens, slots, 4, 0.2)
    plan = experts.sort_tokens(dev, 4)
    g = torch.Generator().manual_seed(9)
    x, dy, u = (torch.randn(tokens, width, generator=g).cuda() for _ in range(3))
    s = torch.randn(tokens * slots, 1, generator=g).cuda()
    weights, v = torch.rand(tokens, slots, generator=g).cuda(), torch.randn(tokens, slots, generator=g).cuda()

    def loss(x, weights):
        return (experts.combine(experts.dispatch(x, plan) * s, plan, weights).double() * dy.double()).sum()
    ys = experts.dispatch(x, plan) * s
    dys, dweights = experts.combine_backward(dy, ys, plan, weights)
    dx = experts.dispatch_backward(dys * s, plan)
    for got, want in (((dx.double() * u.double()).sum(), (loss(x + u, weights) - loss(x - u, weights)) / 2),
                      ((dweights.double() * v.double()).sum(), (loss(x, weights + v) - loss(x, weights - v)) / 2)):
        assert abs(got - want) <= 2.0 ** -24 * 4 * 2 * tokens * slots * width


def test_non_finite_values_reach_their_token_alone():
    ids = np.array([[0, 1], [1, 2], [2, 0]])
    plan = experts.sort_tokens(torch.from_numpy(ids).cuda(), 3)
    rows = ref.plan(ids, 3)[1]
    ys = torch.ones(6, 40, device="cuda")
    ys[rows[1, 0], 3] = float("inf")
    ys[rows[1, 1], 4] = float("nan")
    y = experts.combine(ys, plan, torch.full((3, 2), 0.5, device="cuda"))
    want = torch.ones(3, 40)
    want[1, 3], want[1, 4] = float("inf"), float("nan")
    assert torch.equal(torch.nan_to_num(y.cpu(), nan=-7.0), torch.nan_to_num(want, nan=-7.0))


def test_rows_of_another_plan():
    """Rows past the batch's count as left out, and nothing is written for them."""
    rows = torch.tensor([[0, 6], [2, -8], [1, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    plan = experts.Plan(None, rows, None)
    x = torch.arange(3.0, device="cuda")[:, None].repeat(1, 16) + 1
    y = experts.combine(torch.ones(6, 16, device="cuda"), plan, torch.full((3, 2), 2.0, device="cuda"))
    assert torch.equal(y, torch.full((3, 16), 2.0, device="cuda"))
    xs = experts.dispatch(x, plan)
    assert torch.equal(xs[[0, 2, 1], 0].cpu(), torch.tensor([1.0, 2.0, 3.0]))
    dys, dw = experts.combine_backward(x, torch.ones(6, 16, device="cuda"), plan, torch.full((3, 2), 2.0, device="cuda"))
    assert torch.equal(dw.cpu(), torch.tensor([[16.0, 0.0], [32.0, 0.0], [48.0, 0.0]]))


def test_offsets_past_32_bits():
    tokens, slots, width = 140000, 8, 2048  # 2.3e9 elements of sorted rows
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, 16, (tokens, slots), generator=g, device="cuda")
    plan = experts.sort_tokens(ids, 16)
    x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
    xs = experts.dispatch(x, plan)
    for t in (0, 1, 77777, tokens - 1):
        for j in range(slots):
            assert torch.equal(xs[plan.rows[t, j].item()], x[t])
    assert torch.equal(xs[-1], x[plan.source[-1].item() // slots])
    y = experts.combine(xs, plan)
    assert torch.equal(y, x * 8)  # a sum of eight equal bf16 values is exact
    del y
    dys, dw = experts.combine_backward(x, xs, plan, torch.ones(tokens, slots, device="cuda"))
    assert torch.equal(dys, xs)
    want = x[-5:].double().square().sum(1, keepdim=True).expand(5, slots)
    assert ((dw[-5:].double() - want).abs() <= (width + 2) * 2.0 ** -24 * want).all()


def test_more_tokens_than_a_launch_has_threads_for():
    """2^26 tokens and some, four to a workgroup of 256: over 2^32 threads in all. (In torch too an index of so many rows
    gives five rows and nothing else: the rows are taken in parts.)"""
    tokens, width = 2 ** 26 + 5, 8
    log(f"routes {tokens} x 1 x {width}")
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(-1, 4, (tokens, 1), generator=g, device="cuda", dtype=torch.int32)
    plan = experts.sort_tokens(ids, 4)
    x = torch.randint(-4, 5, (tokens, width), generator=g, device="cuda").bfloat16()
    want = torch.cat([x[torch.where(s < 0, ~s, s)] * (s >= 0)[:, None] for s in plan.source.long().split(2 ** 24)])
    assert torch.equal(plan.offsets[1:].long(), torch.stack([(ids[:, 0] == e).sum() for e in range(4)]).cumsum(0))
    xs = experts.dispatch(x, plan)
    assert torch.equal(xs, want)
    kept = x * (ids >= 0)
    assert torch.equal(experts.combine(xs, plan), kept)
    dys, dw = experts.combine_backward(x, xs, plan, torch.full((tokens, 1), 2.0, device="cuda"))
    assert torch.equal(dys, 2 * want)
    assert torch.equal(dw[:, 0], kept.float().square().sum(1))  # small integers: exact


def test_streams_and_graphs():
    """On another stream, and captured into a graph that is replayed with eager work between."""
    ids, dev = make_ids(3, 3000, 2, 8, 0.1)
    x = torch.randn(3000, 128, device="cuda").bfloat16()
    weights = torch.rand(3000, 2, device="cuda")

    def run():
        plan = experts.sort_tokens(dev, 8)
        xs = experts.dispatch(x, plan)
        return (*plan, xs, experts.combine(xs, plan, weights), *experts.combine_backward(x, xs, plan, weights))
    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = run()
    for turn in range(3):
        x.copy_(torch.randn(3000, 128, device="cuda").bfloat16())
        dev.copy_(torch.from_numpy(make_ids(10 + turn, 3000, 2, 8, 0.1)[0]).cuda())
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, run())), turn
