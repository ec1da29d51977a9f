"""The measured cases of the experts' path of a feed-forward block: tokens sorted by expert and back, with weights applied, and the
matrix product in 8-bit floating point with a scale for each block of 128, dense or one matrix an expert; forward and backward.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once at the end), or, where `own` is
true, by the framework's entry points in `blocked_shampoo_preconditioning_amd.experts`."""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a 1B-class decoder while it is sampled from: to its two experts and back, latency alone
        {"name": "sort_one_token_bf16", "op": "sort", "train": False, "tokens": 1, "slots": 2, "experts": 8, "d": 2048, "left_out": 0.0,
         "dtype": "bf16"},
        # training on four sequences of 2048, two of eight experts for each token
        {"name": "sort_train_bf16", "op": "sort", "train": True, "tokens": 8192, "slots": 2, "experts": 8, "d": 2048, "left_out": 0.0,
         "dtype": "bf16"},
        # many small experts, eight of 64 for each token: eight copies of every row
        {"name": "sort_many_experts_bf16", "op": "sort", "train": True, "tokens": 16384, "slots": 8, "experts": 64, "d": 2048,
         "left_out": 0.0, "dtype": "bf16"},
        # packed sequences of uneven length, an odd width, slots that a capacity limit has left out
        {"name": "sort_ragged_f32", "op": "sort", "train": True, "tokens": 3001, "slots": 3, "experts": 13, "d": 777, "left_out": 0.05,
         "dtype": "f32"},
        # one token through one dense 8-bit matrix: its weights are read for one row
        {"name": "product_one_token_bf16", "op": "product", "train": False, "tokens": 1, "slots": 0, "experts": 0, "in": 2048, "out": 8192,
         "left_out": 0.0, "dtype": "bf16"},
        # a small batch of requests on eight experts: a few rows each, every expert's weights read
        {"name": "product_experts_few_bf16", "op": "product", "train": False, "tokens": 16, "slots": 2, "experts": 8, "in": 2048,
         "out": 8192, "left_out": 0.0, "dtype": "bf16"},
        # two prompts of 2048 through the second matrix of a 1B-class block
        {"name": "product_prompt_bf16", "op": "product", "train": False, "tokens": 4096, "slots": 0, "experts": 0, "in": 8192, "out": 2048,
         "left_out": 0.0, "dtype": "bf16"},
        # prompts on many small experts, eight of 64 for each token
        {"name": "product_experts_prompt_bf16", "op": "product", "train": False, "tokens": 2048, "slots": 8, "experts": 64, "in": 2048,
         "out": 768, "left_out": 0.0, "dtype": "bf16"},
        # the training step of one matrix of the 1B-class set on four sequences of 2048: new weights in 8 bits, forward, both gradients
        {"name": "product_train_1b_bf16", "op": "product", "train": True, "tokens": 8192, "slots": 0, "experts": 0, "in": 2048,
         "out": 8192, "left_out": 0.0, "dtype": "bf16"},
        # the same at GPT-small width on one sequence of 1024: too few tiles to fill the card
        {"name": "product_train_small_bf16", "op": "product", "train": True, "tokens": 1024, "slots": 0, "experts": 0, "in": 768,
         "out": 2048, "left_out": 0.0, "dtype": "bf16"},
        # the experts' training step: eight matrices, two for each token
        {"name": "product_experts_train_bf16", "op": "product", "train": True, "tokens": 8192, "slots": 2, "experts": 8, "in": 2048,
         "out": 2048, "left_out": 0.0, "dtype": "bf16"},
        # fp32, widths that are no multiple of anything, uneven experts, slots left out
        {"name": "product_ragged_f32", "op": "product", "train": True, "tokens": 1537, "slots": 1, "experts": 5, "in": 1001, "out": 2730,
         "left_out": 0.05, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width over its logarithm: mostly a multiple of 64, some of 8, some of nothing."""
    n = _log(rng, lo, hi)
    step = rng.choice((64, 64, 64, 8, 1))
    return min(hi, max(step, n // step * step))


def draw(rng):
    op = rng.choice(("sort", "sort", "serve", "serve", "train", "train"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    left_out = rng.choice((0.0, 0.0, 0.05))
    experts = _log(rng, 2, 64 if op == "sort" else 16)
    slots = rng.randint(1, min(8, experts))
    if op == "sort":
        return {"op": "sort", "train": rng.random() < 0.7, "tokens": _log(rng, 1, 16384), "slots": slots, "experts": experts,
                "d": _width(rng, 64, 2048), "left_out": left_out, "dtype": dtype}
    if rng.random() < 0.4:
        experts, slots, left_out = 0, 0, 0.0
    tokens = _log(rng, 1, 4096 // max(1, slots) if op == "serve" else 8192 // max(1, slots))
    return {"op": "product", "train": op == "train", "tokens": tokens, "slots": slots, "experts": experts, "in": _width(rng, 64, 2048),
            "out": _width(rng, 64, 2048 if experts else 8192), "left_out": left_out, "dtype": dtype}


def _rows(case):
    return case["tokens"] * max(1, case["slots"])


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    n, k, e = case["tokens"], case["slots"], case["experts"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    s = {"case": case}
    if e:  # a router's choice: the likeliest experts of each token, some experts liked more than others, some slots left out
        logits = torch.randn(n, e, generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
        top, ids = logits.softmax(1).topk(k, dim=1)
        s["weights"] = top / top.sum(1, keepdim=True)
        s["ids"] = torch.where(torch.rand(n, k, generator=g, device="cuda") < case["left_out"], -1, ids)
    if case["op"] == "sort":
        d = case["d"]
        s["x"], s["ys"] = normal(n, d), normal(n * k, d, std=0.5)
        if case["train"]:
            s["dy"], s["dxs"] = normal(n, d, std=1e-2), normal(n * k, d, std=1e-2)
        return s
    # activations with a few wide features, as they are behind a norm with weights
    s["x"] = (normal(n, case["in"]).float() * torch.exp(torch.randn(case["in"], generator=g, device="cuda"))).to(dt)
    w = normal(*((e,) if e else ()), case["in"], case["out"], std=case["in"] ** -0.5)
    if case["train"]:
        s["w"], s["dy"] = w, normal(_rows(case), case["out"], std=1e-2)
    else:  # a serving program keeps the 8-bit weights alone
        s["w8"] = _laid_out(w)
    return s


def _laid_out(w):
    """8-bit weights as they are kept: values [.., out, in rounded up to 128], a scale for each 128 x 128 block."""
    v = w.float().reshape(-1, *w.shape[-2:]).transpose(1, 2)  # [e, out, in]
    e, out, cols = v.shape
    ob, kb = -(-out // BLOCK), -(-cols // BLOCK)
    p = torch.zeros(e, ob * BLOCK, kb * BLOCK, device=w.device)
    p[:, :out, :cols] = v
    p = p.view(e, ob, BLOCK, kb, BLOCK)
    power = _power(p.abs().amax((2, 4)))
    q = torch.ldexp(p, -power[:, :, None, :, None]).to(torch.float8_e4m3fn).view(e, ob * BLOCK, kb * BLOCK)[:, :out].contiguous()
    scales = torch.full((e, ob, -(-kb // 4) * 4), 127, dtype=torch.uint8, device=w.device)
    scales[:, :, :kb] = (power + 127).to(torch.uint8)
    lead = w.shape[:-2]
    return q.view(*lead, out, -1), scales.view(torch.float8_e8m0fnu).view(*lead, ob, -1)


# ----------------------------------------------------------------------- run
def run(s):
    if own:
        return _run_own(s)
    return _plain_sort(s) if s["case"]["op"] == "sort" else _plain_product(s)


def _run_own(s):
    from blocked_shampoo_preconditioning_amd import experts
    c = s["case"]
    plan = experts.sort_tokens(s["ids"], c["experts"]) if c["experts"] else None
    if c["op"] == "sort":
        out = {"offsets": plan.offsets, "rows": plan.rows, "source": plan.source, "xs": experts.dispatch(s["x"], plan),
               "y": experts.combine(s["ys"], plan, s["weights"])}
        if c["train"]:
            out["dys"], out["dweights"] = experts.combine_backward(s["dy"], s["ys"], plan, s["weights"])
            out["dx"] = experts.dispatch_backward(s["dxs"], plan)
        return out
    if not c["train"]:
        return {"y": experts.product8_forward(s["x"], experts.Weight8(*s["w8"], c["in"], c["out"]), plan, gather=plan is not None)}
    w8 = experts.quantize_weight(s["w"], backward=True)
    y, saved = experts.product8_forward(s["x"], w8, plan, gather=plan is not None, save=True)
    dx, dw = experts.product8_backward(s["dy"], w8, saved, plan)
    return {"y": y, "dx": dx, "dw": dw}


# --------------------------------------------------------------- plain forms
def _plain_plan(ids, experts):
    """Offsets of the experts' rows, each slot's row (~row where it is left out, behind the others), each row's slot."""
    key = ids.reshape(-1)
    kept = (key >= 0) & (key < experts)
    key = torch.where(kept, key, experts)
    order = torch.argsort(key, stable=True)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(torch.bincount(key, minlength=experts + 1)[:experts], 0)
    return offsets, torch.where(kept, rows, ~rows), torch.where(kept[order], order, ~order)


def _plain_sort(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    n, k, d = c["tokens"], c["slots"], c["d"]
    offsets, rows, source = _plain_plan(s["ids"], c["experts"])
    out = {"offsets": offsets.int(), "rows": rows.view(n, k).int(), "source": source.int()}
    slot = torch.where(source >= 0, source, ~source)
    kept_row = (source >= 0)[:, None]
    at = torch.where(rows >= 0, rows, ~rows)
    kept = (rows >= 0).view(n, k)
    out["xs"] = torch.where(kept_row, s["x"].float()[slot // k], 0.0).to(dt)
    ys = torch.where(kept[:, :, None], s["ys"].float()[at].view(n, k, d), 0.0)
    out["y"] = (ys * s["weights"][:, :, None]).sum(1).to(dt)
    if c["train"]:
        dy = s["dy"].float()
        out["dys"] = torch.where(kept_row, dy[slot // k] * s["weights"].reshape(-1)[slot][:, None], 0.0).to(dt)
        out["dweights"] = (ys * dy[:, None, :]).sum(2)
        out["dx"] = torch.where(kept[:, :, None], s["dxs"].float()[at].view(n, k, d), 0.0).sum(1).to(dt)
    return out


def _power(amax):
    """The exponent of a block's scale: the smallest e >= -126 with amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)
    return torch.clamp(torch.where(m > 0.875, x - 8, x - 9), min=-126)


def _plain_quantized(x):
    """x [.., k] in 8 bits by blocks of 128 along its last axis, as the values that these stand for."""
    k = x.shape[-1]
    p = torch.nn.functional.pad(x, (0, -k % BLOCK)).view(*x.shape[:-1], -1, BLOCK)
    power = _power(p.abs().amax(-1, keepdim=True))
    q = torch.ldexp(torch.ldexp(p, -power).to(torch.float8_e4m3fn).float(), power)
    return q.view(*x.shape[:-1], -1)[..., :k]


def _plain_kept_weight(s):
    """[e, in, out] values of the 8-bit weights."""
    c = s["case"]
    values, scales = s["w8"] if "w8" in s else _laid_out(s["w"])
    values = values.float().view(-1, c["out"], values.shape[-1])
    power = scales.view(torch.uint8).int().view(values.shape[0], -1, scales.shape[-1]) - 127
    power = power.repeat_interleave(BLOCK, 1)[:, :c["out"]].repeat_interleave(BLOCK, 2)[:, :, :values.shape[2]]
    return torch.ldexp(values, power)[:, :, :c["in"]].transpose(1, 2).contiguous()


def _plain_product(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    n, e = _rows(c), max(1, c["experts"])
    x = s["x"].float()
    w = _plain_kept_weight(s)
    # rows by expert in a padded batch [e, cap, ..]: `place` of each sorted row that belongs to one
    if c["experts"]:
        offsets, _, source = _plain_plan(s["ids"], e)
        kept = source >= 0
        row = torch.arange(n, device=x.device)
        of = torch.clamp(torch.searchsorted(offsets, row, right=True) - 1, max=e - 1)
        cap = -(-int((offsets[1:] - offsets[:-1]).max()) // BLOCK) * BLOCK or BLOCK
        place = (of * cap + row - offsets[of])[kept]
        x = torch.where(kept[:, None], x[torch.where(kept, source, ~source) // c["slots"]], 0.0)
    else:
        kept = torch.ones(n, dtype=torch.bool, device=x.device)
        cap = -(-n // BLOCK) * BLOCK
        place = torch.arange(n, device=x.device)

    def batch(rows):
        return torch.zeros(e * cap, rows.shape[1], device=rows.device).index_copy_(0, place, rows[kept]).view(e, cap, -1)

    def back(batched):
        out = torch.zeros(n, batched.shape[2], device=batched.device)
        out[kept] = batched.reshape(e * cap, -1)[place]
        return out.to(dt)

    def quantized_columns(t):
        return _plain_quantized(t.transpose(1, 2).contiguous())

    xb = batch(x)
    out = {"y": back(torch.bmm(_plain_quantized(xb), w))}
    if c["train"]:
        dyb = batch(s["dy"].float())
        out["dx"] = back(torch.bmm(_plain_quantized(dyb), w.transpose(1, 2).contiguous()))
        dw = torch.bmm(quantized_columns(xb), quantized_columns(dyb).transpose(1, 2).contiguous())
        out["dw"] = dw.to(dt).view(s["w"].shape)
    return out


# --------------------------------------------------------------------- exact
def _exact_quantized(x, dims):
    """8-bit values of float64 x by blocks of 128 along `dims` together, from the format's definition: three bits behind the leading
    one, exponents from -6, ties to even, the largest 448."""
    shape = list(x.shape)
    split, block_dims = [], []
    pads = []
    for i, m in enumerate(shape):
        if i in [d % x.dim() for d in dims]:
            split += [-(-m // BLOCK), BLOCK]
            block_dims.append(len(split) - 1)
            pads.append(-m % BLOCK)
        else:
            split.append(m)
            pads.append(0)
    p = torch.zeros([m + q for m, q in zip(shape, pads)], dtype=torch.float64, device=x.device)
    p[tuple(slice(0, m) for m in shape)] = x
    p = p.view(split)
    amax = p.abs().amax(block_dims, keepdim=True)
    e = torch.ceil(torch.log2(amax / 448.0))
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, e)
    scale = torch.exp2(torch.clamp(e, min=-126.0))
    v = p / scale
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs())), min=-6.0) - 3)
    q = torch.round(v / step) * step * scale
    return q.reshape([m + t for m, t in zip(shape, pads)])[tuple(slice(0, m) for m in shape)]


def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    s = prepare(case, seed)
    n, k, e = case["tokens"], case["slots"], case["experts"]
    dev = s["x"].device
    if e:  # (expert, slot number) pairs in order; those left out keep their order behind the others
        ids = s["ids"].cpu().numpy().reshape(-1)
        group = np.where((ids < 0) | (ids >= e), e, ids)
        order = np.lexsort((np.arange(ids.size), group))
        counts = np.array([(group == i).sum() for i in range(e)])
        kept = int(counts.sum())
    if case["op"] == "sort":
        at = np.empty(ids.size, np.int64)
        at[order] = np.arange(ids.size)
        rows = np.where(group < e, at, -1 - at).reshape(n, k)
        whole = {"offsets": np.concatenate([[0], np.cumsum(counts)]), "rows": rows, "source": np.where(np.arange(ids.size) < kept, order, -1 - order)}
        out = {name: torch.from_numpy(v.astype(np.int32)).to(dev) for name, v in whole.items()}
        token = torch.from_numpy(order[:kept] // k).to(dev)
        w = s["weights"].double().reshape(-1)[torch.from_numpy(order[:kept]).to(dev)][:, None]
        ys = s["ys"][:kept].double()
        out["xs"] = torch.zeros(n * k, case["d"], dtype=torch.float64, device=dev)
        out["xs"][:kept] = s["x"].double()[token]
        out["y"] = torch.zeros(n, case["d"], dtype=torch.float64, device=dev).index_add_(0, token, ys * w)
        if case["train"]:
            dy = s["dy"].double()[token]
            out["dys"] = torch.zeros_like(out["xs"])
            out["dys"][:kept] = dy * w
            dots = torch.zeros(n * k, dtype=torch.float64, device=dev)
            dots[torch.from_numpy(order[:kept]).to(dev)] = (dy * ys).sum(1)
            out["dweights"] = dots.view(n, k)
            out["dx"] = torch.zeros_like(out["y"]).index_add_(0, token, s["dxs"][:kept].double())
        return out
    if case["train"]:
        w = _exact_quantized(s["w"].double(), (-2, -1))
    else:
        values, scales = s["w8"]
        power = torch.exp2(scales.view(torch.uint8).double() - 127)
        grid = torch.kron(power.reshape(-1, scales.shape[-1]), torch.ones(BLOCK, BLOCK, dtype=torch.float64, device=dev))
        grid = grid.view(*values.shape[:-2], -1, scales.shape[-1] * BLOCK)
        w = (values.double() * grid[..., :case["out"], :values.shape[-1]])[..., :case["in"]].transpose(-1, -2)
    x = s["x"].double()
    if e:
        bounds = np.concatenate([[0], np.cumsum(counts)])
        parts = [(i, slice(int(bounds[i]), int(bounds[i + 1]))) for i in range(e)]
        xs = torch.zeros(n * k, case["in"], dtype=torch.float64, device=dev)
        xs[:kept] = x[torch.from_numpy(order[:kept] // k).to(dev)]
        x = xs
    else:
        parts, w = [(0, slice(0, n))], w[None]
    out = {"y": torch.zeros(x.shape[0], case["out"], dtype=torch.float64, device=dev)}
    if case["train"]:
        dy = s["dy"].double()
        out["dx"], out["dw"] = torch.zeros_like(x), torch.zeros(w.shape, dtype=torch.float64, device=dev)
    for i, part in parts:
        if part.stop == part.start:
            continue
        out["y"][part] = _exact_quantized(x[part], (1,)) @ w[i]
        if case["train"]:
            out["dx"][part] = _exact_quantized(dy[part], (1,)) @ w[i].t()
            out["dw"][i] = _exact_quantized(x[part], (0,)).t() @ _exact_quantized(dy[part], (0,))
    if case["train"]:
        out["dw"] = out["dw"].view(s["w"].shape)
    return out


# ---------------------------------------------------------------------- work
def work(case):
    """What a pass cannot do without: inputs read once, outputs written once, the products' operations."""
    size = 2 if case["dtype"] == "bf16" else 4
    n, k, e, train = case["tokens"], case["slots"], case["experts"], case["train"]
    rows = _rows(case)
    plan = 8 * n * k
    if case["op"] == "sort":
        d = case["d"]
        plan += 4 * (e + 1) + 8 * n * k + 4 * n * k  # offsets, rows, source, weights
        tokens, sorted_rows = (4, 4) if train else (2, 2)  # x, y, dy, dx; xs, ys, dys, dxs
        return {"bytes": plan + (4 * n * k if train else 0) + (tokens * n + sorted_rows * rows) * d * size, "flops": (6 if train else 2) * rows * d}
    i, o = case["in"], case["out"]
    matrices = max(1, min(e, rows)) * i * o  # at most a matrix a row is needed
    if not train:
        return {"bytes": plan + n * i * size + matrices + rows * o * size, "flops": 2 * rows * i * o}
    # w, x, dy; y, dx, dw
    return {"bytes": plan + (2 * max(1, e) * i * o + (n + rows) * i + 2 * rows * o) * size, "flops": 6 * rows * i * o}
