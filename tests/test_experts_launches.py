"""Which kernels the calls of the GPU tests launch, without a GPU (tests/launch_recorder.cpp): the cases that are there for a kernel
launch it, and every kernel of the experts' path has a case."""
import ctypes
import os
import re
import subprocess

import pytest

from blocked_shampoo_preconditioning_amd import experts as X
from blocked_shampoo_preconditioning_amd import shampoo as S
from tests import test_gpu_experts_paths as paths
from tests import test_gpu_experts_product as products
from tests import test_gpu_experts_route as routes
from tests.test_experts_host import FAKE, PRODUCT, ROUTE, SORT, WEIGHT

TYPES = {"f32": S.SHAMPOO_F32, "bf16": S.SHAMPOO_BF16}


@pytest.fixture(scope="module")
def launched(tmp_path_factory):
    """launched(calls): the kernels' names of each (function, with a workspace, arguments)."""
    if not os.path.exists(S.LIB_PATH):
        from blocked_shampoo_preconditioning_amd import build
        build.build()
    exe = str(tmp_path_factory.mktemp("recorder") / "launch_recorder")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["g++", "-std=c++17", "-O1", "-rdynamic", os.path.join(here, "launch_recorder.cpp"), "-ldl", "-o", exe], check=True)

    def run(calls):
        text = "".join(f"{name} {int(workspace)} {args.hex()}\n" for name, workspace, args in calls)
        lines = subprocess.run([exe, S.LIB_PATH], input=text, text=True, capture_output=True, check=True).stdout.splitlines()
        assert len(lines) == len(calls)
        got = []
        for line in lines:
            status, *kernels = line.split(" | ")
            assert status == "0", line
            got.append([re.sub(r"( \d+){3}$", "", k) for k in kernels])
        return got
    return run


def product(rows, n_in, n_out, dtype, n_experts=0, slots=1, gather=False, **over):
    """The arguments of a product as the binding gives them."""
    args = {**PRODUCT, "rows": rows, "n_in": n_in, "n_out": n_out, "experts": max(1, n_experts), "dtype": TYPES[dtype], "offsets": FAKE if n_experts else 0,
            "source": FAKE if gather else 0, "x_rows": rows // slots, "slots": slots, "slot_rows": FAKE if n_experts else 0, "ld_x": n_in, "ld_y": n_out,
            "ld_dy": n_out, "ld_dx": n_in, "ld_dw": n_out, "stride_dw": n_in * n_out, **over}
    return X._PRODUCT.pack(*args.values())


def calls_of(rows, n_in, n_out, dtype, n_experts=0, slots=1, gather=False):
    """y alone, y saving x, dx alone, dx and dW of one shape."""
    shape = (rows, n_in, n_out, dtype, n_experts, slots)
    return [("shampoo_product8_forward", True, product(*shape, gather, saved=0)), ("shampoo_product8_forward", True, product(*shape, gather)),
            ("shampoo_product8_backward", True, product(*shape, dw=0)), ("shampoo_product8_backward", True, product(*shape))]


def rows_of(counts, left):
    return counts if isinstance(counts, int) else sum(counts.values()) + left


def parameters(test, first):
    return next(m.args[1] for m in test.pytestmark if m.name == "parametrize" and m.args[0].split(",")[0] == first)


@pytest.mark.parametrize("dtype,n_experts,counts,left,n_in,n_out,kernel,back_kernel", paths.FEW)
def test_few_rows(launched, dtype, n_experts, counts, left, n_in, n_out, kernel, back_kernel):
    rows = rows_of(counts, left)
    assert rows <= 64
    y, _, dx, _ = launched(calls_of(rows, n_in, n_out, dtype, n_experts))
    assert y == [kernel] and dx == [back_kernel]


@pytest.mark.parametrize("dtype,n_experts,counts,left,n_in,n_out,kernel,back_kernel", paths.MORE)
def test_more_rows(launched, dtype, n_experts, counts, left, n_in, n_out, kernel, back_kernel):
    rows = rows_of(counts, left)
    slots = 2 if rows % 2 == 0 and n_experts else 1
    y, kept, _, back = launched(calls_of(rows, n_in, n_out, dtype, n_experts, slots, n_experts > 0))
    assert y[-1] == kept[-1] == kernel and back[-1] == back_kernel


@pytest.mark.parametrize("tokens,slots", paths.SCATTER)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_slots(launched, tokens, slots, dtype):
    y, kept, _, _ = launched(calls_of(tokens * slots, 200, 136, dtype, 20, slots, True))
    assert y[0].startswith("scatter_kernel" if slots <= 16 else "quantize_kernel") and kept[0].startswith("quantize_kernel")


def test_some_expert_is_in_front_of_dx():
    """UNEVEN has experts whose sums of dW are longer than a row's of dx (out / 128 blocks), and such whose are not."""
    for out in (390, 512, 999, 1200):
        longer = [rows for rows in paths.UNEVEN.values() if -(-rows // 128) > -(-out // 128)]
        assert len(longer) < len(paths.UNEVEN) and longer


def test_every_kernel_has_a_case(launched):
    calls = [("shampoo_quantize_weight", False, X._WEIGHT.pack(*{**WEIGHT, "dtype": t}.values())) for t in TYPES.values()]
    for tokens, slots, n_experts, *_ in parameters(routes.test_sort, "tokens") + paths.SORT:
        calls.append(("shampoo_sort_tokens", True, X._SORT.pack(*{**SORT, "tokens": tokens, "slots": slots, "experts": n_experts, "ld_ids": slots}.values())))
    for tokens, slots, width, dtype, pad in parameters(routes.test_routes, "tokens") + paths.ROUTES:
        args = {**ROUTE, "tokens": tokens, "slots": slots, "width": width, "dtype": TYPES[dtype], "ld_x": width + pad, "ld_ys": width + pad, "ld_y": width, "ld_xs": width}
        calls += [(f"shampoo_{name}", False, X._ROUTE.pack(*args.values())) for name in ("dispatch", "combine", "combine_backward")]
    for dtype in TYPES:
        for rows, n_in, n_out, _ in parameters(products.test_dense, "rows"):
            calls += calls_of(rows, n_in, n_out, dtype)
    for rows, n_in, n_out in parameters(products.test_dense_large_tiles, "rows"):
        calls += calls_of(rows, n_in, n_out, "bf16")
    for dtype, n_experts, counts, left, n_in, n_out, *_ in paths.FEW + paths.MORE:
        calls += calls_of(rows_of(counts, left), n_in, n_out, dtype, n_experts)
    for tokens, slots in paths.SCATTER:
        for dtype in TYPES:
            calls += calls_of(tokens * slots, 200, 136, dtype, 20, slots, True)
    seen = {name for kernels in launched(calls) for name in kernels}
    listing = subprocess.run(["nm", "-C", S.LIB_PATH], capture_output=True, text=True, check=True).stdout
    kernels = set(re.findall(r"__device_stub__(.*)\(she::\w+Args\)|__device_stub__(.*)\(she::Products\)", listing))
    kernels = {re.sub(r"she::|\(anonymous namespace\)::", "", a or b) for a, b in kernels}
    assert len(kernels) >= 30
    assert kernels <= seen, sorted(kernels - seen)


def test_rows_that_need_no_workspace():
    """The binding asks for none up to _FEW_ROWS, the library from there on."""
    lib, size = X.load_library(), ctypes.c_size_t()
    for rows, some in ((X._FEW_ROWS, False), (X._FEW_ROWS + 1, True)):
        assert lib.shampoo_product8_workspace_size(product(rows, 200, 300, "bf16", saved=0), 0, ctypes.byref(size)) == 0
        assert (size.value > 0) == some
