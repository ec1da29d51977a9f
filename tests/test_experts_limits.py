"""Host-side limits of the experts' path (no GPU): which layouts of several matrices are taken."""
import os

import pytest

from blocked_shampoo_preconditioning_amd import experts as X
from blocked_shampoo_preconditioning_amd import shampoo as S
from tests.test_experts_host import FAKE, INVALID, MISALIGNED, PRODUCT, WEIGHT


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(S.LIB_PATH):
        from blocked_shampoo_preconditioning_amd import build
        build.build()
    return X.load_library()


@pytest.mark.parametrize("ld,stride,taken", [
    (300, 60000, True), (300, 59999, False), (320, 199 * 320 + 300, True), (300, 1 << 40, True), (300, (1 << 40) + 1, False),
    # side by side: two matrices' rows of 300 in one of ld elements
    (600, 300, True), (700, 300, True), (700, 400, True), (700, 401, False), (600, 299, False), (599, 300, False), (600, 0, False), (600, -300, False)])
def test_matrices_of_experts(lib, ld, stride, taken):
    """Two matrices of 200 x 300 that share no element are read and written where they lie. A call that takes them is refused for its
    workspace or the alignment of its results, before any GPU work."""
    code = lib.shampoo_quantize_weight(X._WEIGHT.pack(*{**WEIGHT, "ld_w": ld, "stride_w": stride, "values": FAKE + 8}.values()), None)
    assert code == (MISALIGNED if taken else INVALID)
    code = lib.shampoo_product8_backward(X._PRODUCT.pack(*{**PRODUCT, "ld_dw": ld, "stride_dw": stride}.values()), FAKE + 16, 1 << 30, None)
    assert code == (MISALIGNED if taken else INVALID)
    assert ("overlap" in lib.shampoo_last_error().decode()) != taken
