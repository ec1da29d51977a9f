"""Host-side limits of the layer operators and their binding (no GPU)."""
import ctypes
import os

import pytest

from blocked_shampoo_preconditioning_amd import layer as L
from blocked_shampoo_preconditioning_amd import shampoo as S
from tests.test_layer_host import DROP, FAKE, FFN, INVALID, NORM


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(S.LIB_PATH):
        from blocked_shampoo_preconditioning_amd import build
        build.build()
    return L.load_library()


def test_table_of_sizes_is_bounded():
    """A program whose calls never repeat a size: the table of byte counts does not grow with them, and every count is right."""
    L._sizes.clear()
    for n in range(1, 6000):
        fields = (n, 16, 32, 1, 0, FAKE, FAKE, FAKE, FAKE, 16, 32, 32, 16)
        assert L._saved_size(fields) >= 3 * n * 32 * 2
    assert 0 < len(L._sizes) <= 4096
    for n in range(1, 6000):
        args = {**NORM, "rows": n}
        head = tuple(args.values())[:11]
        size = L._norm_workspace(head, L._NORM.pack(*args.values()))
        assert size == L._size("shampoo_norm_workspace_size", L._NORM.pack(*args.values()))
    assert 0 < len(L._sizes) <= 4096
    L._sizes.clear()


LARGEST, LD = (1 << 31) - 1024, 1 << 21


@pytest.mark.parametrize("over,code", [(dict(tokens=LARGEST), 0), (dict(tokens=LARGEST + 1), INVALID), (dict(d_model=LD), 0),
                                       (dict(d_model=LD + 1), INVALID), (dict(d_hidden=LD), 0), (dict(d_hidden=LD + 1), INVALID)])
def test_largest_sizes_of_the_block(lib, over, code):
    """The last size that is taken and the first that is refused, as the header and the message state them."""
    out = ctypes.c_size_t()
    assert lib.shampoo_ffn_saved_size(L._FFN.pack(*{**FFN, **over}.values()), ctypes.byref(out)) == code
    header = open(L.LAYER_HEADER_PATH).read()
    assert "0 <= tokens <= 2^31 - 1024" in header and "in [1, 2^21]" in header
    if code:
        assert "[0, 2^31 - 1024]" in lib.shampoo_last_error().decode() and "[1, 2^21]" in lib.shampoo_last_error().decode()


def test_largest_sizes_of_dropout(lib):
    # no row: the largest width is checked and nothing runs
    assert lib.shampoo_dropout(L._DROP.pack(*{**DROP, "rows": 0, "cols": LARGEST}.values()), None) == 0
    assert lib.shampoo_dropout(L._DROP.pack(*{**DROP, "rows": 0, "cols": LARGEST + 1}.values()), None) == INVALID
    assert "[0, 2^31 - 1024]" in lib.shampoo_last_error().decode()
    assert "0 <= cols <= 2^31 - 1024" in open(L.LAYER_HEADER_PATH).read()
