"""Host-side limits of the layer operators and their binding (no GPU)."""
import ctypes
import os

import pytest

from blocked_shampoo_preconditioning_amd import layer as L
from blocked_shampoo_preconditioning_amd import shampoo as S
from tests.test_layer_host import DROP, FAKE, FFN, INVALID, MISALIGNED, NORM, SMALL, UNSUPPORTED


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


# the norm alone that made a block's x
BEFORE = {**NORM, **dict(z=0, post_kind=0, post_weight=0, gate=0, r=0, dtype=1, dr=0, dn=0, dx=0, dz=0, d_post_weight=0, d_gate=0, d_next_weight=0)}


@pytest.mark.parametrize("over,norm,code", [
    ({}, {}, 0), (dict(activation=2), {}, 0), ({}, dict(z=FAKE), INVALID), ({}, dict(rows=5), INVALID), ({}, dict(width=8), INVALID),
    ({}, dict(dtype=0), INVALID), ({}, dict(next_kind=0, next_weight=0), INVALID), ({}, dict(stats=0), INVALID), ({}, dict(stats=FAKE + 8), MISALIGNED),
    ({}, dict(x=0), INVALID), ({}, dict(ld_x=15), INVALID), ({}, dict(next_kind=3), UNSUPPORTED), (dict(x=0), {}, INVALID),
    (dict(activation=3), {}, UNSUPPORTED)])
def test_refusals_of_the_block_behind_a_norm(lib, over, norm, code):
    out = ctypes.c_size_t()
    args = L._FFN.pack(*{**FFN, "activation": 2, **over}.values()), L._NORM.pack(*{**BEFORE, **norm}.values())
    assert lib.shampoo_ffn_normed_workspace_size(*args, ctypes.byref(out)) == code
    if code:
        assert lib.shampoo_last_error().decode()
        assert lib.shampoo_ffn_forward_normed(*args, FAKE, 1 << 30, None) == code


def test_workspace_of_the_block_behind_a_norm(lib):
    """The second term costs workspace with ReLU and bf16 alone; a NULL norm and a small workspace are refused."""
    def size(name, *args):
        out = ctypes.c_size_t()
        assert getattr(lib, name)(*args, ctypes.byref(out)) == 0
        return out.value
    for activation, dtype in ((2, 1), (0, 1), (2, 0)):
        ffn = L._FFN.pack(*{**FFN, "tokens": 100, "activation": activation, "dtype": dtype}.values())
        norm = L._NORM.pack(*{**BEFORE, "rows": 100, "dtype": dtype}.values())
        with_norm, without = size("shampoo_ffn_normed_workspace_size", ffn, norm), size("shampoo_ffn_workspace_size", ffn, 0)
        assert (with_norm > without) == (activation == 2 and dtype == 1)
    ffn, norm = L._FFN.pack(*{**FFN, "tokens": 100, "activation": 2}.values()), L._NORM.pack(*{**BEFORE, "rows": 100}.values())
    need = size("shampoo_ffn_normed_workspace_size", ffn, norm)
    assert lib.shampoo_ffn_normed_workspace_size(ffn, norm, None) == INVALID
    assert lib.shampoo_ffn_normed_workspace_size(ffn, None, ctypes.byref(ctypes.c_size_t())) == INVALID
    assert lib.shampoo_ffn_forward_normed(ffn, norm, None, need, None) == INVALID
    assert lib.shampoo_ffn_forward_normed(ffn, norm, FAKE + 8, need, None) == MISALIGNED
    assert lib.shampoo_ffn_forward_normed(ffn, norm, FAKE, need - 1, None) == SMALL
