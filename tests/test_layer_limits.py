"""Host-side limits of the layer operators' binding (no GPU)."""
import os

import pytest

from blocked_shampoo_preconditioning_amd import layer as L
from blocked_shampoo_preconditioning_amd import shampoo as S
from tests.test_layer_host import FAKE, NORM


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
