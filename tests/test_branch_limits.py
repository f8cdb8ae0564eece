"""CPU tests of what the operators for branching and long generation take of memory."""

import pytest

from paged_kv_gb300 import pkv


@pytest.mark.parametrize("n,heads,cols,ps", [(1, 1, 1, 1), (16, 8, 36864, 16), (4096, 8, 36864, 16),
                                             (4096, 8, 36863, 1), (3, 5, 1001, 7)])
def test_selection_takes_8_bytes_a_page_and_8_a_head(n, heads, cols, ps):
    need = pkv.load().pkv_select_pages_workspace_bytes(n, heads, cols, ps)
    pages = n * heads * -(-cols // ps)
    assert 8 * pages <= need <= 8 * pages + 8 * n * heads + 8 * n + 64
