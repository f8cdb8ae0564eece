"""pkv.compact_pages with so many moves that warps take whole pages, and with just too few:
every byte of every layer's pages, scales and bounds."""

import pytest
import torch

import branch_reference as ref
from test_gpu_fork import check_collect

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["heads", "slots", "rows"])
@pytest.mark.parametrize("heads,dim,ps", [(3, 80, 20), (8, 128, 4), (5, 32, 27)])
@pytest.mark.parametrize("more", [True, False])
def test_moves_past_the_number_of_warps(more, heads, dim, ps, layout):
    """300, 256 and 270 vectors a page: a piece and a bit, one piece, a piece and a bit."""
    warps = torch.cuda.get_device_properties(0).multi_processor_count * 6 * 8
    layers = 32
    moves = -(-warps // (2 * layers)) + (7 if more else -1)
    # One row whose pages all lie past as many free ones.
    held = 2 * moves
    rows, table = torch.tensor([1], dtype=torch.int32), torch.full((2, held * ps), -5, dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    pages = held + moves + 5
    low = torch.randperm(held, generator=g)[:moves]
    high = held + torch.randperm(pages - held, generator=g)[:moves]
    at = torch.cat([low, high])[torch.randperm(held, generator=g)]
    table[1] = (at[:, None] * ps + torch.arange(ps)).flatten().to(torch.int32)
    assert int((at >= held).sum()) == moves and ((moves * 2 * layers >= warps) == more)
    check_collect(rows, [held * ps - 3], ps, pages, table,
                  ref.caches(layers, pages, ps, heads, dim, layout, 4, bounds=True))
