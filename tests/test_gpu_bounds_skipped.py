"""pkv.update_bounds with long stretches of skipped tokens before, within and after a run."""

import pytest
import torch

import branch_reference as ref
import serving_reference as sref
from paged_kv_gb300 import pkv
from test_gpu_append import make_cache
from test_gpu_sparse import f8

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("gap", [1, 31, 32, 33, 1000, 70001])
@pytest.mark.parametrize("every", [1, 2, 5, 13])
def test_skipped_tokens_part_no_run(gap, every):
    """After every few of the tokens as many skipped ones: runs of a page go on behind them."""
    p = sref.page_problem([3, 0, 11], [30, 17, 60], 8, 2, 32, 22)
    loc, skipped = p["out_loc"], torch.full((gap,), -1, dtype=torch.int32)
    parts = [skipped]
    for x in loc.split(every if gap < 10000 else 40):
        parts += [x, skipped]
    bounds = torch.full((p["num_pages"], 2, 2, 32), 3, dtype=torch.uint8)
    got, st = f8(bounds), torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.update_bounds(make_cache(p), got, torch.cat(parts).to(DEV), status=st)
    k, last = p["k"].contiguous().view(torch.uint8), {}
    for x in loc.tolist():
        last[x // 8] = x % 8
    for page, slot in last.items():
        bounds[page] = ref.page_bounds(k[page], slot + 1)
    assert int(st) == pkv.ST_ROW_OOB and torch.equal(got.view(torch.uint8).cpu(), bounds)
