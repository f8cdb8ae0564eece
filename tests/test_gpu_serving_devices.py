"""The serving operators' binding on tensors of another GPU than the cache's: refused."""

import pytest
import torch

import serving_reference as ref
from paged_kv_gb300 import pkv
from test_gpu_append import make_cache
from test_gpu_attention import DEV, queries

pytestmark = pytest.mark.gpu


def test_tensors_on_another_gpu_than_the_caches():
    p = ref.page_problem([20], [3], 16, 1, 64, 1)
    cache = make_cache(p)
    q = queries(3, 2, 64, torch.bfloat16, 2).to(DEV)
    k = queries(3, 1, 64, torch.bfloat16, 3).to(DEV)
    dev = {x: p[x].to(DEV) for x in ("cached_len", "device_len", "table_idx", "page_table",
                                     "positions", "out_loc")}
    out = torch.full_like(q, 5.0)
    before = cache.k.view(torch.uint8).clone()
    cache._index += 1  # as a cache on the next GPU has it
    # (With the stream given, nothing is asked of that GPU.)
    s = torch.cuda.current_stream()
    with pytest.raises(ValueError, match="cuda:"):
        pkv.paged_attention(q, cache, dev["cached_len"], dev["device_len"], dev["table_idx"],
                            dev["page_table"], 3, out=out, stream=s)
    with pytest.raises(ValueError, match="cuda:"):
        pkv.append_kv(cache, k, k, dev["positions"], dev["out_loc"], stream=s)
    torch.cuda.synchronize()
    assert bool((out == 5.0).all()) and torch.equal(cache.k.view(torch.uint8), before)
