"""pkv.select_pages' choice where its sums are taken again."""

import pytest
import torch

import branch_reference as ref
import serving_reference as sref
from test_gpu_sparse import check_select, cpu_bounds

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def exact_queries(n, heads, dim, dt, seed):
    """Queries of a few bits (multiples of 1/64 below 2): their products with codes, and the sums
    of those, are exact in fp64."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(-127, 128, (n, heads, dim), generator=g) / 64).to(dt)


def vector_select(p, q, bounds, budget, sink, recent):
    """The definition for one request, all pages of a token at once."""
    ps, hkv = p["k"].shape[1], p["k"].shape[2]
    n, hq, _ = q.shape
    group = hq // hkv
    row = p["page_table"][int(p["table_idx"][0])]
    first = int(p["cached_len"][0])
    pages = torch.full((n, hkv, budget), -1, dtype=torch.int32)
    lengths = torch.zeros(n, dtype=torch.int32)
    value = ref.value(bounds)
    for j in range(n):
        pos = first + j
        mine = row[:pos + 1:ps].long() // ps
        m = len(mine)
        lengths[j] = (min(m, budget) - 1) * ps + pos % ps + 1
        for h in range(hkv):
            keep = torch.arange(m)
            if m > budget:
                x = q[j, h * group:(h + 1) * group].double()
                lo, hi = value[mine, h, 0], value[mine, h, 1]
                s = torch.maximum(x[:, None] * lo, x[:, None] * hi).sum(-1).amax(0)
                s = s * p["k_scale"][mine, h].double()
                order = torch.sort(s[sink:m - recent], descending=True, stable=True).indices + sink
                keep = torch.cat([torch.arange(sink), order[:budget - sink - recent],
                                  torch.arange(m - recent, m)]).sort().values
            pages[j, h, :len(keep)] = mine[keep].to(torch.int32)
    return pages, lengths


def problem(count, ps, new, hkv, dim, seed):
    p = sref.page_problem([count * ps - 1], [new], ps, hkv, dim, seed)
    p["k_scale"] = torch.exp2(torch.randint(-6, -3, p["k_scale"].shape,
                                            generator=torch.Generator().manual_seed(seed)).float())
    return p


def run(p, q, bounds, budget, sink=1, recent=1):
    check_select(p, q, bounds, budget, sink, recent,
                 want=vector_select(p, q, bounds, budget, sink, recent))


@pytest.mark.parametrize("size", [2.0 ** 126, 2.0 ** 120, 2.0 ** -126, 2.0 ** -132])
def test_queries_at_the_ends_of_bf16(size):
    """Finite queries whose products with codes leave fp32's range, and pages whose scores are
    so near one another that their sums are taken again."""
    p = problem(400, 4, 1, 2, 32, 59)
    p["k_scale"].fill_(0.25)
    q = exact_queries(1, 4, 32, FP16, 60).float()
    q = (torch.sign(q) * torch.exp2(torch.round(torch.log2(q.abs() + 2.0 ** -6)))).clamp(-1.9, 1.9)
    b = cpu_bounds(p)
    for some in (b, b[:1].expand_as(b).contiguous()):
        b2 = some.clone()
        g = torch.Generator().manual_seed(61)
        b2[:, :, 1, 5] = torch.randint(8, 40, b2[:, :, 1, 5].shape, generator=g).to(torch.uint8)
        b2[:, :, 0, 5] = b2[:, :, 1, 5]
        # (A power of two less: the other queries keep their bits at both ends.)
        x = q.clone()
        x[..., 5] = 2.0 ** -6
        scaled = (x.double() * size).to(torch.float32).to(BF16)
        for budget in (9, 100):
            want = vector_select(p, scaled, b2, budget, 1, 1)
            check_select(p, scaled, b2, budget, want=want)
