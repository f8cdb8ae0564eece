"""pkv.select_pages' choice among many pages: more equal or nearly equal scores than are ranked
at once, more pages than are held in shared memory, few and many (token, head)s, sums that are
taken again."""

import pytest
import torch

import branch_reference as ref
import serving_reference as sref
from paged_kv_gb300 import pkv
from test_gpu_sparse import check_select, cpu_bounds, f8, on_gpu
from test_gpu_append import make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"
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


# (new tokens, cache heads): a CTA of 1024 threads a (token, head), and of 256 where there
# are more of them than SMs.
CELLS = [(1, 2), (170, 1)]


def problem(count, ps, new, hkv, dim, seed):
    p = sref.page_problem([count * ps - 1], [new], ps, hkv, dim, seed)
    p["k_scale"] = torch.exp2(torch.randint(-6, -3, p["k_scale"].shape,
                                            generator=torch.Generator().manual_seed(seed)).float())
    return p


def run(p, q, bounds, budget, sink=1, recent=1):
    check_select(p, q, bounds, budget, sink, recent,
                 want=vector_select(p, q, bounds, budget, sink, recent))


@pytest.mark.parametrize("dt", [BF16, FP16], ids=str)
@pytest.mark.parametrize("new,hkv", CELLS)
@pytest.mark.parametrize("count", [300, 700, 4090, 4300, 6000])
def test_distinct_scores(count, new, hkv, dt):
    p = problem(count, 1, new, hkv, 32, 50)
    q = exact_queries(new, 2 * hkv, 32, dt, 51)
    b = cpu_bounds(p)
    for budget in (3, 60, 299, min(count - 5, 4097)):
        run(p, q, b, budget)


@pytest.mark.parametrize("new,hkv", CELLS)
@pytest.mark.parametrize("count", [300, 1500, 4098, 5001])
def test_equal_scores_on_more_pages_than_are_ranked_at_once(count, new, hkv):
    p = problem(count, 2, new, hkv, 32, 52)
    p["k_scale"].fill_(0.25)
    q = exact_queries(new, 4 * hkv, 32, BF16, 53)
    b = cpu_bounds(p)
    same = b[:1].expand_as(b).contiguous()
    some = b.clone()
    some[::3] = b[0]
    for budget in (2, 40, 290):
        run(p, q, same, budget, 0, 1)
        run(p, q, same, budget, 1, 1)
        run(p, q, some, budget, 0, 2)
        run(p, torch.zeros_like(q), b, budget)


@pytest.mark.parametrize("new,hkv", CELLS)
@pytest.mark.parametrize("count", [600, 5001])
@pytest.mark.parametrize("scale", [0.25, 0.3])
def test_nearly_equal_scores_on_more_pages_than_are_ranked_at_once(count, new, hkv, scale):
    """Scores that differ far below their fp32 error: with a scale of a few bits the sums' lower
    halves are often zero, with another they are not."""
    p = problem(count, 1, new, hkv, 32, 54)
    p["k_scale"].fill_(scale)
    q = exact_queries(new, 2 * hkv, 32, BF16, 55).abs() + 0.25
    q[..., 7] = 2.0 ** -24
    b = cpu_bounds(p)
    near = b[:1].expand_as(b).contiguous()
    g = torch.Generator().manual_seed(56)
    for codes in ((8, 10), (8, 60)):  # many ties, few
        near[:, :, 1, 7] = torch.randint(*codes, near[:, :, 1, 7].shape, generator=g).to(torch.uint8)
        near[:, :, 0, 7] = near[:, :, 1, 7]
        for budget in (2, 200, 500):
            run(p, q.to(BF16), near, budget)
    # Every other page is far above or below: sure ones beside those in doubt.
    mixed = near.clone()
    mixed[::5, :, :, :4] = 0x7E
    mixed[1::5, :, :, :4] = 0xFE
    for budget in (100, 500):
        run(p, q.to(BF16), mixed, budget)


@pytest.mark.parametrize("new,hkv", CELLS)
def test_nan_bounds_on_many_pages(new, hkv):
    p = problem(1200, 1, new, hkv, 32, 57)
    q = exact_queries(new, 2 * hkv, 32, FP16, 58)
    b = cpu_bounds(p)
    row = p["page_table"][int(p["table_idx"][0])].long()
    for logical in range(100, 800, 2):
        b[row[logical], :, :, 3] = 0x7F
    for budget in (20, 349, 600):  # fewer than those pages, and more
        pages, lengths = vector_select(p, q, torch.where((b & 127) == 127, 0, b), budget, 1, 1)
        nan = torch.arange(100, 800, 2)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = pkv.select_pages(q.to(DEV), make_cache(p), f8(b), *on_gpu(p), new, budget, status=st)
        assert int(st) == 0 and torch.equal(got[1].cpu(), lengths)
        have = got[0].cpu()
        for j in range(new):
            for h in range(hkv):
                taken = set(have[j, h].tolist())
                assert len(taken) == budget
                first = row[nan[:budget - 2]].tolist()  # the lowest come first
                assert taken.issuperset(first)
                assert len(taken & set(row[nan].tolist())) == min(budget - 2, len(nan))


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
