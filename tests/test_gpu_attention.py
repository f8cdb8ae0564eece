"""pkv_paged_attention on the GPU against the fp64 restatement: single tokens,
draft tokens, prompt chunks, ragged lengths, head groups, page sizes, windows,
rows that see nothing, values in places that are not seen, errors, long caches."""

import math

import pytest
import torch

import serving_reference as ref
from paged_kv_gb300 import pkv
from test_gpu_append import dev_like, make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


def queries(n, heads, d, dt, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, d, generator=g) * gain).to(dt)


def call(p, cache, q, **kw):
    dev = lambda t: t.to(DEV)  # noqa: E731
    lse = torch.full((q.shape[0], q.shape[1]), 9.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = {k: dev(x) if isinstance(x, torch.Tensor) else x for k, x in kw.items()}
    max_q_len = kw.pop("max_q_len", p["max_q_len"])
    out = pkv.paged_attention(dev(q), cache, dev(p["cached_len"]), dev(p["device_len"]),
                              dev(p["table_idx"]), dev(p["page_table"]), max_q_len, lse=lse,
                              status=status, **kw)
    torch.cuda.synchronize()
    return out.cpu().double(), lse.cpu().double(), int(status.item())


def check(p, q, got, lse, sm_scale=None, **kw):
    d = q.shape[2]
    want = ref.attend(p, q, d ** -0.5 if sm_scale is None else sm_scale, **kw)
    tol, lse_tol = ref.attend_tolerance(want, q.dtype, d)
    err = (got - want["out"]).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    empty = want["lse"] == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    e = (lse - want["lse"]).abs()[~empty]
    assert bool((e <= lse_tol[~empty]).all()), float((e / lse_tol[~empty]).max())
    assert not got[empty].any()


CASES = [
    # cached, new, ps, hkv, group, d, dt, window
    ([0], [1], 1, 1, 1, 16, torch.bfloat16, 0),
    ([0, 1, 15, 16, 17, 63, 64, 65], [1] * 8, 16, 2, 2, 128, torch.bfloat16, 0),
    ([700, 33, 129, 0], [1, 1, 1, 1], 5, 1, 5, 80, torch.float16, 0),
    ([300, 21, 64], [1, 1, 1], 64, 2, 8, 64, torch.float16, 0),
    ([257, 90], [1, 1], 3, 1, 16, 96, torch.bfloat16, 0),
    ([90, 0], [1, 1], 7, 1, 20, 32, torch.bfloat16, 0),
    ([40, 0, 200, 77], [4, 3, 1, 0], 16, 2, 2, 128, torch.float16, 0),
    ([40, 0, 200], [5, 3, 1], 1, 3, 1, 64, torch.float16, 33),
    ([500, 10], [2, 1], 100, 1, 3, 112, torch.bfloat16, 1),
    ([100, 0, 3], [61, 130, 1], 16, 2, 2, 128, torch.bfloat16, 0),
    ([0, 70], [129, 200], 32, 1, 4, 64, torch.float16, 0),
    ([5, 150], [140, 33], 3, 1, 3, 96, torch.bfloat16, 50),
    ([64, 0], [128, 257], 16, 1, 1, 128, torch.float16, 0),
    ([11], [300], 20, 1, 16, 80, torch.bfloat16, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"q{max(c[1])}ps{c[2]}g{c[4]}d{c[5]}w{c[7]}")
@pytest.mark.parametrize("head_major", [True, False])
def test_matches_fp64(case, head_major):
    cached, new, ps, hkv, group, d, dt, window = case
    p = ref.page_problem(cached, new, ps, hkv, d, 21, head_major=head_major)
    q = queries(sum(new), hkv * group, d, dt, 4)
    out, lse, status = call(p, make_cache(p), q, window=window)
    assert status == 0
    check(p, q, out, lse, window=window)


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    g = torch.Generator().manual_seed(seed)
    pick = lambda xs: xs[int(torch.randint(0, len(xs), (1,), generator=g))]  # noqa: E731
    b = pick([1, 2, 5, 9])
    most = pick([1, 1, 6, 40, 150])
    cached = torch.randint(0, pick([3, 100, 900]), (b,), generator=g).tolist()
    new = torch.randint(0, most + 1, (b,), generator=g).tolist()
    new[0] = most
    hkv, group, d = pick([1, 2, 3]), pick([1, 2, 3, 8]), pick([16, 48, 64, 80, 128])
    window = pick([0, 0, 1, 17, 100])
    dt = pick([torch.bfloat16, torch.float16])
    p = ref.page_problem(cached, new, pick([1, 2, 16, 24, 64]), hkv, d, seed + 50)
    q = queries(sum(new), hkv * group, d, dt, seed, gain=2.0)
    out, lse, status = call(p, make_cache(p), q, window=window, sm_scale=0.2)
    assert status == 0
    check(p, q, out, lse, sm_scale=0.2, window=window)


def test_many_requests_share_ctas_and_long_ones_are_split():
    g = torch.Generator().manual_seed(3)
    cached = torch.randint(0, 60, (500,), generator=g).tolist()
    cached[77], cached[499] = 3000, 1500
    p = ref.page_problem(cached, [1] * 500, 16, 1, 32, 22)
    q = queries(500, 2, 32, torch.bfloat16, 5)
    out, lse, status = call(p, make_cache(p), q)
    assert status == 0
    check(p, q, out, lse)


@pytest.mark.parametrize("new", [1, 3, 140])
def test_one_long_request_and_equal_bits(new):
    p = ref.page_problem([20000], [new], 64, 1, 64, 23)
    q = queries(new, 1, 64, torch.float16, 6)
    cache = make_cache(p)
    out, lse, status = call(p, cache, q)
    assert status == 0
    rows = sorted({0, new // 2, new - 1})
    small = dict(p, cached_len=p["cached_len"] + rows[0])
    for r in rows:
        one = dict(small, cached_len=p["cached_len"] + r, device_len=p["cached_len"] + r + 1)
        check(one, q[r:r + 1], out[r:r + 1], lse[r:r + 1])
    for _ in range(3):
        again, lse2, _ = call(p, cache, q)
        assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("new", [[1, 1, 1], [4, 2, 3], [150, 3, 140]])
def test_rows_that_see_nothing(new):
    p = ref.page_problem([50, 20, 0], new, 16, 2, 64, 24)
    q = queries(sum(new), 4, 64, torch.bfloat16, 7)
    begin = torch.tensor([10, 22, 100000], dtype=torch.int32)
    out, lse, status = call(p, make_cache(p), q, kv_begin=begin, window=0)
    assert status == 0
    check(p, q, out, lse, kv_begin=begin)
    out, lse, status = call(p, make_cache(p), q, kv_begin=begin, window=9)
    check(p, q, out, lse, kv_begin=begin, window=9)


@pytest.mark.parametrize("value", [0x7F, 0xFF, 0x7E])
@pytest.mark.parametrize("new", [[1, 1], [3, 2], [140, 33]])
def test_places_that_are_not_seen_do_not_reach_a_row(value, new):
    # Everything outside the seen places becomes a NaN (or the largest code), scales too.
    cached, ps, window = [40, 21], 8, 11
    p = ref.page_problem(cached, new, ps, 2, 64, 25, extra_cols=16)
    q = queries(sum(new), 4, 64, torch.float16, 8)
    want, want_lse, _ = call(p, make_cache(p), q, window=window)
    seen = torch.zeros(p["num_pages"], ps, dtype=torch.bool)
    for i, (c, m) in enumerate(zip(cached, new)):
        loc = p["page_table"][int(p["table_idx"][i]), max(0, c - window + 1):c + m].long()
        seen[loc // ps, loc % ps] = True
    dirty = dict(p)
    for name in "kv":
        bits = p[name].view(torch.uint8).clone()
        bits[~seen] = value
        dirty[name] = bits.view(torch.float8_e4m3fn)
        scale = p[name + "_scale"].clone()
        scale[~seen.any(1)] = float("nan")
        dirty[name + "_scale"] = scale
    out, lse, status = call(dirty, make_cache(dirty), q, window=window)
    assert status == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("new", [4, 140])
@pytest.mark.parametrize("which", ["k", "v"])
def test_a_nan_reaches_exactly_the_rows_that_see_it(which, new):
    p = ref.page_problem([30], [new], 16, 1, 64, 26)
    q = queries(new, 2, 64, torch.bfloat16, 9)
    clean, clean_lse, _ = call(p, make_cache(p), q)
    at = 30 + new // 2  # a later query's own position
    loc = int(p["page_table"][int(p["table_idx"][0]), at])
    bits = p[which].view(torch.uint8).clone()
    bits[loc // 16, loc % 16, 0, 5] = 0x7F
    bad = dict(p, **{which: bits.view(torch.float8_e4m3fn)})
    out, lse, _ = call(bad, make_cache(bad), q)
    before = slice(0, new // 2)
    after = slice(new // 2, None)
    assert torch.equal(out[before], clean[before]) and torch.equal(lse[before], clean_lse[before])
    if which == "k":
        assert bool(torch.isnan(out[after]).all()) and bool(torch.isnan(lse[after]).all())
    else:
        assert bool(torch.isnan(out[after][..., 5]).all())
        rest = [i for i in range(64) if i != 5]
        assert torch.equal(out[after][..., rest], clean[after][..., rest])
        assert torch.equal(lse, clean_lse)


def test_scales_far_apart():
    p = ref.page_problem([200, 70], [1, 2], 8, 1, 64, 27)
    g = torch.Generator().manual_seed(1)
    p["v_scale"] = torch.exp2(torch.randint(-60, 61, p["v_scale"].shape, generator=g).float())
    q = queries(3, 2, 64, torch.bfloat16, 10)
    out, lse, status = call(p, make_cache(p), q)
    assert status == 0
    check(p, q, out, lse)


@pytest.mark.parametrize("new", [1, 130])
def test_scores_far_apart(new):
    p = ref.page_problem([150], [new], 16, 1, 64, 28)
    q = queries(new, 1, 64, torch.float16, 11, gain=60.0)
    out, lse, status = call(p, make_cache(p), q)
    assert status == 0
    check(p, q, out, lse)


def test_strided_queries_and_outputs_and_a_scale_that_is_no_power_of_two():
    p = ref.page_problem([60, 5], [1, 6], 16, 2, 64, 29)
    p["k_scale"], p["v_scale"] = p["k_scale"] * 1.37, p["v_scale"] * 0.81
    q = queries(7, 8, 64, torch.bfloat16, 12)
    wide = torch.zeros(7, 20, 64, dtype=torch.bfloat16, device=DEV)
    view = wide[:, 2:18:2]
    view.copy_(q)
    keep = torch.full((7, 11, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    cache = make_cache(p)
    dev = [p[x].to(DEV) for x in ("cached_len", "device_len", "table_idx", "page_table")]
    out = pkv.paged_attention(view, cache, *dev, 6, out=keep[:, 1:9])
    assert out.data_ptr() == keep[:, 1:9].data_ptr()
    want = ref.attend(p, q, 64 ** -0.5)
    tol, _ = ref.attend_tolerance(want, q.dtype, 64)
    assert bool(((keep[:, 1:9].cpu().double() - want["out"]).abs() <= tol).all())
    assert bool((keep[:, 0] == 3.0).all()) and bool((keep[:, 9:] == 3.0).all())


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [130, 2, 131, 140]])
def test_bad_requests_get_zeros_and_status_bits(new):
    p = ref.page_problem([20, 9, 30, 4], new, 16, 1, 64, 30)
    n = sum(new)
    q = queries(n, 2, 64, torch.float16, 13)
    cache = make_cache(p)
    good, good_lse, _ = call(p, cache, q)
    span = [slice(sum(new[:i]), sum(new[:i + 1])) for i in range(4)]
    for what, bit in (("table", pkv.ST_ROW_OOB), ("cached", pkv.ST_COL_OOB)):
        bad = dict(p)
        if what == "table":
            bad["table_idx"] = p["table_idx"].clone()
            bad["table_idx"][1] = 999
        else:
            shift = p["page_table"].shape[1]
            for name in ("cached_len", "device_len"):
                bad[name] = p[name].clone()
                bad[name][1] += shift
        out, lse, status = call(bad, cache, q)
        assert status == bit
        for i in (0, 2, 3):
            assert torch.equal(out[span[i]], good[span[i]])
            assert torch.equal(lse[span[i]], good_lse[span[i]])
        assert not out[span[1]].any() and bool((lse[span[1]] == -math.inf).all())


def test_more_query_tokens_than_the_bound():
    p = ref.page_problem([20, 9], [1, 5], 16, 1, 64, 31)
    q = queries(6, 2, 64, torch.float16, 14)
    good, _, _ = call(p, make_cache(p), q)
    out, lse, status = call(p, make_cache(p), q, max_q_len=2)
    assert status == pkv.ST_TOKEN_CAP
    assert torch.equal(out[0], good[0]) and not out[1:].any()
    # The lengths ask for more packed rows than there are.
    out, lse, status = call(p, make_cache(p), q[:4], max_q_len=5)
    assert status & pkv.ST_TOKEN_CAP and torch.equal(out[0], good[0])


def test_a_location_outside_the_cache_reads_as_zeros():
    p = ref.page_problem([20], [1], 16, 1, 64, 32)
    q = queries(1, 2, 64, torch.float16, 15)
    row = int(p["table_idx"][0])
    loc = int(p["page_table"][row, 5])
    bad = dict(p, page_table=p["page_table"].clone())
    bad["page_table"][row, 5] = 1 << 30
    out, lse, status = call(bad, make_cache(p), q)
    assert status == pkv.ST_ROW_OOB
    zero = dict(p)
    for name in "kv":
        x = p[name].float().clone()
        x[loc // 16, loc % 16] = 0.0
        zero[name] = x.to(torch.float8_e4m3fn)
    check(zero, q, out, lse)


def test_cache_past_four_gigabytes():
    ps, hkv, d = 64, 8, 128
    pages = (5 << 30) // (ps * hkv * d)
    p = ref.page_problem([130], [1], ps, hkv, d, 33)
    cache = pkv.KVCache.empty(pages, ps, hkv, d)
    shift = pages - p["num_pages"]
    for name in "kv":
        getattr(cache, name)[shift:] = dev_like(p[name])
        getattr(cache, name + "_scale")[shift:] = p[name + "_scale"].to(DEV)
    q = queries(1, 8, d, torch.bfloat16, 16)
    moved = dict(p, page_table=p["page_table"] + shift * ps)
    out, lse, status = call(moved, cache, q)
    assert status == 0
    check(p, q, out, lse)


@pytest.mark.parametrize("new", [1, 150])
def test_two_streams_with_their_own_workspaces_and_a_graph(new):
    p = ref.page_problem([900, 40], [new, 1], 16, 2, 128, 34)
    q = queries(new + 1, 4, 128, torch.bfloat16, 17)
    cache = make_cache(p)
    want, _, _ = call(p, cache, q)
    dev = [p[x].to(DEV) for x in ("cached_len", "device_len", "table_idx", "page_table")]
    qd = q.to(DEV)
    need = pkv.paged_attention_workspace_bytes(2, new + 1, new, 4, 2, 128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, works = [], [torch.zeros(need, dtype=torch.uint8, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, w in zip(streams, works):
            with torch.cuda.stream(s):
                outs.append(pkv.paged_attention(qd, cache, *dev, new, workspace=w))
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu().double(), want) for o in outs)
    out = torch.empty_like(qd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_attention(qd, cache, *dev, new, out=out, workspace=works[0])
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu().double(), want)


def test_calls_of_different_shapes_share_a_workspace():
    # Each leaves the workspace ready for the next, whatever its shape.
    problems = []
    for i, (cached, new, hkv, group, d) in enumerate([
            ([9000], [1], 1, 16, 128), ([5000], [300], 1, 1, 64), ([4000, 9], [2, 5], 1, 4, 64),
            ([3000], [200], 2, 1, 128), ([7000], [1], 1, 1, 64)]):
        p = ref.page_problem(cached, new, 16, hkv, d, 60 + i)
        q = queries(sum(new), hkv * group, d, torch.bfloat16, i)
        problems.append((p, make_cache(p), q))
    size = max(pkv.paged_attention_workspace_bytes(len(p["cached_len"]), q.shape[0], p["max_q_len"],
                                                   q.shape[1], c.kv_heads, q.shape[2])
               for p, c, q in problems)
    fresh = [call(p, c, q, workspace=torch.zeros(size, dtype=torch.uint8))[0] for p, c, q in problems]
    shared = torch.zeros(size, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for (p, c, q), want in zip(problems, fresh):
            assert torch.equal(call(p, c, q, workspace=shared)[0], want)


@pytest.mark.parametrize("new,long", [(40, 700), (1, 60), ((1, 40), 150)], ids=str)
def test_short_blocks_beside_a_long_one(new, long):
    # The ranges of equal cost end within and at blocks' starts; both kernels in one call.
    b = 36
    new = [new] * b if isinstance(new, int) else [new[i % 2] for i in range(b)]
    cached = [(7 * i) % 5 for i in range(b)]
    new[b // 2] = long
    cached[b - 1] = 3000
    p = ref.page_problem(cached, new, 16, 2, 64, 71)
    q = queries(sum(new), 2, 64, torch.bfloat16, 72)
    cache = make_cache(p)
    got, lse, status = call(p, cache, q)
    assert status == 0
    check(p, q, got, lse)
    for _ in range(3):
        again, lse2, _ = call(p, cache, q)
        assert torch.equal(again, got) and torch.equal(lse2, lse)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("new", [1, 3, 130])
@pytest.mark.parametrize("rising", [True, False])
def test_scores_that_rise_or_fall_along_the_keys(dt, new, rising):
    # Keys grow (or shrink) from page to page, so that a reference taken from the first
    # ones is far from the last ones, by more than the largest power of two of fp32.
    p = ref.page_problem([400], [new], 16, 1, 64, 70)
    q = queries(new, 1, 64, dt, 18, gain=3.0)
    pages = (p["page_table"][int(p["table_idx"][0]), ::16] // 16).long()
    e = torch.linspace(-8.0, 2.0, len(pages)).round()
    p["k_scale"][pages, 0] = torch.exp2(e if rising else e.flip(0))
    p["v_scale"][pages, 0] = torch.exp2((-e if rising else e) * 3.0)
    out, lse, status = call(p, make_cache(p), q)
    assert status == 0
    check(p, q, out, lse)
