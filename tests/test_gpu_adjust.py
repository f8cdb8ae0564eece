"""pkv_adjust_logits on the GPU against the fp64 restatement: each rule and all
together, in place and out of place, odd sizes and strides, skipped entries."""

import math

import pytest
import torch

import serving_reference as ref
from paged_kv_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def problem(b, v, hist, nbias, seed, dt, rules="rpfbm"):
    g = torch.Generator().manual_seed(seed)
    p = {}
    length = torch.randint(0, hist + 1, (b,), generator=g)
    if b > 2:
        length[0], length[1] = 0, hist
    if any(x in rules for x in "rpf"):
        pool = (torch.rand(b + 3, hist, generator=g) ** 3 * v).to(torch.int32)
        pool[torch.rand(pool.shape, generator=g) < 0.02] = -1
        pool[torch.rand(pool.shape, generator=g) < 0.02] = v
        p.update(token_pool=pool, table_idx=torch.randperm(b + 3, generator=g)[:b].to(torch.int32),
                 prompt_len=(length * torch.rand(b, generator=g)).to(torch.int32),
                 device_len=length.to(torch.int32))
    if "r" in rules:
        p["repetition"] = 0.7 + torch.rand(b, generator=g)
    if "p" in rules:
        p["presence"] = torch.randn(b, generator=g)
    if "f" in rules:
        p["frequency"] = torch.randn(b, generator=g) * 0.3
    if "b" in rules:
        count = torch.randint(0, nbias + 1, (b,), generator=g)
        p["bias_ptr"] = torch.cat([torch.zeros(1, dtype=torch.long), count.cumsum(0)]).to(torch.int32)
        n = int(count.sum())
        p["bias_ids"] = torch.randint(0, min(v, 40), (n,), generator=g).to(torch.int32)  # repeats
        p["bias_values"] = torch.randn(n, generator=g) * 3
    if "m" in rules:
        m = torch.randint(-2 ** 31, 2 ** 31, (b, (v + 31) // 32), generator=g)
        m[torch.rand(m.shape, generator=g) < 0.3] = -1
        m[torch.rand(m.shape, generator=g) < 0.2] = 0
        if b > 1:
            m[b - 1] = 0  # a row whose grammar allows nothing
        p["mask"] = m.to(torch.int32)
    logits = (torch.randn(b, v, generator=g) * 4).to(dt)
    return logits, p


def check(got, logits, p):
    want, size = ref.adjust(logits, **p)
    got = got.cpu().double()
    hidden = want == -math.inf
    assert torch.equal(got == -math.inf, hidden)
    eps = 2.0 ** -8 if logits.dtype == torch.bfloat16 else 0.0
    # fp32: a few roundings of terms no larger than their sum of magnitudes (counts up to
    # thousands are exact in fp32, the rest of a term is one product).
    tol = eps * want.abs() + 2.0 ** -20 * size + 1e-30
    err = (got - want).abs()
    assert bool((err <= tol)[~hidden].all()), float((err / tol)[~hidden].max())


def dev(p):
    return {k: x.to(DEV) for k, x in p.items()}


SIZES = [(1, 1, 1, 1), (3, 31, 5, 3), (4, 32000, 30, 5), (2, 1025, 2000, 64), (5, 5003, 333, 300),
         (3, 151936, 2512, 64)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("rules", ["rpfbm", "r", "p", "f", "b", "m", "rpf"])
def test_matches_fp64(size, dt, rules):
    b, v, hist, nbias = size
    logits, p = problem(b, v, hist, nbias, 41, dt, rules)
    x = logits.to(DEV)
    out = pkv.adjust_logits(x, out=torch.full_like(x, 5.0), **dev(p))
    check(out, logits, p)
    assert torch.equal(x.cpu(), logits)
    # In place the same rules give the same bits.
    assert pkv.adjust_logits(x, **dev(p)) is x
    assert torch.equal(x.cpu(), out.cpu())


@pytest.mark.parametrize("inplace", [True, False])
def test_long_histories_use_wide_counts(inplace):
    logits, p = problem(3, 700, 40000, 8, 42, torch.float32)
    p["token_pool"][int(p["table_idx"][1])] = 17  # one token 40000 times
    p["prompt_len"][1] = 100
    x = logits.to(DEV)
    out = pkv.adjust_logits(x, out=None if inplace else torch.empty_like(x), **dev(p))
    check(out, logits, p)


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("spread", [20, 5000, 70000])
@pytest.mark.parametrize("many", [512, 513, 3000])
def test_long_bias_lists(many, spread, inplace):
    """More biases than a slice gathers, in one slice and over several, with repeats."""
    logits, p = problem(2, 70000, 50, 3, 45, torch.float32)
    g = torch.Generator().manual_seed(46)
    p["bias_ptr"] = torch.tensor([0, 2, 2 + many], dtype=torch.int32)
    p["bias_ids"] = torch.randint(0, spread, (2 + many,), generator=g).to(torch.int32)
    p["bias_values"] = torch.randn(2 + many, generator=g)
    x = logits.to(DEV)
    out = pkv.adjust_logits(x, out=None if inplace else torch.empty_like(x), **dev(p)).cpu().double()
    want, size = ref.adjust(logits, **p)
    hidden = want == -math.inf
    assert torch.equal(out == -math.inf, hidden)
    # A rounding for each addend of a token, and a few before them.
    most = int(torch.bincount(p["bias_ids"].long()).max())
    assert bool(((out - want).abs() <= (most + 8) * 2.0 ** -24 * size)[~hidden].all())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_strides_that_are_not_aligned(dt):
    logits, p = problem(4, 2050, 100, 20, 43, dt)
    wide = torch.full((4, 2061), 9.0, dtype=dt, device=DEV)
    x = wide[:, 3:2053]
    x.copy_(logits)
    keep = torch.full((4, 2057), 8.0, dtype=dt, device=DEV)
    mask = torch.zeros(4, 70, dtype=torch.int32, device=DEV)
    q = dev(p)
    mask[:, :65] = q["mask"]
    q["mask"] = mask[:, :65]
    out = pkv.adjust_logits(x, out=keep[:, 1:2051], **q)
    check(out, logits, p)
    assert bool((keep[:, 0] == 8.0).all()) and bool((keep[:, 2051:] == 8.0).all())
    pkv.adjust_logits(x, **q)
    assert torch.equal(x, out)
    assert bool((wide[:, :3] == 9.0).all()) and bool((wide[:, 2053:] == 9.0).all())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("at", range(8))
@pytest.mark.parametrize("v", [1, 6, 37, 2049, 40003])
def test_rows_that_begin_anywhere(v, at, dt):
    """In and out at the same distance from a 16-byte boundary, and at another."""
    logits, p = problem(3, v, 60, 5, 47, dt)
    stride = v + 9
    src = torch.full((4 * stride,), 9.0, dtype=dt, device=DEV)
    x = src.as_strided((3, v), (stride, 1), at)
    x.copy_(logits)
    first = None
    for o in (at, at + 1):
        dst = torch.full((4 * stride,), 8.0, dtype=dt, device=DEV)
        out = pkv.adjust_logits(x, out=dst.as_strided((3, v), (stride, 1), o), **dev(p))
        check(out, logits, p)
        first = out.clone() if first is None else first
        assert torch.equal(out, first)
        touched = torch.zeros(4 * stride, dtype=torch.bool, device=DEV)
        touched.as_strided((3, v), (stride, 1), o).fill_(True)
        assert bool((dst[~touched] == 8.0).all())


@pytest.mark.parametrize("inplace", [True, False])
def test_values_that_are_not_finite(inplace):
    logits, p = problem(2, 300, 20, 4, 44, torch.float32)
    logits[0, :40] = float("nan")
    logits[0, 40:60] = float("inf")
    logits[1, 7], logits[1, 9] = -float("inf"), torch.finfo(torch.float32).min
    x = logits.to(DEV)
    got = pkv.adjust_logits(x, out=None if inplace else torch.empty_like(x), **dev(p)).cpu().double()
    want, _ = ref.adjust(logits, **p)
    assert torch.equal(got == -math.inf, want == -math.inf)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got == math.inf, want == math.inf)


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_what_no_rule_names_keeps_its_bits(dt, inplace):
    # NaNs of every payload and sign beside named tokens, in every place of a vector.
    v = 4096
    bits = torch.arange(v, dtype=torch.int32)
    if dt == torch.bfloat16:
        raw = (0x7F81 + bits % 126 + (bits % 2) * 0x8000).to(torch.int32).to(torch.int16)
    else:
        raw = (0x7F800001 + bits * 1021) | torch.where(bits % 2 == 1, -2 ** 31, 0).to(torch.int32)
    named = torch.arange(0, v, 3, dtype=torch.int32)
    logits = raw.view(dt)[None].clone()
    p = dict(token_pool=named[None].contiguous(), table_idx=torch.zeros(1, dtype=torch.int32),
             prompt_len=torch.tensor([700], dtype=torch.int32),
             device_len=torch.tensor([named.numel()], dtype=torch.int32),
             repetition=torch.tensor([1.5]), frequency=torch.tensor([0.5]),
             presence=torch.tensor([0.25]))
    x = logits.to(DEV)
    got = pkv.adjust_logits(x, out=None if inplace else torch.empty_like(x), **dev(p)).cpu()
    other = torch.ones(v, dtype=torch.bool)
    other[named.long()] = False
    assert torch.equal(got.view(raw.dtype)[0, other], raw[other])
    assert bool(torch.isnan(got).all())


def test_bad_rows_are_reported_and_skipped():
    logits, p = problem(4, 500, 40, 6, 45, torch.float32, "rpfb")
    good = dict(p)
    p = {k: x.clone() for k, x in p.items()}
    p["table_idx"][0] = 77
    p["device_len"][1] = 41
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = logits.to(DEV)
    out = pkv.adjust_logits(x, out=torch.empty_like(x), status=status, **dev(p))
    assert int(status.item()) == pkv.ST_ROW_OOB | pkv.ST_COL_OOB
    good["device_len"] = good["device_len"].clone()
    good["device_len"][:2] = 0
    check(out, logits, good)
    # A bias id outside the vocabulary, a list that does not ascend.
    q = {k: x.clone() for k, x in good.items()}
    q["bias_ptr"] = torch.tensor([0, 2, 1, 3, 3], dtype=torch.int32)
    q["bias_ids"] = torch.tensor([5, 500, 7], dtype=torch.int32)
    q["bias_values"] = torch.tensor([1.0, 2.0, 3.0])
    status.zero_()
    out = pkv.adjust_logits(x, out=torch.empty_like(x), status=status, **dev(q))
    assert int(status.item()) == pkv.ST_COL_OOB
    fair = dict(q, bias_ptr=torch.tensor([0, 1, 1, 3, 3], dtype=torch.int32),
                bias_ids=torch.tensor([5, 500, 7], dtype=torch.int32))
    fair["bias_ptr"][2] = 1
    check(out, logits, fair)


def test_equal_bits_each_time_another_stream_and_a_graph():
    logits, p = problem(6, 20000, 500, 50, 46, torch.bfloat16)
    x, q = logits.to(DEV), dev(p)
    first = pkv.adjust_logits(x, out=torch.empty_like(x), **q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(4):
            again = pkv.adjust_logits(x, out=torch.empty_like(x), **q)
    s.synchronize()
    assert torch.equal(first, again)
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.adjust_logits(x, out=out, **q)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
