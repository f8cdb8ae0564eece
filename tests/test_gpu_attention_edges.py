"""pkv_paged_attention on the GPU at its edges: tables whose locations are no runs of a
page, references that move several times a unit, requests past their bound, queries
and scales at the ends of their ranges."""

import math

import pytest
import torch

import serving_reference as ref
from paged_kv_gb300 import pkv
from test_gpu_append import make_cache
from test_gpu_attention import DEV, call, queries

pytestmark = pytest.mark.gpu


def attend(p, q, sm_scale):
    """ref.attend's values for causal calls, a (request, head) at a time."""
    ps, hkv = p["k"].shape[1], p["k"].shape[2]
    n, hq, d = q.shape
    group = hq // hkv
    out = {x: torch.zeros(n, hq, d, dtype=torch.float64) for x in ("out", "mass", "tail")}
    out.update({x: torch.zeros(n, hq, dtype=torch.float64) for x in ("lse", "prod")})
    at = 0
    for i in range(len(p["cached_len"])):
        c, e = int(p["cached_len"][i]), int(p["device_len"][i])
        loc = p["page_table"][int(p["table_idx"][i]), :e].long()
        page, off = loc // ps, loc % ps
        rows = slice(at, at + e - c)
        at += e - c
        hide = torch.arange(e) > torch.arange(c, e)[:, None]
        for h in range(hkv):
            k, v = (p[x].float()[page, off, h].double()
                    * p[x + "_scale"][page, h].double()[:, None] for x in "kv")
            for g in range(h * group, (h + 1) * group):
                x = q[rows, g].double()
                s = (x @ k.T * sm_scale).masked_fill(hide, -math.inf)
                top = s.amax(1, keepdim=True)
                w = torch.exp(s - top)
                z = w.sum(1, keepdim=True)
                out["out"][rows, g] = (w @ v) / z
                out["lse"][rows, g] = (top + z.log())[:, 0]
                out["mass"][rows, g] = (w @ v.abs()) / z
                out["tail"][rows, g] = ((~hide).double() @ v.abs()) / z
                # (A sum over seen keys' channels bounds their largest product.)
                out["prod"][rows, g] = (x.abs() @ k.abs().T * abs(sm_scale)).masked_fill(
                    hide, 0.0).amax(1)
    return out


def check(want, q, got, lse):
    tol, lse_tol = ref.attend_tolerance(want, q.dtype, q.shape[2])
    err = (got - want["out"]).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    err = (lse - want["lse"]).abs()
    assert bool((err <= lse_tol).all()), float((err / lse_tol).max())


def set_channel(p, name, positions, channel, value):
    """Channel ``channel`` of the keys or values at the first request's positions."""
    loc = p["page_table"][int(p["table_idx"][0]), positions].long()
    ps = p[name].shape[1]
    x = p[name].float().clone()
    x[loc // ps, loc % ps, :, channel] = torch.as_tensor(value)[..., None]
    p[name] = x.to(torch.float8_e4m3fn)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("odd_units", [(0, 1, 2, 3), (0,), (1, 6, 11), (3, 4, 9, 15)], ids=str)
@pytest.mark.parametrize("bad", [False, True])
def test_tables_that_are_no_runs_in_some_units(dt, odd_units, bad):
    """Units of 128 positions whose groups of 16 mix pages (or begin with a location outside
    the cache) among units of whole pages: each unit takes its own way."""
    requests, cached, new, ps, hkv, d = 12, 2000, 150, 16, 8, 64
    p = ref.page_problem([cached], [new], ps, hkv, d, 81)
    g = torch.Generator().manual_seed(82)
    for name in "kv":  # neighbouring pages differ by much
        p[name + "_scale"] = torch.exp2(torch.randint(-9, -2, p[name + "_scale"].shape,
                                                      generator=g).float())
    row = int(p["table_idx"][0])
    used = set((p["page_table"][row] // ps).tolist())
    spare = next(x for x in range(p["num_pages"]) if x not in used)
    for name in "kv":
        x = p[name].float().clone()
        x[spare] = 0.0
        p[name] = x.to(torch.float8_e4m3fn)
    given = dict(p, page_table=p["page_table"].clone())
    p["page_table"] = p["page_table"].clone()
    for u in odd_units:
        span = slice(128 * u, 128 * u + 128)
        if bad:
            at = torch.arange(128 * u, 128 * u + 128, 16)
            given["page_table"][row, at] = 1 << 30
            p["page_table"][row, at] = spare * ps  # a zero key and value
        else:
            order = torch.randperm(128, generator=g)
            for t in (p, given):
                t["page_table"][row, span] = t["page_table"][row, span][order]
    q = queries(new, 2 * hkv, d, dt, 83)
    want = attend(p, q, d ** -0.5)
    many = dict(given)  # the same request again and again: every CTA has many units
    for name in ("cached_len", "device_len", "table_idx"):
        many[name] = given[name].repeat(requests)
    cache = make_cache(p)
    for _ in range(4):
        out, lse, status = call(many, cache, q.repeat(requests, 1, 1))
        assert status == (pkv.ST_ROW_OOB if bad else 0)
        for i in range(requests):
            check(want, q, out[i * new:(i + 1) * new], lse[i * new:(i + 1) * new])


@pytest.mark.parametrize("dt,small", [(torch.bfloat16, 2.0 ** -11), (torch.float16, 2.0 ** -7)],
                         ids=["bf16", "fp16"])
def test_small_query_elements_beside_a_large_one_in_prompt_chunks(dt, small):
    """The largest element of a query meets zeros; the scores are the small ones'."""
    p = ref.page_problem([200], [140], 16, 2, 64, 86)
    p["k_scale"][:] = 1.0
    set_channel(p, "k", torch.arange(340), 0, torch.zeros(340))
    g = torch.Generator().manual_seed(87)
    q = small * (1 + torch.rand(140, 4, 64, generator=g))
    q = (q * torch.where(torch.rand(q.shape, generator=g) < 0.5, -1.0, 1.0)).to(dt)
    q[..., 0] = 1.0
    sm_scale = 5 / (small * 384)
    want = attend(p, q, sm_scale)
    out, lse, status = call(p, make_cache(p), q, sm_scale=sm_scale)
    assert status == 0
    check(want, q, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("new", [5, 130, 300])
def test_references_that_move_in_every_quarter_of_a_unit(dt, new):
    """Scores rise by 32 (46 powers of two) every 32 positions: what a unit has summed, and
    the weights that it has stored, are scaled down several times before it ends."""
    p = ref.page_problem([448], [new], 16, 1, 64, 84)
    q = queries(new, 1, 64, dt, 85, gain=0.05)
    q[..., 0] = 8.0
    p["k_scale"][:] = 1.0
    step = (torch.arange(448 + new) // 32).clamp_max(14) * 32.0
    set_channel(p, "k", torch.arange(448 + new), 0, step)
    want = attend(p, q, 0.125)
    cache = make_cache(p)
    for _ in range(4):
        out, lse, status = call(p, cache, q, sm_scale=0.125)
        assert status == 0
        check(want, q, out, lse)


@pytest.mark.parametrize("group,new,most", [(16, [1, 3, 1, 40], 1), (2, [2, 100, 1], 2),
                                            (1, [33, 4, 4000], 4), (8, [2, 5], 4)], ids=str)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_requests_of_many_rows_past_the_bound_get_zeros(dt, group, new, most):
    """However many rows they have, and whichever kernels the bound asks for."""
    p = ref.page_problem([20 * i for i in range(len(new))], new, 16, 2, 64, 88)
    q = queries(sum(new), 2 * group, 64, dt, 89)
    cache = make_cache(p)
    out = torch.full(q.shape, 5.0, dtype=dt, device=DEV)
    got, lse, status = call(p, cache, q, max_q_len=most, out=out)
    assert status == pkv.ST_TOKEN_CAP
    want = attend(p, q, 64 ** -0.5)
    at = 0
    for n in new:
        rows = slice(at, at + n)
        at += n
        if n > most:
            assert not got[rows].any() and bool((lse[rows] == -math.inf).all())
        else:
            check({x: y[rows] for x, y in want.items()}, q[rows], got[rows], lse[rows])


@pytest.mark.parametrize("small", [2.0 ** -16, 2.0 ** -27], ids=["2^-16", "2^-27"])
def test_small_query_elements_beside_a_large_one_in_decoding(small):
    p = ref.page_problem([200, 31], [1, 3], 16, 2, 64, 90)
    p["k_scale"][:] = 1.0
    bits = p["k"].float().clone()
    bits[..., 0] = 0.0
    p["k"] = bits.to(torch.float8_e4m3fn)
    g = torch.Generator().manual_seed(91)
    q = small * (1 + torch.rand(4, 4, 64, generator=g))
    q = (q * torch.where(torch.rand(q.shape, generator=g) < 0.5, -1.0, 1.0)).to(torch.bfloat16)
    q[..., 0] = 1.0
    sm_scale = 5 / (small * 384)
    want = attend(p, q, sm_scale)
    out, lse, status = call(p, make_cache(p), q, sm_scale=sm_scale)
    assert status == 0
    check(want, q, out, lse)


@pytest.mark.parametrize("new", [1, 5])
@pytest.mark.parametrize("power", [-133, -126, -119, -100, 126, 127])
def test_queries_at_the_ends_of_bf16(new, power):
    """The largest magnitudes, the smallest and subnormal ones, under a scale that makes
    their scores ordinary ones."""
    p = ref.page_problem([150], [new], 16, 1, 64, 92)
    p["k_scale"][:] = 2.0 ** (-6 if power > 0 else 20)
    g = torch.Generator().manual_seed(93)
    q = torch.where(torch.rand(new, 2, 64, generator=g) < 0.5, -1.0, 1.0)
    q = (q * 2.0 ** max(power, -133)).to(torch.bfloat16)
    # Scores of some units: 48 * sqrt(64) * |q| * scales.
    sm_scale = 2.0 ** (-power - 8 + 6) if power > 0 else 2.0 ** min(-power - 8 - 20, 100)
    want = attend(p, q, sm_scale)
    out, lse, status = call(p, make_cache(p), q, sm_scale=sm_scale)
    assert status == 0
    check(want, q, out, lse)


@pytest.mark.parametrize("new", [1, 4, 130])
@pytest.mark.parametrize("power", [-64, -20, 100, 112, 119])
def test_value_scales_at_the_ends_of_their_range(new, power):
    """One position leads by e^8, and thousands of others hold as much together: none of
    their weights may be lost under any scale."""
    p = ref.page_problem([3000], [new], 16, 1, 64, 94)
    p["k_scale"][:] = 1.0
    p["v_scale"][:] = 2.0 ** power
    q = queries(new, 1, 64, torch.bfloat16, 95, gain=0.01)
    q[..., 0] = 1.0
    code = torch.zeros(3000 + new)
    code[0] = 64.0
    set_channel(p, "k", torch.arange(3000 + new), 0, code)
    want = attend(p, q, 0.125)
    out, lse, status = call(p, make_cache(p), q, sm_scale=0.125)
    assert status == 0
    check(want, q, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("new", [1, 4, 130])
@pytest.mark.parametrize("others", [-64, -6])
def test_scores_that_rise_after_values_of_nothing(dt, new, others):
    """The first page's values are zeros under the least scale (as pkv_append_kv leaves them);
    later scores are larger by 2^53 in weight."""
    p = ref.page_problem([3000], [new], 16, 1, 64, 96)
    p["k_scale"][:] = 1.0
    p["v_scale"][:] = 2.0 ** others
    q = queries(new, 1, 64, dt, 97, gain=0.01)
    q[..., 0] = 1.03125
    code = torch.full((3000 + new,), 288.0)
    code[:32] = 0.0
    set_channel(p, "k", torch.arange(3000 + new), 0, code)
    first = p["page_table"][int(p["table_idx"][0]), [0, 16]].long() // 16
    bits = p["v"].float().clone()
    bits[first] = 0.0
    p["v"] = bits.to(torch.float8_e4m3fn)
    p["v_scale"][first] = 2.0 ** -64
    want = attend(p, q, 0.125)
    out, lse, status = call(p, make_cache(p), q, sm_scale=0.125)
    assert status == 0
    check(want, q, out, lse)


def test_many_scores_that_rise_under_the_least_value_scale():
    """As above for long ranges: sums of weights that the least scale makes large."""
    requests, cached, new, hkv = 12, 3000, 130, 8
    p = ref.page_problem([cached], [new], 16, hkv, 64, 98)
    p["k_scale"][:] = 1.0
    p["v_scale"][:] = 2.0 ** -64
    q = queries(new, hkv, 64, torch.bfloat16, 99, gain=0.0005)
    q[..., 0] = 1.0546875
    code = torch.full((cached + new,), 288.0)  # 2^54.8 in weight
    code[:32] = 0.0
    set_channel(p, "k", torch.arange(cached + new), 0, code)
    want = attend(p, q, 0.125)
    many = dict(p)
    for name in ("cached_len", "device_len", "table_idx"):
        many[name] = p[name].repeat(requests)
    out, lse, status = call(many, make_cache(p), q.repeat(requests, 1, 1), sm_scale=0.125)
    assert status == 0
    for i in range(requests):
        check(want, q, out[i * new:(i + 1) * new], lse[i * new:(i + 1) * new])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("new", [1, 5, 140])
@pytest.mark.parametrize("sm_scale", [0.0, 2.0 ** -120, -(2.0 ** -60)])
@pytest.mark.parametrize("ps", [16, 5])
def test_no_scores_to_speak_of_and_keys_of_nothing(dt, new, sm_scale, ps):
    """Products that fall below fp32's range, under the least key scale: a plain average of
    what each row sees, and nothing of what it does not."""
    p = ref.page_problem([150, 0], [new, 2], ps, 1, 64, 100)
    p["k_scale"][::2] = 2.0 ** -64
    q = queries(new + 2, 2, 64, dt, 101)
    want = attend(p, q, sm_scale)
    out, lse, status = call(p, make_cache(p), q, sm_scale=sm_scale)
    assert status == 0
    check(want, q, out, lse)


@pytest.mark.parametrize("power", [-133, -126, -119, -100, 126, 127])
def test_prompt_queries_at_the_ends_of_bf16(power):
    test_queries_at_the_ends_of_bf16(140, power)
