"""pkv_append_kv on the GPU against the fp64 restatement: rotation, page scales,
codes, re-rounding of begun pages, strides, and what it refuses or skips."""

import pytest
import torch

import serving_reference as ref
from paged_kv_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make_cache(p):
    return pkv.KVCache(*(dev_like(p[x]) for x in ("k", "v")),
                       p["k_scale"].to(DEV), p["v_scale"].to(DEV))


def dev_like(t):
    """On the device with the same strides (a dense permuted tensor)."""
    perm = sorted(range(t.dim()), key=lambda i: -t.stride(i))
    back = [perm.index(i) for i in range(t.dim())]
    return t.permute(perm).contiguous().to(DEV).permute(back)


def tokens(n, heads, d, dt, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, d, generator=g) * gain).to(dt)


def check(p, cache, want, dt, before):
    for name in "kv":
        w = want[name]
        scale = getattr(cache, name + "_scale").cpu().double()
        assert torch.equal(scale, w["scale"]), name + "_scale"
        got = getattr(cache, name).cpu().to(torch.float32).double() * scale[:, None, :, None]
        y = w["value"] / w["scale"][:, None, :, None]
        # Half a spacing; fp32 arithmetic before it moves a value by 2^-22 of its pair.
        tol = (0.5 * ref.e4m3_spacing(y) + 2.0 ** -20 * (y.abs() + 448 * 2 ** -4)) \
            * w["scale"][:, None, :, None]
        fresh = torch.zeros(got.shape, dtype=torch.bool)
        for page, slot in w["written"]:
            fresh[page, slot] = True
        for page, slot, h in w["again"]:
            fresh[page, slot, h] = True
        err = (got - w["value"]).abs()
        assert bool((err <= tol)[fresh].all()), (name, float((err / tol)[fresh].max()))
        same = getattr(cache, name).cpu().contiguous().view(torch.uint8)
        old = before[name].contiguous().view(torch.uint8)
        assert torch.equal(same[~fresh], old[~fresh]), name + " written elsewhere"


def check_q(got, want, dt):
    for j, x in want["q"].items():
        tol = (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -10) * x.abs() + 1e-5
        assert bool(((got[j].cpu().double() - x).abs() <= tol).all())


CASES = [
    # cached, new, ps, hkv, group, d, rot, interleaved, dt
    ([0], [1], 1, 1, 1, 16, 16, False, torch.bfloat16),
    ([5, 0, 16, 31], [1, 1, 1, 1], 16, 8, 2, 128, 128, False, torch.bfloat16),
    ([3, 0, 7], [40, 5, 0], 4, 2, 3, 64, 64, True, torch.float16),
    ([1, 9, 100], [70, 33, 17], 64, 3, 1, 80, 40, False, torch.float16),
    ([2, 6], [150, 21], 100, 1, 4, 96, 8, True, torch.bfloat16),
    ([0, 1, 2, 3, 4], [9, 8, 7, 6, 5], 5, 2, 2, 32, 32, False, torch.float16),
    ([33], [129], 48, 4, 1, 128, 64, False, torch.bfloat16),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"ps{c[2]}d{c[5]}rot{c[6]}")
@pytest.mark.parametrize("head_major", [True, False])
def test_matches_fp64(case, head_major):
    cached, new, ps, hkv, group, d, rot, inter, dt = case
    p = ref.page_problem(cached, new, ps, hkv, d, 5, head_major=head_major)
    n = p["positions"].numel()
    k, v, q = (tokens(n, h, d, dt, s, g) for h, s, g in ((hkv, 1, 3.0), (hkv, 2, 0.7),
                                                         (hkv * group, 3, 1.0)))
    cs = ref.rope_table(max(int(x) for x in p["device_len"]), rot)
    want = ref.append(p, k, v, q, cs, inter)
    cache = make_cache(p)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pkv.append_kv(cache, k.to(DEV), v.to(DEV), p["positions"].to(DEV), p["out_loc"].to(DEV),
                        cos_sin=cs.to(DEV), interleaved=inter, q=q.to(DEV), status=status)
    check(p, cache, want, dt, p)
    check_q(got, want, dt)
    assert int(status.item()) == 0


def test_slices_of_one_projection_and_in_place_queries():
    p = ref.page_problem([3, 20], [30, 1], 16, 2, 64, 6)
    n = p["positions"].numel()
    qkv = tokens(n, 8, 64, torch.bfloat16, 9).to(DEV)
    cpu = qkv.cpu()
    cs = ref.rope_table(64, 64)
    want = ref.append(p, cpu[:, 4:6], cpu[:, 6:], cpu[:, :4], cs)
    cache = make_cache(p)
    got = pkv.append_kv(cache, qkv[:, 4:6], qkv[:, 6:], p["positions"].to(DEV), p["out_loc"].to(DEV),
                        cos_sin=cs.to(DEV), q=qkv[:, :4], q_out=qkv[:, :4])
    check(p, cache, want, torch.bfloat16, p)
    check_q(got, want, torch.bfloat16)
    assert torch.equal(qkv[:, 4:].cpu(), cpu[:, 4:])


def test_without_rotation_and_queries():
    p = ref.page_problem([4], [7], 8, 2, 48, 7)
    k, v = tokens(7, 2, 48, torch.float16, 1), tokens(7, 2, 48, torch.float16, 2)
    cache = make_cache(p)
    assert pkv.append_kv(cache, k.to(DEV), v.to(DEV), p["positions"].to(DEV),
                         p["out_loc"].to(DEV)) is None
    check(p, cache, ref.append(p, k, v), torch.float16, p)


def test_a_page_filled_token_by_token_keeps_its_earlier_tokens():
    # Growing values raise the page's scale at nearly every step.
    ps, d = 8, 32
    p = ref.page_problem([0], [ps], ps, 1, d, 8)
    cache = make_cache(p)
    k = torch.stack([torch.linspace(-1, 1, d) * 3.0 ** t for t in range(ps)])[:, None].half()
    for t in range(ps):
        pkv.append_kv(cache, k[t:t + 1].to(DEV), k[t:t + 1].to(DEV),
                      p["positions"][t:t + 1].to(DEV), p["out_loc"][t:t + 1].to(DEV))
    page = int(p["out_loc"][0]) // ps
    scale = float(cache.k_scale[page, 0])
    assert scale == ref.power_scale(float(k.abs().max()))
    got = cache.k[page, :, 0].cpu().float().double() * scale
    want = k[:, 0].double()
    # One rounding a token while its scale holds, and a subnormal one for each growth.
    tol = 2.0 ** -4 * want.abs() + ps * 2.0 ** -10 * scale
    assert bool(((got - want).abs() <= tol).all())


def test_total_tokens_on_the_device_and_one_more_stream():
    p = ref.page_problem([0, 5], [6, 9], 4, 2, 64, 9)
    n = 15
    k, v, q = (tokens(n, 2, 64, torch.bfloat16, s) for s in (1, 2, 3))
    cs = ref.rope_table(16, 64)
    want = ref.append(p, k, v, q, cs, n=9)
    cache = make_cache(p)
    args = [t.to(DEV) for t in (k, v, p["positions"], p["out_loc"], cs, q)]
    total = torch.tensor([9], dtype=torch.int64, device=DEV)
    out = torch.full((n, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pkv.append_kv(cache, *args[:4], cos_sin=args[4], q=args[5], q_out=out, total_tokens=total)
    s.synchronize()
    check(p, cache, want, torch.bfloat16, p)
    check_q(out, want, torch.bfloat16)
    assert bool((out[9:] == 7.0).all())


def test_skipped_tokens_and_status_bits():
    p = ref.page_problem([2], [20], 8, 1, 32, 10)
    loc, pos = p["out_loc"].clone(), p["positions"].clone()
    loc[3], loc[11], pos[6] = -1, p["num_pages"] * 8, 4000
    p["out_loc"], p["positions"] = loc, pos
    k, v, q = (tokens(20, 1, 32, torch.float16, s) for s in (1, 2, 3))
    cs = ref.rope_table(64, 32)
    want = ref.append(p, k, v, q, cs)
    cache = make_cache(p)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((20, 1, 32), 5.0, dtype=torch.float16, device=DEV)
    pkv.append_kv(cache, k.to(DEV), v.to(DEV), pos.to(DEV), loc.to(DEV), cos_sin=cs.to(DEV),
                  q=q.to(DEV), q_out=out, status=status)
    check(p, cache, want, torch.float16, p)
    check_q(out, want, torch.float16)
    assert all(bool((out[j] == 5.0).all()) for j in (3, 6, 11))
    assert int(status.item()) == pkv.ST_ROW_OOB | pkv.ST_COL_OOB


def test_values_that_are_not_finite_or_too_large():
    p = ref.page_problem([0], [4], 4, 1, 16, 11)
    k = tokens(4, 1, 16, torch.bfloat16, 1)
    k[1, 0, 3], k[2, 0, 4], k[2, 0, 5] = float("nan"), float("inf"), -float("inf")
    v = torch.full((4, 1, 16), 3e38, dtype=torch.bfloat16)
    cache = make_cache(p)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.append_kv(cache, k.to(DEV), v.to(DEV), p["positions"].to(DEV), p["out_loc"].to(DEV),
                  status=status)
    assert int(status.item()) == pkv.ST_NONFINITE
    page = int(p["out_loc"][0]) // 4
    got = cache.k[page, :, 0].cpu().float()
    assert bool(torch.isnan(got[1, 3])) and int(torch.isnan(got).sum()) == 1
    assert float(got[2, 4]) == 448.0 and float(got[2, 5]) == -448.0
    assert float(cache.v_scale[page, 0]) == 2.0 ** 119
    # 3e38 of 448 * 2^119 (2.98e38) is limited to the largest code.
    assert bool((cache.v[page].cpu().float() == 448.0).all())


def test_zeros_take_the_least_scale():
    p = ref.page_problem([0], [2], 2, 1, 16, 12)
    z = torch.zeros(2, 1, 16, dtype=torch.float16, device=DEV)
    cache = make_cache(p)
    pkv.append_kv(cache, z, z, p["positions"].to(DEV), p["out_loc"].to(DEV))
    page = int(p["out_loc"][0]) // 2
    assert float(cache.k_scale[page, 0]) == 2.0 ** -64 and not cache.k[page].float().any()


def test_pages_past_four_gigabytes():
    ps, hkv, d = 64, 8, 128
    pages = (5 << 30) // (ps * hkv * d)
    p = ref.page_problem([60], [9], ps, hkv, d, 13)
    cache = pkv.KVCache.empty(pages, ps, hkv, d)
    page = p["out_loc"] // ps
    first = int(page.min())
    loc = (pages - 1 - (page - first).abs()) * ps + p["out_loc"] % ps
    k, v = tokens(9, hkv, d, torch.bfloat16, 1), tokens(9, hkv, d, torch.bfloat16, 2)
    pkv.append_kv(cache, k.to(DEV), v.to(DEV), p["positions"].to(DEV), loc.to(torch.int32).to(DEV))
    got = cache.k.view(torch.uint8)[(loc // ps).to(DEV), (loc % ps).to(DEV)]
    got = got.view(torch.float8_e4m3fn).float().cpu()
    got = got * cache.k_scale[(loc // ps).to(DEV)].cpu()[..., None]
    assert bool(((got - k.float()).abs() <= 2.0 ** -4 * k.float().abs() + 2.0 ** -8).all())


def test_replays_in_a_graph():
    p = ref.page_problem([3, 8], [1, 1], 4, 2, 64, 14)
    cache = make_cache(p)
    k, v = (tokens(2, 2, 64, torch.bfloat16, s).to(DEV) for s in (1, 2))
    pos, loc = p["positions"].to(DEV), p["out_loc"].to(DEV)
    pkv.append_kv(cache, k, v, pos, loc)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.append_kv(cache, k, v, pos, loc)
    fresh = tokens(2, 2, 64, torch.bfloat16, 3)
    k.copy_(fresh)
    g.replay()
    torch.cuda.synchronize()
    page, off = p["out_loc"].long() // 4, p["out_loc"].long() % 4
    got = cache.k.cpu().float()[page, off] * cache.k_scale.cpu()[page][..., None]
    assert bool(((got - fresh.float()).abs() <= 2.0 ** -4 * fresh.float().abs() + 2.0 ** -6).all())
