"""What is measured of the serving operators: the paged 8-bit KV cache (append with
rotation, attention over it) and the logit adjustment before the sampler.

Three operators, each in a plain form (elementary torch operations, fp32) and as a
user calls the framework:

  * ``append``  -- ``pkv.append_kv``: rotate q and k, quantise k and v into the pages
    ``out_loc`` names, one power-of-two scale per (page, kv head);
  * ``attend``  -- ``pkv.paged_attention``: attention of a step's packed query tokens
    over those pages;
  * ``adjust``  -- ``pkv.adjust_logits``: penalties for repeated tokens, biases and
    grammar masks.

Sizes follow the repository's workloads: the mixed batch (256 requests, pages of 16,
up to 2000 cached and 512 new tokens, V=151936), the large batch (pages of 64, up to
36863 tokens, V=256000), the four-request example (V=32000) and the heads of
Qwen3-0.6B (16 query, 8 key/value, 128 wide); other head layouts are generic.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0
EMIN, EMAX = -64, 119  # exponents a page scale may take


# ------------------------------------------------------------------ cases


def listed():
    heads = dict(hq=16, hkv=8, d=128)
    return [
        # One decode step of the mixed batch: a token per request, most pages part full.
        dict(name="append_decode", op="append", b=256, cached=2000, new=1, fixed_new=True, ps=16,
             dt="bf16", rot=128, inter=False, **heads),
        # The mixed batch's prompt chunks (about 65 thousand tokens in one step).
        dict(name="append_chunks", op="append", b=256, cached=2000, new=512, fixed_new=False,
             ps=16, dt="bf16", rot=128, inter=False, **heads),
        # An odd small batch: fp16, pages of 5, narrow heads, partial interleaved rotation.
        dict(name="append_odd", op="append", b=7, cached=333, new=45, fixed_new=False, ps=5,
             dt="fp16", rot=32, inter=True, hq=9, hkv=3, d=64),
        # A single conversation decoding: the call's latency.
        dict(name="attend_one", op="attend", b=1, cached=700, new=1, fixed_new=True, ps=16,
             dt="bf16", window=0, full=True, **heads),
        # The mixed batch decoding, ragged lengths.
        dict(name="attend_decode", op="attend", b=256, cached=2512, new=1, fixed_new=True, ps=16,
             dt="bf16", window=0, full=False, **heads),
        # Long contexts in pages of 64, wider groups of query heads.
        dict(name="attend_long", op="attend", b=16, cached=36863, new=1, fixed_new=True, ps=64,
             dt="fp16", window=0, full=False, hq=32, hkv=4, d=128),
        # Draft tokens verified against pages of one token under a sliding window.
        dict(name="attend_verify", op="attend", b=61, cached=2001, new=5, fixed_new=False, ps=1,
             dt="fp16", window=777, full=False, hq=12, hkv=12, d=64),
        # Two long prompts in chunks of up to 4096 tokens on top of what is cached.
        dict(name="attend_chunks", op="attend", b=2, cached=4096, new=4096, fixed_new=True, ps=16,
             dt="bf16", window=0, full=True, **heads),
        # Short prompt chunks of the mixed batch: ragged, rows of many requests at once.
        dict(name="attend_mixed", op="attend", b=48, cached=2000, new=512, fixed_new=False, ps=16,
             dt="bf16", window=0, full=False, **heads),
        # Four requests with every adjustment on fp32 logits: latency.
        dict(name="adjust_small", op="adjust", b=4, v=32000, dt="fp32", hist=30, bias=5,
             mask=0.5),
        # The mixed batch: histories of up to 2512 tokens, a third of the rows under a grammar.
        dict(name="adjust_mixed", op="adjust", b=256, v=151936, dt="bf16", hist=2512, bias=64,
             mask=0.33),
        # The large batch: histories of up to 36863 tokens.
        dict(name="adjust_large", op="adjust", b=1024, v=256000, dt="bf16", hist=36863, bias=300,
             mask=0.33),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "attend", "adjust",
                     "adjust"])
    if op == "adjust":
        b, v = _log(rng, 1, 1024), _log(rng, 1000, 256000)
        return dict(op=op, b=b, v=v, dt=rng.choice(["bf16", "fp32"]) if b * v < 1 << 27 else "bf16",
                    hist=_log(rng, 1, 36863), bias=rng.choice([0, _log(rng, 1, 300)]),
                    mask=rng.choice([0.0, 0.33, 1.0]))
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    d = rng.choice([64, 80, 96, 128, 128])
    case = dict(op=op, hq=hq, hkv=hkv, d=d, ps=rng.choice([1, 3, 4, 16, 16, 32, 64, 100]),
                dt=rng.choice(["bf16", "fp16"]))
    if op == "append":
        b = _log(rng, 1, 256)
        new = rng.choice([1, _log(rng, 1, 4096)])
        new = max(1, min(new, 60000 * 16 // (b * max(16, hq + 2 * hkv))))
        return dict(case, b=b, cached=_log(rng, 1, 4096), new=new, fixed_new=new == 1,
                    rot=rng.choice([d, d, d // 2]), inter=rng.choice([False, True]))
    shape = rng.choice(["decode", "decode", "verify", "chunks"])
    new = {"decode": 1, "verify": rng.randint(2, 8), "chunks": _log(rng, 16, 4096)}[shape]
    cached = _log(rng, 1, 36863 if shape == "decode" else 4096)
    total = cached + new
    # As many requests as keep the keys of the padded batch under 2^28 values and its scores
    # under 3 * 2^28.
    most = min((1 << 28) // (total * hkv * d), (3 << 28) // (total * new * hq), 256)
    while most < 1:  # long chunks of many heads: fewer new tokens
        new = max(1, new // 2)
        total = cached + new
        most = min((1 << 28) // (total * hkv * d), (3 << 28) // (total * new * hq), 256)
    return dict(case, b=_log(rng, 1, most), cached=cached, new=new,
                fixed_new=rng.choice([True, False]), full=rng.choice([True, False, False]),
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))


# ------------------------------------------------------------------ inputs


def _lengths(case):
    """New and cached tokens of each request: from the case alone, so that its work is too."""
    g = torch.Generator().manual_seed(1009 * case["b"] + case["cached"])
    b = case["b"]
    new = torch.randint(1, case["new"] + 1, (b,), generator=g)
    cached = torch.randint(0, case["cached"] + 1, (b,), generator=g)
    if case["fixed_new"]:
        new.fill_(case["new"])
    if case.get("full"):
        cached.fill_(case["cached"])
    new[0], cached[b - 1] = case["new"], case["cached"]
    return cached, new


def _pages(case, seed):
    """Lengths, a page table over shuffled pages, and the packed positions and locations."""
    cached, new = _lengths(case)
    b, ps = case["b"], case["ps"]
    total = cached + new
    need = (total + ps - 1) // ps
    g = torch.Generator().manual_seed(seed)
    pages = int(need.sum()) + 3
    order = torch.randperm(pages, generator=g)
    width = int(need.max()) * ps
    table = torch.zeros(b + 1, (width + 31) // 32 * 32, dtype=torch.int32)
    rows = torch.randperm(b + 1, generator=g)[:b]
    at = 0
    for i in range(b):
        n = int(need[i])
        locs = order[at:at + n, None] * ps + torch.arange(ps)
        table[rows[i], :n * ps] = locs.reshape(-1).to(torch.int32)
        at += n
    pos = torch.cat([torch.arange(int(c), int(c + m)) for c, m in zip(cached, new)])
    req = torch.repeat_interleave(torch.arange(b), new)
    loc = table[rows[req], pos]
    i32 = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    return dict(cached_len=i32(cached), device_len=i32(total), table_idx=i32(rows),
                page_table=table.cuda(), positions=i32(pos), out_loc=i32(loc),
                num_pages=pages, max_q_len=int(new.max()), max_len=int(total.max()))


def _spread(shape, g, dt, loud):
    """Activations: normal, a few channels ``loud`` times larger, tokens of varying size."""
    x = torch.randn(shape, generator=g, device="cuda")
    gain = torch.ones(shape[-1], device="cuda")
    gain[torch.randperm(shape[-1], generator=g, device="cuda")[:max(1, shape[-1] // 32)]] = loud
    size = torch.exp(0.3 * torch.randn(shape[:-2] + (1, 1), generator=g, device="cuda"))
    return (x * gain * size).to(dt)


def _cache(case, s, g):
    """A filled cache: codes of normal values under scales that vary by page and head."""
    shape = (s["num_pages"], case["hkv"], case["ps"], case["d"])
    out = {}
    for name, loud in (("k", 4.0), ("v", 1.5)):
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
        step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
        gain = torch.ones(shape[-1], device="cuda")
        gain[:max(1, shape[-1] // 32)] = loud
        for p in range(0, shape[0], step):
            part = torch.randn((min(step, shape[0] - p),) + shape[1:], generator=g, device="cuda")
            codes[p:p + step] = (part * gain * 64.0).clamp_(-E4M3_MAX, E4M3_MAX).to(codes.dtype)
        # A page's tokens lie next to one another for each head; the view names token before head.
        out[name] = codes.permute(0, 2, 1, 3)
        e = torch.randint(-8, -4, (shape[0], shape[1]), generator=g, device="cuda")
        out[name + "_scale"] = torch.exp2(e.float())
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dt"]]
    if case["op"] == "adjust":
        s = _prepare_adjust(case, g, dt)
    else:
        s = _pages(case, seed)
        s.update(_cache(case, s, g))
        n, hq, hkv, d = s["positions"].numel(), case["hq"], case["hkv"], case["d"]
        if case["op"] == "append":
            # One fused projection's output, as the model leaves it: q, k and v side by side.
            qkv = _spread((n, hq + 2 * hkv, d), g, dt, 4.0)
            s.update(q=qkv[:, :hq], k_new=qkv[:, hq:hq + hkv], v_new=qkv[:, hq + hkv:])
            half = case["rot"] // 2
            freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
            ang = torch.arange(s["max_len"], dtype=torch.float64)[:, None] * freq
            s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
            s["q_out"] = torch.empty(n, hq, d, dtype=dt, device="cuda")
        else:
            s["q"] = _spread((n, hq, d), g, dt, 2.0)
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(n, hq, device="cuda")
        if own:
            from paged_kv_gb300 import pkv

            s["cache"] = pkv.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    s["case"] = case
    return s


def _prepare_adjust(case, g, dt):
    b, v, hist = case["b"], case["v"], case["hist"]
    dev = "cuda"
    s = dict(logits=(torch.randn(b, v, generator=g, device=dev) * 3.0).to(dt))
    s["out"] = torch.empty_like(s["logits"])
    length, prompt = _histories(case)
    s["device_len"], s["prompt_len"] = length.to(torch.int32).to(dev), prompt.to(torch.int32).to(dev)
    # Text repeats its tokens: ranks fall off as a power, the ranks' tokens differ by row.
    rank = torch.rand(b + 1, hist, generator=g, device=dev).pow_(6.0).mul_(v).long()
    shift = torch.randint(0, v, (b + 1, 1), generator=g, device=dev)
    s["token_pool"] = ((rank * 7919 + shift) % v).to(torch.int32)
    s["table_idx"] = torch.randperm(b + 1, generator=g, device=dev)[:b].to(torch.int32)
    u = torch.rand(3, b, generator=g, device=dev)
    s["repetition"] = 1.0 + 0.3 * u[0]
    s["presence"], s["frequency"] = 1.5 * u[1], 0.8 * u[2] - 0.2
    count = _bias_counts(case)
    s["bias_ptr"] = torch.cat([torch.zeros(1, dtype=torch.long), count.cumsum(0)]).to(torch.int32).to(dev)
    nnz = int(count.sum())
    s["bias_ids"] = torch.randint(0, v, (nnz,), generator=g, device=dev).to(torch.int32)
    s["bias_values"] = 4.0 * torch.randn(nnz, generator=g, device=dev)
    s["mask"] = None
    if case["mask"] > 0:
        words = (v + 31) // 32
        # A grammar allows few tokens: one word in eight has some; other rows allow all.
        bits = torch.randint(-2**31, 2**31, (b, words), generator=g, device=dev)
        some = torch.rand(b, words, generator=g, device=dev) < 0.125
        free = torch.rand(b, 1, generator=g, device=dev) >= case["mask"]
        s["mask"] = torch.where(free, torch.full_like(bits, -1),
                                torch.where(some, bits, torch.zeros_like(bits))).to(torch.int32)
    return s


def _histories(case):
    g = torch.Generator().manual_seed(31 * case["b"] + case["hist"])
    length = torch.randint(1, case["hist"] + 1, (case["b"],), generator=g)
    prompt = (length * torch.rand(case["b"], generator=g)).long()
    return length, prompt


def _bias_counts(case):
    g = torch.Generator().manual_seed(17 * case["b"] + case["bias"])
    return torch.randint(0, case["bias"] + 1, (case["b"],), generator=g)


# ------------------------------------------------------------------ one pass


def run(s):
    case = s["case"]
    if case["op"] == "append":
        return _append_own(s) if own else _append_plain(s)
    if case["op"] == "attend":
        return _attend_own(s) if own else _attend_plain(s)
    return _adjust_own(s) if own else _adjust_plain(s)


def _append_own(s):
    from paged_kv_gb300 import pkv

    pkv.append_kv(s["cache"], s["k_new"], s["v_new"], s["positions"], s["out_loc"],
                  cos_sin=s["cos_sin"], interleaved=s["case"]["inter"], q=s["q"],
                  q_out=s["q_out"])
    return dict(q=s["q_out"], k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _attend_own(s):
    from paged_kv_gb300 import pkv

    pkv.paged_attention(s["q"], s["cache"], s["cached_len"], s["device_len"], s["table_idx"],
                        s["page_table"], s["max_q_len"], window=s["case"]["window"],
                        out=s["out"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def _adjust_own(s):
    from paged_kv_gb300 import pkv

    return pkv.adjust_logits(s["logits"], out=s["out"], token_pool=s["token_pool"],
                             table_idx=s["table_idx"], prompt_len=s["prompt_len"],
                             device_len=s["device_len"], repetition=s["repetition"],
                             presence=s["presence"], frequency=s["frequency"],
                             bias_ptr=s["bias_ptr"], bias_ids=s["bias_ids"],
                             bias_values=s["bias_values"], mask=s["mask"])


def _rotate(x, cos, sin, rot, inter):
    x = x.float()
    part, rest = x[..., :rot], x[..., rot:]
    c, n = cos[:, None], sin[:, None]
    if inter:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, rest], -1)


def _power_scale(amax):
    """2^e with the least e such that amax <= 448 * 2^e."""
    f, x = torch.frexp(amax)
    e = torch.where(f <= 0.875, x - 9, x - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, EMIN)).clamp(EMIN, EMAX)
    return torch.ldexp(torch.ones_like(amax), e)


def _append_plain(s):
    case = s["case"]
    half, ps = case["rot"] // 2, case["ps"]
    cs = s["cos_sin"][s["positions"].long()]
    cos, sin = cs[:, :half], cs[:, half:]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, case["rot"], case["inter"]))
    loc = s["out_loc"].long()
    page, off = loc // ps, loc % ps
    new = s["device_len"].long() - s["cached_len"].long()
    first = new.cumsum(0) - new                   # each request's first packed token
    start = loc[first] // ps                      # the page that it goes to,
    begun = off[first]                            # and how much of it is taken
    for name, x in (("k", _rotate(s["k_new"], cos, sin, case["rot"], case["inter"])),
                    ("v", s["v_new"].float())):
        codes, scale = s[name].view(torch.uint8), s[name + "_scale"]
        top = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(-1, scale.shape[1]),
                                                      x.abs().amax(-1), "amax")
        need = _power_scale(top)
        old = scale[start]
        grown = torch.where((begun > 0)[:, None], torch.maximum(old, need[start]), need[start])
        was = codes[start].view(torch.float8_e4m3fn).float()
        again = (was * (old / grown)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        kept = torch.arange(ps, device=loc.device) < begun[:, None]
        codes[start] = torch.where(kept[:, :, None, None], again, codes[start])
        scale[page] = need[page]
        scale[start] = grown
        y = (x / scale[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        codes[page, off] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    return dict(q=s["q_out"], k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _attend_plain(s):
    case = s["case"]
    hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["ps"]
    b, lmax, qmax = case["b"], s["max_len"], s["max_q_len"]
    cached, total = s["cached_len"].long(), s["device_len"].long()
    new = total - cached
    first = new.cumsum(0) - new
    step = torch.arange(qmax, device="cuda")
    live = step < new[:, None]                                       # [b, qmax]
    at = torch.where(live, first[:, None] + step, torch.zeros_like(first)[:, None])
    q = s["q"][at].float().view(b, qmax, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    loc = s["page_table"][s["table_idx"].long(), :lmax].long()
    page, off = loc // ps, loc % ps
    k = s["k"].view(torch.uint8)[page, off].view(torch.float8_e4m3fn).float()
    k = k * s["k_scale"][page][..., None]                            # [b, lmax, hkv, d]
    w = q.reshape(b, hkv, -1, d) @ k.permute(0, 2, 3, 1)             # [b, hkv, g * qmax, lmax]
    del k
    w = w.view(b, hkv, hq // hkv, qmax, lmax).mul_(1.0 / math.sqrt(d))
    j, i = torch.arange(lmax, device="cuda"), cached[:, None] + step
    seen = j <= i[..., None]
    if case["window"] > 0:
        seen &= j > i[..., None] - case["window"]
    w.masked_fill_(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = w.sub_(top).exp_()
    total_w = w.sum(-1, keepdim=True)
    v = s["v"].view(torch.uint8)[page, off].view(torch.float8_e4m3fn).float()
    v = (v * s["v_scale"][page][..., None]).masked_fill_((j >= total[:, None])[..., None, None], 0.0)
    o = w.view(b, hkv, -1, lmax) @ v.permute(0, 2, 1, 3)
    o = o.view(b, hkv, hq // hkv, qmax, d) / total_w.clamp_min(torch.finfo(torch.float32).tiny)
    lse = (top + total_w.log()).squeeze(-1)
    req = torch.repeat_interleave(torch.arange(b, device="cuda"), new,
                                  output_size=s["q"].shape[0])
    t = torch.arange(s["q"].shape[0], device="cuda") - first[req]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4)[req, t].reshape(-1, hq, d))
    s["lse"].copy_(lse.permute(0, 3, 1, 2)[req, t].reshape(-1, hq))
    return dict(out=s["out"], lse=s["lse"])


def _adjust_plain(s):
    b, v = s["logits"].shape
    hist = s["token_pool"][s["table_idx"].long()].long()
    at = torch.arange(hist.shape[1], device="cuda")
    past = at < s["device_len"][:, None]
    made = past & (at >= s["prompt_len"][:, None])
    count = torch.zeros(b, v, device="cuda").scatter_add_(1, hist, made.float())
    seen = torch.zeros(b, v, device="cuda").scatter_add_(1, hist, past.float()) > 0
    x = s["logits"].float()
    r = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    n = s["bias_ids"].numel()
    row = torch.searchsorted(s["bias_ptr"][1:], torch.arange(n, device="cuda", dtype=torch.int32),
                             right=True)
    x.index_put_((row, s["bias_ids"].long()), s["bias_values"], accumulate=True)
    if s["mask"] is not None:
        bit = (s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        x.masked_fill_(bit.view(b, -1)[:, :v] == 0, -math.inf)
    return s["out"].copy_(x)


# ------------------------------------------------------------------ work and exact results


def work(case):
    """Bytes read and written once, and the products' operations."""
    elt = 4 if case["dt"] == "fp32" else 2
    if case["op"] == "adjust":
        b, v = case["b"], case["v"]
        length, _ = _histories(case)
        words = (v + 31) // 32 if case["mask"] > 0 else 0
        return {"bytes": 2 * b * v * elt + 4 * int(length.sum()) + 8 * int(_bias_counts(case).sum())
                + 4 * b * words, "flops": 4 * b * v}
    cached, new = _lengths(case)
    n, hq, hkv, d, ps = int(new.sum()), case["hq"], case["hkv"], case["d"], case["ps"]
    if case["op"] == "append":
        pages = int(((cached + new + ps - 1) // ps - cached // ps).sum())
        return {"bytes": n * d * elt * (2 * hq + 2 * hkv) + 2 * n * hkv * d + 8 * n
                + 8 * pages * hkv + 4 * case["rot"] * int((cached + new).max()),
                "flops": 3 * n * case["rot"] * (hq + hkv)}
    total = cached + new
    if case["window"] > 0:
        w = case["window"]
        kept = torch.minimum(total, new + w - 1)
        pairs = sum(int(torch.arange(int(c) + 1, int(t) + 1).clamp(max=w).sum())
                    for c, t in zip(cached, total))
    else:
        kept = total
        pairs = int((new * cached + new * (new + 1) // 2).sum())
    keys = int(kept.sum())
    return {"bytes": 2 * keys * hkv * d + 8 * (keys // ps) * hkv + 4 * keys
            + 2 * n * hq * d * elt + 4 * n * hq, "flops": 4 * d * hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _append_exact(case, s)
    if case["op"] == "attend":
        return _attend_exact(case, s)
    return _adjust_exact(case, s)


def _append_exact(case, s):
    """Rotation by complex products; the codes' values before their rounding."""
    rot, half, ps = case["rot"], case["rot"] // 2, case["ps"]
    cs = s["cos_sin"][s["positions"].long()].double()
    turn = torch.complex(cs[:, :half], cs[:, half:])[:, None]

    def rotated(x):
        x = x.double().clone()
        if case["inter"]:
            z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], half, 2).contiguous())
            x[..., :rot] = torch.view_as_real(z * turn).flatten(-2)
        else:
            z = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous()) * turn
            x[..., :half], x[..., half:rot] = z.real, z.imag
        return x

    loc = s["out_loc"].long()
    # Blocks of packed tokens that share a page: every one begins where the page changes.
    page = loc // ps
    head = torch.ones_like(page, dtype=torch.bool)
    head[1:] = page[1:] != page[:-1]
    block = head.long().cumsum(0) - 1
    begin = head.nonzero().squeeze(1)
    out = {"q": rotated(s["q"])}
    for name, x in (("k", rotated(s["k_new"])), ("v", s["v_new"].double())):
        codes = s[name].float().double().contiguous()
        scale = s[name + "_scale"].double()
        amax = torch.zeros(begin.numel(), x.shape[1], dtype=torch.float64, device="cuda")
        amax.index_reduce_(0, block, x.abs().amax(-1), "amax")
        # log2 of an exact power may come out a little above it.
        e = torch.ceil(torch.log2(amax / E4M3_MAX) - 1e-12).clamp(EMIN, EMAX)
        want = torch.exp2(e)
        p, o = page[begin], loc[begin] % ps
        old = scale[p]
        now = torch.where((o > 0)[:, None], torch.maximum(old, want), want)
        keep = torch.arange(ps, device="cuda") < o[:, None]
        held = codes[p]
        codes[p] = torch.where(keep[:, :, None, None], held * (old / now)[:, None, :, None], held)
        scale[p] = now
        codes[page, loc % ps] = x / now[block][:, :, None]
        out[name], out[name + "_scale"] = codes, scale
    return out


def _attend_exact(case, s):
    """One request and one group of heads at a time, in fp64."""
    hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["ps"]
    group = hq // hkv
    cached, new = _lengths(case)
    if 4 * d * hq * int((new * (cached + new)).sum()) > 6e12:
        return None
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    k8, v8 = s["k"].view(torch.uint8), s["v"].view(torch.uint8)
    rows = s["table_idx"].tolist()
    at = 0
    for i in range(case["b"]):
        c, m = int(cached[i]), int(new[i])
        low = max(0, c - case["window"] + 1) if case["window"] > 0 else 0
        loc = s["page_table"][rows[i], low:c + m].long()
        j = torch.arange(low, c + m, device="cuda")
        k = k8[loc // ps, loc % ps].view(torch.float8_e4m3fn).double() * s["k_scale"][loc // ps].double()[..., None]
        v = v8[loc // ps, loc % ps].view(torch.float8_e4m3fn).double() * s["v_scale"][loc // ps].double()[..., None]
        gap = torch.arange(c, c + m, device="cuda")[:, None] - j
        hide = gap < 0
        if case["window"] > 0:
            hide |= gap >= case["window"]
        for h in range(hq):
            z = s["q"][at:at + m, h].double() @ k[:, h // group].T / math.sqrt(d)
            z = z.masked_fill(hide, -math.inf)
            lse[at:at + m, h] = torch.logsumexp(z, 1)
            out[at:at + m, h] = torch.softmax(z, 1) @ v[:, h // group]
        at += m
    return {"out": out, "lse": lse}


def _adjust_exact(case, s):
    """A row at a time, touching only the tokens that a rule names."""
    if case["b"] * case["v"] > 1 << 26:
        return None
    x = s["logits"].double()
    length, prompt = _histories(case)
    ptr = s["bias_ptr"].tolist()
    rows = s["table_idx"].tolist()
    for i in range(case["b"]):
        past = s["token_pool"][rows[i], :int(length[i])].long()
        seen = past.unique()
        r = s["repetition"][i].double()
        y = x[i, seen]
        x[i, seen] = torch.where(y > 0, y / r, y * r)
        made, count = past[int(prompt[i]):].unique(return_counts=True)
        x[i, made] -= s["frequency"][i].double() * count + s["presence"][i].double()
        some = slice(ptr[i], ptr[i + 1])
        x[i].index_add_(0, s["bias_ids"][some].long(), s["bias_values"][some].double())
    if s["mask"] is not None:
        word = torch.arange(case["v"], device="cuda")
        bit = (s["mask"].long()[:, word // 32] >> (word % 32)) & 1
        x = torch.where(bit == 1, x, torch.full_like(x, -math.inf))
    return x
