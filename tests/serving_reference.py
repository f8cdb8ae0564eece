"""Plain fp64 restatements of the serving operators on the CPU (the paged 8-bit
KV cache's append and attention, the logit adjustment), and seeded small
problems for them.  Written from the definitions in include/pkv.h, one token or
one row at a time; they share no code with the library."""

import math

import numpy as np
import torch

E4M3_MAX = 448.0


def e4m3_spacing(y):
    """Distance between neighbouring e4m3 values around |y|, y a float64 tensor."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    return torch.exp2(e.clamp_max(8.0) - 3.0)


def page_problem(lengths, new, ps, hkv, d, seed, spare_pages=2, head_major=True, extra_cols=0):
    """Lengths, a shuffled page table, packed positions and locations, and a cache of
    random codes under random power-of-two scales.  ``lengths`` are the cached ones."""
    g = torch.Generator().manual_seed(seed)
    cached = torch.tensor(lengths, dtype=torch.int32)
    total = cached + torch.tensor(new, dtype=torch.int32)
    b = len(lengths)
    need = [(int(t) + ps - 1) // ps for t in total]
    pages = sum(need) + spare_pages
    order = torch.randperm(pages, generator=g).tolist()
    cols = max(max(need), 1) * ps + extra_cols
    table = torch.full((b + 2, cols), -5, dtype=torch.int32)
    rows = torch.randperm(b + 2, generator=g)[:b].to(torch.int32)
    at = 0
    for i in range(b):
        for p in range(need[i]):
            start = order[at] * ps
            at += 1
            table[rows[i], p * ps:(p + 1) * ps] = torch.arange(start, start + ps, dtype=torch.int32)
    pos = [torch.arange(int(c), int(t), dtype=torch.int32) for c, t in zip(cached, total)]
    loc = [table[r, int(c):int(t)] for r, c, t in zip(rows.tolist(), cached, total)]
    shape = (pages, hkv, ps, d) if head_major else (pages, ps, hkv, d)
    out = dict(cached_len=cached, device_len=total, table_idx=rows, page_table=table,
               positions=torch.cat(pos), out_loc=torch.cat(loc).contiguous(), num_pages=pages,
               max_q_len=max(int(max(new)), 1))
    for name in "kv":
        x = (torch.randn(shape, generator=g) * 48).clamp(-E4M3_MAX, E4M3_MAX)
        x = x.to(torch.float8_e4m3fn)
        out[name] = x.permute(0, 2, 1, 3) if head_major else x
        e = torch.randint(-8, -3, (pages, hkv), generator=g)
        out[name + "_scale"] = torch.exp2(e.float())
    return out


def rope_table(max_pos, rot):
    half = rot // 2
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * (
        10000.0 ** (-torch.arange(half, dtype=torch.float64) / half))
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def rotate(x, row, rot, interleaved):
    """x [heads, d] fp64 by one row of the fp32 table."""
    y = x.clone()
    half = rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        c, s = float(row[i]), float(row[half + i])
        y[:, a] = x[:, a] * c - x[:, b] * s
        y[:, b] = x[:, b] * c + x[:, a] * s
    return y


def power_scale(amax):
    if amax == 0:
        return 2.0 ** -64
    e = -64
    while amax > E4M3_MAX * 2.0 ** e and e < 119:
        e += 1
    return 2.0 ** e


def append(p, k_new, v_new, q=None, cos_sin=None, interleaved=False, n=None):
    """Values the cache stands for after the call, before their last rounding.

    Returns q' (fp64), and for k and v: ``value`` [pages, ps, hkv, d] (the new tokens'
    exact values; earlier slots' dequantised values), ``scale`` [pages, hkv], and the
    sets of written and of re-rounded (page, slot)."""
    rot = 0 if cos_sin is None else cos_sin.shape[1]
    ps = p["k"].shape[1]
    n = k_new.shape[0] if n is None else n
    pos, loc = p["positions"].tolist(), p["out_loc"].tolist()
    slots = p["num_pages"] * ps

    def turned(x, j):
        x = x[j].double()
        return rotate(x, cos_sin[pos[j]], rot, interleaved) if rot else x

    ok = [0 <= loc[j] < slots and (rot == 0 or 0 <= pos[j] < cos_sin.shape[0]) for j in range(n)]
    out = {}
    if q is not None:
        out["q"] = {j: turned(q, j) for j in range(n) if ok[j]}
    for name, x in (("k", k_new), ("v", v_new)):
        new = {j: (turned(x, j) if name == "k" else x[j].double()) for j in range(n) if ok[j]}
        scale = p[name + "_scale"].double().clone()
        value = p[name].to(torch.float32).double() * p[name + "_scale"].double()[:, None, :, None]
        written, again = {}, set()
        pages = {}
        for j in new:
            pages.setdefault(loc[j] // ps, []).append(j)
        for page, js in pages.items():
            first = min(loc[j] % ps for j in js)
            for h in range(x.shape[1]):
                mags = torch.stack([new[j][h] for j in js]).abs()
                finite = mags[torch.isfinite(mags)]
                s = power_scale(float(finite.max()) if finite.numel() else 0.0)
                if first > 0:
                    s = max(s, float(scale[page, h]))
                    if s != float(scale[page, h]):
                        again |= {(page, o, h) for o in range(first)}
                scale[page, h] = s
            for j in js:
                value[page, loc[j] % ps] = new[j]
                written[(page, loc[j] % ps)] = j
        out[name] = dict(value=value, scale=scale, written=written, again=again)
    return out


def attend(p, q, sm_scale, window=0, kv_begin=None):
    """out and lse (fp64), and each row's sum of |p v| and largest |q||k| products, for
    tolerances.  One query row at a time; what a row does not see is never read."""
    ps, hkv = p["k"].shape[1], p["k"].shape[2]
    n, hq, d = q.shape
    group = hq // hkv
    k_all, v_all = p["k"].to(torch.float32), p["v"].to(torch.float32)
    out = torch.zeros(n, hq, d, dtype=torch.float64)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64)
    mass = torch.zeros(n, hq, d, dtype=torch.float64)
    tail = torch.zeros(n, hq, d, dtype=torch.float64)
    prod = torch.zeros(n, hq, dtype=torch.float64)
    j = 0
    for i in range(len(p["cached_len"])):
        c, e = int(p["cached_len"][i]), int(p["device_len"][i])
        low = 0 if kv_begin is None else max(0, int(kv_begin[i]))
        for pos in range(c, e):
            lo = max(low, pos - window + 1) if window > 0 else low
            if lo <= pos and j < n:
                loc = p["page_table"][int(p["table_idx"][i]), lo:pos + 1].long()
                page, off = loc // ps, loc % ps
                for h in range(hkv):
                    k = k_all[page, off, h].double() * p["k_scale"][page, h].double()[:, None]
                    v = v_all[page, off, h].double() * p["v_scale"][page, h].double()[:, None]
                    for g in range(h * group, (h + 1) * group):
                        x = q[j, g].double()
                        s = (k @ x) * sm_scale
                        top = s.max()
                        w = torch.exp(s - top)
                        z = w.sum()
                        out[j, g] = (w @ v) / z
                        lse[j, g] = top + z.log()
                        mass[j, g] = (w @ v.abs()) / z
                        tail[j, g] = v.abs().sum(0) / z
                        prod[j, g] = (k.abs() @ x.abs()).max() * sm_scale
            j += 1
    return dict(out=out, lse=lse, mass=mass, tail=tail, prod=prod)


def attend_tolerance(want, dt, d):
    """Weights of at least 8 significant bits, with an absolute floor of 2^-19 of the
    largest; fp32 scores (a sum of d products) through an exponential; one rounding of
    the result."""
    score = 2.0 ** -24 * (d + 8) * want["prod"] + 1e-6 * (8 + want["prod"])
    last = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -10
    out = ((2.0 ** -8 + 2 * score)[..., None] * want["mass"] + 2.0 ** -19 * want["tail"]
           + last * want["out"].abs() + (6.2e-8 if dt == torch.float16 else 1e-30))
    return out, score + 1e-6 * (1 + want["lse"].abs().nan_to_num(0.0, 0.0, 0.0))


def adjust(logits, token_pool=None, table_idx=None, prompt_len=None, device_len=None,
           repetition=None, presence=None, frequency=None, bias_ptr=None, bias_ids=None,
           bias_values=None, mask=None):
    """fp64 result, and the sum of the magnitudes that went into each element."""
    b, v = logits.shape
    x = logits.double().clone()
    size = x.abs()
    for i in range(b):
        if token_pool is not None:
            n = int(device_len[i])
            prompt = min(max(int(prompt_len[i]), 0), n)
            hist = token_pool[int(table_idx[i]), :n].tolist()
            made = {}
            for t in hist[prompt:]:
                made[t] = made.get(t, 0) + 1
            for t in set(hist):
                if not 0 <= t < v:
                    continue
                if repetition is not None:
                    r = float(repetition[i])
                    x[i, t] = x[i, t] / r if x[i, t] > 0 else x[i, t] * r
                    size[i, t] = x[i, t].abs()
                c = made.get(t, 0)
                if c and frequency is not None:
                    x[i, t] -= float(frequency[i]) * c
                    size[i, t] += abs(float(frequency[i])) * c
                if c and presence is not None:
                    x[i, t] -= float(presence[i])
                    size[i, t] += abs(float(presence[i]))
        if bias_ptr is not None:
            for e in range(int(bias_ptr[i]), int(bias_ptr[i + 1])):
                t = int(bias_ids[e])
                if 0 <= t < v:
                    x[i, t] += float(bias_values[e])
                    size[i, t] += abs(float(bias_values[e]))
    if mask is not None:
        words = mask.numpy().view(np.uint32)
        bit = (words[:, np.arange(v) // 32] >> (np.arange(v) % 32).astype(np.uint32)) & 1
        x[torch.from_numpy(bit == 0)] = -math.inf
    return x, size
