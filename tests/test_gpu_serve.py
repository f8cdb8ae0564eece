"""The example engine: its last step against a plain fp64 forward pass over what
its caches hold, chunked prompts against whole ones, and what its rules promise."""

import math

import pytest
import torch

import serving_reference as ref
from paged_kv_gb300 import serve

pytestmark = pytest.mark.gpu


def requests(vocab, new=5):
    g = torch.Generator().manual_seed(3)

    def prompt(n):
        return torch.randint(0, vocab, (n,), generator=g).tolist()

    return [serve.Request(prompt(1), new), serve.Request(prompt(150), new, temperature=0.7),
            serve.Request(prompt(37), new, repetition=1.3, presence=0.4, frequency=0.2),
            serve.Request(prompt(64), new, bias=[(3, 50.0), (9, 1.0), (3, -100.0)]),
            serve.Request(prompt(16), new, allowed=[5, 6, 7, 100, 511])]


def plain(engine, row, position):
    """fp64 logits after ``position``, the sums of a step's roundings left out: the
    keys and values up to it are read from the caches."""
    m, c = engine.model, engine.model.cfg
    token = int(engine.token_pool[row, position])
    slots = engine.page_table[row, :position + 1].cpu().long()
    x = m.embed[token].cpu().double()

    def norm(x):
        return x / torch.sqrt((x * x).mean() + 1e-5)

    for i, (w, cache) in enumerate(zip(m.layers, engine.caches)):
        w = {k: t.cpu().double() for k, t in w.items()}
        q = (w["qkv"] @ norm(x))[:c.q_heads * c.head_dim].view(c.q_heads, c.head_dim)
        q = ref.rotate(q, m.cos_sin[position].cpu(), c.head_dim, False)
        page, at = slots // cache.page_size, slots % cache.page_size
        k = cache.k.float().cpu()[page, at].double() * cache.k_scale.cpu()[page].double()[..., None]
        v = cache.v.float().cpu()[page, at].double() * cache.v_scale.cpu()[page].double()[..., None]
        first = max(0, position + 1 - m.window(i)) if m.window(i) else 0
        k, v = k[first:].repeat_interleave(c.q_heads // c.kv_heads, 1), v[first:].repeat_interleave(
            c.q_heads // c.kv_heads, 1)
        p = torch.softmax(torch.einsum("hd,thd->ht", q, k) * c.head_dim ** -0.5, 1)
        x = x + w["out"] @ torch.einsum("ht,thd->hd", p, v).flatten()
        h = w["up"] @ norm(x)
        x = x + w["down"] @ (h * torch.sigmoid(h))
    return m.embed.cpu().double() @ norm(x)


@pytest.mark.parametrize("page_size,chunk,window", [(16, 64, 0), (8, 13, 20), (64, 512, 48)])
def test_logits_of_a_step_match_a_plain_forward_pass(page_size, chunk, window):
    cfg = serve.Config(window=window)
    reqs = requests(cfg.vocab)
    engine = serve.Engine(serve.Model(cfg), reqs, page_size, chunk)
    for _ in range(200):
        before = list(engine.known)
        got = engine.step()
        if got is None:
            break
        rows, logits, tokens = got
        if len(rows) < 2:
            continue
        for j, row in enumerate(rows):
            n = before[row]
            want = plain(engine, row, n - 1)
            r = reqs[row]
            past = engine.token_pool[row, :n].cpu().long().tolist()
            for t in set(past):
                want[t] = want[t] / r.repetition if want[t] > 0 else want[t] * r.repetition
                made = past[len(r.prompt):].count(t)
                want[t] -= r.frequency * made + r.presence * (made > 0)
            for t, x in r.bias:
                want[t] += x
            have = logits[j].cpu().double()
            if r.allowed is not None:
                hidden = torch.ones(cfg.vocab, dtype=torch.bool)
                hidden[list(r.allowed)] = False
                assert bool((have[hidden] == -math.inf).all())
                have, want = have[~hidden], want[~hidden]
            # bf16 activations: some 8 roundings of 2^-9 a layer on values of order 1, and the
            # logits' own; the sum over the width leaves them of order 1 too.
            assert float((have - want).abs().max()) <= 24 * 2.0 ** -9 * max(
                1.0, float(want.abs().max())), (row, n)
            if r.temperature == 0.0:
                assert int(tokens[j]) == int(logits[j].argmax())
    assert engine.known == engine.goal and int(engine.status.item()) == 0


def test_a_run_repeats_and_keeps_its_rules():
    cfg = serve.Config()
    model = serve.Model(cfg)
    a = serve.Engine(model, requests(cfg.vocab, 12), chunk=32).run()
    b = serve.Engine(model, requests(cfg.vocab, 12), chunk=32).run()
    assert a == b and all(len(x) == 12 for x in a)
    assert set(a[4]) <= {5, 6, 7, 100, 511}
    assert 3 not in a[3]  # a bias of -50 in all


def test_refusals():
    model = serve.Model(serve.Config(max_pos=32))
    with pytest.raises(ValueError):
        serve.Engine(model, [serve.Request([])])
    with pytest.raises(ValueError):
        serve.Engine(model, [serve.Request([1] * 30, 3)])


def test_the_command_runs(capsys):
    serve.main(["3", "2"])
    assert capsys.readouterr().out.count("request") == 3
