"""pkv.beam_select's order where sums' roundings could change it: equal beams at any place in
memory, scores that cancel logits' gaps, equal candidates of beams with other scores, scores
far from zero."""

import math
from fractions import Fraction

import pytest
import torch

import branch_reference as ref
from paged_kv_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP32 = torch.bfloat16, torch.float32
# A log-sum-exp is off by less than 3e-6, a sum of two fp32 values by some 2^-46 of the largest
# term, and a score is rounded once.
ERR, PAIR, STEP = 3e-6, 2.0 ** -44, 2.0 ** -24


def select(x, scores, n, eos=-1):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pkv.beam_select(x, scores.to(DEV), n, eos=eos, status=st)
    assert int(st) == 0
    return got


def check(x, gpu, scores, n, want=None, eos=-1):
    want = ref.beam_select(x, scores, n, eos) if want is None else want
    got = select(gpu, scores, n, eos)
    assert torch.equal(got[0].cpu(), want[0])
    assert torch.equal(got[1].cpu(), want[1])
    y, z = got[2].cpu().double(), want[2]
    assert torch.equal(y == -math.inf, z == -math.inf)
    fine = z > -math.inf
    tol = ERR + PAIR * scores.double().abs().max() + STEP * z.abs()
    assert bool(((y - z).abs() <= tol)[fine].all())
    if eos >= 0:
        assert torch.equal(got[3].cpu() == -math.inf, want[3] == -math.inf)


# ------------------------------------------------------------------ equal beams


@pytest.mark.parametrize("dt", [BF16, FP32], ids=str)
def test_equal_beams_wherever_their_rows_begin(dt):
    """Four beams of one request with the same logits and scores: rows of odd sizes one after
    another begin at different distances from a 16-byte boundary."""
    g = torch.Generator().manual_seed(1)
    per = 8 if dt == BF16 else 4
    for trial in range(24):
        v = int(torch.randint(9000, 30000, (1,), generator=g)) | 1
        row = (torch.randn(v, generator=g) * 3).to(dt)
        scores = -torch.rand(1, 1, generator=g).expand(1, per).contiguous() * 5
        x = row.repeat(per, 1)
        lead = trial % per
        buf = torch.zeros(lead + per * v, dtype=dt, device=DEV)
        gpu = buf[lead:].view(per, v)
        gpu.copy_(x)
        check(x, gpu, scores, per + 1, eos=int(row.argmax()))
        check(x, gpu, scores, 3)


@pytest.mark.parametrize("dt", [BF16, FP32], ids=str)
def test_flat_equal_beams_wherever_their_rows_begin(dt):
    """The same where more candidates are equal than the list holds."""
    g = torch.Generator().manual_seed(2)
    per = 8 if dt == BF16 else 4
    for trial in range(12):
        v = int(torch.randint(5000, 20000, (1,), generator=g)) | 1
        row = (torch.randn(v, generator=g) * 2).to(dt)
        row[torch.randperm(v, generator=g)[:1500]] = 9.0
        x = row.repeat(per, 1)
        scores = -torch.rand(1, 1, generator=g).expand(1, per).contiguous() * 5
        check(x, x.to(DEV), scores, 2 * per, eos=int(row.argmax()))


# ------------------------------------------------------------------ scores that cancel


@pytest.mark.parametrize("size", [1e3, 1e4, 1e5, 1e6, 1e8])
@pytest.mark.parametrize("dt", [BF16, FP32], ids=str)
def test_scores_that_cancel_a_gap_of_the_logits(size, dt):
    """One logit is far above the others and the score as far above zero: but for the first,
    candidates are small numbers that are differences of large ones."""
    size = float(torch.tensor(size).to(dt))
    g = torch.Generator().manual_seed(3)
    for trial in range(8):
        v = 20000 + 3 * trial
        x = torch.randn(3, v, generator=g).to(dt)
        x[0, 17 * trial] = size
        x[2, 40 + trial] = size / 2
        one = torch.tensor([[size]])
        check(x[:1], x[:1].to(DEV), one, 4)
        check(x[:1], x[:1].to(DEV), one, 40, eos=3)
        scores = torch.tensor([[size, 9.0, size / 2]])
        for n in (2, 4, 40):
            check(x, x.to(DEV), scores, n, eos=5)


# ------------------------------------------------------------------ the order of real numbers


def exact_select(x, scores, n):
    """The definition by whole fractions, all but the sums' logarithm (fp64)."""
    b, w = scores.shape
    parents = torch.full((b, n), -1, dtype=torch.int32)
    tokens, out = parents.clone(), torch.full((b, n), -math.inf, dtype=torch.float64)
    least = math.inf  # difference of two candidates that are not equal
    for i in range(b):
        cand = []
        for j in range(w):
            row = x[i * w + j].double()
            m = float(row.max())
            log = Fraction(math.log(math.fsum(torch.exp(row - m).tolist())))
            base = Fraction(float(scores[i, j])) - Fraction(m) - log
            edge = float(row.topk(min(n, row.numel())).values[-1])
            cand += [(-(base + Fraction(float(row[t]))), j, t)
                     for t in (row >= edge).nonzero().flatten().tolist()]
        cand.sort()
        for k, (t, j, v) in enumerate(cand[:n]):
            parents[i, k], tokens[i, k], out[i, k] = j, v, float(-t)
            if k and t != cand[k - 1][0]:
                least = min(least, float(t - cand[k - 1][0]))
    return (parents, tokens, out, None), least


@pytest.mark.parametrize("dt", [BF16, FP32], ids=str)
@pytest.mark.parametrize("far", [0.0, -2048.0, 2.0 ** 20])
def test_equal_candidates_of_beams_with_other_scores(far, dt):
    """Beams with the same logits, multiples of 1/8 as the scores are: a lower score meets a
    higher logit, and the two candidates are the same number."""
    g = torch.Generator().manual_seed(4)
    b, w, v = 800, 4, 50
    x = (torch.randint(-40, 41, (b, 1, v), generator=g) / 8).expand(b, w, v).reshape(b * w, v).to(dt)
    scores = far - torch.randint(0, 16, (b, w), generator=g) / 8
    for n in (8, 32):
        want, least = exact_select(x, scores, n)
        assert least >= 0.125
        check(x, x.to(DEV), scores, n, want)


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("score", [-2.0 ** 20, -2.0 ** 27, 2.0 ** 30, -1e9, 1e30])
def test_near_candidates_of_beams_with_far_scores(score, flat):
    """Logits a step of fp32 apart under scores whose own steps are much larger."""
    g = torch.Generator().manual_seed(5)
    for trial in range(6):
        v = 3001 + 2 * trial
        row = -torch.rand(v, generator=g)
        if flat:  # more candidates than the list holds
            row[100:1900] = 1.0
        # The second beam's are the first's in another order, its largest half a step higher.
        row[:24] = 1.0 + torch.randperm(24, generator=g) * 2.0 ** -22
        x = torch.stack([row, row])
        x[1, :24] += 2.0 ** -23
        x[1] = x[1, torch.randperm(v, generator=g)]
        scores = torch.tensor([[score, score]])
        want, least = exact_select(x, scores, 30)
        assert least > 1e-10
        check(x, x.to(DEV), scores, 30, want)
