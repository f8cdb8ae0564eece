"""pkv_adjust_logits on logits and outputs whose rows take turns in one buffer."""

import pytest
import torch

from paged_kv_gb300 import pkv
from test_gpu_adjust import check, dev, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("v", [1000, 517])
@pytest.mark.parametrize("first", [True, False])
def test_rows_that_take_turns(dt, v, first):
    logits, p = problem(5, v, 60, 9, 61, dt)
    buf = torch.full((5, 2 * v + 3), 6.0, dtype=dt, device="cuda")
    halves = buf[:, :v], buf[:, v + 3:]
    x, out = halves if first else halves[::-1]
    x.copy_(logits)
    assert pkv.adjust_logits(x, out=out, **dev(p)) is out
    check(out, logits, p)
    assert torch.equal(x.cpu(), logits) and bool((buf[:, v:v + 3] == 6.0).all())


def test_rows_of_different_strides_that_take_turns():
    logits, p = problem(3, 100, 20, 5, 62, torch.float32)
    buf = torch.full((1200,), 6.0, device="cuda")
    x, out = buf.as_strided((3, 100), (200, 1), 0), buf.as_strided((3, 100), (400, 1), 100)
    x.copy_(logits)
    check(pkv.adjust_logits(x, out=out, **dev(p)), logits, p)
    assert torch.equal(x.cpu(), logits)


@pytest.mark.parametrize("stride,start", [(200, 99), (200, 150), (150, 100), (300, 1), (100, 0)])
def test_rows_that_overlap_are_refused(stride, start):
    logits, p = problem(3, 100, 20, 5, 62, torch.float32)
    buf = torch.zeros(1200, device="cuda")
    x, out = buf.as_strided((3, 100), (200, 1), 0), buf.as_strided((3, 100), (stride, 1), start)
    with pytest.raises(pkv.PkvError):
        pkv.adjust_logits(x, out=out, **dev(p))
    torch.cuda.synchronize()
    assert not buf.any()
