"""The workspace that pkv.paged_attention takes by itself: on side streams, in captured
graphs, after calls of other shapes."""

import pytest
import torch

import serving_reference as ref
from paged_kv_gb300 import pkv
from test_gpu_append import make_cache
from test_gpu_attention import DEV, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def none_yet(monkeypatch):
    """Each test begins without default workspaces (earlier ones stay alive)."""
    torch.cuda.synchronize()
    monkeypatch.setattr(pkv, "_attention_workspaces", {})
    monkeypatch.setattr(pkv, "_capture_workspaces", {})
    yield
    torch.cuda.synchronize()


class Problem:
    """A call of ``new`` tokens a request that splits its long request over the GPU."""

    def __init__(self, new, d, seed):
        p = ref.page_problem([5000, 40], [new, 1], 16, 2, d, seed)
        self.cache, self.new = make_cache(p), new
        self.q = queries(new + 1, 4, d, torch.bfloat16, seed).to(DEV)
        self.dev = [p[x].to(DEV) for x in ("cached_len", "device_len", "table_idx", "page_table")]
        need = pkv.paged_attention_workspace_bytes(2, new + 1, new, 4, 2, d)
        self.want = self(workspace=torch.zeros(need, dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()

    def __call__(self, **kw):
        return pkv.paged_attention(self.q, self.cache, *self.dev, self.new, **kw)

    def good(self, out):
        torch.cuda.synchronize()
        return torch.equal(out, self.want)


def dirty_memory():
    """Leaves freed memory that is not zero, and a stream that is busy for some ms."""
    for mb in (8, 16, 32, 64, 128):
        torch.full((mb << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    torch.cuda._sleep(20_000_000)


@pytest.mark.parametrize("new", [1, 150])
@pytest.mark.parametrize("how", ["object", "handle", "current"])
def test_the_first_call_goes_to_a_side_stream(new, how):
    x = Problem(new, 128, 1)
    side = torch.cuda.Stream()
    out = torch.empty_like(x.q)
    torch.cuda.synchronize()
    dirty_memory()
    if how == "current":
        with torch.cuda.stream(side):
            x(out=out)
    else:
        x(out=out, stream=side if how == "object" else side.cuda_stream)
    assert x.good(out)
    assert x.good(x())  # and on the first stream, by now


@pytest.mark.parametrize("new", [1, 150])
def test_calls_on_several_streams_at_once(new):
    x = Problem(new, 64, 2)
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [torch.empty_like(x.q) for _ in range(32)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        x(out=out, stream=streams[i % 4])
    assert all(x.good(out) for out in outs)


@pytest.mark.parametrize("warm", [False, True])
def test_a_captured_decode_step_outlives_larger_calls(warm):
    step, prompt = Problem(1, 64, 3), Problem(150, 128, 4)
    if warm:
        assert step.good(step())
    out = torch.empty_like(step.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            step(out=out)
    for _ in range(3):
        assert prompt.good(prompt())
        dirty_memory()
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        assert step.good(out)


@pytest.mark.parametrize("new", [1, 150])
def test_calls_before_the_first_replay_and_a_capture_of_two_shapes(new):
    x, y = Problem(new, 64, 5), Problem(200, 128, 6)
    torch.cuda.synchronize()
    dirty_memory()
    torch.cuda.synchronize()
    out, out2 = torch.empty_like(x.q), torch.empty_like(y.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x(out=out)
        y(out=out2)
        x(out=out)
    assert x.good(x()) and y.good(y())
    for _ in range(3):
        out.zero_(), out2.zero_()
        graph.replay()
        assert x.good(out) and y.good(out2)


def test_replays_beside_calls_on_the_capturing_stream():
    x = Problem(150, 128, 7)
    side = torch.cuda.Stream()
    outs = [torch.empty_like(x.q) for _ in range(12)]
    out = torch.empty_like(x.q)
    x(out=out, stream=side)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        for o in outs[:6]:
            x(out=o)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    graph.replay()
    for o in outs[6:]:
        x(out=o, stream=side)
    assert all(x.good(o) for o in outs)


def test_a_workspace_needs_no_more_zeros_than_it_says():
    x = Problem(150, 128, 8)
    need = pkv.paged_attention_workspace_bytes(2, 151, 150, 4, 2, 128)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    ws[:pkv.PKV_ATTENTION_ZERO_BYTES] = 0
    for _ in range(3):
        assert x.good(x(workspace=ws))
    assert not ws[:pkv.PKV_ATTENTION_ZERO_BYTES].any()


@pytest.mark.parametrize("how", ["object", "handle"])
def test_outputs_are_the_call_streams_memory(how):
    """Memory that the current stream has freed and has yet to write is not taken for the
    output of a call on another stream."""
    x = Problem(150, 128, 9)
    n, hkv, d = 151, 2, 128
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    loc = pos.clone()
    cache = pkv.KVCache.empty(40, 16, hkv, d)
    k = torch.zeros(n, hkv, d, dtype=x.q.dtype, device=DEV)
    side = torch.cuda.Stream()
    stream = side if how == "object" else side.cuda_stream
    torch.cuda.synchronize()
    for call, want in ((lambda: x(stream=stream), x.want),
                       (lambda: pkv.append_kv(cache, k, k, pos, loc, q=x.q, stream=stream), x.q)):
        late = torch.empty_like(x.q)
        torch.cuda._sleep(20_000_000)
        late.fill_(7.0)
        del late
        out = call()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
