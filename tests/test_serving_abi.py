"""CPU tests of what the serving operators refuse before any launch, through the
C ABI and through the Python binding."""

import ctypes

import pytest
import torch

from paged_kv_gb300 import pkv

D = ctypes.c_void_p(256)


def cache(**kw):
    a = dict(k=256, v=256, k_scale=256, v_scale=256, num_pages=8, page_stride=4 * 2 * 64,
             token_stride=64, head_stride=4 * 64, page_size=4, kv_heads=2, head_dim=64, reserved=0)
    a.update(kw)
    return pkv._KVCacheStruct(*(a[f[0]] for f in pkv._KVCacheStruct._fields_))


BAD_CACHES = [
    dict(k=None), dict(v_scale=None), dict(k=264), dict(page_size=0), dict(num_pages=0),
    dict(num_pages=1 << 30), dict(kv_heads=0), dict(head_dim=0), dict(head_dim=24),
    dict(head_dim=144), dict(page_stride=8), dict(token_stride=-16), dict(head_stride=1 << 46),
]


def append(**kw):
    a = dict(cache=cache(), k=D, kts=256, khs=64, v=D, vts=256, vhs=64, dt=1, n=3, total=None,
             pos=D, loc=D, cs=D, max_pos=100, rot=64, inter=0, q=D, qts=256, qhs=64, hq=4, qo=D,
             ots=256, ohs=64)
    a.update(kw)
    c = a.pop("cache")
    return pkv.load().pkv_append_kv(ctypes.byref(c) if c is not None else None, *a.values(), None,
                                    None)


def attend(**kw):
    a = dict(cache=cache(), q=D, qts=256, qhs=64, hq=4, dt=1, n=3, out=D, ots=256, ohs=64,
             lse=None, cached=D, device=D, table=D, begin=None, B=2, max_q=2, pt=D, ptr=4, ptc=64,
             scale=0.1, window=0, status=None, ws=D, wsb=1 << 30)
    a.update(kw)
    c = a.pop("cache")
    return pkv.load().pkv_paged_attention(ctypes.byref(c) if c is not None else None, *a.values(),
                                          None)


def adjust(**kw):
    a = dict(x=D, stride=100, dt=0, B=2, V=100, out=ctypes.c_void_p(1 << 20), ostride=100, pool=D,
             pr=4, pc=16, table=D, prompt=D, device=D, rep=D, pres=None, freq=None, ptr=D, ids=D,
             vals=D, nb=3, mask=D, mstride=4)
    a.update(kw)
    return pkv.load().pkv_adjust_logits(*a.values(), None, None)


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(bad):
    for f in (append, attend):
        assert f(cache=cache(**bad)) == pkv.PKV_EINVAL
        assert pkv.last_error() != ""
    assert append(cache=None) == attend(cache=None) == pkv.PKV_EINVAL


@pytest.mark.parametrize("bad", [
    dict(dt=0), dict(dt=7), dict(n=-1), dict(n=1 << 31), dict(rot=4), dict(rot=72), dict(rot=-8),
    dict(cs=None), dict(max_pos=0), dict(cs=ctypes.c_void_p(260)), dict(pos=None), dict(loc=None),
    dict(k=None), dict(v=None), dict(k=ctypes.c_void_p(258)), dict(kts=260), dict(vhs=-64),
    dict(hq=0), dict(q=None), dict(qo=None), dict(qts=4), dict(ohs=63), dict(n=(1 << 31) - 1, hq=60000),
], ids=str)
def test_append_refusals(bad):
    assert append(**bad) == pkv.PKV_EINVAL
    assert pkv.last_error() != ""


def test_append_of_nothing():
    assert append(n=0) == pkv.PKV_OK and pkv.last_error() == ""


@pytest.mark.parametrize("bad", [
    dict(dt=0), dict(B=-1), dict(B=5000), dict(hq=3), dict(hq=0), dict(n=-1), dict(n=1 << 30),
    dict(max_q=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(out=None),
    dict(q=ctypes.c_void_p(264)), dict(qts=100), dict(ohs=-8), dict(cached=None), dict(device=None),
    dict(table=None), dict(pt=None), dict(ptr=0), dict(ptc=0), dict(ptc=(1 << 30) + 1),
    dict(ws=None), dict(wsb=100), dict(ws=ctypes.c_void_p(264)),
], ids=str)
def test_attention_refusals(bad):
    assert attend(**bad) == pkv.PKV_EINVAL
    assert pkv.last_error() != ""


def test_attention_of_nothing_and_its_workspace():
    assert attend(B=0) == pkv.PKV_OK and attend(n=0) == pkv.PKV_OK
    need = pkv.paged_attention_workspace_bytes
    assert need(4, 4, 1, 16, 8, 128) > 0
    assert need(5000, 4, 1, 16, 8, 128) == need(4, 4, 1, 15, 8, 128) == need(4, 4, 0, 16, 8, 128) == 0
    # The workspace that the call asks for is the one the function tells.
    n = need(2, 3, 2, 4, 2, 64)
    assert attend(wsb=n - 1) == pkv.PKV_EINVAL and str(n) in pkv.last_error()


@pytest.mark.parametrize("bad", [
    dict(dt=2), dict(B=-1), dict(B=65536), dict(V=0), dict(stride=99), dict(ostride=99),
    dict(x=None), dict(out=None), dict(out=D, ostride=200), dict(out=ctypes.c_void_p(256 + 16)),
    dict(pool=None), dict(table=None), dict(prompt=None), dict(device=None), dict(pr=0), dict(pc=0),
    dict(pc=1 << 30), dict(ptr=None), dict(ids=None), dict(vals=None), dict(nb=-1), dict(mstride=3),
], ids=str)
def test_adjust_refusals(bad):
    assert adjust(**bad) == pkv.PKV_EINVAL
    assert pkv.last_error() != ""


def test_adjust_limits():
    assert adjust(B=0) == pkv.PKV_OK
    assert adjust(V=300000, stride=300000, ostride=300000) == pkv.PKV_EUNSUPPORTED


def test_binding_refuses_wrong_tensors():
    f8 = torch.zeros(2, 4, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(2, 2)
    with pytest.raises(TypeError):
        pkv.KVCache(f8, f8, s, s)  # not on the GPU
    with pytest.raises(ValueError):
        pkv.adjust_logits(torch.zeros(2, 8))


class HostCache:
    """Stands in for a KVCache where a call is refused before any launch."""

    def __init__(self):
        self._struct = cache()
        self._ref, self._index = ctypes.addressof(self._struct), 0
        self.device = torch.device("cpu")


def test_binding_checks_every_tensor_before_the_call():
    c = HostCache()
    x, i = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for bad in (x, x.float(), 5, None):
        with pytest.raises(TypeError):
            pkv.append_kv(c, bad, x, i, i)
        with pytest.raises(TypeError):
            pkv.paged_attention(bad if isinstance(bad, torch.Tensor) else x, c, i, i, i, i, 1)
    with pytest.raises(TypeError):
        pkv._bind().append_kv(c._ref, 0)
