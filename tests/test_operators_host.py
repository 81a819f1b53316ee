"""Argument checks of the router's, the products' and the gradients' C entry points: all of
these are refused on the host, before any launch (no GPU needed)."""
import ctypes

import pytest

from unpermute_ep_dispatch_gb300 import _binding, build

INVALID = _binding.EPD_ERR_INVALID_ARG
FAKE = ctypes.c_void_p(0x10000)        # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10004)         # 4-aligned, not 16-aligned


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _binding.load_library()


def caller(fn, ok):
    return lambda **kw: fn(*dict(ok, **kw).values())


def test_route_rejects_bad_args(lib):
    call = caller(lib.ep_route, dict(l=FAKE, dt=2, bias=None, T=4, k=2, E=16, G=4, keep=2, gs=0, sc=0, re=1,
                                     scale=1.0, idx=FAKE, w=FAKE, st=FAKE, s=None))
    for kw in (dict(dt=1), dict(dt=9), dict(T=-1), dict(k=0), dict(k=17), dict(E=0), dict(E=4097), dict(G=3),
               dict(G=0), dict(keep=5), dict(keep=0), dict(gs=2), dict(sc=2), dict(l=None), dict(idx=None),
               dict(w=None), dict(st=None), dict(idx=ODD), dict(l=ctypes.c_void_p(0x10002)),
               dict(k=65, E=128), dict(T=1 << 30, k=4)):
        assert call(**kw) == INVALID, kw
    assert call(E=130, G=65, keep=1) == _binding.EPD_ERR_UNSUPPORTED
    assert call(T=0, l=None, idx=None, w=None) == _binding.EPD_OK


def test_route_backward_rejects_bad_args(lib):
    call = caller(lib.ep_route_backward, dict(g=FAKE, l=FAKE, dt=0, idx=FAKE, T=4, k=2, E=16, sc=1, re=0,
                                              scale=1.0, d=FAKE, st=FAKE, s=None))
    for kw in (dict(dt=1), dict(T=-1), dict(k=0), dict(k=65), dict(E=0), dict(sc=7), dict(g=None), dict(l=None),
               dict(idx=None), dict(d=None), dict(st=None), dict(idx=ODD)):
        assert call(**kw) == INVALID, kw
    assert call(T=0, g=None, l=None, idx=None, d=None) == _binding.EPD_OK


def rows(E=2, cap=16, rect=0, start=0x10000, count=0x10000):
    return ctypes.byref(_binding.ExpertRows(E, cap, rect, start, count))


BAD_ROWS = [dict(E=0), dict(E=5000), dict(cap=-1), dict(cap=1 << 31), dict(count=None), dict(count=0x10001),
            dict(start=0x10002), dict(start=None, rect=9), dict(start=None, rect=-1)]


def test_expert_matmul_rejects_bad_args(lib):
    call = caller(lib.ep_expert_matmul, dict(r=rows(), x=FAKE, dt=0, xs=None, a=0, b=0, c=0, w=FAKE, ws=None, K=64,
                                             N=32, act=0, bias=None, res=None, y=FAKE, pre=None, st=FAKE, s=None))
    for kw in ([dict(r=rows(**b)) for b in BAD_ROWS] + [
            dict(r=None), dict(dt=2), dict(dt=5), dict(K=60), dict(K=0), dict(N=20), dict(N=0), dict(act=5),
            dict(act=-1), dict(act=4, N=20), dict(x=None), dict(x=ODD), dict(w=None), dict(w=ODD), dict(y=None),
            dict(y=ODD), dict(res=ODD), dict(pre=ODD), dict(bias=ctypes.c_void_p(0x10002)), dict(st=None),
            dict(xs=FAKE), dict(ws=FAKE), dict(dt=1), dict(dt=1, xs=FAKE, K=128),
            dict(dt=1, xs=FAKE, ws=FAKE, K=64), dict(dt=1, xs=FAKE, ws=FAKE, K=128, act=4, N=64)]):
        assert call(**kw) == INVALID, kw
    assert call(r=rows(cap=0), x=None, y=None) == _binding.EPD_OK


def test_dgrad_rejects_bad_args(lib):
    call = caller(lib.ep_expert_matmul_dgrad, dict(r=rows(), dy=FAKE, w=FAKE, K=64, N=32, act=0, pre=None, dx=FAKE,
                                                   st=FAKE, s=None))
    for kw in ([dict(r=rows(**b)) for b in BAD_ROWS] + [
            dict(r=None), dict(K=60), dict(N=20), dict(act=9), dict(act=2), dict(pre=FAKE), dict(act=2, pre=ODD),
            dict(dy=None), dict(dy=ODD), dict(w=None), dict(w=ODD), dict(dx=None), dict(dx=ODD), dict(st=None)]):
        assert call(**kw) == INVALID, kw
    assert call(r=rows(cap=0), dy=None, dx=None) == _binding.EPD_OK


def test_wgrad_rejects_bad_args(lib):
    call = caller(lib.ep_expert_matmul_wgrad, dict(r=rows(), dy=FAKE, x=FAKE, K=64, N=32, dw=FAKE, db=None, st=FAKE,
                                                   s=None))
    for kw in ([dict(r=rows(**b)) for b in BAD_ROWS] + [
            dict(r=None), dict(K=60), dict(N=20), dict(dy=None), dict(dy=ODD), dict(x=None), dict(x=ODD),
            dict(dw=None), dict(dw=ODD), dict(db=ctypes.c_void_p(0x10002)), dict(st=None)]):
        assert call(**kw) == INVALID, kw


def test_unpermute_backward_rejects_bad_args(lib):
    call = caller(lib.ep_unpermute_backward, dict(gy=FAKE, eo=FAKE, cap=8, oi=FAKE, w=FAKE, T=4, k=2, H=64, geo=FAKE,
                                                  gw=FAKE, st=FAKE, s=None))
    for kw in (dict(H=60), dict(H=0), dict(T=-1), dict(k=65), dict(cap=-1), dict(cap=1 << 31), dict(gy=None),
               dict(gy=ODD), dict(eo=ODD), dict(eo=None), dict(geo=None), dict(geo=ODD), dict(oi=None), dict(w=None),
               dict(gw=None), dict(st=None)):
        assert call(**kw) == INVALID, kw
    assert call(T=0, gy=None, eo=None, oi=None, w=None, geo=None, gw=None) == _binding.EPD_OK


def test_new_status_code_has_a_name(lib):
    assert "logit" in _binding.status_string(_binding.EPD_ERR_NONFINITE)


def test_wgrad_rejects_features_beyond_half_of_32_bits(lib):
    call = caller(lib.ep_expert_matmul_wgrad, dict(r=rows(), dy=FAKE, x=FAKE, K=64, N=32, dw=FAKE, db=None, st=FAKE,
                                                   s=None))
    assert call(K=1 << 30) == _binding.EPD_ERR_UNSUPPORTED
    assert call(N=(1 << 31) - 8) == _binding.EPD_ERR_UNSUPPORTED
