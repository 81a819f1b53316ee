"""Argument checks of the norm's C entry points: refused on the host, before any launch (no GPU needed)."""
import ctypes

import pytest

from unpermute_ep_dispatch_gb300 import _binding, build

INVALID, UNSUPPORTED, OK = _binding.EPD_ERR_INVALID_ARG, _binding.EPD_ERR_UNSUPPORTED, _binding.EPD_OK
FAKE = ctypes.c_void_p(0x10000)        # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10004)         # 4-aligned, not 16-aligned


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _binding.load_library()


def test_norm_rejects_bad_args(lib):
    ok = dict(x=FAKE, dt=0, r=None, w=None, b=None, T=4, H=256, eps=1e-5, kind=0, sum=None, y=FAKE, q=None, qs=None,
              mean=None, rstd=None, s=None)
    call = lambda **kw: lib.ep_layer_norm(*dict(ok, **kw).values())  # noqa: E731
    for kw in (dict(dt=1), dict(dt=9), dict(kind=2), dict(T=-1), dict(H=0), dict(H=252), dict(eps=-1.0),
               dict(eps=float("nan")), dict(x=None), dict(y=None), dict(q=FAKE), dict(qs=FAKE),
               dict(q=FAKE, qs=FAKE, H=136), dict(sum=FAKE), dict(x=ODD), dict(y=ODD), dict(r=ODD), dict(w=ODD),
               dict(b=ODD), dict(r=FAKE, sum=ODD), dict(q=ODD, qs=FAKE), dict(mean=ctypes.c_void_p(0x10002)),
               dict(rstd=ctypes.c_void_p(0x10002))):
        assert call(**kw) == INVALID, kw
    assert call(H=16392) == UNSUPPORTED
    assert call(T=0, x=None, y=None) == OK


def test_norm_backward_rejects_bad_args(lib):
    ok = dict(dy=FAKE, x=FAKE, dt=0, w=None, mean=FAKE, rstd=FAKE, gs=None, T=4, H=256, kind=0, ws=FAKE, dx=FAKE,
              dw=FAKE, db=None, s=None)
    call = lambda **kw: lib.ep_layer_norm_backward(*dict(ok, **kw).values())  # noqa: E731
    for kw in (dict(dt=1), dict(kind=-1), dict(T=-1), dict(H=12), dict(dy=None), dict(x=None), dict(mean=None),
               dict(rstd=None), dict(dx=None), dict(ws=None), dict(dy=ODD), dict(x=ODD), dict(gs=ODD), dict(dx=ODD),
               dict(dw=ODD), dict(db=ODD), dict(w=ODD), dict(ws=ODD), dict(mean=ctypes.c_void_p(0x10002))):
        assert call(**kw) == INVALID, kw
    assert call(H=16392) == UNSUPPORTED
    assert call(T=0, dy=None, x=None, mean=None, rstd=None, dx=None, dw=None, ws=None) == OK


def test_norm_workspace_holds_every_block(lib):
    for H in (8, 1000, 1032, 7168, 8192, 8200, 16384):
        n = lib.epd_norm_workspace_bytes(H)
        assert n >= 152 * 2 * H * 4 and n % 16 == 0
    assert [lib.epd_norm_workspace_bytes(H) for H in (0, -8, 12, 16392)] == [0] * 4
