"""Argument checks of the rotary positions' and the cache's C entry points: refused on the host,
before any launch (no GPU needed)."""
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


def cache(dt=0, KH=2, D=64, page=16, P=4, k=0x10000, v=0x10000, ks=None, vs=None, sp=2048, st=128, sh=64, cp=0, ct=0,
          ch=0, table=0x10000, S=4, M=3, ts=3):
    return ctypes.byref(_binding.KVCache(dt, KH, D, page, P, k, v, ks, vs, sp, st, sh, cp, ct, ch, table, S, M, ts))


BAD_CACHES = [dict(dt=2), dict(KH=0), dict(D=0), dict(D=60), dict(page=0), dict(P=-1), dict(P=1 << 31), dict(k=None),
              dict(v=None), dict(k=0x10004), dict(v=0x10008), dict(ks=0x10000), dict(vs=0x10000), dict(sp=-8),
              dict(st=4), dict(sh=12), dict(table=None), dict(table=0x10002), dict(S=-1), dict(M=-1), dict(ts=2),
              dict(page=1 << 30, M=2, ts=2), dict(dt=1), dict(dt=1, ks=0x10000, vs=0x10000, D=72),
              dict(dt=1, ks=0x10000, vs=0x10000, sh=72), dict(dt=1, ks=0x10002, vs=0x10000)]


def test_rotary_rejects_bad_args(lib):
    ok = dict(x=FAKE, ts=128, hs=64, pos=FAKE, steps=FAKE, T=4, N=2, D=64, R=64, inter=0, scale=1.0, inv=0, out=FAKE,
              ots=128, ohs=64, s=None)
    call = lambda **kw: lib.ep_rotary(*dict(ok, **kw).values())  # noqa: E731
    for kw in (dict(T=-1), dict(N=-1), dict(D=0), dict(D=60), dict(R=0), dict(R=3), dict(R=66), dict(R=-2), dict(x=None),
               dict(out=None), dict(pos=None), dict(steps=None), dict(x=ODD), dict(out=ODD), dict(ts=4), dict(hs=-8),
               dict(ots=12), dict(ohs=4), dict(scale=float("nan")), dict(pos=ctypes.c_void_p(0x10002)), dict(steps=ODD)):
        assert call(**kw) == INVALID, kw
    assert call(D=264, R=64) == UNSUPPORTED
    assert call(T=0, x=None, out=None, pos=None) == OK
    assert call(N=0, x=None, out=None) == OK


def test_append_rejects_bad_args(lib):
    ok = dict(c=cache(), q=None, qs=0, QH=0, k=FAKE, ks=128, v=FAKE, vs=128, pos=FAKE, seq=None, T=4, steps=None, R=0,
              inter=0, scale=1.0, qo=None, qos=0, st=FAKE, s=None)
    call = lambda **kw: lib.ep_cache_append(*dict(ok, **kw).values())  # noqa: E731
    for kw in ([dict(c=cache(**b)) for b in BAD_CACHES] + [
            dict(c=None), dict(T=-1), dict(T=5), dict(QH=-1), dict(k=None), dict(v=None), dict(k=ODD), dict(v=ODD),
            dict(ks=4), dict(vs=-8), dict(pos=None), dict(pos=ctypes.c_void_p(0x10002)), dict(st=None), dict(R=64),
            dict(R=3, steps=FAKE), dict(R=66, steps=FAKE), dict(q=FAKE, QH=4, qs=256), dict(q=ODD, QH=4, qs=256, qo=FAKE),
            dict(q=FAKE, QH=4, qs=12, qo=FAKE), dict(seq=ctypes.c_void_p(0x10002))]):
        assert call(**kw) == INVALID, kw
    assert call(c=cache(D=264)) == UNSUPPORTED
    assert call(T=0, k=None, v=None, pos=None) == OK


def test_attention_rejects_bad_args(lib):
    ok = dict(c=cache(), q=FAKE, qs=256, QH=4, lens=FAKE, scale=0.1, window=0, ws=FAKE, out=FAKE, lse=None, st=FAKE,
              s=None)
    call = lambda **kw: lib.ep_decode_attention(*dict(ok, **kw).values())  # noqa: E731
    for kw in ([dict(c=cache(**b)) for b in BAD_CACHES] + [
            dict(c=None), dict(q=None), dict(q=ODD), dict(qs=12), dict(qs=-8), dict(QH=0), dict(QH=3), dict(lens=None),
            dict(lens=ctypes.c_void_p(0x10002)), dict(scale=float("nan")), dict(window=-1), dict(ws=None), dict(ws=ODD),
            dict(out=None), dict(out=ODD), dict(lse=ctypes.c_void_p(0x10002)), dict(st=None)]):
        assert call(**kw) == INVALID, kw
    assert call(c=cache(D=264)) == UNSUPPORTED
    assert call(c=cache(S=0), q=None, out=None, lens=None, ws=None) == OK


def test_attention_workspace_bytes(lib):
    f = lib.epd_attention_workspace_bytes
    assert f(4, 32, 8, 128) >= 152 * 4 + 152 * 2 * 16 * 130 * 4
    assert f(4, 32, 8, 256) > f(4, 32, 8, 128) > f(4, 32, 8, 64) > 0
    for bad in ((-1, 32, 8, 128), (4, 0, 8, 128), (4, 32, 0, 128), (4, 32, 5, 128), (4, 32, 8, 0), (4, 32, 8, 100), (4, 32, 8, 264)):
        assert f(*bad) == 0


def test_shared_rows(lib):
    """A table's row may serve all sequences; what is written lies apart."""
    append = dict(c=cache(), q=None, qs=0, QH=0, k=FAKE, ks=128, v=FAKE, vs=128, pos=FAKE, seq=FAKE, T=0, steps=None, R=0,
                  inter=0, scale=1.0, qo=None, qos=0, st=FAKE, s=None)
    call = lambda **kw: lib.ep_cache_append(*dict(append, **kw).values())  # noqa: E731
    assert call(c=cache(ts=0)) == OK
    fp8 = dict(dt=1, ks=0x10000, vs=0x10000, cp=32, ct=2, ch=1)
    assert call(c=cache(**fp8)) == OK
    for kw in (dict(sp=0), dict(st=0), dict(sh=0), dict(fp8, cp=0), dict(fp8, ct=0), dict(fp8, ch=0), dict(fp8, sh=0)):
        assert call(c=cache(**kw)) == INVALID, kw
    assert call(c=cache(sp=0, st=0, sh=0, P=1, page=1, KH=1)) == OK
    assert call(q=FAKE, QH=4, qs=256, qo=FAKE, qos=0, T=2) == INVALID
    rotary = dict(x=FAKE, ts=128, hs=64, pos=FAKE, steps=FAKE, T=4, N=2, D=64, R=64, inter=0, scale=1.0, inv=0, out=FAKE,
                  ots=0, ohs=64, s=None)
    assert lib.ep_rotary(*rotary.values()) == INVALID
    assert lib.ep_rotary(*dict(rotary, ots=128, ohs=0).values()) == INVALID
    # reading is not writing: heads that share their rows
    attention = dict(c=cache(S=0, sh=0, ts=0), q=None, qs=256, QH=4, lens=None, scale=0.1, window=0, ws=None, out=None, lse=None,
                     st=FAKE, s=None)
    assert lib.ep_decode_attention(*attention.values()) == OK


def test_frequencies_refuse_what_has_no_blend():
    """The blend's ends are logarithms to the base of turns over the original length."""
    f = _binding.rotary_frequencies
    for bad in (dict(base=1.0), dict(base=0.5), dict(beta_fast=0.0), dict(beta_slow=0.0), dict(beta_slow=-1.0), dict(original_length=0),
                dict(base=float("nan")), dict(base=float("inf")), dict(factor=float("inf")), dict(beta_fast=0.5)):
        with pytest.raises(ValueError):
            f(64, **{**dict(scaling="yarn", factor=4.0), **bad})
    for bad in (dict(base=float("inf")), dict(factor=float("inf"), scaling="linear"), dict(factor=float("inf"), scaling="ntk")):
        with pytest.raises(ValueError):
            f(64, **bad)
    assert float(f(64, base=0.5)[0][0]) == 1.0  # (without a blend any positive base does)
