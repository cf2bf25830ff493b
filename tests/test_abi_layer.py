"""Host-side checks of the calls around an attention layer (no GPU needed):
bad arguments are refused before any launch."""
import ctypes
import math
import os

import pytest

from exact_second_order_gb300 import flashbob as fb

INVALID, UNSUPPORTED, MISALIGNED = (fb.FLASHBOB_ERR_INVALID_ARG, fb.FLASHBOB_ERR_UNSUPPORTED,
                                    fb.FLASHBOB_ERR_MISALIGNED)
BIG = 1 << 40


@pytest.fixture(scope="session")
def lib():
    if not os.path.exists(fb.LIB_PATH):
        from exact_second_order_gb300.build import build
        build()
    return fb.load_library()


def ptrs(n, stride=1 << 24, base=1 << 36):
    # distinct, 16-byte aligned addresses, never dereferenced
    return [base + i * stride for i in range(n)]


def each_bad_pointer(call, n, optional):
    ok = ptrs(n)
    for i in range(n):
        p = list(ok)
        p[i] += 4
        assert call(p) == MISALIGNED, i
        if i not in optional:
            p[i] = None
            assert call(p) == INVALID, i


def attention(lib, p, tau=0.1, cap=0.0, ws=BIG, B=1, H=2, Hkv=1, Nq=8, Nk=4096, d=64, causal=0,
              dtype=1):
    return lib.flashbob_attention(*p[:6], tau, cap, p[6], p[7], p[8], ws, B, H, Hkv, Nq, Nk, d,
                                  causal, dtype, None)


def grad(lib, p, tau=0.1, cap=0.0, ws=BIG, B=1, H=2, Hkv=1, Nq=8, Nk=8, d=64, causal=0, dtype=1):
    return lib.flashbob_attention_grad(*p[:9], tau, cap, *p[9:13], ws, B, H, Hkv, Nq, Nk, d, causal,
                                       dtype, None)


BAD_SIZES = [dict(B=0), dict(H=-1), dict(Hkv=0), dict(Nq=0), dict(Nk=0), dict(d=0), dict(H=3, Hkv=2),
             dict(tau=0.0), dict(tau=math.nan), dict(tau=math.inf), dict(cap=-1.0),
             dict(cap=math.nan), dict(cap=math.inf), dict(causal=2), dict(dtype=5),
             dict(tau=1e-42), dict(cap=1e-42), dict(tau=1e37), dict(cap=1e37),
             dict(tau=1e-20, cap=1e20)]
TOO_LARGE = [dict(d=129), dict(B=70000), dict(H=65535, Nq=2 ** 20), dict(Nk=2 ** 31 - 1000)]


def test_attention_refuses(lib):
    each_bad_pointer(lambda p: attention(lib, p), 9, optional=(3, 4, 5))
    each_bad_pointer(lambda p: grad(lib, p), 13, optional=(6, 7, 8))
    for call, n in ((attention, 9), (grad, 13)):
        for kw in BAD_SIZES:
            assert call(lib, ptrs(n), **kw) == INVALID, kw
        for kw in TOO_LARGE:
            assert call(lib, ptrs(n), **kw) == UNSUPPORTED, kw
        assert call(lib, ptrs(n), ws=64) == INVALID
    for i in (6, 7, 8):  # an output on an input
        p = ptrs(9)
        p[i] = p[1] + 4096
        assert attention(lib, p) == INVALID
    for i in (9, 10, 11, 12):  # outputs on each other
        p = ptrs(13)
        p[i] = p[9 if i > 9 else 10]
        assert grad(lib, p) == INVALID


def test_attention_workspace(lib):
    # Many rows need none forward; few rows over a long cache do.
    assert fb.flashbob_attention_workspace(1, 8, 8, 16384, 16384, 64, 1)[0] == 0
    one = fb.flashbob_attention_workspace(1, 8, 1, 1, 65536, 128, 1)[0]
    assert one >= 8 * 128 * 4
    assert fb.flashbob_attention_workspace(2, 8, 4, 100, 100, 80, 0)[1] >= 2 * 8 * 100 * 24
    with pytest.raises(fb.FlashbobError):
        fb.flashbob_attention_workspace(1, 3, 2, 1, 1, 64, 1)
    n = ctypes.c_size_t()
    assert lib.flashbob_attention_workspace(1, 1, 1, 1, 1, 64, 1, None, ctypes.byref(n)) == 0


def test_ranges_refuse(lib):
    def call(p, B=2, M=3, Nq=8, Nk=8, causal=1):
        return lib.flashbob_attention_ranges(*p, B, M, Nq, Nk, causal, None)

    each_bad_pointer(call, 5, optional=(0, 1, 2, 4))
    for kw in (dict(B=0), dict(M=0), dict(M=-1), dict(Nq=0), dict(Nk=0), dict(causal=3)):
        assert call(ptrs(5), **kw) == INVALID, kw
    assert call(ptrs(5), B=70000) == UNSUPPORTED
    p = ptrs(5)
    p[0] = None  # documents counted, or with prefixes, but not given
    assert call(p) == INVALID
    assert call(p, M=0) == INVALID
    p = ptrs(5)
    p[4] = p[3]
    assert call(p) == INVALID


def test_norm_refuses(lib):
    def call(p, eps=1e-6, B=2, N=8, H=4, Hkv=2, Nk=8, d=64, R=64, axes=1, inter=0, dtype=1):
        return lib.flashbob_qk_norm_rope(*p[:6], eps, *p[6:9], B, N, H, Hkv, Nk, d, R, axes, inter,
                                         dtype, None)

    def back(p, eps=1e-6, ws=BIG, B=2, N=8, H=4, Hkv=2, d=64, R=64, axes=1, inter=0, dtype=1,
             gtype=0):
        return lib.flashbob_qk_norm_rope_grad(*p[:5], eps, *p[5:12], ws, B, N, H, Hkv, d, R, axes,
                                              inter, dtype, gtype, None)

    each_bad_pointer(call, 9, optional=(4, 5))
    each_bad_pointer(back, 12, optional=(4,))
    for f, n in ((call, 9), (back, 12)):
        for kw in (dict(B=0), dict(N=0), dict(H=0), dict(Hkv=0), dict(d=0), dict(R=-2), dict(R=3),
                   dict(R=66), dict(axes=0), dict(inter=2), dict(dtype=4), dict(eps=0.0),
                   dict(eps=math.nan), dict(eps=math.inf)):
            assert f(ptrs(n), **kw) == INVALID, kw
        for kw in (dict(d=130, R=64), dict(axes=5), dict(H=70000), dict(Hkv=70000),
                   dict(B=65536, N=65536)):
            assert f(ptrs(n), **kw) == UNSUPPORTED, kw
        p = ptrs(n)
        p[4] = None  # no positions: one axis only
        assert f(p, axes=2) == INVALID
        p = ptrs(n)
        p[1] = None  # one gain without the other
        assert f(p) == INVALID
    p = ptrs(9)
    p[5] = None  # no rows given, and fewer rows than tokens
    assert call(p, Nk=7) == INVALID
    p = ptrs(9)
    p[8] = p[7]
    assert call(p) == INVALID
    assert back(ptrs(12), ws=64) == INVALID
    assert back(ptrs(12), gtype=2) == INVALID
    p = ptrs(12)
    p[1] = p[2] = None  # gradients of gains that are not there
    assert back(p) == INVALID
