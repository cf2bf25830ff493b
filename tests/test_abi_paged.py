"""Host-side checks of the calls on a paged cache (no GPU needed): bad arguments are
refused before any launch."""
import math
import os

import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests.test_abi_layer import BIG, INVALID, UNSUPPORTED, each_bad_pointer, ptrs


@pytest.fixture(scope="session")
def lib():
    if not os.path.exists(fb.LIB_PATH):
        from exact_second_order_gb300.build import build
        build()
    return fb.load_library()


def append(lib, p, eps=0.0, B=2, N=8, H=4, Hkv=2, P=9, T=16, M=4, d=64, R=64, axes=1, inter=0, dtype=1, cache=2):
    return lib.flashbob_cache_append(*p[:8], eps, *p[8:13], B, N, H, Hkv, P, T, M, d, R, axes, inter, dtype, cache, None)


def bare(lib, p, **kw):  # no gains, which need a norm
    return append(lib, p[:1] + [None, None] + p[3:], **kw)


def read(lib, p, B=2, Hkv=2, P=9, T=16, M=4, Nk=64, d=64, cache=2, dtype=1):
    return lib.flashbob_cache_read(*p, B, Hkv, P, T, M, Nk, d, cache, dtype, None)


def attention(lib, p, tau=0.1, cap=0.0, ws=BIG, B=1, H=2, Hkv=1, Nq=8, P=99, T=16, M=3000, d=64, causal=0, dtype=1, cache=2):
    return lib.flashbob_attention_paged(*p[:9], tau, cap, p[9], p[10], p[11], ws, B, H, Hkv, Nq, P, T, M, d, causal, dtype, cache,
                                        None)


BAD_PAGES = [dict(P=0), dict(T=0), dict(T=-16), dict(M=0), dict(d=0), dict(B=0), dict(Hkv=0), dict(dtype=2), dict(dtype=5), dict(cache=0),
             dict(cache=3), dict(dtype=0, cache=1)]
TOO_LARGE = [dict(P=2 ** 30, Hkv=2, H=2), dict(T=8), dict(T=48), dict(T=256), dict(T=2 ** 31 - 1), dict(M=2 ** 27), dict(d=129)]


def test_append_refuses(lib):
    each_bad_pointer(lambda p: append(lib, p, eps=1e-6), 13, optional=(4, 5, 6))
    for kw in BAD_PAGES + [dict(N=0), dict(H=0), dict(R=-2), dict(R=3), dict(R=66), dict(axes=0), dict(inter=2), dict(eps=-1.0),
                           dict(eps=math.nan), dict(eps=math.inf)]:
        assert bare(lib, ptrs(13), **kw) == INVALID, kw
    for kw in TOO_LARGE + [dict(axes=5), dict(H=70000), dict(Hkv=70000), dict(B=65535, N=65536), dict(N=2 ** 31 - 1, B=1)]:
        assert bare(lib, ptrs(13), **kw) == UNSUPPORTED, kw
    assert append(lib, ptrs(13)) == INVALID  # gains without a norm
    p = ptrs(13)
    p[1] = None  # one gain without the other
    assert append(lib, p, eps=1e-6) == INVALID
    p = ptrs(13)
    p[4] = None  # no positions: one axis only
    assert bare(lib, p, axes=2) == INVALID
    p = ptrs(13)
    p[3] = None  # nothing to turn by
    assert bare(lib, p) == INVALID
    assert bare(lib, ptrs(13), cache=1) == INVALID  # scales of a cache that has none
    for i, j in ((8, 0), (9, 0), (9, 7), (10, 9), (11, 12), (11, 9), (12, 8)):
        p = ptrs(13)
        p[i] = p[j]
        assert bare(lib, p) == INVALID, (i, j)


def test_read_refuses(lib):
    each_bad_pointer(lambda p: read(lib, p), 8, optional=(5,))
    for kw in BAD_PAGES + [dict(Nk=0), dict(Nk=65)]:
        assert read(lib, ptrs(8), **kw) == INVALID, kw
    for kw in TOO_LARGE + [dict(Hkv=70000), dict(B=70000)]:
        kw = {k: v for k, v in kw.items() if k != "H"}
        assert read(lib, ptrs(8), **kw) == UNSUPPORTED, kw
    assert read(lib, ptrs(8), cache=1) == INVALID
    for i, j in ((6, 0), (7, 1), (7, 6), (6, 4)):
        p = ptrs(8)
        p[i] = p[j]
        assert read(lib, p) == INVALID, (i, j)


def test_attention_refuses(lib):
    each_bad_pointer(lambda p: attention(lib, p), 12, optional=(6, 7, 8))
    for kw in BAD_PAGES + [dict(H=-1), dict(Nq=0), dict(H=3, Hkv=2), dict(tau=0.0), dict(tau=math.nan), dict(tau=math.inf), dict(cap=-1.0),
                           dict(cap=math.nan), dict(causal=2), dict(tau=1e-42), dict(tau=1e37), dict(tau=1e-20, cap=1e20)]:
        assert attention(lib, ptrs(12), **kw) == INVALID, kw
    for kw in TOO_LARGE + [dict(H=65535, Nq=2 ** 20), dict(B=70000)]:
        assert attention(lib, ptrs(12), **kw) == UNSUPPORTED, kw
    assert attention(lib, ptrs(12), ws=64) == INVALID
    assert attention(lib, ptrs(12), cache=1) == INVALID
    for i, j in ((9, 0), (9, 1), (10, 5), (11, 2), (11, 9)):
        p = ptrs(12)
        p[i] = p[j]
        assert attention(lib, p) == INVALID, (i, j)


def test_workspace(lib):
    # Many rows need none; few rows over a long cache do.
    assert fb.flashbob_attention_paged_workspace(1, 8, 8, 16384, 64, 256, 64, 1, 2) == 0
    assert fb.flashbob_attention_paged_workspace(1, 8, 1, 1, 64, 65536, 128, 1, 2) >= 8 * 128 * 4
    with pytest.raises(fb.FlashbobError):
        fb.flashbob_attention_paged_workspace(1, 3, 2, 1, 16, 4, 64, 1, 2)
    for at in range(7):
        sizes = [1, 1, 1, 8, 16, 8, 64]
        sizes[at] = 2 ** 32 + 5
        with pytest.raises(ValueError):
            fb.flashbob_attention_paged_workspace(*sizes, 1, 2)


def test_a_cache_is_of_cuda_tensors():
    x = torch.zeros((2, 1, 16, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fb.PagedCache(x, x)


@pytest.mark.gpu
def test_the_binding_refuses():
    E4M3, BF, F32, I = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32
    K, V = (torch.zeros((5, 2, 16, 64), dtype=E4M3, device="cuda") for _ in range(2))
    s = torch.ones((5, 2), device="cuda")
    cache = fb.PagedCache(K, V, s, s.clone())
    plain = fb.PagedCache(K.to(BF), V.to(BF))
    table = torch.zeros((3, 2), dtype=I, device="cuda")
    x = torch.zeros((3, 4, 8, 64), dtype=BF, device="cuda")
    Q = torch.zeros((3, 4, 1, 64), dtype=BF, device="cuda")
    bad = [
        (ValueError, lambda: fb.PagedCache(K, V)),
        (ValueError, lambda: fb.PagedCache(K, V, s)),
        (ValueError, lambda: fb.PagedCache(K, V[:4], s, s)),
        (TypeError, lambda: fb.PagedCache(K, V.to(BF), s, s)),
        (TypeError, lambda: fb.PagedCache(K, V, s.double(), s)),
        (TypeError, lambda: fb.PagedCache(K.to(torch.float16), V.to(torch.float16))),
        (ValueError, lambda: fb.PagedCache(K.to(BF), V.to(BF), s, s)),
        (ValueError, lambda: fb.PagedCache(K.transpose(0, 1), V, s, s)),
        (ValueError, lambda: fb.PagedCache.empty(4, 2, 48, 64)),
        (ValueError, lambda: fb.cache_append(x, 3, cache, table)),
        (ValueError, lambda: fb.cache_append(x, 0, cache, table)),
        (ValueError, lambda: fb.cache_append(x[..., :32].contiguous(), 4, cache, table)),
        (ValueError, lambda: fb.cache_append(x, 4, cache, table[:2])),
        (TypeError, lambda: fb.cache_append(x, 4, cache, table.long())),
        (TypeError, lambda: fb.cache_append(x.float(), 4, plain, table)),
        (TypeError, lambda: fb.cache_append(x, 4, (K, V), table)),
        (ValueError, lambda: fb.cache_append(x, 4, cache, table, wq=s[0], wk=s[0])),
        (ValueError, lambda: fb.cache_append(x, 4, cache, table, eps=0.0)),
        (TypeError, lambda: fb.cache_append(x, 4, cache, table, kv_start=torch.zeros(3, device="cuda"))),
        (ValueError, lambda: fb.cache_append(x, 4, cache, table, counts=torch.zeros(2, dtype=I, device="cuda"))),
        (ValueError, lambda: fb.cache_append(x, 4, cache, table.cpu())),
        (ValueError, lambda: fb.cache_read(cache, table, 33)),
        (ValueError, lambda: fb.cache_read(cache, table, 0)),
        (TypeError, lambda: fb.cache_read(cache, table, 8, dtype=torch.float16)),
        (TypeError, lambda: fb.cache_read(plain, table, 8, dtype=F32)),
        (ValueError, lambda: fb.cache_read(cache, table[0], 8)),
        (ValueError, lambda: fb.cache_read(cache, table.t(), 8)),
        (ValueError, lambda: fb.attention_paged(Q[..., :32].contiguous(), cache, table, 1.0)),
        (ValueError, lambda: fb.attention_paged(Q[:2], cache, table, 1.0)),
        (TypeError, lambda: fb.attention_paged(Q.float(), plain, table, 1.0)),
        (TypeError, lambda: fb.attention_paged(Q.half(), cache, table, 1.0)),
        (ValueError, lambda: fb.attention_paged(Q, cache, table, 1.0, ranges=table)),
        (ValueError, lambda: fb.attention_paged(Q, cache, table, 1.0, slopes=s[0])),
        (ValueError, lambda: fb.attention_paged(Q[:, ::2], cache, table, 1.0)),
        (fb.FlashbobError, lambda: fb.attention_paged(Q[:, :3].contiguous(), cache, table, 1.0)),
        (fb.FlashbobError, lambda: fb.attention_paged(Q, cache, table, 0.0)),
    ]
    for k, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {k} was accepted")
    # A fp32 call on an 8-bit cache is fine.
    fb.attention_paged(Q.float(), cache, table, 1.0)
