"""Calls of the C interface whose tensors start 16 bytes into an allocation, as far
aligned as the header asks, give the bits of calls on fresh ones."""
import itertools

import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests import paged_reference as pag

pytestmark = pytest.mark.gpu

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
CODE = {F32: fb.FLASHBOB_F32, BF: fb.FLASHBOB_BF16, E4M3: fb.FLASHBOB_E4M3}


def shifted(t, shift):
    """A copy of t whose address is `shift` modulo 256."""
    n = t.numel() * t.element_size()
    out = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    at = (shift - out.data_ptr()) % 256
    out = out[at:at + n].view(t.dtype).view(t.shape)
    out.view(torch.uint8).copy_(t.contiguous().view(torch.uint8))
    assert out.data_ptr() % 256 == shift
    return out


def ptr(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("dtype,cache", [(BF, E4M3), (F32, E4M3), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("d", [16, 64, 80, 128])
def test_read(dtype, cache, d):
    B, Hkv, M, T, Nk = 2, 3, 5, 16, 77
    pools, values = pag.pools(B * M, Hkv, T, d, cache)
    table = pag.table_of(B, M, B * M)
    want = [pag.dense(x, table)[:, :, :Nk] for x in values]
    for at in itertools.product((0, 16, 32, 48), repeat=2):
        out = [shifted(torch.zeros((B, Hkv, Nk, d), dtype=dtype, device="cuda"), s) for s in at]
        p = [x if x is None else shifted(x, 16) for x in pools]
        st = fb.load_library().flashbob_cache_read(
            *(ptr(x) for x in p), table.data_ptr(), None, *(ptr(x) for x in out), B, Hkv, B * M, T, M, Nk, d,
            CODE[cache], CODE[dtype], torch.cuda.current_stream().cuda_stream)
        assert st == fb.FLASHBOB_OK
        for x, w in zip(out, want):
            assert torch.equal(x.double(), w), at


@pytest.mark.parametrize("cache", [E4M3, BF])
@pytest.mark.parametrize("d,R,N", [(64, 64, 20), (128, 128, 200), (80, 60, 33), (128, 64, 1)])
def test_append(cache, d, R, N):
    B, H, Hkv, T, M = 2, 4, 2, 32, 9
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((B, N, H + 2 * Hkv, d), generator=g, device="cuda").to(BF)
    gains = 1 + torch.rand((2, d), generator=g, device="cuda")
    freqs = torch.rand((1, R // 2), generator=g, device="cuda")
    start = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    pools, _ = pag.pools(B * M, Hkv, T, d, cache)
    table = pag.table_of(B, M, B * M)
    results = []
    for s in (0, 16):
        p = [t if t is None else shifted(t, s) for t in pools]
        Q = shifted(torch.zeros((B, H, N, d), dtype=BF, device="cuda"), s)
        *ins, first = [shifted(t, s) for t in (x, gains[0], gains[1], freqs, start)]
        st = fb.load_library().flashbob_cache_append(
            *(ptr(t) for t in ins), None, ptr(first), None, table.data_ptr(), 1e-5, ptr(Q),
            *(ptr(t) for t in p), B, N, H, Hkv, B * M, T, M, d, R, 1, 0, CODE[BF], CODE[cache],
            torch.cuda.current_stream().cuda_stream)
        assert st == fb.FLASHBOB_OK
        torch.cuda.synchronize()
        results.append([Q] + [t for t in p if t is not None])
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("cache", [E4M3, BF])
@pytest.mark.parametrize("d,H,Nq", [(64, 4, 1), (128, 8, 1), (128, 4, 60), (64, 4, 200), (96, 4, 3)])
def test_attention(cache, d, H, Nq):
    B, Hkv, T, M = 2, 2, 64, 30
    pools, _ = pag.pools(B * M, Hkv, T, d, cache)
    table = pag.table_of(B, M, B * M)
    Q = torch.randn((B, H, Nq, d), device="cuda").to(BF)
    need = fb.flashbob_attention_paged_workspace(B, H, Hkv, Nq, T, M, d, CODE[BF], CODE[cache])
    results = []
    for s in (0, 16):
        p, q = [t if t is None else shifted(t, s) for t in pools], shifted(Q, s)
        O = shifted(torch.zeros_like(Q), s)
        L = shifted(torch.zeros((B, H, Nq), device="cuda"), s)
        w = shifted(torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda"), s)
        st = fb.load_library().flashbob_attention_paged(
            ptr(q), *(ptr(t) for t in p), table.data_ptr(), None, None, None, 0.1, 0.0, ptr(O), ptr(L),
            ptr(w), need, B, H, Hkv, Nq, B * M, T, M, d, 0, CODE[BF], CODE[cache],
            torch.cuda.current_stream().cuda_stream)
        assert st == fb.FLASHBOB_OK
        torch.cuda.synchronize()
        results.append((O, L))
    for a, b in zip(*results):
        assert torch.equal(a, b)
