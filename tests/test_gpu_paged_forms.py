"""The forms of the paged kernels that larger calls choose: prompts in blocks of 256 rows,
appends with two tokens a slot, heads that turn in part; each case says which form it
is meant for, and by how much it is beyond the rule that chooses it."""
import math

import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests import paged_reference as pag
from tests import test_gpu_paged_attention as attn
from tests import test_gpu_paged_cache as cache

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
SMS = 152

# 256 rows a block: at d = 128 from 114 such blocks on, at d = 64 with codes from 228 on
# (160 and more, 320 and more here).
# Groups of one head and of several; rows that fill the blocks and rows that do not; heads
# that straddle blocks and heads of whole blocks, whose blocks take turns; keys of a part of
# a tile, and of so many tiles that every ring goes round.
BLOCKS = [attn.case(*c) for c in (
    (4, 40, 40, 130, 3, 64, 128), (4, 40, 40, 256, 5, 16, 128), (10, 32, 16, 256, 4, 32, 128), (5, 48, 16, 111, 2, 128, 128),
    (2, 80, 80, 200, 19, 64, 128), (4, 40, 40, 130, 3, 64, 128, BF, BF), (10, 32, 16, 256, 4, 32, 128, BF, BF),
    (2, 80, 80, 200, 40, 16, 128, BF, BF), (8, 40, 40, 130, 3, 64, 64), (20, 32, 8, 129, 2, 128, 64),
    (10, 32, 16, 512, 9, 16, 64), (4, 80, 80, 200, 31, 32, 64))]


def blocks(c):
    rows = c["H"] // c["Hkv"] * c["Nq"]
    return c["B"] * c["Hkv"] * -(-rows // 256)


def test_the_cases_are_beyond_the_rule():
    for c in BLOCKS:
        assert c["H"] // c["Hkv"] * c["Nq"] > 128
        assert blocks(c) >= (1 if c["d"] == 128 else 2) * SMS, c
        assert c["d"] == 128 or c["cache"] is E4M3
    for c in attn.PROMPTS:  # and those are on its other side
        assert c["H"] // c["Hkv"] * c["Nq"] <= 128 or 2 * blocks(c) < SMS


# The reference of a case holds [B, H, Nq, Nk] numbers of 64 bits several times over.
@pytest.mark.gpu
@pytest.mark.parametrize("c", BLOCKS, ids=attn.name)
@pytest.mark.parametrize("mask", ["chunk", "window", "random", "none"])
def test_blocks_of_256_rows(c, mask):
    attn.check(c, mask=mask)


@pytest.mark.gpu
@pytest.mark.parametrize("c", [BLOCKS[i] for i in (0, 2, 3, 5, 6, 8, 10)], ids=attn.name)
@pytest.mark.parametrize("cap,bias", [(20.0, False), (0.0, True), (50.0, True), (0.3, False), (1e4, True)])
def test_blocks_of_256_rows_with_caps_and_biases(c, cap, bias):
    attn.check(c, cap=cap, bias=bias, seed=3)
    attn.check(c, cap=cap, bias=bias, mask="random", seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("c", [BLOCKS[i] for i in (1, 3, 5, 9)], ids=attn.name)
def test_blocks_of_256_rows_at_the_ends(c):
    attn.check(c, mask="one", seed=5)
    attn.check(c, mask="nothing", seed=5)
    attn.check(c, mask="none", seed=6, causal=True)
    attn.check(c, tau=4.0, seed=7)
    if c["cache"] is E4M3:
        attn.check(c, seed=8, spread=8.0, tau=1e-3)


@pytest.mark.gpu
@pytest.mark.parametrize("c", [BLOCKS[1], BLOCKS[6], BLOCKS[8]], ids=attn.name)
def test_blocks_of_256_rows_on_another_stream_and_replayed(c):
    attn.test_same_bits_on_another_stream_and_replayed(c)


# Two tokens a slot, from pages of 128 tokens and 65 new ones on; types of the cache and of
# the projection; halves of the whole head, heads that turn in part, neighbouring pairs;
# one eight of elements a lane (heads of up to 64) and two.
APPENDS = [  # B, N, H, Hkv, d, T, R, axes, interleaved, dtype, cache, norm
    (2, 200, 4, 2, 128, 128, 128, 1, False, BF, E4M3, False), (1, 300, 8, 2, 128, 128, 128, 1, False, BF, E4M3, True),
    (2, 200, 4, 2, 64, 128, 64, 1, False, BF, E4M3, True), (2, 200, 3, 1, 64, 128, 32, 1, False, BF, E4M3, False),
    (1, 150, 4, 2, 48, 128, 16, 1, False, BF, E4M3, True), (2, 200, 4, 2, 64, 128, 64, 1, True, BF, E4M3, False),
    (2, 200, 4, 2, 128, 128, 96, 1, True, BF, E4M3, True), (2, 200, 4, 2, 128, 128, 64, 2, False, BF, E4M3, False),
    (2, 200, 4, 2, 128, 128, 128, 1, False, BF, BF, False), (2, 200, 4, 2, 64, 128, 64, 1, False, BF, BF, True),
    (2, 200, 4, 2, 64, 128, 32, 1, False, BF, BF, False), (2, 200, 4, 2, 128, 128, 64, 1, False, BF, BF, True),
    (2, 200, 4, 2, 96, 128, 96, 1, True, BF, BF, False), (3, 20, 4, 2, 64, 32, 32, 1, False, BF, BF, True),
    (3, 20, 4, 2, 128, 64, 64, 1, False, BF, BF, False), (3, 20, 4, 2, 80, 64, 80, 1, True, BF, BF, False),
    (2, 200, 3, 1, 80, 128, 60, 3, False, BF, BF, True), (2, 200, 4, 2, 128, 128, 128, 1, False, F32, E4M3, True),
    (2, 200, 4, 2, 64, 128, 32, 1, True, F32, F32, False), (2, 200, 3, 1, 90, 128, 50, 1, False, F32, F32, True),
    (1, 1, 4, 2, 128, 128, 64, 1, False, F32, F32, False), (1, 129, 70, 70, 128, 128, 128, 1, False, BF, E4M3, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("c", APPENDS, ids=cache.name)
def test_appends(c):
    a = cache.make(*c)
    cache.check(*a, H=c[2], inter=c[8], norm=c[11])


@pytest.mark.gpu
@pytest.mark.parametrize("c", [APPENDS[i] for i in (0, 2, 3, 5, 6, 8, 11, 17)], ids=cache.name)
@pytest.mark.parametrize("first", [0, 1, 64, 65, 127])
def test_appends_at_any_row(c, first):
    c = (2,) + c[1:]
    a = cache.make(*c, starts=[first, first + 70], counts=[c[1], c[1] // 2], seed=first)
    cache.check(*a, H=c[2], inter=c[8], norm=c[11])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kind,H,d,N", [(BF, E4M3, 4, 64, 200), (BF, BF, 4, 128, 40), (F32, E4M3, 2, 80, 30)])
def test_second_order_over_cached_keys(dtype, kind, H, d, N):
    """The tangent of attention over what a cache holds, against differences of the
    definition in 64 bits."""
    B, Hkv, T, M = 2, 2, 32, 5
    Nk = 137
    pools, values = pag.pools(B * M, Hkv, T, d, kind)
    table = pag.table_of(B, M, B * M)
    g = torch.Generator(device="cuda").manual_seed(5)
    K, V = fb.cache_read(fb.PagedCache(*pools), table, Nk, dtype=dtype)
    Q, UQ = (torch.randn((B, H, N, d), generator=g, device="cuda").to(dtype) for _ in range(2))
    UK, UV = (torch.randn((B, Hkv, Nk, d), generator=g, device="cuda").to(dtype) for _ in range(2))
    tau = 1 / math.sqrt(d)
    O, L, Od, Ld = fb.attention_jvp(Q, K, V, UQ, UK, UV, tau)

    def definition(t):
        q = Q.double() + t * UQ.double()
        k, v = ((pag.dense(x, table)[:, :, :Nk] + t * u.double()).repeat_interleave(H // Hkv, dim=1)
                for x, u in zip(values, (UK, UV)))
        z = q @ k.transpose(2, 3) * tau
        return torch.softmax(z, dim=3) @ v, torch.logsumexp(z, dim=3)

    # Of fourth order: an error of h^4 = 1e-12 and 1e-16 / h = 1e-13 times a few.
    h = 1e-3
    parts = [definition(t * h) for t in (-2, -1, 1, 2)]
    want = [(a - 8 * b + 8 * c - e) / (12 * h) for a, b, c, e in zip(*parts)]
    # Weights in 16 bits in the tensor-core form (half a step, 2^-8, of terms whose sum of
    # squares the norm is of, and as much again for U_V); 32 bits elsewhere.
    tol = 2 * 2.0 ** -8 if dtype is BF else 1e-5
    for got, w in zip((Od, Ld), want):
        assert float((got.double() - w).norm() / w.norm()) <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("kind,P", [(E4M3, (1 << 32) // (2 * 128 * 128) + 4), (BF, (1 << 31) // (2 * 128 * 128) + 4)])
def test_appends_past_32_bit_offsets(kind, P):
    """Pages behind 2^32 bytes and 2^31 elements get what pages of a small pool get."""
    Hkv, T, d, N = 2, 128, 128, 300
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((1, N, 4 + 2 * Hkv, d), generator=g, device="cuda").to(BF)
    start = torch.tensor([50], dtype=torch.int32, device="cuda")
    at = torch.tensor([[P - 1, 0, P - 3]], dtype=torch.int32, device="cuda")
    small, far = fb.PagedCache.empty(3, Hkv, T, d, dtype=kind), fb.PagedCache.empty(P, Hkv, T, d, dtype=kind)
    local = torch.arange(3, device="cuda")[None].int()
    Q = [fb.cache_append(x, 4, c, t, kv_start=start) for c, t in ((small, local), (far, at))]
    assert torch.equal(*Q)
    for a, b in ((small.K, far.K), (small.V, far.V), (small.k_scale, far.k_scale), (small.v_scale, far.v_scale)):
        if a is not None:
            for i, p in enumerate(at[0].tolist()):
                assert torch.equal(a[i].view(torch.uint8), b[p].view(torch.uint8))
    for a, b in zip(fb.cache_read(small, local, 350), fb.cache_read(far, at, 350)):
        assert torch.equal(a, b)
    # and nothing else has been touched
    assert not far.K.view(torch.uint8)[1:P - 3].any() and not far.V.view(torch.uint8)[P - 2].any()
