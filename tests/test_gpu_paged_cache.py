"""Appending to a paged cache and reading it, against the 64-bit definition; a run of
the paged operators as a served model uses them."""
import math

import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests import layer_reference as ref
from tests import paged_reference as pag

pytestmark = pytest.mark.gpu

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-5


def make(B, N, H, Hkv, d, T, R, axes, inter, dtype, cache, norm, seed=0, starts=None, counts=None):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s, t=F32):
        return torch.randn(s, generator=g, device="cuda").to(t)

    M = (N + 200) // T + 2
    P = B * M + 2
    pools, _ = pag.pools(P, Hkv, T, d, cache, seed)
    table = pag.table_of(B, M, P, seed)
    form = dict(wq=None, wk=None, freqs=None, positions=None)
    if norm:
        form["wq"], form["wk"] = 1 + 0.2 * r(d), 1 + 0.2 * r(d)
    if R:
        freqs = (10000.0 ** (-torch.arange(R // 2, device="cuda") / max(1, R // 2))).expand(axes, -1)
        axis = torch.arange(R // 2, device="cuda") % axes
        form["freqs"] = torch.where(axis == torch.arange(axes, device="cuda")[:, None], freqs,
                                    0.0).contiguous()
        if axes > 1:
            form["positions"] = torch.randint(0, 5000, (axes, B, N), generator=g, device="cuda").int()
    elif axes > 1:
        raise AssertionError
    x = r(B, N, H + 2 * Hkv, d) * torch.exp(r(B, N, 1, 1))
    if starts is None:
        starts = torch.randint(0, M * T - N + 1, (B,), generator=g, device="cuda").int()
    else:
        starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
    if counts is not None:
        counts = torch.tensor(counts, dtype=torch.int32, device="cuda")
    return x.to(dtype), pools, table, form, starts, counts


def check(x, pools, table, form, starts, counts, H, inter, norm):
    """One append against the definition; returns the cache and Q."""
    B, N, heads, d = x.shape
    P, Hkv, T, _ = pools[0].shape
    M = table.shape[1]
    codes = pools[2] is not None
    before = [t.clone() if t is not None else None for t in pools]
    cache = fb.PagedCache(*pools)
    Q = fb.cache_append(x, H, cache, table, kv_start=starts, counts=counts, **form,
                        eps=EPS if norm else None, interleaved=inter)
    torch.cuda.synchronize()
    positions = form["positions"]
    if positions is None:
        positions = (starts[:, None].long() + torch.arange(N, device="cuda"))[None]
    if norm:
        want = ref.norm_rope(x, H, form["wq"], form["wk"], form["freqs"], positions, EPS, inter)
    else:  # the rotation alone: of rows of norm sqrt(d), whose norm is 1 / r = 1
        size = x.double().square().mean(dim=3, keepdim=True).sqrt()
        want = [t * s for t, s in zip(
            ref.norm_rope(x.double() / size, H, None, None, form["freqs"], positions, 0.0, inter),
            (size[:, :, :H].transpose(1, 2), size[:, :, H:H + Hkv].transpose(1, 2), 1.0))]
        want[2] = x[:, :, H + Hkv:].double().transpose(1, 2)
    # fp32 arithmetic as in the dense call: (d + 16) 2^-24 of the norm of the row.
    e = (d + 16) * 2.0 ** -24
    u = torch.finfo(x.dtype).eps / 2
    assert bool(((Q.double() - want[0]).abs() <= u * want[0].abs()
                 + e * want[0].norm(dim=3, keepdim=True)).all())
    touched = torch.zeros((P, T), dtype=torch.bool, device="cuda")
    table_, starts_ = table.tolist(), starts.tolist()
    counts_ = [N] * B if counts is None else [max(0, min(N, c)) for c in counts.tolist()]
    for which in range(2):
        new, pool, old = want[1 + which], pools[which], before[which]
        err = e * new.norm(dim=3, keepdim=True) * (1 if which == 0 else 0)
        scales = pools[2 + which]
        changed = torch.zeros((P,), dtype=torch.bool, device="cuda")
        for b in range(B):
            n = 0
            while n < counts_[b]:
                p = starts_[b] + n
                m = min(T - p % T, counts_[b] - n)
                page = table_[b][p // T] if 0 <= p // T < M else -1
                if not 0 <= page < P:
                    n += m
                    continue
                row, y, w = p % T, new[b, :, n:n + m], err[b, :, n:n + m]
                n += m
                touched[page, row:row + m] = True
                got = pool[page, :, row:row + m].double()
                if not codes:
                    v = torch.finfo(pool.dtype).eps / 2
                    assert bool(((got - y).abs() <= v * y.abs() + w).all())
                    continue
                changed[page] = True
                s = scales[page].double()[:, None, None]
                most = y.abs().amax(dim=(1, 2))
                top = w.amax(dim=(1, 2))
                for h in range(Hkv):
                    fits = {pag.scale_for(float(most[h] - top[h])), pag.scale_for(float(most[h] + top[h]))}
                    if row:
                        fits = {max(f, float(before[2 + which][page, h])) for f in fits}
                    assert float(scales[page, h]) in fits
                # Half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below 2^-6 of it.
                assert bool(((got * s - y).abs() <= torch.maximum(y.abs() * 2.0 ** -4,
                                                                  s * 2.0 ** -10) + w).all())
                if which == 1:
                    assert torch.equal(got, pag.nearest(y / s))
                if row:  # what it held, in the new scale
                    touched[page, :row] = True
                    held = old[page, :, :row].double() * before[2 + which][page].double()[:, None, None]
                    assert torch.equal(pool[page, :, :row].double(), pag.nearest(held / s))
        a = pool.view(torch.uint8) if codes else pool
        z = old.view(torch.uint8) if codes else old
        keep = ~touched[:, None, :, None].expand(a.shape)
        assert torch.equal(a[keep], z[keep])
        if codes:
            assert torch.equal(scales[~changed], before[2 + which][~changed])
    return cache, Q


CASES = [  # B, N, H, Hkv, d, T, R, axes, interleaved, dtype, cache, norm
    (1, 1, 1, 1, 64, 16, 64, 1, False, BF, E4M3, False), (5, 1, 8, 2, 128, 64, 128, 1, False, BF, E4M3, False),
    (2, 3, 4, 4, 64, 32, 32, 1, True, BF, E4M3, True), (3, 33, 6, 2, 80, 32, 60, 3, True, BF, E4M3, True),
    (1, 300, 4, 1, 128, 16, 128, 1, False, BF, E4M3, False), (2, 200, 2, 2, 64, 128, 64, 2, False, BF, E4M3, False),
    (2, 130, 4, 2, 128, 128, 64, 1, True, BF, E4M3, False), (1, 500, 3, 1, 128, 64, 128, 1, False, F32, E4M3, True),
    (2, 70, 2, 1, 34, 16, 34, 1, False, BF, E4M3, False), (1, 40, 1, 1, 1, 16, 0, 1, False, F32, E4M3, False),
    (2, 20, 5, 1, 127, 128, 126, 1, True, F32, E4M3, False), (3, 50, 2, 2, 96, 64, 48, 1, False, F32, F32, False),
    (4, 1, 12, 12, 64, 16, 64, 1, False, BF, BF, True), (2, 260, 4, 2, 128, 64, 128, 1, False, BF, BF, False),
    (2, 5, 3, 3, 33, 32, 32, 1, True, BF, BF, False), (40, 2, 4, 2, 128, 16, 128, 1, False, BF, E4M3, False),
]


def name(c):
    return "-".join(str(v).replace("torch.", "") for v in c)


@pytest.mark.parametrize("c", CASES, ids=name)
def test_append_matches_the_definition(c):
    a = make(*c)
    check(*a, H=c[2], inter=c[8], norm=c[11])


@pytest.mark.parametrize("c", [CASES[2], CASES[4], CASES[6], CASES[13]], ids=name)
@pytest.mark.parametrize("first", [0, 1, 15, 16, 63, 127, 128, 129])
def test_append_at_any_row(c, first):
    c = (2,) + c[1:]
    a = make(*c, starts=[first, first + 5], counts=[c[1], c[1] // 2], seed=first)
    check(*a, H=c[2], inter=c[8], norm=c[11])


def test_append_drops_what_has_no_place():
    c = (6, 40) + CASES[4][2:]
    M = (40 + 200) // 16 + 2
    a = make(*c, starts=[-10, M * 16 - 7, -400, 2 ** 31 - 20, 8, 24], counts=[40, 40, 40, 40, 0, -3])
    a[2][4, 0], a[2][5, 3] = -1, 10 ** 6  # pages outside the pool
    check(*a, H=c[2], inter=c[8], norm=c[11])
    a = make(*c, starts=[0, 3, 16, 17, 30, 0])
    a[2][0, 0], a[2][1, 1], a[2][5, 2] = -1, 2 ** 31 - 1, -2 ** 31
    check(*a, H=c[2], inter=c[8], norm=c[11])


def test_pages_that_fill_token_by_token():
    """Values that grow: the scale follows, and what the page holds with it."""
    B, Hkv, d, T, n = 2, 2, 64, 16, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((B, n, 1 + 2 * Hkv, d), generator=g, device="cuda") * torch.exp2(
        torch.arange(n, device="cuda") % 13 - 4.0)[:, None, None]
    table = torch.tensor([[2, 0, 5], [1, 4, 3]], dtype=torch.int32, device="cuda")
    cache = fb.PagedCache.empty(7, Hkv, T, d)
    cache.k_scale.fill_(math.nan)  # what a page has before its first token does not matter
    cache.v_scale.fill_(math.inf)
    held = {}
    for i in range(n):
        fb.cache_append(x[:, i:i + 1].contiguous(), 1, cache, table,
                        kv_start=torch.full((B,), i, dtype=torch.int32, device="cuda"))
        for b in range(B):
            for h in range(Hkv):
                for w, r in enumerate((1, 1 + Hkv)):
                    y = x[b, i, r + h].double()
                    s = pag.scale_for(float(y.abs().max()))
                    old = held.get((b, h, w))
                    if i % T:
                        s = max(s, old[1])
                        rows = torch.cat([pag.nearest(old[0] * old[1] / s), pag.nearest(y / s)[None]])
                    else:
                        rows = pag.nearest(y / s)[None]
                    held[b, h, w] = rows, s
                    page = int(table[b, i // T])
                    pool, scale = ((cache.K, cache.k_scale), (cache.V, cache.v_scale))[w]
                    assert float(scale[page, h]) == s
                    assert torch.equal(pool[page, h, :i % T + 1].double(), rows)


def test_values_at_the_ends():
    """Zeros, infinities, NaN and values beyond the reach of the scales."""
    Hkv, d, T = 1, 64, 16
    cache = fb.PagedCache.empty(3, Hkv, T, d)
    table = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    x = torch.zeros((1, 48, 3, d), device="cuda")
    x[0, 16:32, 1:] = torch.linspace(-3, 3, d, device="cuda")
    x[0, 17, 1:, 5], x[0, 18, 1:, 6], x[0, 19, 1:, 7] = math.inf, -math.inf, math.nan
    x[0, 32:, 1:] = 1e30
    x[0, 33, 1:] = 1e-30
    fb.cache_append(x, 1, cache, table)
    for pool, scale in ((cache.K, cache.k_scale), (cache.V, cache.v_scale)):
        assert scale[:, 0].tolist() == [2.0 ** -60, 2.0 ** -7, 2.0 ** 60]
        v = pool[:, 0].double()
        assert bool((v[0] == 0).all())
        assert v[1, 1, 5] == 448 and v[1, 2, 6] == -448 and bool(v[1, 3, 7].isnan())
        fine = torch.ones((16, d), dtype=torch.bool, device="cuda")
        fine[1, 5] = fine[2, 6] = fine[3, 7] = False
        assert torch.equal(v[1][fine], pag.nearest(x[0, 16:32, 1].double() * 2.0 ** 7)[fine])
        assert bool((v[2, 0] == 448).all()) and bool((v[2, 1] == 0).all())


@pytest.mark.parametrize("dtype,cache", [(BF, E4M3), (F32, E4M3), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("B,Hkv,M,T,d,Nk", [(1, 1, 1, 16, 1, 1), (3, 2, 5, 16, 80, 77), (2, 4, 3, 128, 128, 384),
                                            (5, 1, 9, 32, 33, 250), (1, 3, 40, 64, 64, 2100), (2, 2, 2, 64, 48, 100)])
def test_read(B, Hkv, M, T, d, Nk, dtype, cache):
    P = B * M + 1
    pools, values = pag.pools(P, Hkv, T, d, cache)
    table = pag.table_of(B, M, P)
    lens = torch.tensor([(Nk * (b + 1)) // B - (b == 1) for b in range(B)], dtype=torch.int32, device="cuda")
    if M > 4:
        table[0, 1] = -7
    for n in (None, lens, torch.zeros_like(lens), lens + 10 ** 6, lens - 10 ** 6):
        K, V = fb.cache_read(fb.PagedCache(*pools), table, Nk, lens=n, dtype=dtype)
        for got, x in ((K, values[0]), (V, values[1])):
            want = pag.dense(x, table)[:, :, :Nk]
            if n is not None:
                want = want * (torch.arange(Nk, device="cuda") < n[:, None])[:, None, :, None]
            assert got.dtype is dtype and torch.equal(got.double(), want)  # powers of two: exact


def test_calls_are_replayed_and_ordered_on_their_stream():
    c = CASES[1]
    x, pools, table, form, starts, counts = make(*c)
    other = [t.clone() for t in pools]
    side = torch.cuda.Stream()
    a, z = fb.PagedCache(*pools), fb.PagedCache(*other)
    Q = fb.cache_append(x, c[2], a, table, kv_start=starts, **form)
    K, V = fb.cache_read(a, table, 100)
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q2 = fb.cache_append(x, c[2], z, table, kv_start=starts, **form)
        K2, V2 = fb.cache_read(z, table, 100)
    graph.replay()
    graph.replay()  # the same tokens to the same places: the same cache
    Q3 = fb.cache_append(x, c[2], a, table, kv_start=starts, **form, stream=side)
    K3, V3 = fb.cache_read(a, table, 100, stream=side)
    torch.cuda.synchronize()
    for p, q, r in ((Q, Q2, Q3), (K, K2, K3), (V, V2, V3)):
        assert torch.equal(p, q) and torch.equal(p, r)
    for p, q in zip(pools, other):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("cache_dtype,d", [(E4M3, 128), (BF, 64), (E4M3, 64), (E4M3, 80)])
def test_a_served_model(cache_dtype, d):
    """Prompts of a padded batch, a second part of one of them, then single tokens: the
    cache that grows by appends, and attention over it, against dense attention of what
    the cache stands for."""
    B, H, Hkv, T, M = 3, 4, 2, 16, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = fb.PagedCache.empty(B * M, Hkv, T, d, dtype=cache_dtype)
    table = pag.table_of(B, M, B * M)
    freqs = (10000.0 ** (-torch.arange(d // 2, device="cuda") / (d // 2)))[None].float().contiguous()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    tau = 1 / math.sqrt(d)
    for n, counts in ((50, [50, 17, 33]), (9, [9, 9, 2]), (1, [1, 1, 1]), (1, [1, 0, 1])):
        x = torch.randn((B, n, H + 2 * Hkv, d), generator=g, device="cuda").to(BF)
        new = torch.tensor(counts, dtype=torch.int32, device="cuda")
        Q = fb.cache_append(x, H, cache, table, kv_start=lens, counts=new, freqs=freqs)
        ranges, q_pos = fb.attention_ranges(B, n, M * T, q_start=lens, causal=True)
        live = torch.arange(n, device="cuda") < new[:, None]
        ranges *= live[..., None]
        O, L = fb.attention_paged(Q, cache, table, tau, ranges=ranges, q_pos=q_pos)
        lens = lens + new
        K, V = fb.cache_read(cache, table, M * T, lens=lens)
        O2, L2 = fb.attention(Q, K, V, tau, ranges=ranges, q_pos=q_pos)
        val, bound = ref.attention(Q, K, V, tau, ranges=ranges, q_pos=q_pos)
        for o, l in ((O, L), (O2, L2)):
            # The paged call works on the same numbers: its bounds are the dense call's
            # and 2^-25 a weight (of at most 1) times the values' sizes.
            more = 2.0 ** -25 * V.double().abs().sum(dim=2).repeat_interleave(H // Hkv, dim=1)[:, :, None] * 64
            assert ref.worst(o, val["O"], bound["O"] + more) <= 1
            assert ref.worst(l, val["L"], bound["L"] + 1e-6) <= 1
        # Second order over the cached keys, as over any others.
        if n == 9 and d != 80:
            Od, Ld = fb.attention_jvp(Q, K, V, Q, K, V, tau)[2:]
            assert bool(Od.isfinite().all()) and bool(Ld.isfinite().all())
