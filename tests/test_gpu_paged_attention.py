"""Attention over a paged cache against the 64-bit definition, element by element
within the bounds of its roundings."""
import math

import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests import layer_reference as ref
from tests import paged_reference as pag

pytestmark = pytest.mark.gpu

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def make(B, H, Hkv, Nq, M, T, d, dtype, cache, mask="chunk", bias=False, seed=0, spread=1.0, **_):
    g = torch.Generator(device="cuda").manual_seed(seed)
    P, Nk = B * M + 2, M * T
    pools, values = pag.pools(P, Hkv, T, d, cache, seed, spread)
    table = pag.table_of(B, M, P, seed)
    Q = torch.randn((B, H, Nq, d), generator=g, device="cuda").to(dtype)
    form = dict(slopes=None, ranges=None, q_pos=None)
    if bias:
        form["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    i = torch.arange(Nq, device="cuda")
    if mask == "chunk":  # the last tokens of requests of several lengths
        last = torch.randint(min(Nq, Nk), Nk + 1, (B, 1), generator=g, device="cuda")
        pos = (last - Nq + i).int()
        form["q_pos"] = pos
        form["ranges"] = torch.stack([torch.zeros_like(pos), pos + 1], dim=2).contiguous()
    elif mask == "window":  # of 37 keys, in a padded batch
        pos = (Nk - Nq + i).expand(B, Nq).int().contiguous()
        live = i < torch.randint(1, Nq + 1, (B, 1), generator=g, device="cuda")
        form["q_pos"] = pos
        form["ranges"] = torch.where(live[..., None], torch.stack([pos - 36, pos + 1], dim=2),
                                     0).int().contiguous()
    elif mask == "random":  # any ranges at all: long, short, empty, beyond the ends
        lo = torch.randint(-5, Nk, (B, Nq), generator=g, device="cuda")
        n = torch.randint(-3, Nk + 5, (B, Nq), generator=g, device="cuda")
        form["ranges"] = torch.stack([lo, lo + n], dim=2).int()
        form["q_pos"] = torch.randint(-4, Nk + 4, (B, Nq), generator=g, device="cuda").int()
    elif mask == "one":  # one key
        lo = torch.randint(0, Nk, (B, Nq), generator=g, device="cuda")
        form["ranges"] = torch.stack([lo, lo + 1], dim=2).int()
    elif mask == "nothing":
        form["ranges"] = torch.zeros((B, Nq, 2), dtype=torch.int32, device="cuda")
    return Q, pools, values, table, form


def poison(Q, pools, table, form, causal):
    """NaN wherever the mask leaves nothing: rows that see no key, keys outside the run
    that the batch entry's queries see, and the pages that nobody has."""
    B, H, Nq, d = Q.shape
    P, Hkv, T, _ = pools[0].shape
    M = table.shape[1]
    see, _ = ref.visible(B, Nq, M * T, form["ranges"], form["q_pos"], causal)
    seen = see.any(dim=1)
    j = torch.arange(M * T, device="cuda")
    lo = torch.where(seen, j, M * T).amin(dim=1, keepdim=True)
    hi = torch.where(seen, j, -1).amax(dim=1, keepdim=True)
    free = torch.ones((P, T), dtype=torch.bool, device="cuda")
    free[table.long()] = ((j < lo) | (j > hi)).view(B, M, T)
    Q = Q.masked_fill(~see.any(dim=2)[:, None, :, None], math.nan)
    out = []
    for x in pools[:2]:
        wipe = free[:, None, :, None].expand(x.shape)
        if x.dtype is E4M3:
            out.append(x.view(torch.uint8).masked_fill(wipe, 0x7F).view(E4M3))
        else:
            out.append(x.masked_fill(wipe, math.nan))
    return Q, out + pools[2:]


def check(case, tau=None, cap=0.0, causal=False, poisoned=True, **kw):
    Q, pools, values, table, form = make(**case, **kw)
    tau = 1 / math.sqrt(Q.shape[3]) if tau is None else tau
    q, p = poison(Q, pools, table, form, causal) if poisoned else (Q, pools)
    cache = fb.PagedCache(*p)
    O, L = fb.attention_paged(q, cache, table, tau, cap=cap, causal=causal, **form)
    torch.cuda.synchronize()
    assert fb.flashbob_last_device_error() == fb.FLASHBOB_OK
    k, v = (pag.dense(x, table) for x in values)
    codes = scales = None
    if pools[2] is not None:
        T = pools[0].shape[2]
        scales = pools[3][table.long()].transpose(1, 2).double().repeat_interleave(T, dim=2)
        codes = v / scales[..., None]
    val, bound = pag.attention(Q, k, v, codes, scales, tau, cap=cap, causal=causal, **form)
    assert O.dtype is Q.dtype and L.dtype is F32
    assert ref.worst(O, val["O"], bound["O"]) <= 1
    assert ref.worst(L, val["L"], bound["L"]) <= 1


def case(B, H, Hkv, Nq, M, T, d, dtype=BF, cache=E4M3):
    return dict(B=B, H=H, Hkv=Hkv, Nq=Nq, M=M, T=T, d=d, dtype=dtype, cache=cache)


def name(c):
    return "-".join(str(v).replace("torch.", "") for v in c.values())


TOKENS = [case(*c) for c in (
    (1, 1, 1, 1, 1, 16, 64), (1, 12, 12, 1, 9, 16, 64), (3, 8, 2, 1, 5, 64, 128),
    (2, 8, 1, 1, 40, 32, 128), (5, 4, 4, 2, 3, 128, 64), (2, 16, 1, 1, 11, 16, 128),
    (1, 8, 2, 4, 70, 64, 128), (2, 32, 1, 1, 3, 32, 64), (1, 8, 1, 4, 9, 128, 128),
    (2, 6, 2, 5, 17, 16, 64), (1, 3, 1, 7, 33, 64, 128), (1, 4, 4, 1, 300, 16, 128),
    (1, 8, 8, 1, 129, 128, 128), (1, 2, 1, 1, 1, 128, 128), (2, 31, 1, 1, 10, 32, 128),
    (3, 8, 2, 1, 5, 64, 128, BF, BF), (1, 8, 2, 4, 70, 64, 64, BF, BF), (2, 32, 1, 1, 9, 16, 128, BF, BF),
    (1, 12, 12, 1, 61, 16, 64, BF, BF), (1, 4, 1, 3, 40, 128, 128, BF, BF))]
PROMPTS = [case(*c) for c in (
    (1, 2, 2, 40, 3, 16, 64), (2, 4, 2, 129, 5, 64, 128), (1, 8, 2, 100, 9, 32, 128),
    (3, 3, 1, 77, 40, 16, 64), (1, 4, 4, 300, 4, 128, 128), (1, 2, 1, 513, 17, 64, 128),
    (2, 12, 4, 256, 30, 32, 64), (1, 1, 1, 33, 200, 16, 128), (1, 16, 16, 640, 11, 64, 128),
    (2, 4, 2, 129, 5, 64, 128, BF, BF), (1, 6, 2, 200, 40, 16, 64, BF, BF),
    (1, 8, 8, 700, 7, 128, 128, BF, BF))]
# Requests of unequal length whose keys are shared out evenly among the blocks.
SHARED = [case(*c) for c in (
    (7, 8, 2, 1, 20, 64, 128), (3, 32, 2, 2, 130, 16, 64), (40, 4, 4, 1, 16, 64, 64), (9, 8, 8, 3, 9, 128, 128),
    (2, 3, 1, 5, 64, 16, 128), (130, 2, 1, 1, 64, 16, 64), (4, 16, 1, 1, 17, 64, 128, BF, BF), (6, 24, 2, 2, 40, 32, 64, BF, BF))]
OTHERS = [case(*c) for c in (
    (1, 1, 1, 1, 1, 16, 1, F32, E4M3), (2, 3, 3, 33, 5, 16, 80, F32, E4M3), (1, 4, 2, 3, 20, 64, 64, F32, F32),
    (2, 2, 1, 65, 3, 128, 128, F32, E4M3), (1, 6, 3, 5, 9, 32, 34, BF, E4M3), (2, 2, 2, 70, 9, 32, 96, BF, BF),
    (1, 5, 1, 9, 3, 16, 127, F32, F32))]
ALL = TOKENS + SHARED + PROMPTS + OTHERS


@pytest.mark.parametrize("c", ALL, ids=name)
@pytest.mark.parametrize("mask", ["chunk", "window", "random"])
def test_matches_the_definition(c, mask):
    check(c, mask=mask)


@pytest.mark.parametrize("c", TOKENS[2:8] + TOKENS[15:18] + PROMPTS[1:4] + PROMPTS[9:11] + OTHERS[1:3],
                         ids=name)
@pytest.mark.parametrize("cap,bias", [(20.0, False), (0.0, True), (50.0, True), (0.3, False)])
def test_caps_and_biases(c, cap, bias):
    check(c, cap=cap, bias=bias, seed=3)
    check(c, cap=cap, bias=bias, mask="random", seed=4)


@pytest.mark.parametrize("c", [TOKENS[3], TOKENS[16], SHARED[0], SHARED[7], PROMPTS[1], PROMPTS[9], OTHERS[1]], ids=name)
@pytest.mark.parametrize("mask", ["none", "one", "nothing"])
def test_few_and_all_keys(c, mask):
    check(c, mask=mask, seed=5)
    check(c, mask=mask, seed=6, causal=True)


@pytest.mark.parametrize("c", [TOKENS[2], TOKENS[6], TOKENS[15], PROMPTS[2], PROMPTS[5], OTHERS[1]], ids=name)
def test_large_scores_and_scales_far_apart(c):
    """Scores of hundreds, and pages whose values differ by many powers of two."""
    check(c, tau=4.0, seed=7)
    check(c, seed=8, spread=8.0, tau=1e-3)
    check(c, seed=9, spread=8.0, tau=1e-3, mask="random")


@pytest.mark.parametrize("c", [TOKENS[2], PROMPTS[1], OTHERS[1]], ids=name)
def test_pages_outside_the_pool_are_zeros(c):
    Q, pools, values, table, form = make(**c, mask="none")
    table[0, -1], table[-1, 0] = -1, pools[0].shape[0]
    if table.shape[1] > 2:
        table[0, 1] = 2 ** 31 - 1
    tau = 0.1
    O, L = fb.attention_paged(Q, fb.PagedCache(*pools), table, tau)
    k, v = (pag.dense(x, table) for x in values)
    T = pools[0].shape[2]
    ok = (table >= 0) & (table < pools[0].shape[0])
    scales = torch.where(ok[:, :, None], pools[3][table.clamp(0, pools[0].shape[0] - 1).long()], 1.0)
    scales = scales.transpose(1, 2).double().repeat_interleave(T, dim=2)
    val, bound = pag.attention(Q, k, v, v / scales[..., None], scales, tau)
    assert ref.worst(O, val["O"], bound["O"]) <= 1 and ref.worst(L, val["L"], bound["L"]) <= 1


@pytest.mark.parametrize("c", [TOKENS[6], PROMPTS[1], OTHERS[1]], ids=name)
def test_pages_of_zeros_beside_others(c):
    """A page that holds only zeros has the least scale; its keys still count."""
    Q, pools, values, table, form = make(**c, mask="none")
    page = int(table[0, 0])
    for i in range(2):
        pools[i].view(torch.uint8)[page] = 0
        pools[2 + i][page] = 2.0 ** -60
        values[i][page] = 0
    tau = 0.1
    O, L = fb.attention_paged(Q, fb.PagedCache(*pools), table, tau)
    k, v = (pag.dense(x, table) for x in values)
    scales = pools[3][table.long()].transpose(1, 2).double().repeat_interleave(pools[0].shape[2], dim=2)
    val, bound = pag.attention(Q, k, v, v / scales[..., None], scales, tau)
    assert ref.worst(O, val["O"], bound["O"]) <= 1 and ref.worst(L, val["L"], bound["L"]) <= 1


def test_the_same_as_dense_keys():
    """A 16-bit cache holds what the dense call reads: the same definition."""
    c = case(2, 4, 2, 50, 6, 32, 64, BF, BF)
    Q, pools, values, table, form = make(**c)
    O, L = fb.attention_paged(Q, fb.PagedCache(*pools), table, 0.125, **form)
    K, V = (pag.dense(x, table).to(BF).contiguous() for x in values)
    O2, L2 = fb.attention(Q, K, V, 0.125, **form)
    assert float((L - L2).abs().max()) <= 2e-5 and float((O.float() - O2.float()).abs().max()) <= 2e-2


@pytest.mark.parametrize("c", [TOKENS[6], TOKENS[12], SHARED[0], SHARED[7], PROMPTS[1], OTHERS[1]], ids=name)
def test_same_bits_on_another_stream_and_replayed(c):
    Q, pools, _, table, form = make(**c)
    cache = fb.PagedCache(*pools)

    def run(stream=None):
        return fb.attention_paged(Q, cache, table, 0.1, cap=30.0, stream=stream, **form)

    a = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = run(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = run()
    for t in g:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, g):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_caches_past_32_bit_offsets():
    """Pages behind 2^31 elements, and 2^32."""
    P, Hkv, T, d = (1 << 32) // (2 * 128 * 128) + 4, 2, 128, 128
    cache = fb.PagedCache.empty(P, Hkv, T, d)
    pools, values = pag.pools(4, Hkv, T, d, E4M3, 11)
    at = [P - 1, 0, P // 2 + 3, P - 3]
    for k, p in enumerate(at):
        for x, y in zip((cache.K, cache.V), pools):
            x.view(torch.uint8)[p] = y.view(torch.uint8)[k]
        cache.k_scale[p], cache.v_scale[p] = pools[2][k], pools[3][k]
    table = torch.tensor([at], dtype=torch.int32, device="cuda")
    local = torch.arange(4, device="cuda")[None].int()
    for Nq in (1, 100):
        Q = torch.randn((1, 4, Nq, d), device="cuda").to(BF)
        O, L = fb.attention_paged(Q, cache, table, 0.1)
        O2, L2 = fb.attention_paged(Q, fb.PagedCache(*pools), local, 0.1)
        assert torch.equal(O, O2) and torch.equal(L, L2)
    K, V = fb.cache_read(cache, table, 4 * T, dtype=F32)
    for x, y in ((K, values[0]), (V, values[1])):
        assert torch.equal(x.double(), pag.dense(y, local))
