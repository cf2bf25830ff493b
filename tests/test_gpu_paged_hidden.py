"""What a mask hides reaches nothing, not even a last bit, with the keys in pages: calls
whose hidden queries, keys, values and pages hold zeros, large numbers, infinities or NaN
give the same bits."""
import math

import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests import layer_reference as ref
from tests import paged_reference as pag

pytestmark = pytest.mark.gpu

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
# B, H, Hkv, Nq, M, T, d, dtype, cache: single and drafted tokens; prompts in blocks of 128
# rows, some cut along the keys; in blocks of 256 (160 of them at d = 128, 320 at d = 64);
# and on CUDA cores.
TOKENS = [(3, 8, 2, 1, 40, 16, 128, BF, E4M3), (2, 16, 4, 4, 20, 64, 64, BF, E4M3), (3, 16, 2, 3, 9, 64, 128, BF, BF)]
PROMPTS = [(2, 4, 2, 100, 30, 32, 128, BF, E4M3), (3, 6, 2, 150, 40, 16, 64, BF, E4M3), (2, 3, 3, 200, 9, 128, 64, BF, BF),
           (4, 40, 40, 200, 6, 64, 128, BF, E4M3), (4, 80, 40, 120, 12, 32, 128, BF, BF), (8, 40, 40, 200, 24, 16, 64, BF, E4M3)]
OTHERS = [(2, 4, 2, 70, 9, 32, 96, BF, E4M3), (2, 4, 2, 5, 9, 32, 64, F32, E4M3)]


def build(c, seed=3):
    """Padded requests of several lengths behind a cached part: some queries see nothing,
    and pages at both ends, and the last page's rest, are nobody's."""
    B, H, Hkv, Nq, M, T, d, dtype, cache = c
    g = torch.Generator(device="cuda").manual_seed(seed)
    pools, _ = pag.pools(B * M + 2, Hkv, T, d, cache, seed)
    table = pag.table_of(B, M, B * M + 2, seed)
    Q = torch.randn((B, H, Nq, d), generator=g, device="cuda").to(dtype)
    i = torch.arange(Nq, device="cuda")
    new = torch.randint(Nq // 2, Nq + 1, (B, 1), generator=g, device="cuda")
    if Nq <= 4:
        new[0] = 0  # a request that takes no part
    last = torch.randint(Nq + (M * T - Nq) // 2, M * T - 3, (B, 1), generator=g, device="cuda")
    pos = last - Nq + i
    ranges = torch.stack([torch.full_like(pos, T + 5), pos + 1], dim=2)
    ranges = torch.where((i < new)[..., None], ranges, 0).int().contiguous()
    return Q, pools, table, dict(ranges=ranges, q_pos=pos.int().contiguous())


def fill(Q, pools, table, form, value, code):
    """Copies with `value` (and its nearest code) wherever nothing is seen."""
    B, H, Nq, d = Q.shape
    P, Hkv, T, _ = pools[0].shape
    M = table.shape[1]
    see, _ = ref.visible(B, Nq, M * T, form["ranges"], form["q_pos"], False)
    seen = see.any(dim=1)
    j = torch.arange(M * T, device="cuda")
    first = torch.where(seen, j, M * T).amin(dim=1, keepdim=True)
    last = torch.where(seen, j, -1).amax(dim=1, keepdim=True)
    free = torch.ones((P, T), dtype=torch.bool, device="cuda")
    free[table.long()] = ((j < first) | (j > last)).view(B, M, T)
    Q = Q.masked_fill(~see.any(dim=2)[:, None, :, None], value)
    out = []
    for x in pools[:2]:
        wipe = free[:, None, :, None].expand(x.shape)
        out.append(x.view(torch.uint8).masked_fill(wipe, code).view(E4M3) if x.dtype is E4M3 else x.masked_fill(wipe, value))
    for s in pools[2:]:
        out.append(None if s is None else s.masked_fill(free.all(dim=1)[:, None], value))
    return Q, out


@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (20.0, True), (1e4, False)])
@pytest.mark.parametrize("c", TOKENS + PROMPTS + OTHERS, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_the_same_bits_whatever_hidden_rows_hold(c, cap, bias):
    Q, pools, table, form = build(c)
    if bias:
        form["slopes"] = torch.exp2(-4.0 - torch.arange(c[1], device="cuda") % 8)
    want = None
    for value, code in ((0.0, 0), (300.0, 0x79), (1e30, 0x7E), (-math.inf, 0xFE), (math.nan, 0x7F)):
        q, p = fill(Q, pools, table, form, value, code)
        got = fb.attention_paged(q, fb.PagedCache(*p), table, 1 / math.sqrt(c[6]), cap=cap, **form)
        want = got if want is None else want
        assert bool(got[0].isfinite().all())
        for x, y in zip(got, want):
            assert torch.equal(x, y), value
