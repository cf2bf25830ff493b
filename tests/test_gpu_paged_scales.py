"""Attention over pages whose scales lie as far apart as they may, 2^-60 beside 2^60: a key
counts by its score, whatever the scale of the values beside it."""
import math

import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests import layer_reference as ref
from tests import paged_reference as pag

pytestmark = pytest.mark.gpu

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
# B, H, Hkv, Nq, M, T, d, dtype: tokens whose keys are cut into no runs, clusters of them,
# clusters and parts, parts alone, with 8, 16 and 32 rows; prompts in blocks of 128 rows,
# cut and whole, and in blocks of 256; CUDA cores.
CASES = [(2, 8, 2, 1, 6, 16, 128, BF), (2, 6, 2, 2, 40, 64, 64, BF), (1, 8, 1, 1, 200, 64, 128, BF),
         (20, 32, 8, 1, 40, 64, 128, BF), (20, 16, 8, 1, 64, 32, 64, BF), (3, 32, 2, 1, 40, 64, 128, BF),
         (2, 8, 1, 4, 130, 16, 64, BF), (1, 4, 2, 100, 30, 32, 128, BF), (1, 6, 2, 200, 60, 16, 64, BF),
         (9, 8, 8, 200, 10, 64, 128, BF), (5, 32, 32, 160, 8, 64, 128, BF), (8, 40, 40, 150, 24, 16, 64, BF),
         (2, 4, 2, 9, 20, 16, 96, BF), (1, 4, 2, 70, 20, 16, 64, F32)]


def build(c, kind, seed=1):
    """Scales of the values: 2^60 on the first page and the seventh, elsewhere 2^-60 and
    zeros ("zeros"); by page, or by runs of six pages, any of five; all of them 2^-60."""
    B, H, Hkv, Nq, M, T, d, dtype = c
    g = torch.Generator(device="cuda").manual_seed(seed)
    pools, values = pag.pools(B * M, Hkv, T, d, E4M3, seed, spread=0.0)
    table = pag.table_of(B, M, B * M, seed)
    some = torch.tensor([-60.0, -45.0, -20.0, 0.0, 60.0], device="cuda")
    page = torch.arange(M, device="cuda")
    if kind == "zeros":
        e = torch.where(page % 7 == 0, 60.0, -60.0)[None, :, None].expand(B, M, Hkv)
    elif kind == "least":
        e = torch.full((B, M, Hkv), -60.0, device="cuda")
    else:
        of = page // (6 if kind == "runs" else 1)
        e = some[torch.randint(0, 5, (B, M, Hkv), generator=g, device="cuda")][:, of]
    pools[3][table.long()] = torch.exp2(e)
    if kind == "zeros":
        none = (pools[3] < 1)[..., None, None]
        pools[1] = pools[1].view(torch.uint8).masked_fill(none, 0).view(E4M3)
    values[1] = pools[1].double() * pools[3].double()[..., None, None]
    # Scores of several nats, so that gaps of six binades and more are common.
    Q = (3 * torch.randn((B, H, Nq, d), generator=g, device="cuda")).to(dtype)
    i = torch.arange(Nq, device="cuda")
    last = torch.randint(max(Nq, M * T - T), M * T + 1, (B, 1), generator=g, device="cuda")
    pos = (last - Nq + i).int()
    return Q, pools, values, table, dict(q_pos=pos, ranges=torch.stack([torch.zeros_like(pos), pos + 1], dim=2).contiguous())


@pytest.mark.parametrize("kind", ["zeros", "pages", "runs", "least"])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, True), (15.0, False), (0.0, True)])
@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_every_key_counts(c, cap, bias, kind):
    Q, pools, values, table, form = build(c, kind)
    if bias:
        form["slopes"] = torch.exp2(-7.0 - torch.arange(c[1], device="cuda") % 4)
    tau = 1 / math.sqrt(c[6])
    O, L = fb.attention_paged(Q, fb.PagedCache(*pools), table, tau, cap=cap, **form)
    k, v = (pag.dense(x, table) for x in values)
    scales = pools[3][table.long()].transpose(1, 2).double().repeat_interleave(c[5], dim=2)
    val, bound = pag.attention(Q, k, v, v / scales[..., None], scales, tau, cap=cap, **form)
    # An exponent of up to 60 more comes and goes in 32 bits: four roundings of sums of at
    # most 256 are 2^-16 each of a half.
    bound["L"] = bound["L"] + 4 * 2.0 ** -17
    assert bool(O.isfinite().all())
    assert ref.worst(L, val["L"], bound["L"]) <= 1
    assert ref.worst(O, val["O"], bound["O"]) <= 1


@pytest.mark.parametrize("c", [(3, 6, 2, 150, 10, 16, 64, BF), (1, 4, 2, 100, 30, 32, 128, BF), (2, 8, 2, 1, 30, 16, 128, BF),
                               (1, 8, 1, 3, 90, 64, 64, BF)], ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
@pytest.mark.parametrize("kind", [E4M3, BF])
def test_a_key_far_ahead_has_all(c, kind):
    """Scores hundreds above all others': what the others' values would add is no number of
    32 bits, so an element of 0 stays 0."""
    B, H, Hkv, Nq, M, T, d, dtype = c
    pools, _ = pag.pools(B * M, Hkv, T, d, kind, spread=0.0)
    table = pag.table_of(B, M, B * M)
    page = table[:, M // 2].long()
    Q = torch.ones((B, H, Nq, d), device="cuda").to(dtype)
    for t in pools[:2]:  # token 3 of a page in the middle: keys of 2, values of 0 and 2
        rows = torch.full((B, Hkv, d), 2.0, device="cuda")  # at most 448 scales, as a page's largest is above 1.75
        if t is pools[1]:
            rows = 2.0 * (torch.arange(d, device="cuda") % 2).expand(B, Hkv, d)
        if kind is E4M3:
            scale = (pools[2] if t is pools[0] else pools[3])[page][..., None]
            t.view(torch.uint8)[page, :, 3] = (rows / scale).to(E4M3).view(torch.uint8)
        else:
            t[page, :, 3] = rows.to(BF)
    O, L = fb.attention_paged(Q, fb.PagedCache(*pools), table, 3.0)
    want = (2.0 * (torch.arange(d, device="cuda") % 2)).expand(O.shape)
    assert torch.equal(O.float(), want)
    # 3 times 2 d, with the sums of products and log2 e rounded in 32 bits.
    assert bool(((L - 6.0 * d).abs() <= 6.0 * d * (d + 8) * 2.0 ** -24).all())
