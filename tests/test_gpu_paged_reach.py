"""Attention over pages at the ends of what tau, cap and the queries' size may be, against
the 64-bit definition."""
import math

import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests import layer_reference as ref
from tests import paged_reference as pag

pytestmark = pytest.mark.gpu

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
# B, H, Hkv, Nq, M, T, d, dtype, cache: tokens, prompts in blocks of 128 and of 256 rows.
CASES = [(2, 8, 2, 1, 40, 16, 128, BF, E4M3), (2, 8, 1, 3, 9, 64, 64, BF, E4M3), (1, 4, 2, 100, 20, 32, 128, BF, E4M3),
         (5, 32, 32, 160, 6, 64, 128, BF, E4M3), (8, 40, 40, 150, 6, 64, 64, BF, E4M3), (2, 4, 2, 100, 9, 64, 64, BF, BF),
         (2, 4, 2, 9, 20, 16, 96, BF, E4M3)]
IDS = ["-".join(str(v).replace("torch.", "") for v in c) for c in CASES]


def build(c, q, k, seed=1):
    """Queries of size 2^q and keys of size 2^k."""
    B, H, Hkv, Nq, M, T, d, dtype, cache = c
    pools, values = pag.pools(B * M, Hkv, T, d, cache, seed)
    table = pag.table_of(B, M, B * M, seed)
    values[0] = values[0] * 2.0 ** k
    if cache is E4M3:
        pools[2] = pools[2] * 2.0 ** k
        assert 2.0 ** -60 <= float(pools[2].min()) and float(pools[2].max()) <= 2.0 ** 60
    else:
        pools[0] = pools[0] * 2.0 ** k
    g = torch.Generator(device="cuda").manual_seed(seed)
    Q = (torch.randn((B, H, Nq, d), generator=g, device="cuda") * 2.0 ** q).to(dtype)
    return Q, pools, values, table


def check(c, Q, pools, values, table, tau, cap):
    O, L = fb.attention_paged(Q, fb.PagedCache(*pools), table, tau, cap=cap)
    k, v = (pag.dense(x, table) for x in values)
    codes = scales = None
    if pools[2] is not None:
        scales = pools[3][table.long()].transpose(1, 2).double().repeat_interleave(c[5], dim=2)
        codes = v / scales[..., None]
    val, bound = pag.attention(Q, k, v, codes, scales, tau, cap=cap)
    if cap:  # the reference counts an error of tanh as an absolute one of 2^-21; near 0 it is relative
        small, bound_small = pag.attention(Q, k, v, codes, scales, tau)
        z = float((Q.double().abs().amax() * k.abs().amax() * c[6] * tau))
        if z < cap * 2.0 ** -14:  # then the cap changes a score by less than 2^-28 of it
            val, bound = small, bound_small
    assert ref.worst(L, val["L"], bound["L"]) <= 1
    assert ref.worst(O, val["O"], bound["O"]) <= 1


@pytest.mark.parametrize("c", CASES, ids=IDS)
@pytest.mark.parametrize("e,q,k,cap", [(100, -55, -45, 0), (-100, 55, 45, 0), (0, -40, 43, 0), (0, 45, -45, 0), (0, 45, -45, 30.0),
                                       (60, -100, 40, 20.0), (0, -50, 50, 2.0 ** 110), (0, -36, 40, 2.0 ** 100),
                                       (0, -36, 36, 2.0 ** 90), (0, 45, -45, 2.0 ** 110), (30, -60, 30, 2.0 ** 119),
                                       (0, -30, 30, 2.0 ** 70), (0, -45, 45, 2.0 ** 80), (-60, 30, 30, 2.0 ** 50)])
def test_scores_of_order_one(c, e, q, k, cap):
    """tau = 2^e / sqrt(d) with queries and keys that make up for it, and caps that are none."""
    check(c, *build(c, q, k), 2.0 ** e / math.sqrt(c[6]), cap)


@pytest.mark.parametrize("c", CASES, ids=IDS)
@pytest.mark.parametrize("e,q,cap", [(50, 8, 0), (100, -45, 0), (30, 28, 0), (-100, 120, 0), (50, 8, 30.0), (100, -45, 2.0 ** 30),
                                     (90, -35, 2.0 ** 79)])
def test_keys_of_zero(c, e, q, cap):
    """Their scores are 0, with queries times tau up to 2^60."""
    Q, pools, values, table = build(c, q, 0)
    pools[0], values[0] = torch.zeros_like(pools[0]), torch.zeros_like(values[0])
    check(c, Q, pools, values, table, 2.0 ** e, cap)


@pytest.mark.parametrize("e,q,k,cap,bias", [(12, 0, 0, 0, 0), (21, 0, 0, 0, 0), (12, 0, 0, 2.0 ** 20, 0), (12, 0, 0, 0, 2.0 ** 10),
                                            (27, 0, 0, 0, 0), (27, 0, 0, 2.0 ** 60, 0), (40, 10, 0, 0, 0), (40, 10, 0, 0, 2.0 ** 40),
                                            (40, 10, 0, 2.0 ** 60, 0), (20, 20, 40, 0, 0), (20, 20, 40, 0, 2.0 ** 40)])
@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_scores_far_apart(c, e, q, k, cap, bias):
    """Scores that fp32 holds to several units: the largest has all the weight."""
    Q, pools, values, table = build(c, q, k)
    B, H, Hkv, Nq, M, T, d = c[:7]
    if c[8] is not E4M3 and e + q + k > 25:
        return  # beyond what is asked of a 16-bit cache, as of dense keys
    slopes = torch.full((H,), bias, device="cuda") if bias else None
    q_pos = (M * T + torch.arange(Nq, device="cuda")).expand(B, Nq).int().contiguous()  # behind all keys
    tau = 2.0 ** e
    O, L = fb.attention_paged(Q, fb.PagedCache(*pools), table, tau, cap=cap, slopes=slopes, q_pos=q_pos)
    ks, vs = (pag.dense(x, table).repeat_interleave(H // Hkv, dim=1) for x in values)
    z = Q.double() @ ks.transpose(2, 3) * tau
    # What 32-bit sums of the products and their roundings lose, here with a bias too.
    err = (d + 8) * 2.0 ** -23 * (Q.double().abs() @ ks.abs().transpose(2, 3) * tau).amax(dim=3)
    if cap:
        z = cap * torch.tanh(z / cap)
        err = err + z.abs().amax(dim=3) * 2.0 ** -20  # tanh's, relative (2^-21), and its factors'
    if bias:
        far = bias * (q_pos[:, None, :, None] - torch.arange(M * T, device="cuda")).double()
        z = z - far
        err = err + far.amax(dim=3) * 2.0 ** -22
    top, at = z.topk(2, dim=3)
    sure = top[..., 0] - top[..., 1] > 2 * err + 25
    assert bool(sure.float().mean() > 0.5)
    assert bool(((L.double() - top[..., 0]).abs() <= err + top[..., 0].abs() * 2.0 ** -21 + 12).all())
    want = torch.gather(vs, 2, at[..., :1].expand(*at.shape[:3], vs.shape[3]))
    assert bool(O.isfinite().all())
    # The others' part: a weight of e^-25 at most each.
    rest = M * T * math.exp(-25) * vs.abs().amax(dim=2)[:, :, None]
    assert bool(((O.double() - want).abs() <= 2.0 ** -7 * want.abs() + rest)[sure].all())
