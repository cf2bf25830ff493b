"""Attention with large caps (the usual way to switch capping off) and with a
few scores near the cap, against the 64-bit definition.

The error of a capped score is relative to the score, whatever the cap: tanh is
off by 2^-21 relative (a polynomial for |z / cap| <= 1/2, whose first term is
exact; beyond, an absolute error of 2^-22 of a value above 0.46), its argument
and the cap add three roundings of 2^-24, so 2^-20 |c| in all.  An uncapped
score's bound e holds 2^-22 |z| of z = tau q . k, |c| <= |z| and the slope of
tanh is at most 1, so a capped score is off by at most e + 4 e, and L by five
times the bound of the uncapped call.

O is two roundings of the type deep (the weights, O itself), a gradient four (the
weights or score gradients, O within D, O within the products, itself), each
at most u = eps / 2 and taken as independent: 2 u and 4 u of the norm."""
import math

import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests import layer_reference as ref
from tests.test_gpu_attention import BF, F32, check, make, run

pytestmark = pytest.mark.gpu

FORMS = [
    dict(B=1, H=2, Hkv=2, Nq=300, Nk=300, d=64, dtype=BF, causal=True),
    dict(B=1, H=2, Hkv=1, Nq=200, Nk=1300, d=64, dtype=BF),
    dict(B=1, H=2, Hkv=2, Nq=300, Nk=300, d=64, dtype=BF, mask="docs", bias=True),
    dict(B=1, H=2, Hkv=2, Nq=300, Nk=300, d=128, dtype=BF, causal=True),
    dict(B=2, H=2, Hkv=1, Nq=200, Nk=250, d=128, dtype=BF, mask="random", bias=True),
    dict(B=1, H=2, Hkv=2, Nq=150, Nk=150, d=96, dtype=BF, causal=True),
    dict(B=1, H=2, Hkv=2, Nq=150, Nk=150, d=40, dtype=F32, causal=True),
    dict(B=3, H=8, Hkv=2, Nq=1, Nk=900, d=64, dtype=BF, mask="token"),
    dict(B=3, H=8, Hkv=2, Nq=1, Nk=2500, d=64, dtype=BF, mask="token"),
    dict(B=3, H=8, Hkv=2, Nq=1, Nk=900, d=128, dtype=BF, mask="token"),
]


def agree(x, form, tau, cap, causal, got):
    args = (x["Q"], x["K"], x["V"], tau)
    val, _ = ref.attention(*args, cap=cap, causal=causal, dO=x["dO"], **form)
    _, bound = ref.attention(*args, causal=causal, **form)
    check({"L": got["L"]}, {"L": val["L"]}, {"L": 5 * bound["L"]})
    u = torch.finfo(x["Q"].dtype).eps / 2 if x["Q"].dtype == BF else 1e-5
    for k in ("O", "dQ", "dK", "dV"):
        off = float((got[k].double() - val[k]).norm() / val[k].norm())
        assert off <= (2 if k == "O" else 4) * u, f"{k}: {off:.2e}"


@pytest.mark.parametrize("cap", [1e4, 1e6, 1e9, 1e30])
@pytest.mark.parametrize("shape", FORMS, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_a_large_cap_changes_nothing(shape, cap):
    causal = shape.get("causal", False)
    x, form = make(**shape)
    tau = 1 / math.sqrt(shape["d"])
    got = run(x, form, tau, cap, causal)
    agree(x, form, tau, cap, causal, got)
    plain = run(x, form, tau, 0.0, causal)
    u = torch.finfo(x["Q"].dtype).eps / 2 if x["Q"].dtype == BF else 1e-5
    for k in ("O", "dQ", "dK", "dV"):  # each side within its roundings of the definition
        assert float((got[k].double() - plain[k].double()).norm()) <= 8 * u * float(
            plain[k].double().norm()), k


@pytest.mark.parametrize("tau,cap", [(2.0 ** -80, 2.0 ** 36), (2.0 ** 60, 2.0 ** -8),
                                     (2.0 ** -60, 2.0 ** 60), (2.0 ** 40, 2.0 ** 50)])
@pytest.mark.parametrize("d", [64, 128])
def test_ends_of_the_range_of_tau_over_cap(d, tau, cap):
    """Inputs scaled so that the scores stay of order one where the cap allows it."""
    x, form = make(1, 2, 2, 200, 200, d, BF, mask="docs")
    x["Q"] = (x["Q"].double() / (tau * math.sqrt(d))).to(BF)
    O, L = fb.attention(x["Q"], x["K"], x["V"], tau, cap=cap, **form)
    args = (x["Q"], x["K"], x["V"], tau)
    val, _ = ref.attention(*args, cap=cap, **form)
    _, bound = ref.attention(*args, **form)
    check({"L": L}, {"L": val["L"]}, {"L": 5 * bound["L"]})
    off = float((O.double() - val["O"]).norm() / val["O"].norm())
    assert off <= 2 * torch.finfo(BF).eps / 2


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_beside_a_row_near_the_cap(d, bias):
    """One row in eight has scores around the cap; the others, which share its
    tiles, stay as good as without: L and O everywhere, dQ in the other rows.
    In the rows near the cap one key takes nearly all (P = 1 - p), so dP - D is
    of order p |dP| while D = dO . O carries u |dO| |O| from the rounding of O: the
    relative error of their dS is u / p, without a limit, and dK, dV sum those
    rows, times q of 1e4.  So these two are held to the element-wise bounds, which
    count that term."""
    cap, tau = 1e4, 1 / math.sqrt(d)
    x, form = make(1, 2, 2, 256, 300, d, BF, bias=bias)
    x["Q"][:, :, ::8] *= 1e4
    got = run(x, form, tau, cap, False)
    args = (x["Q"], x["K"], x["V"], tau)
    val, bound = ref.attention(*args, cap=cap, dO=x["dO"], **form)
    _, plain = ref.attention(*args, **form)
    check(got, val, bound | {"L": 5 * plain["L"]})
    others = torch.arange(256, device="cuda") % 8 != 0
    for k, n in (("O", 2), ("dQ", 4)):
        a, b = got[k][:, :, others].double(), val[k][:, :, others]
        assert float((a - b).norm() / b.norm()) <= n * torch.finfo(BF).eps / 2, k
