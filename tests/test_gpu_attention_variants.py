"""Variants of the tensor-core attention kernels that only larger calls reach,
against the 64-bit definition with NaN and infinities in the masked places."""
import math

import pytest

from tests import layer_reference as ref
from tests.test_gpu_attention import C, check, ident, make, poison, run

pytestmark = pytest.mark.gpu

CASES = [
    # forward with 256 rows a block at d = 128: 304 such blocks at least
    dict(B=8, H=10, Hkv=10, Nq=1000, Nk=1000, d=128, causal=True),
    dict(B=8, H=20, Hkv=10, Nq=500, Nk=700, d=128, mask="random"),
    dict(B=8, H=10, Hkv=10, Nq=1000, Nk=1000, d=128, mask="docs", cap=4.0),
    dict(B=16, H=20, Hkv=20, Nq=257, Nk=300, d=128, mask="random", bias=True),
    dict(B=8, H=20, Hkv=10, Nq=500, Nk=500, d=128, mask="prefix", cap=4.0, bias=True),
    dict(B=40, H=8, Hkv=8, Nq=130, Nk=130, d=128, mask="nothing"),
    # dQ in large blocks at d = 64: more than 2048 keys
    dict(H=2, Hkv=2, Nq=2300, Nk=2300, causal=True), dict(H=2, Hkv=1, Nq=900, Nk=2100, mask="random"),
    dict(B=2, H=2, Hkv=2, Nq=500, Nk=2177, mask="random", cap=4.0, bias=True),
    # dK, dV with two blocks to a cluster, and with eight
    dict(H=32, Hkv=8, Nq=1000, Nk=1100, mask="random"),
    dict(H=32, Hkv=8, Nq=1000, Nk=1100, d=128, mask="random", cap=4.0, bias=True),
    dict(H=8, Hkv=1, Nq=1500, Nk=300, causal=True, bias=True),
    dict(H=8, Hkv=1, Nq=1500, Nk=300, d=128, mask="random"),
    # capped tokens at d = 64, in small blocks and in large ones
    dict(B=3, H=8, Hkv=2, Nq=1, Nk=1000, mask="token", cap=4.0),
    dict(B=3, H=8, Hkv=2, Nq=2, Nk=1500, mask="token", cap=4.0, bias=True),
]


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_matches_the_definition(case):
    c = C | case
    x, form = make(**c)
    x = poison(x, form, c["causal"])
    tau = 1.3 / math.sqrt(c["d"])
    got = run(x, form, tau, c["cap"], c["causal"])
    val, bound = ref.attention(x["Q"], x["K"], x["V"], tau, cap=c["cap"], causal=c["causal"],
                               dO=x["dO"], **form)
    check(got, val, bound)
