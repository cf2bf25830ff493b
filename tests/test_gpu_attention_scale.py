"""Attention at the ends of tau's range, against the 64-bit definition: inputs
scaled against tau, so that the scores stay of order one, with lengths that
leave padding in the last tile and biases of either sign."""
import math

import pytest
import torch

from tests import layer_reference as ref
from tests.test_gpu_attention import BF, F32, check, make, run

pytestmark = pytest.mark.gpu


def scaled(shape, e, slope, far=0):
    """tau = 2^e / sqrt(d), Q and K times 2^(-e / 2) each; queries `far` keys
    behind their index."""
    x, form = make(**shape)
    x["Q"] *= 2.0 ** (-(e // 2))
    x["K"] *= 2.0 ** (-(e - e // 2))
    if slope:
        form["slopes"] = torch.full((shape["H"],), slope, device="cuda")
    if far:
        form["q_pos"] = (torch.arange(shape["Nq"], device="cuda").expand(shape["B"], -1)
                         + far).int().contiguous()
    return x, form, 2.0 ** e / math.sqrt(shape["d"])


def shape_rows(x):
    """Query rows that share a key head."""
    return x["Q"].shape[1] // x["K"].shape[1] * x["Q"].shape[2]


@pytest.mark.parametrize("slope,far", [(0.0, 0), (-0.7, 0), (1.0, 0), (1.0, 3000)])
@pytest.mark.parametrize("e", [-115, -61, -40, 40, 61, 115])
@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64)])
def test_ends_of_the_range_of_tau(dtype, d, e, slope, far):
    x, form, tau = scaled(dict(B=1, H=2, Hkv=1, Nq=150, Nk=200, d=d, dtype=dtype), e, slope, far)
    got = run(x, form, tau, 0.0, False)
    val, bound = ref.attention(x["Q"], x["K"], x["V"], tau, dO=x["dO"], **form)
    # The sums of dS k and dS^T q are formed before the factor tau, from keys and
    # queries of 2^(-e / 2): a product below 2^-126, the smallest normal number of
    # fp32, may be flushed to 0, 2^-126 absolute for each of the sum's terms, and
    # tau multiplies it (at e = 115 weights below 2^-69 are lost that way).  The
    # results, scaled by 2^(e / 2), may be flushed once more.
    for k, n in (("dQ", x["K"].shape[2]), ("dK", shape_rows(x))):
        bound[k] = bound[k] + (n * tau + 1) * 2.0 ** -126
    check(got, val, bound)


@pytest.mark.parametrize("slope", [-1.0, 0.0])
def test_rows_behind_the_last_add_nothing(slope):
    """The padding of the last tile of rows, where exp of a score below every
    other one is not 0: tau near 2^-100 and a bias that grows with the distance."""
    x, form, tau = scaled(dict(B=1, H=1, Hkv=1, Nq=70, Nk=600, d=64, dtype=BF), -100, slope)
    got = run(x, form, tau, 0.0, False)
    val, bound = ref.attention(x["Q"], x["K"], x["V"], tau, dO=x["dO"], **form)
    check(got, val, bound)
