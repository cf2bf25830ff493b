"""Attention at the ends of tau's range, against the 64-bit definition: inputs
scaled against tau, so that the scores stay of order one, with lengths that
leave padding in the last tile and biases of either sign."""
import math

import pytest
import torch

from tests import layer_reference as ref
from tests.test_gpu_attention import BF, check, make, run

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


@pytest.mark.parametrize("slope", [-1.0, 0.0])
def test_rows_behind_the_last_add_nothing(slope):
    """The padding of the last tile of rows, where exp of a score below every
    other one is not 0: tau near 2^-100 and a bias that grows with the distance."""
    x, form, tau = scaled(dict(B=1, H=1, Hkv=1, Nq=70, Nk=600, d=64, dtype=BF), -100, slope)
    got = run(x, form, tau, 0.0, False)
    val, bound = ref.attention(x["Q"], x["K"], x["V"], tau, dO=x["dO"], **form)
    check(got, val, bound)
