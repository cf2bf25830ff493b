"""What a mask hides reaches nothing, not even a last bit: calls whose hidden
rows hold zeros, large numbers, infinities or NaN give the same bits."""
import math

import pytest
import torch

from tests import layer_reference as ref
from tests.test_gpu_attention import BF, F32, make, run

pytestmark = pytest.mark.gpu


def fill(x, form, causal, value):
    """x with `value` in the rows that see nothing and in the keys outside the
    run that the batch entry's queries see."""
    B, H, Nq, _ = x["Q"].shape
    Nk = x["K"].shape[2]
    see, _ = ref.visible(B, Nq, Nk, form["ranges"], form["q_pos"], causal)
    dead = ~see.any(dim=2)[:, None]
    j = torch.arange(Nk, device="cuda")
    first = torch.where(see, j, Nk).amin(dim=(1, 2))[:, None]
    last = torch.where(see, j, -1).amax(dim=(1, 2))[:, None]
    out = ((j < first) | (j > last))[:, None]
    y = {k: v.clone() for k, v in x.items()}
    for n, rows in (("Q", dead), ("dO", dead), ("K", out), ("V", out)):
        y[n][rows.expand(B, y[n].shape[1], -1)] = value
    return y


CASES = [dict(B=2, H=4, Hkv=2, Nq=1, Nk=700, mask="token"), dict(B=3, H=4, Hkv=2, Nq=1, Nk=1500, mask="token"),
         dict(B=2, H=2, Hkv=2, Nq=300, Nk=300, mask="docs"), dict(B=1, H=2, Hkv=1, Nq=200, Nk=1300, mask="token"),
         dict(B=2, H=2, Hkv=2, Nq=250, Nk=250, mask="random", bias=True)]


@pytest.mark.parametrize("cap", [0.0, 30.0, 1e4])
@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (BF, 96), (F32, 64)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_the_same_bits_whatever_hidden_rows_hold(case, dtype, d, cap):
    x, form = make(d=d, dtype=dtype, seed=3, **case)
    want = run(fill(x, form, False, 0.0), form, 1 / math.sqrt(d), cap, False)
    for value in (300.0, math.inf, math.nan):
        got = run(fill(x, form, False, value), form, 1 / math.sqrt(d), cap, False)
        for k in want:
            assert torch.equal(got[k], want[k]), (k, value)
