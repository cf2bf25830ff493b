"""Sizes that do not fit the C ABI's int are refused, not cut to 32 bits."""
import pytest
import torch

from exact_second_order_gb300 import flashbob as fb

BIG = 2 ** 32 + 5  # its low 32 bits are a fine size


@pytest.mark.parametrize("at", range(6))
def test_attention_workspace(at):
    sizes = [1, 1, 1, 8, 8, 64]
    sizes[at] = BIG
    with pytest.raises(ValueError):
        fb.flashbob_attention_workspace(*sizes, 1)


@pytest.mark.parametrize("at", range(5))
def test_norm_workspace(at):
    sizes = [1, 8, 2, 1, 64]
    sizes[at] = BIG
    with pytest.raises(ValueError):
        fb.flashbob_qk_norm_rope_workspace(*sizes, 1)


@pytest.mark.gpu
def test_ranges_and_caches():
    with pytest.raises(ValueError):
        fb.attention_ranges(1, 4, BIG)
    # 2^31 rows and some of one element, all in one place: refused by shape alone
    row = torch.zeros((1, 1, 1, 1), dtype=torch.bfloat16, device="cuda")
    long = row.expand(1, 1, BIG, 1)
    with pytest.raises(ValueError):
        fb.attention(row, long, long, 1.0)
    x = torch.zeros((1, 1, 3, 1), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="sizes"):
        fb.qk_norm_rope(x, 1, K=long, V=long)
