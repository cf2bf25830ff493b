"""The stream argument of the layer's operators: a torch stream, a handle, or
the handle 0 of the default stream, as in the calls of the C ABI."""
import pytest
import torch

from exact_second_order_gb300 import flashbob as fb

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def calls():
    """Every operator's call as a function of the stream."""
    Q = torch.randn(1, 2, 40, 64, device="cuda").to(BF)
    O, L = fb.attention(Q, Q, Q, 0.1)
    x = torch.randn(1, 40, 6, 64, device="cuda").to(BF)
    off = torch.tensor([[0, 20, 40]], dtype=torch.int32, device="cuda")
    o, l, r = torch.empty_like(O), torch.empty_like(L), torch.empty((1, 40, 2), dtype=torch.int32,
                                                                    device="cuda")
    return [
        lambda s: fb.attention(Q, Q, Q, 0.1, stream=s),
        lambda s: fb.attention_grad(Q, Q, Q, O, L, Q, 0.1, stream=s),
        lambda s: fb.attention_ranges(1, 40, 40, doc_offsets=off, stream=s),
        lambda s: fb.qk_norm_rope(x, 2, stream=s),
        lambda s: fb.qk_norm_rope_grad(x, Q, Q, Q, stream=s),
        lambda s: fb.flashbob_attention(Q, Q, Q, None, None, None, 0.1, 0.0, o, l, None, stream=s),
        lambda s: fb.flashbob_attention_ranges(off, None, None, r, None, 40, stream=s),
    ]


def test_the_stream_that_is_given_is_the_one_that_works(monkeypatch):
    ready, used = calls(), []
    inner = fb._raw_stream
    monkeypatch.setattr(fb, "_raw_stream", lambda index: used.append(inner(index)) or used[-1])
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for k, call in enumerate(ready):
        with torch.cuda.stream(other):
            for given, handle in ((None, other.cuda_stream), (0, 0), (side, side.cuda_stream),
                                  (side.cuda_stream, side.cuda_stream),
                                  (torch.cuda.default_stream(), 0)):
                used.clear()
                call(given)
                torch.cuda.synchronize()
                assert used == [handle], (k, given)
                assert torch.cuda.current_stream() == other


def test_a_stream_of_another_device_is_refused():
    class Elsewhere:
        cuda_stream, device = 0, torch.device("cuda", 1)

    for k, call in enumerate(calls()):
        with pytest.raises(ValueError):
            call(Elsewhere())
