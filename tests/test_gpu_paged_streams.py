"""Streams of the calls on a paged cache: the one that is given works, and calls that
run at the same time, in streams or replayed graphs, do not meet."""
import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests import paged_reference as pag

pytestmark = pytest.mark.gpu

BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def calls():
    """Every call as a function of the stream."""
    pools, _ = pag.pools(6, 2, 16, 64, E4M3)
    cache = fb.PagedCache(*pools)
    table = pag.table_of(2, 3, 6)
    x = torch.randn((2, 3, 8, 64), device="cuda").to(BF)
    Q = torch.randn((2, 4, 20, 64), device="cuda").to(BF)
    return [
        lambda s: fb.cache_append(x, 4, cache, table, stream=s),
        lambda s: fb.cache_read(cache, table, 40, stream=s),
        lambda s: fb.attention_paged(Q, cache, table, 0.1, stream=s),
        lambda s: fb.attention_paged(Q[:, :, :1].contiguous(), cache, table, 0.1, stream=s),
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

    for call in calls():
        with pytest.raises(ValueError):
            call(Elsewhere())


@pytest.mark.parametrize("Nq,B,Hkv", [(1, 1, 1), (1, 30, 8), (3, 2, 2), (40, 1, 2), (200, 2, 2)])
def test_calls_at_the_same_time(Nq, B, Hkv):
    """Split calls have workspaces of their own, on two streams and in two graphs."""
    M, T, d = 128, 64, 128
    pools, _ = pag.pools(B * M, Hkv, T, d, E4M3)
    cache, table = fb.PagedCache(*pools), pag.table_of(B, M, B * M)
    Q = [torch.randn((B, 4 * Hkv, Nq, d), device="cuda").to(BF) for _ in range(2)]
    lens = torch.randint(M * T // 4, M * T + 1, (B, 1), device="cuda")
    hi = (lens - Nq + 1 + torch.arange(Nq, device="cuda")).int()
    ranges = torch.stack([torch.zeros_like(hi), hi], dim=2).contiguous()
    want = [fb.attention_paged(q, cache, table, 0.1, ranges=ranges) for q in Q]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [fb.attention_paged(q, cache, table, 0.1, ranges=ranges, stream=s)
               for q, s in zip(Q, side)]
    torch.cuda.synchronize()
    graphs, out = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for q, graph in zip(Q, graphs):
        with torch.cuda.graph(graph):
            out.append(fb.attention_paged(q, cache, table, 0.1, ranges=ranges))
    for _ in range(5):
        for graph, s in zip(graphs, side):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for w, a, b in zip(want, got, out):
        for x, y, z in zip(w, a, b):
            assert torch.equal(x, y) and torch.equal(x, z)
