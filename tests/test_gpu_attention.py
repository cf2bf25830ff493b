"""Attention with capped scores, a distance bias and key ranges against the
64-bit definition, element by element within the bounds of its roundings."""
import math

import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def offsets(B, M, used, seed=0):
    g = torch.Generator().manual_seed(seed)
    cut = (torch.rand((B, M + 1), generator=g).sort(dim=1).values * used).int()
    cut[:, 0], cut[:, M] = 0, used
    return cut.cuda()


def make(B, H, Hkv, Nq, Nk, d, dtype, mask="none", bias=False, seed=0, **_):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=g, device="cuda").to(dtype)

    x = dict(Q=r(B, H, Nq, d), K=r(B, Hkv, Nk, d), V=r(B, Hkv, Nk, d), dO=r(B, H, Nq, d))
    form = dict(slopes=None, ranges=None, q_pos=None)
    if bias:
        form["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    if mask in ("docs", "prefix"):
        off = offsets(B, 4, max(1, Nk - Nk // 8), seed)
        pre = ((off[:, 1:] - off[:, :-1]) // 3).contiguous() if mask == "prefix" else None
        form["ranges"], form["q_pos"] = fb.attention_ranges(B, Nq, Nk, doc_offsets=off, prefix=pre,
                                                            causal=True)
    elif mask == "random":  # any ranges at all: long, short, empty, beyond the ends
        lo = torch.randint(-5, Nk, (B, Nq), generator=g, device="cuda")
        n = torch.randint(-3, Nk + 5, (B, Nq), generator=g, device="cuda")
        form["ranges"] = torch.stack([lo, lo + n], dim=2).int()
        form["q_pos"] = torch.randint(-4, Nk + 4, (B, Nq), generator=g, device="cuda").int()
    elif mask == "token":  # the last tokens of requests of several lengths
        last = torch.randint(1, Nk + 1, (B, 1), generator=g, device="cuda")
        pos = (last - Nq + torch.arange(Nq, device="cuda")).int()
        form["q_pos"] = pos
        form["ranges"] = torch.stack([torch.zeros_like(pos), pos + 1], dim=2).contiguous()
    elif mask == "nothing":
        form["ranges"] = torch.zeros((B, Nq, 2), dtype=torch.int32, device="cuda")
    return x, form


def poison(x, form, causal):
    """NaN and infinity wherever the mask leaves nothing: rows that see no
    key, and keys outside the run that the batch entry's queries see."""
    B, H, Nq, d = x["Q"].shape
    Nk = x["K"].shape[2]
    see, _ = ref.visible(B, Nq, Nk, form["ranges"], form["q_pos"], causal)
    dead = ~see.any(dim=2)
    j = torch.arange(Nk, device="cuda")
    first = torch.where(see, j, Nk).amin(dim=(1, 2))[:, None]
    last = torch.where(see, j, -1).amax(dim=(1, 2))[:, None]
    out = (j < first) | (j > last)
    for n, bad in (("Q", math.nan), ("dO", math.inf)):
        x[n][dead[:, None].expand(B, H, Nq)] = bad
    for n, bad in (("K", math.inf), ("V", math.nan)):
        x[n][out[:, None].expand(B, x[n].shape[1], Nk)] = bad
    return x


def run(x, form, tau, cap, causal, stream=None):
    O, L = fb.attention(x["Q"], x["K"], x["V"], tau, cap=cap, causal=causal, stream=stream, **form)
    dQ, dK, dV = fb.attention_grad(x["Q"], x["K"], x["V"], O, L, x["dO"], tau, cap=cap,
                                   causal=causal, stream=stream, **form)
    return dict(O=O, L=L, dQ=dQ, dK=dK, dV=dV)


def check(got, val, bound):
    torch.cuda.synchronize()
    assert fb.flashbob_last_device_error() == fb.FLASHBOB_OK
    for k in val:
        assert got[k].shape == val[k].shape
        share = ref.worst(got[k], val[k], bound[k])
        assert share <= 1.0, f"{k}: {share:.2f} of its bound"


C = dict(B=1, H=1, Hkv=1, Nq=64, Nk=64, d=64, dtype=BF, mask="none", bias=False, cap=0.0,
         causal=False)
CASES = [
    # one token, one key
    dict(Nq=1, Nk=1), dict(Nq=1, Nk=1, dtype=F32, d=3), dict(Nq=1, Nk=1, d=128, mask="nothing"),
    dict(Nq=5, Nk=1, d=128), dict(Nq=1, Nk=300, causal=True),
    # head sizes and types
    dict(B=2, H=2, Hkv=2, Nq=65, Nk=65, dtype=F32, d=1), dict(Nq=100, Nk=70, dtype=F32, d=33),
    dict(Nq=130, Nk=190, d=96), dict(Nq=129, Nk=129, d=80, causal=True, cap=10.0, bias=True),
    dict(Nq=200, Nk=200, dtype=F32, d=128, mask="docs", bias=True),
    dict(Nq=200, Nk=200, dtype=F32, d=64, mask="random", cap=5.0),
    dict(H=4, Hkv=2, Nq=67, Nk=130, dtype=F32, d=40, mask="random", cap=5.0, bias=True),
    # tile ends of the tensor-core kernels
    dict(Nq=128, Nk=128), dict(Nq=129, Nk=127), dict(Nq=127, Nk=257, d=128),
    dict(Nq=256, Nk=64, d=128, causal=True), dict(Nq=64, Nk=600), dict(Nq=600, Nk=64, causal=True),
    dict(Nq=300, Nk=900, d=128), dict(B=2, H=3, Hkv=3, Nq=511, Nk=511, causal=True),
    # shared heads: group rows run across heads inside a tile
    dict(B=2, H=6, Hkv=2, Nq=77, Nk=200, causal=True), dict(H=8, Hkv=1, Nq=45, Nk=333, d=128),
    dict(B=2, H=12, Hkv=3, Nq=130, Nk=130, d=128, mask="docs", bias=True),
    # masks
    dict(B=3, H=2, Hkv=2, Nq=700, Nk=700, mask="docs"),
    dict(B=2, H=4, Hkv=2, Nq=450, Nk=450, mask="prefix", d=128),
    dict(B=2, H=4, Hkv=2, Nq=300, Nk=420, mask="random"),
    dict(B=2, H=4, Hkv=4, Nq=300, Nk=420, mask="random", d=128, causal=True, bias=True),
    dict(Nq=200, Nk=200, mask="nothing"), dict(Nq=200, Nk=200, mask="nothing", dtype=F32),
    # caps and biases, alone and together
    dict(B=2, H=2, Hkv=2, Nq=400, Nk=400, cap=2.0), dict(H=2, Hkv=2, Nq=400, Nk=400, cap=0.05, d=128),
    dict(H=3, Hkv=3, Nq=400, Nk=400, bias=True), dict(H=2, Hkv=1, Nq=333, Nk=333, bias=True, d=128),
    dict(H=2, Hkv=2, Nq=400, Nk=400, cap=3.0, bias=True, causal=True),
    dict(B=2, H=4, Hkv=2, Nq=260, Nk=260, cap=3.0, bias=True, mask="prefix", d=128),
    # tokens over a cache
    dict(B=3, H=8, Hkv=2, Nq=1, Nk=1500, mask="token"),
    dict(B=2, H=8, Hkv=1, Nq=1, Nk=4000, mask="token", d=128, cap=4.0),
    dict(B=4, H=4, Hkv=4, Nq=4, Nk=700, mask="token", bias=True),
    dict(B=1, H=3, Hkv=3, Nq=2, Nk=3000, mask="token", dtype=F32, d=48),
    # long
    dict(H=2, Hkv=1, Nq=3000, Nk=3000, causal=True, cap=8.0),
    dict(H=1, Hkv=1, Nq=2500, Nk=2500, mask="docs", d=128),
    # the large blocks of d = 64, and tokens of many requests
    dict(B=2, H=2, Hkv=2, Nq=1300, Nk=1300, mask="docs", bias=True),
    dict(H=4, Hkv=2, Nq=333, Nk=1200, mask="random", cap=3.0),
    dict(B=2, H=2, Hkv=1, Nq=1100, Nk=1100, mask="prefix", cap=2.0, bias=True),
    dict(H=2, Hkv=2, Nq=1100, Nk=1030, causal=True), dict(Nq=150, Nk=1100, mask="nothing"),
    dict(B=80, H=4, Hkv=2, Nq=1, Nk=1500, mask="token", bias=True),
    # biases at positions in no order
    dict(B=2, H=4, Hkv=2, Nq=300, Nk=420, mask="random", bias=True),
    dict(B=2, H=4, Hkv=2, Nq=300, Nk=420, mask="random", bias=True, cap=3.0),
    dict(H=2, Hkv=1, Nq=260, Nk=2300, mask="random", bias=True),
    dict(B=40, H=8, Hkv=2, Nq=12, Nk=1000, mask="token", bias=True),  # the maxima keep rising
    dict(B=40, H=8, Hkv=2, Nq=12, Nk=1100, mask="token", bias=True, d=128),
]


def ident(c):
    return "-".join(f"{k}{str(v).replace('torch.', '')}" for k, v in c.items())


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


@pytest.mark.parametrize("dtype,d", [(F32, 24), (BF, 64), (BF, 128)])
def test_large_scores_and_saturated_caps(dtype, d):
    """Scores of hundreds (one key takes a row), with and without a cap they saturate."""
    x, form = make(1, 2, 2, 200, 300, d, dtype, mask="random", seed=3)
    x["Q"] *= 30
    for cap in (0.0, 15.0):
        got = run(x, form, 1.0, cap, False)
        val, bound = ref.attention(x["Q"], x["K"], x["V"], 1.0, cap=cap, dO=x["dO"], **form)
        check(got, val, bound)


@pytest.mark.parametrize("d", [16, 64, 128])
def test_gradient_agrees_with_differences(d):
    """The directional derivative of sum(O * dO) along a random direction, by
    central differences of the 64-bit forward, against the kernels' gradient."""
    x, form = make(1, 4, 2, 150, 150, d, F32, mask="prefix", bias=True, seed=5)
    tau, cap = 1 / math.sqrt(d), 6.0
    if d != 16:
        x = {k: v.to(BF) for k, v in x.items()}
    got = run(x, form, tau, cap, False)
    g = torch.Generator(device="cuda").manual_seed(9)
    for name, grad in (("Q", "dQ"), ("K", "dK"), ("V", "dV")):
        u = torch.randn(x[name].shape, generator=g, device="cuda", dtype=torch.float64)
        h, vals = 1e-4, []
        for sign in (1, -1):
            y = {k: v.double() for k, v in x.items()}
            y[name] = y[name] + sign * h * u
            O = ref.attention(y["Q"], y["K"], y["V"], tau, cap=cap, **form)[0]["O"]
            vals.append((O * y["dO"]).sum())
        want = float((vals[0] - vals[1]) / (2 * h))
        have = float((got[grad].double() * u).sum())
        # Random signs: the error of the sum is the error's norm times a normal
        # number (5 taken); each element's relative error is at most 2^-6 (a few
        # roundings), and the difference itself is good to 1e-6.
        eps = 2.0 ** -6 if got[grad].dtype == BF else 1e-4
        assert abs(have - want) <= 5 * eps * float(got[grad].double().norm()) + 1e-6 * abs(want)


@pytest.mark.parametrize("dtype,d", [(F32, 24), (BF, 64), (BF, 128)])
def test_same_bits_every_time_and_on_another_stream(dtype, d):
    x, form = make(2, 4, 2, 333, 333, d, dtype, mask="docs", bias=True, seed=7)
    a = run(x, form, 0.2, 9.0, False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = run(x, form, 0.2, 9.0, False, stream=side)
    c = run(x, form, 0.2, 9.0, False, stream=side.cuda_stream)
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


@pytest.mark.parametrize("dtype,d,Nq", [(F32, 24, 40), (BF, 64, 300), (BF, 128, 300), (BF, 128, 1)])
def test_captured_and_replayed(dtype, d, Nq):
    """Two captured graphs, replayed together on two streams with new inputs
    in the same buffers, give what direct calls give."""
    forms, xs, graphs, outs = [], [], [], []
    for seed in (1, 2):
        x, form = make(2, 4, 2, Nq, 700, d, dtype, mask="token", seed=seed)
        run(x, form, 0.1, 0.0, False)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(x, form, 0.1, 0.0, False)
        forms.append(form), xs.append(x), graphs.append(g), outs.append(out)
    fresh = []
    for seed in (0, 1):
        y, form = make(2, 4, 2, Nq, 700, d, dtype, mask="token", seed=11 + seed)
        for k in y:
            xs[seed][k].copy_(y[k])
        for k in ("ranges", "q_pos"):
            forms[seed][k].copy_(form[k])
        fresh.append(run(y, form, 0.1, 0.0, False))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, fresh):
        for k in want:
            assert torch.equal(out[k], want[k]), k


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 40)])
def test_calls_behind_one_another_on_one_workspace(dtype, d):
    """A gradient's launches overlap; what follows on the stream must find them
    done: the next call on the same workspace, and a kernel that reads dQ."""
    tau, sets = 0.2, []
    for seed in (1, 2):
        x, form = make(2, 6, 2, 700, 700, d, dtype, mask="docs", bias=True, seed=seed)
        O, L = fb.attention(x["Q"], x["K"], x["V"], tau, **form)
        sets.append((x, form, O, L))
    x = sets[0][0]
    bwd = fb.flashbob_attention_workspace(2, 6, 2, 700, 700, d, int(dtype == BF))[1]
    workspace = torch.empty(bwd, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(x[k]) for k in ("Q", "K", "V")]

    def call(k):
        x, form, O, L = sets[k]
        fb.flashbob_attention_grad(x["Q"], x["K"], x["V"], O, L, x["dO"], form["ranges"],
                                   form["q_pos"], form["slopes"], tau, 0.0, *outs, workspace)

    want = []
    for k in (0, 1):
        call(k)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])

    def several():
        got = []
        for n in range(12):
            call(n % 2)
            got.append([t.clone() for t in outs])
        return got

    def same(got):
        torch.cuda.synchronize()
        return all(torch.equal(a, b) for n in range(12) for a, b in zip(got[n], want[n % 2]))

    assert same(several())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = several()
    for _ in range(3):
        graph.replay()
    assert same(got)


@pytest.mark.parametrize("dtype,d", [(F32, 20), (BF, 64), (BF, 128)])
def test_writes_its_outputs_and_nothing_else(dtype, d):
    """Outputs and workspace inside larger buffers: the bytes around them stay."""
    B, H, Hkv, Nq, Nk = 2, 4, 2, 70, 900
    x, form = make(B, H, Hkv, Nq, Nk, d, dtype, mask="token")
    fwd, bwd = fb.flashbob_attention_workspace(B, H, Hkv, Nq, Nk, d, 1 if dtype == BF else 0)
    pads, views = [], []

    def inside(shape, t):
        n = math.prod(shape)
        buf = torch.full((n + 256,), 7, dtype=t, device="cuda")
        pads.append((buf, n))
        views.append(buf[128:128 + n].view(shape))
        return views[-1]

    O, L = inside((B, H, Nq, d), dtype), inside((B, H, Nq), F32)
    dQ, dK, dV = (inside(x[k].shape, dtype) for k in ("Q", "K", "V"))
    w1 = inside((fwd,), torch.uint8) if fwd else None
    w2 = inside((bwd,), torch.uint8)
    args = (form["ranges"], form["q_pos"], None, 0.1, 0.0)
    fb.flashbob_attention(x["Q"], x["K"], x["V"], *args, O, L, w1)
    fb.flashbob_attention_grad(x["Q"], x["K"], x["V"], O, L, x["dO"], *args, dQ, dK, dV, w2)
    torch.cuda.synchronize()
    for buf, n in pads:
        assert (buf[:128] == 7).all() and (buf[128 + n:] == 7).all()
    want = run(x, form, 0.1, 0.0, False)
    for k, v in zip(("O", "L", "dQ", "dK", "dV"), views):
        assert torch.equal(v, want[k]), k


def test_offsets_past_32_bits():
    """A cache of 2.2e9 elements: only 300 keys at the very end of the last
    batch entry are seen, the rest holds NaN."""
    B, H, Hkv, Nk, d, n = 2, 4, 2, 4_300_000, 128, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    K, V = (torch.full((B, Hkv, Nk, d), math.nan, dtype=BF, device="cuda") for _ in range(2))
    for t in (K, V):
        t[:, :, Nk - n:] = torch.randn((B, Hkv, n, d), generator=g, device="cuda").to(BF)
    Q, dO = (torch.randn((B, H, 3, d), generator=g, device="cuda").to(BF) for _ in range(2))
    ranges = torch.tensor([[Nk - n, Nk], [Nk - n, Nk - 1], [Nk, Nk]], dtype=torch.int32,
                          device="cuda").expand(B, 3, 2).contiguous()
    O, L = fb.attention(Q, K, V, 0.1, ranges=ranges)
    dQ, dK, dV = fb.attention_grad(Q, K, V, O, L, dO, 0.1, ranges=ranges)
    k, v = K[:, :, Nk - n:].contiguous(), V[:, :, Nk - n:].contiguous()
    val, bound = ref.attention(Q, k, v, 0.1, ranges=ranges - (Nk - n), dO=dO)
    got = dict(O=O, L=L, dQ=dQ, dK=dK[:, :, Nk - n:], dV=dV[:, :, Nk - n:])
    check(got, val, bound)
    assert not dK[:, :, :Nk - n].any() and not dV[:, :, :Nk - n].any()


def test_ranges_match_their_definition():
    for B, M, Nq, Nk in ((1, 1, 1, 1), (3, 5, 300, 200), (2, 40, 5000, 5000), (1, 9000, 9500, 9500)):
        off = offsets(B, M, Nk - Nk // 10 if Nk > 1 else 1, seed=M)
        if M > 3:
            off[:, 2] = off[:, 1]  # an empty document
            off[0, 0] = min(3, int(off[0, 1]))  # queries before the first
        pre = ((off[:, 1:] - off[:, :-1]) * 2 // 3 + 1).int().contiguous()
        start = torch.arange(B, device="cuda", dtype=torch.int32) * 7 - 3
        for causal in (False, True):
            for prefix in (None, pre):
                for q_start in (None, start):
                    got, pos = fb.attention_ranges(B, Nq, Nk, doc_offsets=off, prefix=prefix,
                                                   q_start=q_start, causal=causal)
                    want_pos = torch.arange(Nq).expand(B, Nq).clone()
                    if q_start is not None:
                        want_pos += q_start.cpu()[:, None]
                    o = off.cpu().long()
                    at = torch.searchsorted(o, want_pos.contiguous(), right=True) - 1
                    ok = (at >= 0) & (at < M) & (want_pos >= 0)
                    at = at.clamp(0, M - 1)
                    lo, end = o.gather(1, at), o.gather(1, at + 1)
                    hi = end
                    if causal:
                        hi = want_pos + 1
                        if prefix is not None:
                            hi = torch.maximum(hi, lo + pre.cpu().long().gather(1, at))
                        hi = torch.minimum(hi, end)
                    hi = hi.clamp(max=Nk)
                    want = torch.stack([torch.where(ok, lo, 0), torch.where(ok, hi, 0)], dim=2)
                    assert torch.equal(got.cpu().long(), want)
                    assert torch.equal(pos.cpu().long(), want_pos)
    got, pos = fb.attention_ranges(2, 3, 10, q_start=torch.tensor([4, -1], dtype=torch.int32).cuda(),
                                   causal=True)
    assert got.tolist() == [[[0, 5], [0, 6], [0, 7]], [[0, 0], [0, 1], [0, 2]]]
    assert fb.attention_ranges(1, 2, 10)[0].tolist() == [[[0, 10], [0, 10]]]

    # without documents every position from 0 on is in the one there is
    got, pos = fb.attention_ranges(1, 4, 5, q_start=torch.tensor([3], dtype=torch.int32).cuda(),
                                   causal=True)
    assert got[0].tolist() == [[0, 4], [0, 5], [0, 5], [0, 5]] and pos[0].tolist() == [3, 4, 5, 6]


def test_wrong_arguments_are_refused():
    x, form = make(1, 2, 1, 8, 8, 64, BF, mask="docs")
    ok = dict(tau=0.1, **form)
    Q, K, V = x["Q"], x["K"], x["V"]
    with pytest.raises(ValueError):
        fb.attention(Q, K, V[:, :, :4].contiguous(), **ok)
    with pytest.raises(TypeError):
        fb.attention(Q, K, V.float(), **ok)
    with pytest.raises(TypeError):
        fb.attention(Q.half(), K.half(), V.half(), **ok)
    with pytest.raises(ValueError):
        fb.attention(Q.transpose(2, 3).contiguous().transpose(2, 3), K, V, **ok)
    with pytest.raises(ValueError):
        fb.attention(Q, K, V, tau=0.1, ranges=form["ranges"][:, :4].contiguous())
    with pytest.raises(TypeError):
        fb.attention(Q, K, V, tau=0.1, ranges=form["ranges"].long())
    with pytest.raises(ValueError):
        fb.attention(Q, K, V, tau=0.1, slopes=torch.ones(3, device="cuda"))
    with pytest.raises(ValueError):
        fb.attention(Q.cpu(), K, V, tau=0.1)
    for kw in (dict(tau=-1.0), dict(tau=0.1, cap=-1.0), dict(tau=0.1, cap=math.inf)):
        with pytest.raises(fb.FlashbobError):
            fb.attention(Q, K, V, **kw)
    O, L = fb.attention(Q, K, V, **ok)
    with pytest.raises(fb.FlashbobError):  # a workspace that is too small
        fb.flashbob_attention_grad(Q, K, V, O, L, x["dO"], form["ranges"], form["q_pos"], None, 0.1,
                                   0.0, *(torch.empty_like(t) for t in (Q, K, V)),
                                   torch.empty(64, dtype=torch.uint8, device="cuda"))
