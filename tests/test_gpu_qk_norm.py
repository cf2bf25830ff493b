"""The norm and rotation of queries and keys against the 64-bit definition,
its gradient against autograd of that, and the whole run of the layer's
operators as a model's training step and as a served request use them."""
import math

import pytest
import torch

from exact_second_order_gb300 import flashbob as fb
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(B, N, H, Hkv, d, R, axes, dtype, gain=True, seed=0, far=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s, t=dtype):
        return torch.randn(s, generator=g, device="cuda").to(t)

    x = r(B, N, H + 2 * Hkv, d)
    w = [1 + 0.2 * r(d, t=F32) if gain else None for _ in range(2)]
    freqs = pos = None
    if R:
        freqs = (10000.0 ** (-torch.arange(R // 2, device="cuda") / max(1, R // 2))).expand(axes, -1)
        axis = torch.arange(R // 2, device="cuda") % axes
        freqs = torch.where(axis == torch.arange(axes, device="cuda")[:, None], freqs, 0.0).contiguous()
        top = 2 ** 31 - 1 if far else 5000
        pos = torch.randint(0, top, (axes, B, N), generator=g, device="cuda").int()
    dz = [r(B, h, N, d) for h in (H, Hkv, Hkv)]
    return x, dict(wq=w[0], wk=w[1], freqs=freqs, positions=pos), dz


CASES = [  # B, N, H, Hkv, d, R, axes, interleaved, dtype, gain
    (1, 1, 1, 1, 64, 64, 1, False, BF, True), (2, 3, 4, 2, 128, 128, 1, True, BF, True),
    (1, 7, 3, 1, 1, 0, 1, False, F32, True), (2, 5, 2, 2, 3, 2, 1, False, F32, True),
    (2, 33, 6, 2, 80, 60, 3, True, BF, True), (2, 33, 6, 2, 80, 60, 3, False, BF, False),
    (1, 700, 5, 1, 128, 64, 2, False, F32, True), (3, 500, 8, 4, 64, 32, 4, True, BF, True),
    (1, 1300, 2, 1, 34, 34, 1, False, BF, True), (1, 50, 33, 1, 127, 126, 1, True, F32, True),
    (2, 1500, 4, 2, 128, 128, 1, False, BF, True), (1, 300, 2, 1, 96, 48, 2, False, F32, False),
    (4, 400, 1, 1, 72, 40, 1, False, BF, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_matches_the_definition(case):
    B, N, H, Hkv, d, R, axes, inter, dtype, gain = case
    x, form, dz = make(B, N, H, Hkv, d, R, axes, dtype, gain, far=R == 34)
    u, eps = torch.finfo(dtype).eps / 2, 1e-5
    got = fb.qk_norm_rope(x, H, **form, eps=eps, interleaved=inter)
    grads = fb.qk_norm_rope_grad(x, *dz, **form, eps=eps, interleaved=inter)
    y = x.double().requires_grad_(True)
    w = [None if form[k] is None else form[k].double().requires_grad_(True) for k in ("wq", "wk")]
    want = ref.norm_rope(y, H, w[0], w[1], form["freqs"], form["positions"], eps, inter)
    wants = torch.autograd.grad(want, [y] + ([] if w[0] is None else w), [t.double() for t in dz])
    torch.cuda.synchronize()
    # fp32 arithmetic: the mean of d squares, the square root, the gain, the
    # angle (2^-24 of a half turn, so pi 2^-24) and the turn: (d + 16) 2^-24
    # of the norm of the row's pairs; then one rounding to the type.
    e = (d + 16) * 2.0 ** -24
    for g, t, name in zip(got, want, "QKV"):
        t = t.detach()
        tol = u * t.abs() + (0.0 if name == "V" else e * t.norm(dim=3, keepdim=True))
        assert bool(((g.double() - t).abs() <= tol).all()), name
    dx, t = grads[0].double(), wants[0]
    # The gradient of a row is a projection of r w dz: its terms are bounded by
    # the norms of the row's gradient and input.
    r = torch.rsqrt((y.detach() ** 2).mean(dim=3, keepdim=True) + eps)
    scale = torch.cat([t.double().transpose(1, 2) for t in dz], dim=2).norm(dim=3, keepdim=True) * 2 * (
        1.0 if not gain else max(float(form["wq"].abs().max()), float(form["wk"].abs().max())))
    scale[:, :, :H + Hkv] *= r[:, :, :H + Hkv]
    assert bool(((dx - t).abs() <= u * t.abs() + 2 * e * scale).all())
    if gain:
        # A sum of n products in fp32, by at most n / 256 + 700 sequential additions.
        for k, (g, t, h) in enumerate(zip(grads[1:], wants[1:], (H, Hkv))):
            xh = (y.detach() * r)[:, :, k * H:k * H + h]
            size = (xh.abs() * dz[k].double().transpose(1, 2).norm(dim=3, keepdim=True)).sum(dim=(0, 1, 2))
            n = B * N * h / 256 + 700 + d
            assert bool(((g.double() - t).abs() <= n * 2.0 ** -24 * size).all())
    else:
        assert grads[1] is None and grads[2] is None


def test_gradients_of_the_second_order_call_are_fp32():
    """fp32 gradients (those of flashbob_bob) of a bf16 projection."""
    x, form, dz = make(2, 40, 4, 2, 64, 64, 1, BF)
    a = fb.qk_norm_rope_grad(x, *dz, **form)
    b = fb.qk_norm_rope_grad(x, *[t.float() for t in dz], **form)
    for s, t in zip(a, b):
        assert torch.equal(s, t)


def test_rows_of_a_cache():
    """Only the rows of the new tokens change; rows outside the cache are dropped."""
    B, N, H, Hkv, d, Nk = 4, 3, 4, 2, 64, 10
    x, form, _ = make(B, N, H, Hkv, d, 64, 1, BF)
    Q, K, V = fb.qk_norm_rope(x, H, **form)
    start = torch.tensor([0, 4, 9, -2], dtype=torch.int32).cuda()
    Kc, Vc = (torch.full((B, Hkv, Nk, d), 5.0, dtype=BF, device="cuda") for _ in range(2))
    Q2, K2, V2 = fb.qk_norm_rope(x, H, **form, K=Kc, V=Vc, kv_start=start)
    assert K2 is Kc and V2 is Vc and torch.equal(Q, Q2)
    for c, new in ((Kc, K), (Vc, V)):
        want = torch.full_like(c, 5.0)
        for b, s in enumerate(start.tolist()):
            for n in range(N):
                if 0 <= s + n < Nk:
                    want[b, :, s + n] = new[b, :, n]
        assert torch.equal(c, want)


def test_same_bits_on_another_stream_and_replayed():
    x, form, dz = make(2, 900, 4, 2, 128, 96, 2, BF)

    def run(stream=None):
        return (*fb.qk_norm_rope(x, 4, **form, stream=stream),
                *fb.qk_norm_rope_grad(x, *dz, **form, stream=stream))

    a = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = run(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = run()
    x2, _, dz2 = make(2, 900, 4, 2, 128, 96, 2, BF, seed=4)
    g.replay()
    torch.cuda.synchronize()
    for s, t, v in zip(a, b, c):
        assert torch.equal(s, t) and torch.equal(s, v)
    x.copy_(x2)
    for s, t in zip(dz, dz2):
        s.copy_(t)
    g.replay()
    want = run()
    torch.cuda.synchronize()
    for s, t in zip(want, c):
        assert torch.equal(s, t)


def test_wrong_arguments_are_refused():
    x, form, dz = make(1, 4, 4, 2, 64, 64, 1, BF)
    with pytest.raises(ValueError):
        fb.qk_norm_rope(x, 3, **form)
    with pytest.raises(ValueError):
        fb.qk_norm_rope(x, 8, **form)
    with pytest.raises(ValueError):
        fb.qk_norm_rope(x, 4, **form, K=torch.empty(1, 2, 4, 64, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        fb.qk_norm_rope(x, 4, **form, kv_start=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        fb.qk_norm_rope(x, 4, **(form | {"positions": form["positions"][:, :, :2].contiguous()}))
    for kw in (dict(eps=0.0), dict(eps=math.nan), dict(wk=None)):
        with pytest.raises(fb.FlashbobError):
            fb.qk_norm_rope(x, 4, **(form | kw))
    with pytest.raises(fb.FlashbobError):  # 2 rows for 4 tokens
        fb.qk_norm_rope(x, 4, **form, K=torch.empty(1, 2, 2, 64, dtype=BF, device="cuda"),
                        V=torch.empty(1, 2, 2, 64, dtype=BF, device="cuda"))
    with pytest.raises(TypeError):
        fb.qk_norm_rope_grad(x, dz[0], dz[1].float(), dz[2], **form)


@pytest.mark.parametrize("dtype,d", [(F32, 48), (BF, 64), (BF, 128)])
def test_training_step_of_a_layer(dtype, d):
    """Projection -> norm and rotation -> ranges -> attention, and all the way
    back, against autograd of the 64-bit definition."""
    B, N, H, Hkv = 2, 300, 4, 2
    x, form, _ = make(B, N, H, Hkv, d, d, 1, dtype, seed=2)
    off = torch.tensor([[0, 90, 90, 260], [0, 1, 200, 300]], dtype=torch.int32).cuda()
    pre = torch.tensor([[20, 0, 170], [1, 50, 0]], dtype=torch.int32).cuda()
    dO = torch.randn((B, H, N, d), device="cuda").to(dtype)
    tau, cap = 1 / math.sqrt(d), 20.0
    ranges, q_pos = fb.attention_ranges(B, N, N, doc_offsets=off, prefix=pre, causal=True)
    Q, K, V = fb.qk_norm_rope(x, H, **form)
    O, L = fb.attention(Q, K, V, tau, cap=cap, ranges=ranges, q_pos=q_pos)
    grads = fb.attention_grad(Q, K, V, O, L, dO, tau, cap=cap, ranges=ranges, q_pos=q_pos)
    dx, dwq, dwk = fb.qk_norm_rope_grad(x, *grads, **form)
    y = x.double().requires_grad_(True)
    w = [form[k].double().requires_grad_(True) for k in ("wq", "wk")]
    q, k, v = ref.norm_rope(y, H, w[0], w[1], form["freqs"], form["positions"], 1e-6, False)
    see, _ = ref.visible(B, N, N, ranges, q_pos, False)
    k, v = (t.repeat_interleave(H // Hkv, dim=1) for t in (k, v))
    s = cap * torch.tanh(q @ k.transpose(2, 3) * tau / cap)
    alive = see.any(dim=2)[:, None, :, None]
    s = torch.where(alive, s.masked_fill(~see[:, None], -math.inf), 0.0)
    o = torch.where(alive, torch.softmax(s, dim=3) @ v, 0.0)
    wants = torch.autograd.grad(o, [y, *w], dO.double())
    torch.cuda.synchronize()
    assert fb.flashbob_last_device_error() == fb.FLASHBOB_OK
    # Each stage rounds its outputs (u) and its two inner operands (u): six
    # roundings deep, taken as independent and of at most u each.
    u = torch.finfo(dtype).eps / 2
    tol = 6 * u if dtype == BF else 1e-4
    for got, want in zip((O, dx, dwq, dwk), (o.detach(), *wants)):
        assert float((got.double() - want).norm() / want.norm()) <= tol


@pytest.mark.parametrize("dtype,d", [(F32, 48), (BF, 64), (BF, 128)])
def test_served_request_token_by_token(dtype, d):
    """A prompt into the cache, then single tokens: the same as one forward
    over the whole sequence; the rest of the cache holds NaN."""
    B, H, Hkv, cap_rows = 2, 4, 2, 200
    lens, new = [37, 120], 4
    freqs = (10000.0 ** (-torch.arange(d // 2, device="cuda") / (d // 2)))[None].contiguous()
    w = dict(wq=torch.linspace(0.5, 1.5, d, device="cuda"), wk=torch.linspace(1.5, 0.5, d, device="cuda"),
             freqs=freqs)
    x = torch.randn((B, max(lens) + new, H + 2 * Hkv, d), device="cuda").to(dtype)
    K, V = (torch.full((B, Hkv, cap_rows, d), math.nan, dtype=dtype, device="cuda") for _ in range(2))
    tau = 1 / math.sqrt(d)
    for b, n in enumerate(lens):  # the prompts
        fb.qk_norm_rope(x[b:b + 1, :n].contiguous(), H, **w, K=K[b:b + 1], V=V[b:b + 1])
    outs = []
    for t in range(new):
        at = torch.tensor([n + t for n in lens], dtype=torch.int32, device="cuda")
        xt = torch.stack([x[b, n + t] for b, n in enumerate(lens)])[:, None].contiguous()
        q, _, _ = fb.qk_norm_rope(xt, H, **w, positions=at[None, :, None].contiguous(), K=K, V=V,
                                  kv_start=at)
        ranges, pos = fb.attention_ranges(B, 1, cap_rows, q_start=at, causal=True)
        outs.append(fb.attention(q, K, V, tau, ranges=ranges, q_pos=pos)[0])
    for b, n in enumerate(lens):
        q, k, v = fb.qk_norm_rope(x[b:b + 1, :n + new].contiguous(), H, **w)
        val, bound = ref.attention(q, k, v, tau, causal=True)
        for t in range(new):
            got = outs[t][b]
            assert ref.worst(got[None], val["O"][:, :, n + t:n + t + 1],
                             bound["O"][:, :, n + t:n + t + 1]) <= 1.0
