"""The operators around one attention layer and the cases that they are measured on.

Three operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and as a user calls it from this package:

* attention with capped scores, a distance bias, and key ranges (documents, prefixes, padding),
  with its gradient for training and with a cache of keys and values for single tokens;
* the norm of queries and keys for each head with the rotation by position, from the packed
  projection to head-major tensors (or into a cache), with its gradient;
* the key ranges of packed documents and prefixes, built on the GPU.
"""
import math

import torch

own = False

INT = torch.int32


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # A batch of packed documents of a small language model's layer: training, every head its own keys.
        dict(name="train_docs_small_layer", op="attn", mode="train", dtype="bf16", B=4, H=12, Hkv=12, Nq=1024, Nk=1024, d=64,
             causal=False, docs=5, prefix=False, pad=0, cap=0.0, bias=False),
        # One long sequence whose scores are capped: the largest training case.
        dict(name="train_capped_long", op="attn", mode="train", dtype="bf16", B=1, H=8, Hkv=8, Nq=16384, Nk=16384, d=64,
             causal=True, docs=0, prefix=False, pad=0, cap=30.0, bias=False),
        # Wide heads, four query heads to a key head, a bias by distance, a length that fills no tile.
        dict(name="train_bias_grouped_wide", op="attn", mode="train", dtype="bf16", B=2, H=16, Hkv=4, Nq=2047, Nk=2047, d=128,
             causal=True, docs=0, prefix=False, pad=0, cap=0.0, bias=True),
        # 32-bit inputs, an odd head size, documents that begin with a prefix seen both ways, padding behind the last one.
        dict(name="train_f32_odd_prefix", op="attn", mode="train", dtype="f32", B=2, H=3, Hkv=3, Nq=333, Nk=333, d=80,
             causal=False, docs=3, prefix=True, pad=14, cap=20.0, bias=True),
        # A long prompt with a prefix that all of it sees: the forward alone (scoring, or the prompt of a served request).
        dict(name="forward_prefix_mid", op="attn", mode="forward", dtype="bf16", B=1, H=12, Hkv=12, Nq=8192, Nk=8192, d=64,
             causal=False, docs=1, prefix=True, pad=0, cap=0.0, bias=False),
        # Serving: one token for each of 32 requests of different lengths over their caches.
        dict(name="token_batch_cache", op="attn", mode="token", dtype="bf16", B=32, H=32, Hkv=8, Nq=1, Nk=8192, d=128,
             causal=False, docs=0, prefix=False, pad=0, cap=50.0, bias=False),
        # Serving: one token of one short request; latency counts.
        dict(name="token_single_short", op="attn", mode="token", dtype="bf16", B=1, H=12, Hkv=12, Nq=1, Nk=1000, d=64,
             causal=False, docs=0, prefix=False, pad=0, cap=0.0, bias=True),
        # The projection of a training batch, forward and backward.
        dict(name="norm_train_large", op="norm", mode="train", dtype="bf16", B=2, N=8192, H=32, Hkv=8, d=128, R=128, axes=1,
             interleaved=False, gain=True),
        # Image tokens with three position axes, neighbouring pairs, a head that is rotated in part; odd sizes.
        dict(name="norm_train_axes_odd", op="norm", mode="train", dtype="bf16", B=3, N=1001, H=6, Hkv=2, d=80, R=60, axes=3,
             interleaved=True, gain=True),
        # Serving: the new tokens of 32 requests, keys and values written into the cache.
        dict(name="norm_token_cache", op="norm", mode="token", dtype="bf16", B=32, N=1, H=32, Hkv=8, d=128, R=128, axes=1,
             interleaved=False, gain=True, Nk=1024),
        # Ranges of a small batch of packed documents, causal.
        dict(name="ranges_docs_small", op="ranges", B=4, Nq=1024, Nk=1024, M=5, causal=True, prefix=False),
        # Ranges of a batch of very long packed sequences with many documents and prefixes.
        dict(name="ranges_prefix_long", op="ranges", B=8, Nq=131072, Nk=131072, M=511, causal=True, prefix=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["train", "train", "f32", "forward", "token", "token", "norm", "norm_token", "ranges"])
    if kind in ("train", "f32", "forward"):
        f32 = kind == "f32"
        d = _log(rng, 8, 128) if f32 else rng.choice([64, 64, 128, 128, 96])
        Hkv = rng.choice([1, 2, 3, 4])
        H = Hkv * rng.choice([1, 1, 2, 4])
        B = rng.choice([1, 1, 2, 3])
        top = 700 if f32 or d == 96 else 4096
        low = 1 if kind == "forward" else 2  # over a single key the scores have no gradient at all
        Nq = _log(rng, low, top)
        if rng.random() < 0.3:  # keys of another length than the queries
            Nk, docs, prefix, pad = _log(rng, low, top), 0, False, 0
            causal = rng.random() < 0.5
        else:
            Nk, docs = Nq, rng.choice([0, 1, 3, 8]) if Nq >= 16 else 0
            prefix, pad = docs > 0 and rng.random() < 0.5, rng.choice([0, Nq // 9]) if docs else 0
            causal = docs == 0 and rng.random() < 0.7
        return dict(op="attn", mode="forward" if kind == "forward" else "train", dtype="f32" if f32 else "bf16", B=B, H=H, Hkv=Hkv,
                    Nq=Nq, Nk=Nk, d=d, causal=causal, docs=docs, prefix=prefix, pad=pad,
                    cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.random() < 0.4)
    if kind == "token":
        Hkv = rng.choice([1, 2, 4, 8, 12])
        return dict(op="attn", mode="token", dtype="bf16", B=_log(rng, 1, 32), H=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv,
                    Nq=rng.choice([1, 1, 1, 2, 4]), Nk=_log(rng, 8, 8192), d=rng.choice([64, 128]), causal=False, docs=0, prefix=False,
                    pad=0, cap=rng.choice([0.0, 0.0, 50.0]), bias=rng.random() < 0.3)
    if kind == "ranges":
        N = _log(rng, 1, 131072)
        return dict(op="ranges", B=rng.choice([1, 2, 5, 8]), Nq=N, Nk=N, M=_log(rng, 1, max(1, min(511, N))), causal=rng.random() < 0.7,
                    prefix=rng.random() < 0.5)
    token = kind == "norm_token"
    d = rng.choice([64, 128, 128, 80, 34])
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op="norm", mode="token" if token else "train", dtype=rng.choice(["bf16", "bf16", "f32"]), B=_log(rng, 1, 32) if token else rng.choice([1, 2]),
             N=rng.choice([1, 1, 3]) if token else _log(rng, 1, 6000), H=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv, d=d,
             R=rng.choice([d, d, d // 4 * 2]), axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4, gain=rng.random() < 0.8)
    if token:
        c["Nk"] = _log(rng, 16, 1024)
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _offsets(gen, B, M, used):
    """Starts of M documents within the first `used` rows of each batch entry, and the end of the last: [B, M + 1]."""
    cut = torch.rand((B, M), generator=gen, device="cuda").sort(dim=1).values
    off = torch.empty((B, M + 1), dtype=INT, device="cuda")
    off[:, :M] = (cut * used).to(INT)
    off[:, 0] = 0
    off[:, M] = used
    return off


def _prefixes(gen, off):
    return ((off[:, 1:] - off[:, :-1]) * torch.rand(off[:, 1:].shape, generator=gen, device="cuda") * 0.6).to(INT)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    B = case["B"]
    s = dict(case=case)
    if case["op"] == "ranges":
        s["off"] = _offsets(gen, B, case["M"], max(1, case["Nk"] - case["Nk"] // 50))
        s["prefix"] = _prefixes(gen, s["off"]) if case["prefix"] else None
        return s
    t = _type(case)
    if case["op"] == "attn":
        H, Hkv, Nq, Nk, d = (case[k] for k in ("H", "Hkv", "Nq", "Nk", "d"))
        s["Q"] = randn(B, H, Nq, d, dtype=t)
        s["K"] = randn(B, Hkv, Nk, d, dtype=t)
        s["V"] = randn(B, Hkv, Nk, d, dtype=t)
        s["dO"] = randn(B, H, Nq, d, dtype=t) if case["mode"] == "train" else None
        s["tau"] = 1.0 / math.sqrt(d)
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H) if case["bias"] else None
        s["ranges"], s["q_pos"] = None, None
        if case["mode"] == "token":  # each request's new tokens see its cache up to themselves
            last = (Nk - torch.rand((B, 1), generator=gen, device="cuda") * 0.75 * (Nk - 1)).to(INT).clamp(1, Nk)
            pos = last - Nq + torch.arange(Nq, device="cuda", dtype=INT)
            s["q_pos"] = pos.contiguous()
            s["ranges"] = torch.stack([torch.zeros_like(pos), (pos + 1).clamp(0, Nk)], dim=2).contiguous()
        elif case["docs"]:
            off = _offsets(gen, B, case["docs"], Nk - case["pad"])
            s["ranges"] = _plain_ranges(off, _prefixes(gen, off) if case["prefix"] else None, True, Nq, Nk)[0].contiguous()
        return s
    N, H, Hkv, d, R = (case[k] for k in ("N", "H", "Hkv", "d", "R"))
    s["QKV"] = randn(B, N, H + 2 * Hkv, d, dtype=t)
    s["wq"] = 1.0 + 0.1 * randn(d) if case["gain"] else None
    s["wk"] = 1.0 + 0.1 * randn(d) if case["gain"] else None
    s["eps"] = 1e-6
    half, A = R // 2, case["axes"]
    base = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(1, half))
    axis = torch.arange(half, device="cuda") * A // max(1, half)  # which axis a pair goes by: one run of pairs for each
    s["freqs"] = (base * (axis == torch.arange(A, device="cuda")[:, None])).to(torch.float32).contiguous()
    if A == 1:
        start = torch.randint(0, 100000, (1, B, 1), generator=gen, device="cuda")
        s["positions"] = (start + torch.arange(N, device="cuda")).to(INT).contiguous()
    else:
        s["positions"] = torch.randint(0, 1000, (A, B, N), generator=gen, device="cuda").to(INT)
    if case["mode"] == "train":
        s["dQ"], s["dK"], s["dV"] = randn(B, H, N, d, dtype=t), randn(B, Hkv, N, d, dtype=t), randn(B, Hkv, N, d, dtype=t)
    else:
        Nk = case["Nk"]
        s["Kc"], s["Vc"] = randn(B, Hkv, Nk, d, dtype=t), randn(B, Hkv, Nk, d, dtype=t)
        s["start"] = torch.randint(0, Nk - N + 1, (B,), generator=gen, device="cuda").to(INT)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain_ranges(off, prefix, causal, Nq, Nk):
    """Key ranges [lo, hi) of every query by documents, and the queries' positions."""
    B, M = off.shape[0], off.shape[1] - 1
    pos = torch.arange(Nq, device=off.device, dtype=INT).expand(B, Nq).contiguous()
    at = torch.searchsorted(off, pos, right=True) - 1  # the last document that starts at or before the query
    inside = (at >= 0) & (at < M)
    at = at.clamp(0, M - 1)
    lo, end = off.gather(1, at), off.gather(1, at + 1)
    hi = end
    if causal:
        hi = pos + 1
        if prefix is not None:
            hi = torch.maximum(hi, lo + prefix.gather(1, at))
        hi = torch.minimum(hi, end)
    hi = hi.clamp(max=Nk)
    zero = torch.zeros_like(lo)
    return torch.stack([torch.where(inside, lo, zero), torch.where(inside, hi, zero)], dim=2), pos


def _plain_mask(s, Nq, Nk, causal):
    """True where a query sees a key: [B or 1, 1, 1, Nq, Nk], or None; and the distances [B or 1, 1, 1, Nq, Nk]."""
    j = torch.arange(Nk, device="cuda", dtype=INT)
    pos = (s["q_pos"] if s["q_pos"] is not None else torch.arange(Nq, device="cuda", dtype=INT)[None])[:, :, None]
    see = None
    if s["ranges"] is not None:
        see = (j >= s["ranges"][:, :, :1]) & (j < s["ranges"][:, :, 1:])
    if causal:
        see = j <= pos if see is None else see & (j <= pos)
    return None if see is None else see[:, None, None], (pos - j).abs()[:, None, None] if s["slopes"] is not None else None


def _plain_attention(s):
    case = s["case"]
    B, H, Hkv, Nq, Nk, d = (case[k] for k in ("B", "H", "Hkv", "Nq", "Nk", "d"))
    G, t, tau, cap = H // Hkv, _type(case), s["tau"], case["cap"]
    q = s["Q"].float().view(B, Hkv, G * Nq, d)
    k, v = s["K"].float(), s["V"].float()
    see, far = _plain_mask(s, Nq, Nk, case["causal"])
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, G, Nq, Nk) * tau
    th = None
    if cap:
        th = torch.tanh(x / cap)
        x = cap * th
    if far is not None:
        x = x - s["slopes"].view(1, Hkv, G, 1, 1) * far
    if see is not None:
        x = torch.where(see, x, -math.inf)
    m = x.amax(dim=4, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    del x
    l = p.sum(dim=4, keepdim=True)
    L = (m + torch.log(l)).view(B, H, Nq)
    p = p / torch.where(l == 0, 1.0, l)
    o = torch.matmul(p.view(B, Hkv, G * Nq, Nk), v).view(B, H, Nq, d)
    out = {"O": o.to(t), "L": L}
    if case["mode"] != "train":
        return out
    do = s["dO"].float().view(B, Hkv, G * Nq, d)
    dp = torch.matmul(do, v.transpose(2, 3)).view(B, Hkv, G, Nq, Nk)
    D = (s["dO"].float() * o).sum(dim=3).view(B, Hkv, G, Nq, 1)
    ds = p * (dp - D)
    del dp
    if cap:
        ds = ds * (1.0 - th * th)
    ds = (ds * tau).view(B, Hkv, G * Nq, Nk)
    out["dQ"] = torch.matmul(ds, k).view(B, H, Nq, d).to(t)
    out["dK"] = torch.matmul(ds.transpose(2, 3), q).to(t)
    out["dV"] = torch.matmul(p.view(B, Hkv, G * Nq, Nk).transpose(2, 3), do).to(t)
    return out


def _pairs(case):
    """The two elements of every rotated pair: two index lists of R / 2."""
    half = case["R"] // 2
    k = torch.arange(half, device="cuda")
    return (2 * k, 2 * k + 1) if case["interleaved"] else (k, k + half)


def _angles(s):
    """cos and sin [B, N, 1, R / 2]: the angle needs 64 bits at far positions, its sine does not."""
    a = torch.einsum("abn,ak->bnk", s["positions"].double(), s["freqs"].double())
    return torch.cos(a).float()[:, :, None], torch.sin(a).float()[:, :, None]


def _plain_norm(s):
    case = s["case"]
    H, Hkv, t = case["H"], case["Hkv"], _type(case)
    x = s["QKV"].float()
    i, j = _pairs(case)
    cos, sin = _angles(s)

    def norm(x, w):
        r = torch.rsqrt((x * x).mean(dim=3, keepdim=True) + s["eps"])
        return x * r, r, (x * r if w is None else x * r * w)

    def rotate(y, sin):
        z = y.clone()
        z[..., i] = y[..., i] * cos - y[..., j] * sin
        z[..., j] = y[..., j] * cos + y[..., i] * sin
        return z

    xq, rq, yq = norm(x[:, :, :H], s["wq"])
    xk, rk, yk = norm(x[:, :, H:H + Hkv], s["wk"])
    Q = rotate(yq, sin).transpose(1, 2).to(t).contiguous()
    K = rotate(yk, sin).transpose(1, 2).to(t).contiguous()
    V = s["QKV"][:, :, H + Hkv:].transpose(1, 2).contiguous()
    if case["mode"] == "token":
        b = torch.arange(case["B"], device="cuda")[:, None]
        rows = s["start"].long()[:, None] + torch.arange(case["N"], device="cuda")
        s["Kc"][b, :, rows] = K.transpose(1, 2)
        s["Vc"][b, :, rows] = V.transpose(1, 2)
        return {"Q": Q, "K": s["Kc"], "V": s["Vc"]}

    def back(dz, xh, r, w):
        dy = rotate(dz.float().transpose(1, 2), -sin)
        dw = (dy * xh).sum(dim=(0, 1, 2), dtype=torch.float64).float()
        g = dy if w is None else dy * w
        return r * (g - xh * (g * xh).mean(dim=3, keepdim=True)), dw

    dq, dwq = back(s["dQ"], xq, rq, s["wq"])
    dk, dwk = back(s["dK"], xk, rk, s["wk"])
    dx = torch.cat([dq.to(t), dk.to(t), s["dV"].transpose(1, 2)], dim=2)
    out = {"Q": Q, "K": K, "V": V, "dQKV": dx}
    if case["gain"]:
        out["dwq"], out["dwk"] = dwq, dwk
    return out


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "attn":
        return _plain_attention(s)
    if case["op"] == "norm":
        return _plain_norm(s)
    ranges, pos = _plain_ranges(s["off"], s["prefix"], case["causal"], case["Nq"], case["Nk"])
    return {"ranges": ranges, "q_pos": pos}


def _own(s, case):
    from exact_second_order_gb300 import flashbob as fb
    if case["op"] == "ranges":
        ranges, pos = fb.attention_ranges(case["B"], case["Nq"], case["Nk"], doc_offsets=s["off"], prefix=s["prefix"], causal=case["causal"])
        return {"ranges": ranges, "q_pos": pos}
    if case["op"] == "attn":
        form = dict(cap=case["cap"], slopes=s["slopes"], ranges=s["ranges"], q_pos=s["q_pos"], causal=case["causal"])
        O, L = fb.attention(s["Q"], s["K"], s["V"], s["tau"], **form)
        if case["mode"] != "train":
            return {"O": O, "L": L}
        dQ, dK, dV = fb.attention_grad(s["Q"], s["K"], s["V"], O, L, s["dO"], s["tau"], **form)
        return {"O": O, "L": L, "dQ": dQ, "dK": dK, "dV": dV}
    form = dict(wq=s["wq"], wk=s["wk"], freqs=s["freqs"], positions=s["positions"], eps=s["eps"], interleaved=case["interleaved"])
    if case["mode"] == "token":
        Q, K, V = fb.qk_norm_rope(s["QKV"], case["H"], **form, K=s["Kc"], V=s["Vc"], kv_start=s["start"])
        return {"Q": Q, "K": K, "V": V}
    Q, K, V = fb.qk_norm_rope(s["QKV"], case["H"], **form)
    dx, dwq, dwk = fb.qk_norm_rope_grad(s["QKV"], s["dQ"], s["dK"], s["dV"], **form)
    out = {"Q": Q, "K": K, "V": V, "dQKV": dx}
    if case["gain"]:
        out["dwq"], out["dwk"] = dwq, dwk
    return out


# ---------------------------------------------------------------------------
# What one pass cannot do without
# ---------------------------------------------------------------------------

def _seen_pairs(case):
    """(query, key) pairs that the mask leaves for one head and batch entry, on average over the inputs' random cuts."""
    Nq, Nk = case["Nq"], case["Nk"]
    if case["mode"] == "token":
        return Nq * max(1.0, 0.625 * Nk)
    if case["docs"]:
        n, m = Nk - case["pad"], case["docs"]
        whole = n * n * 2.0 / (m + 1)  # sum of the squared lengths of the runs between m - 1 random cuts
        return whole * (0.5 + (0.06 if case["prefix"] else 0.0))
    if case["causal"]:
        k = min(Nq, Nk)
        return k * (k + 1) / 2 + (Nq - k) * Nk
    return float(Nq * Nk)


def work(case):
    B = case["B"]
    if case["op"] == "ranges":
        M = case["M"]
        return {"bytes": 4 * B * (M + 1 + (M if case["prefix"] else 0)) + 12 * B * case["Nq"], "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        N, H, Hkv, d = case["N"], case["H"], case["Hkv"], case["d"]
        x = B * N * (H + 2 * Hkv) * d
        moves = 2 if case["mode"] == "token" else 4  # read, write; training: the gradients read and written too
        return {"bytes": moves * x * e + 4 * case["axes"] * B * N, "flops": (10 if case["mode"] == "token" else 30) * x}
    H, Hkv, Nq, Nk, d = (case[k] for k in ("H", "Hkv", "Nq", "Nk", "d"))
    pairs = B * H * _seen_pairs(case)
    rows = B * H * Nq
    kv = B * Hkv * Nk * d * e * 2.0
    if case["mode"] == "token":
        kv *= 0.625
    size = 2 * rows * d * e + kv + 4 * rows + (8 * B * Nq if case["docs"] or case["mode"] == "token" else 0)
    flops = 4.0 * d * pairs
    if case["mode"] == "train":
        size += 2 * rows * d * e + kv  # dO read, dQ, dK and dV written
        flops += 10.0 * d * pairs
    return {"bytes": size, "flops": flops}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ranges":
        return None
    return _exact_attention(s, case) if case["op"] == "attn" else _exact_norm(s, case)


def _exact_attention(s, case):
    """Query head by query head, from the definition: softmax over the keys that a query sees, and the chain rule."""
    B, H, Hkv, Nq, Nk, d = (case[k] for k in ("B", "H", "Hkv", "Nq", "Nk", "d"))
    train = case["mode"] == "train"
    f = dict(dtype=torch.float64, device="cuda")
    O, L = torch.zeros((B, H, Nq, d), **f), torch.zeros((B, H, Nq), **f)
    dQ, dK, dV = torch.zeros((B, H, Nq, d), **f), torch.zeros((B, Hkv, Nk, d), **f), torch.zeros((B, Hkv, Nk, d), **f)
    key = torch.arange(Nk, device="cuda")
    step = max(1, (1 << 26) // Nk)  # query rows at a time
    for b in range(B):
        pos = s["q_pos"][b].long() if s["q_pos"] is not None else torch.arange(Nq, device="cuda")
        for h in range(H):
            g = h // (H // Hkv)
            K, V = s["K"][b, g].double(), s["V"][b, g].double()
            for i in range(0, Nq, step):
                r = slice(i, min(Nq, i + step))
                hidden = torch.zeros((r.stop - r.start, Nk), dtype=torch.bool, device="cuda")
                if s["ranges"] is not None:
                    hidden |= (key[None] < s["ranges"][b, r, 0, None]) | (key[None] >= s["ranges"][b, r, 1, None])
                if case["causal"]:
                    hidden |= key[None] > pos[r, None]
                q = s["Q"][b, h, r].double()
                z = (q @ K.T) / math.sqrt(d) if s["tau"] == 1.0 / math.sqrt(d) else (q @ K.T) * s["tau"]
                slope = 1.0
                if case["cap"]:
                    u = torch.tanh(z / case["cap"])
                    z, slope = case["cap"] * u, 1.0 - u ** 2
                if s["slopes"] is not None:
                    z = z - s["slopes"][h].double() * (pos[r, None] - key[None]).abs()
                z = z.masked_fill(hidden, -math.inf)
                L[b, h, r] = torch.logsumexp(z, dim=1)
                P = torch.exp(z - L[b, h, r, None]).masked_fill(hidden, 0.0)
                O[b, h, r] = P @ V
                if train:
                    w = s["dO"][b, h, r].double()
                    dP = w @ V.T
                    dz = P * (dP - (P * dP).sum(dim=1, keepdim=True)) * slope * s["tau"]
                    dQ[b, h, r] = dz @ K
                    dK[b, g] += dz.T @ q
                    dV[b, g] += P.T @ w
    return {"O": O, "L": L, "dQ": dQ, "dK": dK, "dV": dV} if train else {"O": O, "L": L}


def _exact_norm(s, case):
    """As complex numbers: a pair turns by multiplication with exp(i angle); the gradients by autograd."""
    B, N, H, Hkv, d, R = (case[k] for k in ("B", "N", "H", "Hkv", "d", "R"))
    train = case["mode"] == "train"
    turn = torch.polar(torch.ones((B, N, 1, R // 2), dtype=torch.float64, device="cuda"),
                       sum(s["positions"][a].double()[:, :, None, None] * s["freqs"][a].double() for a in range(case["axes"])))

    def one(x, w):
        y = x / torch.sqrt(x.square().sum(dim=3, keepdim=True) / d + s["eps"])
        y = y if w is None else y * w
        a, rest = y[..., :R], y[..., R:]
        a = a.unflatten(3, (R // 2, 2)) if case["interleaved"] else a.unflatten(3, (2, R // 2)).transpose(3, 4)
        a = torch.view_as_real(torch.view_as_complex(a.contiguous()) * turn)
        a = a if case["interleaved"] else a.transpose(3, 4)
        return torch.cat([a.flatten(3), rest], dim=3).transpose(1, 2)

    with torch.enable_grad():
        x = s["QKV"].double().requires_grad_(train)
        wq, wk = ((s[n].double().requires_grad_(train) if s[n] is not None else None) for n in ("wq", "wk"))
        Q, K = one(x[:, :, :H], wq), one(x[:, :, H:H + Hkv], wk)
        V = x[:, :, H + Hkv:].transpose(1, 2)
        if train:
            want = [x] + ([wq, wk] if case["gain"] else [])
            grads = torch.autograd.grad([Q, K, V], want, [s["dQ"].double(), s["dK"].double(), s["dV"].double()])
    if train:
        out = {"Q": Q.detach(), "K": K.detach(), "V": V.detach(), "dQKV": grads[0]}
        if case["gain"]:
            out["dwq"], out["dwk"] = grads[1], grads[2]
        return out
    Kc, Vc = s["Kc"].double(), s["Vc"].double()
    for b in range(B):
        at = int(s["start"][b])
        Kc[b, :, at:at + N], Vc[b, :, at:at + N] = K[b], V[b]
    return {"Q": Q, "K": Kc, "V": Vc}
