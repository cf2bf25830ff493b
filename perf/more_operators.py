"""A paged cache of keys and values and the cases that its operators are measured on.

The keys and values of all requests lie in pages of T tokens, [pages, Hkv, T, d], and a table
names the pages of each request in order.  A cache in 8 bits (e4m3) has one scale for each page
and head, a power of two.  Three operators, each in a plain form (elementary torch operations in
32 bits, rounded once at the end) and as a user calls it from this package:

* append: from the packed projection, queries and keys turned by position (after their norm, if
  asked for), keys and values written into their pages; a page whose scale has to grow for the
  new tokens gets the tokens it already holds in the new scale;
* attention over the pages (single tokens, a few drafted ones, and prompts behind a cached part),
  with capped scores, a distance bias and key ranges;
* read: pages back to head-major keys and values, for the operators that take those.
"""
import math

import torch

own = False

INT = torch.int32
E4M3 = torch.float8_e4m3fn
LOWEST, HIGHEST = -60, 60  # exponents of a scale


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One new token of one request in a GPT-2-sized layer: latency counts.
        dict(name="append_token_single", op="append", dtype="bf16", cache="e4m3", B=1, N=1, H=12, Hkv=12, d=64, T=16, Nk=1024,
             R=64, axes=1, interleaved=False, norm=False, ragged=False),
        # The new tokens of 32 requests in a grouped-query layer.
        dict(name="append_token_batch", op="append", dtype="bf16", cache="e4m3", B=32, N=1, H=32, Hkv=8, d=128, T=64, Nk=2048,
             R=128, axes=1, interleaved=False, norm=False, ragged=False),
        # Two long prompts, the largest append.
        dict(name="append_prompt_large", op="append", dtype="bf16", cache="e4m3", B=2, N=8192, H=32, Hkv=8, d=128, T=64, Nk=10240,
             R=128, axes=1, interleaved=False, norm=False, ragged=False),
        # Image tokens with three position axes and normed heads, neighbouring pairs, a head that turns in part, a padded batch; odd sizes.
        dict(name="append_prompt_axes_odd", op="append", dtype="bf16", cache="e4m3", B=3, N=333, H=6, Hkv=2, d=80, T=32, Nk=500,
             R=60, axes=3, interleaved=True, norm=True, ragged=True),
        # Serving: one token for each of 32 requests of different lengths over their caches.
        dict(name="token_batch", op="attn", mode="token", dtype="bf16", cache="e4m3", B=32, H=32, Hkv=8, Nq=1, Nk=8192, d=128, T=64,
             cap=0.0, bias=False, window=0),
        # One token of one short request in a GPT-2-sized layer: latency counts.
        dict(name="token_single_short", op="attn", mode="token", dtype="bf16", cache="e4m3", B=1, H=12, Hkv=12, Nq=1, Nk=1000, d=64, T=16,
             cap=0.0, bias=True, window=0),
        # One token of one request with a very long context.
        dict(name="token_long_context", op="attn", mode="token", dtype="bf16", cache="e4m3", B=1, H=32, Hkv=8, Nq=1, Nk=131072, d=128, T=64,
             cap=0.0, bias=False, window=0),
        # Four drafted tokens of 16 requests are checked in one pass, scores capped.
        dict(name="token_draft_capped", op="attn", mode="token", dtype="bf16", cache="e4m3", B=16, H=16, Hkv=4, Nq=4, Nk=4096, d=128, T=32,
             cap=50.0, bias=False, window=0),
        # A prompt's next 2048 tokens behind what is cached already: the largest attention.
        dict(name="prompt_chunk", op="attn", mode="prompt", dtype="bf16", cache="e4m3", B=1, H=32, Hkv=8, Nq=2048, Nk=16384, d=128, T=64,
             cap=0.0, bias=False, window=0),
        # A padded batch of prompts with a sliding window, 16-bit cache, small pages, sizes that fill no tile.
        dict(name="prompt_ragged_window", op="attn", mode="prompt", dtype="bf16", cache="same", B=4, H=12, Hkv=4, Nq=1000, Nk=5000, d=64, T=16,
             cap=0.0, bias=False, window=1024),
        # The cached part of four long requests back to head-major tensors.
        dict(name="read_long", op="read", dtype="bf16", cache="e4m3", B=4, Hkv=8, Nk=32768, d=128, T=64),
        # A few odd ones, to 32 bits.
        dict(name="read_odd_f32", op="read", dtype="f32", cache="e4m3", B=3, Hkv=2, Nk=777, d=80, T=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append_token", "append", "append", "token", "token", "token", "prompt", "prompt", "f32", "read"])
    T = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["e4m3", "e4m3", "e4m3", "same"])
    if kind.startswith("append"):
        token = kind == "append_token"
        d = rng.choice([64, 128, 128, 80, 34])
        Hkv = rng.choice([1, 2, 4, 8])
        N = rng.choice([1, 1, 3]) if token else _log(rng, 2, 4096)
        return dict(op="append", dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), cache=cache, B=_log(rng, 1, 64) if token else rng.choice([1, 2, 3]),
                    N=N, H=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv, d=d, T=T, Nk=N + _log(rng, 1, 1024), R=rng.choice([d, d, d // 4 * 2]),
                    axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.3, ragged=rng.random() < 0.4)
    if kind == "read":
        return dict(op="read", dtype=rng.choice(["bf16", "bf16", "f32"]), cache=cache, B=rng.choice([1, 2, 5, 8]), Hkv=rng.choice([1, 2, 4, 8]),
                    Nk=_log(rng, 1, 16384), d=rng.choice([64, 128, 80, 33]), T=T)
    if kind == "token":
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(op="attn", mode="token", dtype="bf16", cache=cache, B=_log(rng, 1, 32), H=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv,
                    Nq=rng.choice([1, 1, 1, 2, 4]), Nk=_log(rng, 8, 8192), d=rng.choice([64, 128, 128]), T=T, cap=rng.choice([0.0, 0.0, 50.0]),
                    bias=rng.random() < 0.3, window=rng.choice([0, 0, 700]))
    f32 = kind == "f32"
    Hkv = rng.choice([1, 2, 4])
    top = 300 if f32 else 2048
    Nq = _log(rng, 2, top)
    return dict(op="attn", mode="prompt", dtype="f32" if f32 else "bf16", cache=cache, B=rng.choice([1, 1, 2, 4]), H=Hkv * rng.choice([1, 2, 4]),
                Hkv=Hkv, Nq=Nq, Nk=Nq + _log(rng, 1, 500 if f32 else 6000), d=_log(rng, 8, 128) if f32 else rng.choice([64, 128, 128]), T=T,
                cap=rng.choice([0.0, 0.0, 30.0]), bias=rng.random() < 0.3, window=rng.choice([0, 0, 200]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _cache(s, gen, case):
    """Pages in a random order that hold normal values, some channels and pages larger than others."""
    B, Hkv, T, d = (case[k] for k in ("B", "Hkv", "T", "d"))
    M = -(-case["Nk"] // T)
    P = B * M + 3  # a few pages that nobody has

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s["table"] = torch.randperm(P, generator=gen, device="cuda")[:B * M].to(INT).view(B, M).contiguous()
    for name, scale in (("K", "k_scale"), ("V", "v_scale")):
        x = randn(P, Hkv, T, d)
        x *= torch.exp(0.5 * randn(Hkv, 1, d))
        x *= torch.exp(0.3 * randn(P, Hkv, 1, 1))
        if case["cache"] == "e4m3":
            s[scale] = _scale_of(x.abs().amax(dim=(2, 3)))
            s[name] = _code(x, s[scale][:, :, None, None])
        else:
            s[name], s[scale] = x.to(_type(case)), None


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    B, t, s = case["B"], _type(case), dict(case=case)
    _cache(s, gen, case)
    Nk = case["Nk"]
    if case["op"] == "read":
        s["lens"] = (Nk - rand(B) * 0.5 * Nk).to(INT).clamp(1, Nk)
    elif case["op"] == "append":
        N, H, Hkv, d, R, A = (case[k] for k in ("N", "H", "Hkv", "d", "R", "axes"))
        s["QKV"] = randn(B, N, H + 2 * Hkv, d, dtype=t)
        s["start"] = (rand(B) * (Nk - N + 1)).to(INT).clamp(0, Nk - N)
        s["counts"] = (N - rand(B) * 0.5 * N).to(INT).clamp(1, N) if case["ragged"] else None
        s["wq"], s["wk"] = (1.0 + 0.1 * randn(d) if case["norm"] else None for _ in range(2))
        half = R // 2
        base = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(1, half))
        axis = torch.arange(half, device="cuda") * A // max(1, half)  # which axis a pair goes by: one run of pairs for each
        s["freqs"] = (base * (axis == torch.arange(A, device="cuda")[:, None])).to(torch.float32).contiguous()
        # With one axis a token turns by its place in the cache.
        s["positions"] = None if A == 1 else (rand(A, B, N) * 1000).to(INT)
    else:
        H, Nq, d = case["H"], case["Nq"], case["d"]
        s["Q"] = randn(B, H, Nq, d, dtype=t)
        s["tau"] = 1.0 / math.sqrt(d)
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H) if case["bias"] else None
        i = torch.arange(Nq, device="cuda", dtype=INT)
        if case["mode"] == "token":  # each request's new tokens see its cache up to themselves
            last = (Nk - rand(B, 1) * 0.75 * (Nk - 1)).to(INT).clamp(1, Nk)
            pos, live = last - Nq + i, torch.ones((B, Nq), dtype=torch.bool, device="cuda")
        else:  # new tokens at the end of what is cached; a padded batch
            n = (Nq - rand(B, 1) * 0.5 * (Nq - 1)).to(INT).clamp(1, Nq) if B > 1 else torch.full((1, 1), Nq, dtype=INT, device="cuda")
            pos, live = Nk - Nq + i.expand(B, Nq), i < n
        lo = (pos + 1 - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(pos)
        hi = (pos + 1).clamp(0, Nk)
        s["q_pos"] = pos.contiguous()
        s["ranges"] = torch.stack([torch.where(live, lo, 0), torch.where(live, hi, 0)], dim=2).to(INT).contiguous()
    if own:  # the handle that a program makes once for its cache
        from exact_second_order_gb300 import flashbob as fb
        s["cache"] = fb.PagedCache(s["K"], s["V"], s["k_scale"], s["v_scale"])
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _scale_of(most):
    """The least power of two within the range whose 448-fold is no less than `most`."""
    m, e = torch.frexp(most)  # most = m 2^e, 448 = 0.875 2^9
    e = torch.where(most > 0, e - 9 + (m > 0.875).to(e.dtype), LOWEST).clamp(LOWEST, HIGHEST)
    return torch.ldexp(torch.ones_like(most), e)


def _code(x, scale):
    return (x / scale).clamp(-448.0, 448.0).to(E4M3)


def _pages(s, name, scale, table):
    """The pages that a table [..] names, in 32 bits: [.., Hkv, T, d]."""
    pool = s[name]
    if s[scale] is None:
        return pool[table].float()
    return pool.view(torch.uint8)[table].view(E4M3).float() * s[scale][table][..., None, None]


def _dense(s, name, scale):
    """Keys or values of every request, head-major: [B, Hkv, M T, d]."""
    x = _pages(s, name, scale, s["table"].long())
    B, M, Hkv, T, d = x.shape
    return x.transpose(1, 2).reshape(B, Hkv, M * T, d)


def _plain_read(s, case):
    Nk = case["Nk"]
    live = (torch.arange(Nk, device="cuda") < s["lens"][:, None])[:, None, :, None]
    return {n: torch.where(live, _dense(s, n, c)[:, :, :Nk], 0.0).to(_type(case)) for n, c in (("K", "k_scale"), ("V", "v_scale"))}


def _plain_attention(s, case):
    B, H, Hkv, Nq, d = (case[k] for k in ("B", "H", "Hkv", "Nq", "d"))
    G, cap = H // Hkv, case["cap"]
    q = s["Q"].float().view(B, Hkv, G * Nq, d)
    k, v = _dense(s, "K", "k_scale"), _dense(s, "V", "v_scale")
    n = k.shape[2]
    j = torch.arange(n, device="cuda", dtype=INT)
    see = ((j >= s["ranges"][:, :, :1]) & (j < s["ranges"][:, :, 1:]))[:, None, None]
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, G, Nq, n) * s["tau"]
    if cap:
        x = cap * torch.tanh(x / cap)
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, Hkv, G, 1, 1) * (s["q_pos"][:, :, None] - j).abs()[:, None, None]
    x = torch.where(see, x, -math.inf)
    m = x.amax(dim=4, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    del x
    l = p.sum(dim=4, keepdim=True)
    L = (m + torch.log(l)).view(B, H, Nq)
    p = p / torch.where(l == 0, 1.0, l)
    O = torch.matmul(p.view(B, Hkv, G * Nq, n), v).view(B, H, Nq, d)
    return {"O": O.to(_type(case)), "L": L}


def _plain_append(s, case):
    B, N, H, Hkv, d, R, T = (case[k] for k in ("B", "N", "H", "Hkv", "d", "R", "T"))
    t, half = _type(case), R // 2
    n = torch.arange(N, device="cuda")
    start = s["start"].long()
    positions = s["positions"] if s["positions"] is not None else (start[:, None] + n)[None]
    angle = torch.einsum("abn,ak->bnk", positions.double(), s["freqs"].double())  # far positions need 64 bits, the sine does not
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    k = torch.arange(half, device="cuda")
    i, j = (2 * k, 2 * k + 1) if case["interleaved"] else (k, k + half)

    def turn(x, w):
        if case["norm"]:
            x = x * torch.rsqrt((x * x).mean(dim=3, keepdim=True) + 1e-6) * w
        y = x.clone()
        y[..., i] = x[..., i] * cos - x[..., j] * sin
        y[..., j] = x[..., j] * cos + x[..., i] * sin
        return y

    x = s["QKV"].float()
    Q = turn(x[:, :, :H], s["wq"]).transpose(1, 2).to(t).contiguous()
    new = {"K": turn(x[:, :, H:H + Hkv], s["wk"]), "V": x[:, :, H + Hkv:]}
    # The pages that may be touched, S of each request, and what each of their rows gets.
    count = torch.full_like(start, N) if s["counts"] is None else s["counts"].long()
    S = (N + T - 2) // T + 1
    at = (start // T)[:, None] + torch.arange(S, device="cuda")  # [B, S]
    page = s["table"].long().gather(1, at.clamp(max=s["table"].shape[1] - 1))
    token = at[:, :, None] * T + torch.arange(T, device="cuda") - start[:, None, None]  # [B, S, T]
    fresh = (token >= 0) & (token < count[:, None, None])
    kept = (token < 0) & fresh.any(dim=2, keepdim=True)  # what a page that gets tokens holds already
    b, slot, row = torch.nonzero(fresh | kept, as_tuple=True)
    at_row = page[b, slot]
    isnew, isold = (f[:, :, None, :, None] for f in (fresh, kept))
    index = token.clamp(0, N - 1).flatten(1)[:, :, None, None].expand(B, S * T, Hkv, d)
    for name, scale in (("K", "k_scale"), ("V", "v_scale")):
        y = new[name].gather(1, index).view(B, S, T, Hkv, d).transpose(2, 3)  # [B, S, Hkv, T, d]
        if s[scale] is None:
            z = torch.where(isnew, y, _pages(s, name, scale, page)).to(t)
            s[name][at_row, :, row] = z[b, slot, :, row]
            continue
        z = torch.where(isnew, y, torch.where(isold, _pages(s, name, scale, page), 0.0))
        need = _scale_of(torch.where(isnew, y, 0.0).abs().amax(dim=(3, 4)))
        need = torch.where(kept.any(dim=2)[:, :, None], torch.maximum(need, s[scale][page]), need)
        codes = _code(z, need[..., None, None])
        s[name].view(torch.uint8)[at_row, :, row] = codes.view(torch.uint8)[b, slot, :, row]
        touched = fresh.any(dim=2)
        s[scale][page[touched]] = need[touched]
    return _appended(s, Q)


def _appended(s, Q):
    out = {"Q": Q, "K": s["K"], "V": s["V"]}
    if s["k_scale"] is not None:
        out["k_scale"], out["v_scale"] = s["k_scale"], s["v_scale"]
    return out


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return {"append": _plain_append, "attn": _plain_attention, "read": _plain_read}[case["op"]](s, case)


def _own(s, case):
    from exact_second_order_gb300 import flashbob as fb
    if case["op"] == "append":
        Q = fb.cache_append(s["QKV"], case["H"], s["cache"], s["table"], kv_start=s["start"], counts=s["counts"], wq=s["wq"], wk=s["wk"],
                            freqs=s["freqs"], positions=s["positions"], eps=1e-6 if case["norm"] else None, interleaved=case["interleaved"])
        return _appended(s, Q)
    if case["op"] == "read":
        K, V = fb.cache_read(s["cache"], s["table"], case["Nk"], lens=s["lens"], dtype=_type(case))
        return {"K": K, "V": V}
    O, L = fb.attention_paged(s["Q"], s["cache"], s["table"], s["tau"], cap=case["cap"], slopes=s["slopes"], ranges=s["ranges"], q_pos=s["q_pos"])
    return {"O": O, "L": L}


# ---------------------------------------------------------------------------
# What one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    c = 1 if case["cache"] == "e4m3" else e
    if case["op"] == "append":
        N, H = case["N"], case["H"]
        kept = 0.75 if case["ragged"] else 1.0
        return {"bytes": B * N * d * ((H + 2 * Hkv) * e + H * e + kept * 2 * Hkv * c), "flops": 3 * B * N * (H + Hkv) * d}
    if case["op"] == "read":
        return {"bytes": B * Hkv * case["Nk"] * d * 2 * (0.75 * c + e), "flops": 1.5 * B * Hkv * case["Nk"] * d}
    H, Nq, Nk = case["H"], case["Nq"], case["Nk"]
    if case["mode"] == "token":
        keys = max(1.0, 0.625 * Nk)
        keys = min(keys, case["window"]) if case["window"] else keys
        pairs, seen = Nq * keys, keys
    else:
        rows = Nq * (0.75 if B > 1 else 1.0)
        keys = Nk - Nq + rows / 2  # the average query's
        seen = Nk - Nq + rows
        if case["window"]:
            keys, seen = min(keys, case["window"]), min(seen, case["window"] + rows)
        pairs = rows * keys
    return {"bytes": B * (2 * H * Nq * d * e + Hkv * seen * d * 2 * c + 4 * H * Nq + 8 * Nq), "flops": 4.0 * d * B * H * pairs}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _nearest(x):
    """The e4m3 number next to each of x: steps of 2^(e - 3) between 2^e and 2^(e + 1), 2^-9 below 2^-6; ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _held(s, name, b):
    """Keys or values of request b, token by token: [tokens, Hkv, d]."""
    x = torch.cat([s[name][p].double() * (1.0 if s[name[0].lower() + "_scale"] is None else s[name[0].lower() + "_scale"][p].double()[:, None, None])
                   for p in s["table"][b].tolist()], dim=1)
    return x.transpose(0, 1)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attention, "read": _exact_read}[case["op"]](s, case)


def _exact_read(s, case):
    out = {}
    for name in ("K", "V"):
        x = torch.zeros((case["B"], case["Hkv"], case["Nk"], case["d"]), dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            x[b, :, :n] = _held(s, name, b)[:n].transpose(0, 1)
        out[name] = x
    return out


def _exact_attention(s, case):
    """Request by request and key head by key head: softmax over the keys that each query sees."""
    B, H, Hkv, Nq, d = (case[k] for k in ("B", "H", "Hkv", "Nq", "d"))
    G = H // Hkv
    O = torch.zeros((B, H, Nq, d), dtype=torch.float64, device="cuda")
    L = torch.zeros((B, H, Nq), dtype=torch.float64, device="cuda")
    for b in range(B):
        K, V = _held(s, "K", b), _held(s, "V", b)
        key = torch.arange(K.shape[0], device="cuda")
        pos = s["q_pos"][b].long()
        hidden = (key < s["ranges"][b, :, 0, None]) | (key >= s["ranges"][b, :, 1, None])
        for g in range(Hkv):
            h = slice(g * G, (g + 1) * G)
            z = torch.einsum("hid,jd->hij", s["Q"][b, h].double(), K[:, g]) / math.sqrt(d)
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if s["slopes"] is not None:
                z = z - s["slopes"][h].double()[:, None, None] * (pos[:, None] - key).abs()
            z = z.masked_fill(hidden, -math.inf)
            L[b, h] = torch.logsumexp(z, dim=2)
            O[b, h] = torch.exp(z - L[b, h, :, None]).masked_fill(hidden, 0.0) @ V[:, g]
    return {"O": O, "L": L}


def _exact_append(s, case):
    """Pairs as complex numbers that turn by multiplication with exp(i angle); page by page, from the definition of the scales."""
    B, N, H, Hkv, d, R, T = (case[k] for k in ("B", "N", "H", "Hkv", "d", "R", "T"))
    start = s["start"].tolist()
    count = [N] * B if s["counts"] is None else s["counts"].tolist()
    f = s["freqs"].double()
    if s["positions"] is None:
        angle = (s["start"].double()[:, None] + torch.arange(N, device="cuda"))[:, :, None] * f[0]
    else:
        angle = sum(s["positions"][a].double()[:, :, None] * f[a] for a in range(case["axes"]))
    spin = torch.polar(torch.ones_like(angle), angle)[:, :, None]

    def turned(x, w):
        x = x.double()
        if case["norm"]:
            x = x / torch.sqrt(x.square().sum(dim=3, keepdim=True) / d + 1e-6) * w.double()
        a, rest = x[..., :R], x[..., R:]
        a = a.unflatten(3, (R // 2, 2)) if case["interleaved"] else a.unflatten(3, (2, R // 2)).transpose(3, 4)
        a = torch.view_as_real(torch.view_as_complex(a.contiguous()) * spin)
        return torch.cat([(a if case["interleaved"] else a.transpose(3, 4)).flatten(3), rest], dim=3)

    X = s["QKV"]
    out = {"Q": turned(X[:, :, :H], s["wq"]).transpose(1, 2)}
    new = {"K": turned(X[:, :, H:H + Hkv], s["wk"]), "V": X[:, :, H + Hkv:].double()}
    table = s["table"].tolist()
    for name in ("K", "V"):
        pool, scales = s[name].double(), s[name.lower() + "_scale"]
        scales = None if scales is None else scales.double()
        for b in range(B):
            n = 0
            while n < count[b]:
                first = (start[b] + n) % T
                m = min(T - first, count[b] - n)
                p, x = table[b][(start[b] + n) // T], new[name][b, n:n + m].transpose(0, 1)  # [Hkv, m, d]
                n += m
                if scales is None:
                    pool[p, :, first:first + m] = x
                    continue
                need = torch.log2(x.abs().amax(dim=(1, 2)) / 448.0).ceil().clamp(LOWEST, HIGHEST)
                need = torch.exp2(need)
                if first:
                    held = pool[p, :, :first] * scales[p][:, None, None]
                    need = torch.maximum(need, scales[p])
                    pool[p, :, :first] = _nearest(held / need[:, None, None])
                pool[p, :, first:first + m] = _nearest(x / need[:, None, None])
                scales[p] = need
        out[name] = pool
        if scales is not None:
            out[name.lower() + "_scale"] = scales
    return out
