"""64-bit references of the operators around an attention layer, with
element-wise error bounds of the kernels' arithmetic.

A bound counts the roundings that a kernel makes.  u is half a step of the
inputs' type (torch.finfo(t).eps / 2).  Each output is rounded once, |x| u.
The weights P and the score gradients dS are rounded to the type before the
products with V, dO, K and Q, so a sum over them is off by at most u times the
same sum over absolute values.  All else is fp32: a relative error e of P
covers the score's dot product (d + 4 roundings of 2^-24 of the absolute
products, in the forward's score and again in L), the bias, the tanh, the
exponential and the row sum.  D = dO . O is computed from the rounded O.
Numbers below 2^-126, the smallest normal number of fp32 and of bf16, may be
flushed to 0: 2^-126 absolute for each weight that a query gives a key it sees
(and so |dP - D| times that for dS), and for dS itself.
"""
import math

import torch

TINY = 2.0 ** -126


def visible(B, Nq, Nk, ranges, q_pos, causal, device="cuda"):
    """[B, Nq, Nk] truth values, and positions [B, Nq]."""
    j = torch.arange(Nk, device=device)
    pos = q_pos.long() if q_pos is not None else torch.arange(Nq, device=device).expand(B, Nq)
    see = torch.ones((B, Nq, Nk), dtype=torch.bool, device=device)
    if ranges is not None:
        see &= (j >= ranges[:, :, :1]) & (j < ranges[:, :, 1:])
    if causal:
        see &= j <= pos[:, :, None]
    return see, pos


def attention(Q, K, V, tau, cap=0.0, slopes=None, ranges=None, q_pos=None, causal=False, dO=None):
    """(values, bounds): dicts of O, L and, with dO, dQ, dK, dV."""
    t = Q.dtype
    u = torch.finfo(t).eps / 2
    B, H, Nq, d = Q.shape
    Hkv, Nk = K.shape[1], K.shape[2]
    G = H // Hkv
    see, pos = visible(B, Nq, Nk, ranges, q_pos, causal)
    see = see[:, None]
    alive = see.any(dim=3, keepdim=True)  # [B, 1, Nq, 1]
    used = see.any(dim=2)[:, :, :, None]  # [B, 1, Nk, 1]
    # What nobody sees, and the rows that see nothing, take no part.
    q = torch.where(alive, Q.double(), 0.0)
    k = torch.where(used, K.double(), 0.0).repeat_interleave(G, dim=1)
    v = torch.where(used, V.double(), 0.0).repeat_interleave(G, dim=1)
    z = q @ k.transpose(2, 3) * tau
    e = (d + 4) * 2.0 ** -24 * (q.abs() @ k.abs().transpose(2, 3) * tau)
    damp = torch.ones_like(z)
    if cap:
        th = torch.tanh(z / cap)
        z, damp = cap * th, 1 - th * th
        e = e * damp + cap * 2.0 ** -21
    if slopes is not None:
        far = slopes.double()[None, :, None, None] * (pos[:, None, :, None]
                                                       - torch.arange(Nk, device=Q.device)).abs()
        z, e = z - far, e + far * 2.0 ** -22
    e = e + z.abs() * 2.0 ** -22
    z = torch.where(see, z, -math.inf)
    L = torch.logsumexp(z, dim=3, keepdim=True)
    P = torch.where(see, torch.exp(z - torch.where(alive, L, 0.0)), 0.0)
    e = torch.where(see, e, 0.0)
    eL = e.amax(dim=3, keepdim=True) + (Nk + 8) * 2.0 ** -24  # of L, absolute
    eP = e + eL + torch.where(alive, L.abs(), 0.0) * 2.0 ** -22 + 2.0 ** -20  # of P, relative
    bP = torch.where(see, P * (u + eP) + TINY, 0.0)  # of P, absolute
    O = P @ v
    aO = P @ v.abs()
    bO = u * O.abs() + bP @ v.abs()
    val = {"O": O, "L": L[..., 0]}
    bound = {"O": bO, "L": (eL + L.abs() * 2.0 ** -22)[..., 0]}
    if dO is None:
        return val, bound
    w = torch.where(alive, dO.double(), 0.0)
    dP = w @ v.transpose(2, 3)
    D = (w * O).sum(dim=3, keepdim=True)
    eD = (w.abs() * (bO + u * O.abs())).sum(dim=3, keepdim=True) + d * 2.0 ** -24 * (
        w.abs() * aO).sum(dim=3, keepdim=True)
    dS = P * (dP - D) * damp
    # damp = 1 - tanh^2 is off by twice what tanh is (2^-21).
    eS = (P * damp * (eD + (d + 4) * 2.0 ** -24 * (w.abs() @ v.abs().transpose(2, 3)))
          + dS.abs() * (eP + u + 2.0 ** -22) + P * (dP - D).abs() * (2.0 ** -19 if cap else 0.0)
          + torch.where(see, TINY * (1 + (dP - D).abs()), 0.0))

    def shared(x):
        return x.view(B, Hkv, G, Nk, d).sum(dim=2)

    dQ = tau * dS @ k
    dK = shared(tau * dS.transpose(2, 3) @ q)
    dV = shared(P.transpose(2, 3) @ w)
    val |= {"dQ": dQ, "dK": dK, "dV": dV}
    bound |= {"dQ": u * dQ.abs() + tau * eS @ k.abs(),
              "dK": u * dK.abs() + shared(tau * eS.transpose(2, 3) @ q.abs()),
              "dV": u * dV.abs() + shared(bP.transpose(2, 3) @ w.abs())}
    return val, bound


def worst(got, val, bound):
    """The largest error as a share of its bound (infinities and NaN have to agree)."""
    got = got.double()
    same = got == val  # infinities; exact zeros with a bound of zero
    share = (got - val).abs() / bound.clamp(min=1e-36)
    return float(torch.where(same, 0.0, share).max())


def norm_rope(QKV, H, wq, wk, freqs, positions, eps, interleaved):
    """Q, K, V in 64 bits (differentiable), from the definition."""
    B, N, heads, d = QKV.shape
    Hkv = (heads - H) // 2
    R = 0 if freqs is None else 2 * freqs.shape[1]
    x = QKV.double()
    if R:
        if positions is None:
            positions = torch.arange(N, device=QKV.device).expand(1, B, N)
        ang = torch.einsum("abn,ak->bnk", positions.double(), freqs.double())[:, :, None]
        cos, sin = torch.cos(ang), torch.sin(ang)

    def one(x, w):
        y = x * torch.rsqrt((x * x).mean(dim=3, keepdim=True) + eps)
        if w is not None:
            y = y * w.double()
        if R:
            a, rest = y[..., :R], y[..., R:]
            if interleaved:
                a, b = a[..., 0::2], a[..., 1::2]
                turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=4).flatten(3)
            else:
                a, b = a[..., :R // 2], a[..., R // 2:]
                turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=3)
            y = torch.cat([turned, rest], dim=3)
        return y.transpose(1, 2)

    return one(x[:, :, :H], wq), one(x[:, :, H:H + Hkv], wk), x[:, :, H + Hkv:].transpose(1, 2)
