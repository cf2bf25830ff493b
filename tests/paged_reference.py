"""64-bit references of the operators on a paged cache, and caches to test on."""
import math

import torch

from tests import layer_reference as ref

E4M3, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


def nearest(x):
    """The e4m3 number next to each of x (double), ties to the even one, 448 at most."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def scale_for(most: float) -> float:
    """The least power of two s within 2^-60 .. 2^60 with 448 s >= most."""
    if not most > 0:
        return 2.0 ** -60
    m, e = math.frexp(most)
    return 2.0 ** max(-60, min(60, e - 9 + (m > 0.875)))


def pools(P, Hkv, T, d, dtype, seed=0, spread=1.0):
    """K, V, k_scale, v_scale of pages of normal values whose sizes differ by page and
    head (by powers of two, e^spread standard deviation), and their values in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out, values = [], []
    for _ in range(2):
        x = torch.randn((P, Hkv, T, d), generator=g, device="cuda")
        x *= torch.exp(spread * torch.randn((P, Hkv, 1, 1), generator=g, device="cuda"))
        if dtype is E4M3:
            m, e = torch.frexp(x.abs().amax(dim=(2, 3)))
            s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).to(e.dtype))
            c = (x / s[..., None, None]).to(E4M3)
            out.append((c, s))
            values.append(c.double() * s[..., None, None].double())
        else:
            out.append((x.to(dtype), None))
            values.append(x.to(dtype).double())
    (K, ks), (V, vs) = out
    return [K, V, ks, vs], values


def table_of(B, M, P, seed=0):
    g = torch.Generator().manual_seed(seed + 1)
    return torch.randperm(P, generator=g)[:B * M].view(B, M).int().cuda()


def dense(values, table):
    """[B, Hkv, M T, d] of the pools' values; pages outside the pool are zero."""
    P = values.shape[0]
    ok = (table >= 0) & (table < P)
    x = values[table.clamp(0, P - 1).long()] * ok[:, :, None, None, None]
    B, M, Hkv, T, d = x.shape
    return x.transpose(1, 2).reshape(B, Hkv, M * T, d)


def attention(Q, k, v, codes, scales, tau, **form):
    """ref.attention over dense keys and values (double, exact in 32 bits), with what an
    8-bit cache adds to the bounds.  Its products run in 16-bit floating point of 11 bits,
    whose smallest step is 2^-24: Q, scaled so that a row's largest element is between 1
    and 2, loses 2^-25 of that at most; a weight times its page's scale, whose largest in
    a row is at least 1, loses 2^-25, so O 2^-25 max(P s) sum |code|.  Their other
    roundings are 2^-11 and in the bounds already (2^-8 for bf16)."""
    val, bound = ref.attention(Q, k.float(), v.float(), tau, **form)
    if scales is None or Q.dtype is not BF:
        return val, bound
    B, H, Nq, d = Q.shape
    G = H // k.shape[1]
    see, _ = ref.visible(B, Nq, k.shape[2], form.get("ranges"), form.get("q_pos"),
                         form.get("causal", False))
    see = see[:, None]
    used = see.any(dim=2)[..., None]
    ka = torch.where(used, k, 0.0).abs().repeat_interleave(G, dim=1)
    ca = torch.where(used, codes, 0.0).abs().repeat_interleave(G, dim=1)
    alive = see.any(dim=3, keepdim=True)
    q = torch.where(alive, Q.double(), 0.0)
    e = 2.0 ** -25 * q.abs().amax(dim=3, keepdim=True) * ka.sum(dim=3)[:, :, None] * tau
    e = torch.where(see, e, 0.0).amax(dim=3)  # of a score
    # P: the same as a relative error of O's sum, twice (numerator and sum).
    va = torch.where(used, v, 0.0).abs().repeat_interleave(G, dim=1)
    most = torch.where(see, va.amax(dim=3)[:, :, None], 0.0).amax(dim=3)
    top = torch.where(see, scales.repeat_interleave(G, dim=1)[:, :, None], 0.0).amax(dim=3)
    bound["L"] = bound["L"] + e
    bound["O"] = bound["O"] + (2 * e * most)[..., None] + 2.0 ** -25 * (
        top[..., None] * torch.where(see, 1.0, 0.0).to(ca) @ ca)
    return val, bound
