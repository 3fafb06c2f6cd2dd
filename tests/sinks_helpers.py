"""64-bit references of the norm and rotation of queries and keys, and of attention with first positions that stay visible,
written from the header's formulas, with the tolerances that their tests share."""
import math

import numpy as np
import torch

from tests import attn_helpers as ah


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def normal(seed, shape, dtype, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * spread).to(dtype)


# ---- attention -------------------------------------------------------------------------------------------------

def sees(pos, L, window, sinks):
    """bool [Lq, L]: the keys that queries at pos [Lq] see."""
    j, p = torch.arange(L, device=pos.device)[None], pos[:, None]
    return (j <= p) & ((j > p - window) | (j < sinks)) if window else j <= p


def attend(q, k, v, scale, seen):
    """As attn_helpers.attend, of q [Lq, H, Dh], k, v [L, Hkv, Dh] and a mask [Lq, L]."""
    H, Hkv = q.shape[1], k.shape[1]
    y, a = torch.zeros_like(q), torch.zeros_like(q)
    big = torch.zeros(q.shape[0], H, 1, dtype=q.dtype, device=q.device)
    if k.shape[0] == 0:
        return y, a, big
    k, v = (torch.where(seen.any(0)[:, None, None], x, 0.0) for x in (k, v))
    for h in range(H):
        kk, vv = k[:, h // (H // Hkv)].contiguous(), v[:, h // (H // Hkv)].contiguous()
        s = (scale * (q[:, h] @ kk.t().contiguous())).masked_fill(~seen, -math.inf)
        mag = abs(scale) * (q[:, h].abs() @ kk.abs().t().contiguous())
        w = torch.where(seen, torch.exp(s - s.amax(1, keepdim=True).clamp(min=-1e300)), 0.0)
        p = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        y[:, h], a[:, h] = p @ vv, p @ vv.abs()
        big[:, h] = torch.where(seen, mag, 0.0).amax(1, keepdim=True)
    return y, a, big


def check_decode(y, q, k, v, lens, Tq, scale, window, sinks, hidden=None, prefix=0):
    """y [B * Tq, H, Dh] against each sequence's k[b], v[b] (float64 arrays); hidden[b]: bool [len], keys of bad pages.
    Over a shared prefix a weight is two fp16 parts of 2^11 times itself: what is left of the first, rounded again, is off
    by 2^-24 of it (inside attn_helpers' 2^-18) or by half of fp16's least step, 2^-25, so the weight by 2^-36.  It
    is divided by a sum of at least one (the key with the running maximum has weight one): 2^-36 of each |v|."""
    for b, n in enumerate(lens):
        kk, vv = (torch.from_numpy(np.ascontiguousarray(x[b])).cuda() for x in (k, v))
        rows = slice(b * Tq, (b + 1) * Tq)
        seen = sees(n - Tq + torch.arange(Tq, device="cuda"), n, window, sinks)
        if hidden is not None and b in hidden:
            seen = seen & ~hidden[b][None]
        ref, a, big = attend(q[rows].double(), kk, vv, scale, seen)
        err, lim = (y[rows].double() - ref).abs(), ah.decode_tolerance(a, big, n, q.shape[2])
        if prefix:
            lim = lim + 2.0**-36 * vv[:prefix].abs().sum(0).repeat_interleave(q.shape[1] // kk.shape[1], 0)
        assert bool((err <= lim).all()), "sequence %d (%d positions): %.3g of the tolerance" % (b, n, float((err / lim).max()))


# ---- norm and rotation -----------------------------------------------------------------------------------------

def rope(x, w, pos, freq, eps, neighbours):
    """float64 x [n, heads, Dh], w [Dh] or None, pos [n], freq [R/2].  Returns y and what its tolerance is made of: the
    sum of the pair's magnitudes before the turn, and the angle's."""
    u = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        u = u * w
    y, pair, angle = u.clone(), u.abs(), torch.zeros_like(u)
    t = pos[:, None, None] * freq
    half = freq.shape[0]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + half)
        c, s = torch.cos(t[..., i]), torch.sin(t[..., i])
        y[..., a], y[..., b] = u[..., a] * c - u[..., b] * s, u[..., b] * c + u[..., a] * s
        pair[..., a] = pair[..., b] = u[..., a].abs() + u[..., b].abs()
        angle[..., a] = angle[..., b] = t[..., i].abs()
    return y, pair, angle


def rope_tolerance(y, pair, angle, dtype):
    """Largest error.  The sum of Dh squares: 16 one after another, four steps between lanes, eps; half of that remains
    under the root, which is rounded, as are its inverse and the products with it and w: 15 * 2^-24.  Sine and cosine: the
    rest of the angle rounded (2^-25), the series' last steps (2 * 2^-24) and end (2^-28), the angle in 64 bits.  The turn:
    one product rounded and the sum: 2 * 2^-24 of the pair.  Other types round once, or are subnormal; fp32 may be too."""
    lim = (20 * 2.0**-24 + 2 * 2.0**-53 * angle) * pair * (1 + 2.0**-20) + 2.0**-126
    if dtype == torch.float32:
        return lim
    least = 2.0**-25 if dtype == torch.float16 else 2.0**-134
    return lim + torch.finfo(dtype).eps / 2 * (y.abs() + lim) + least
