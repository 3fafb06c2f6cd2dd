"""References in 64 bits for the FP4 cache and the attention calls, written from the header's formulas, and the
problems that the tests of them share."""
import math

import numpy as np
import torch

TYPES = {0: torch.float32, 1: torch.float16, 2: torch.bfloat16}
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])


def quantize(x):
    """(codes uint8 [..., Dh], scale bytes uint8 [..., Dh/32]) of float64 x, by search among the values."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(b).max(-1)
    e = np.full(amax.shape, -120)
    while True:
        low = amax > 6.0 * np.exp2(e.astype(np.float64))
        if not low.any():
            break
        e = e + low
    a = np.abs(b) / np.exp2(e.astype(np.float64))[..., None]
    mids = (E2M1[:7] + E2M1[1:8]) / 2
    code = np.zeros(a.shape, np.uint8)
    for i, m in enumerate(mids):  # past a midpoint, or on it and the code above is even
        code += (a > m) | ((a == m) & ((i + 1) % 2 == 0))
    code |= np.signbit(b).astype(np.uint8) << 3
    return code.reshape(x.shape), (e + 127).astype(np.uint8)


def values(codes, scales):
    """float64 of codes and scale bytes."""
    v = E2M1[codes].reshape(*scales.shape, 32) * np.exp2(scales.astype(np.float64) - 127)[..., None]
    return v.reshape(codes.shape)


def page_bytes(page, Hkv, Dh):
    return Hkv * page * Dh * 17 // 16


def write(kv, page, Hkv, Dh, pid, off, which, codes, scales):
    """One token's codes [Hkv, Dh] and scales [Hkv, Dh/32] into the cache's bytes [num_pages, page_bytes]."""
    region = page * Dh * 17 // 16
    for h in range(Hkv):
        r = kv[pid, h * region:(h + 1) * region]
        for c in range(0, Dh, 2):
            byte = codes[h, c] | codes[h, c + 1] << 4
            if which == 0:
                r[off * (Dh // 2) + c // 2] = byte
            else:
                r[page * Dh // 2 + ((off // 4 * (Dh // 8) + c // 8) * 4 + off % 4) * 4 + c % 8 // 2] = byte
        for s in range(Dh // 32):
            if which == 0:
                r[page * Dh + off * (Dh // 32) + s] = scales[h, s]
            else:
                r[page * Dh + page * Dh // 32 + (off // 4 * (Dh // 32) + s) * 4 + off % 4] = scales[h, s]


class Cache:
    """A cache with every byte that no sequence owns set to 0xFF (NaN scales), pages in a random order and table
    entries behind a sequence out of range.  fill() draws codes and scales; k, v are what they stand for."""

    def __init__(self, lens, Hkv, Dh, page, seed, spare=3, max_pages=None):
        g = np.random.default_rng(seed)
        self.lens, self.Hkv, self.Dh, self.page = list(lens), Hkv, Dh, page
        need = [-(-n // page) for n in lens]
        self.max_pages = max_pages or max(max(need), 1) + 1
        self.num_pages = sum(need) + spare
        order = g.permutation(self.num_pages)
        self.table = np.full((len(lens), self.max_pages), 1 << 30, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.bytes = np.full((self.num_pages, page_bytes(page, Hkv, Dh)), 0xFF, np.uint8)
        self.k = self.v = None

    def places(self, b, n=None):
        pos = np.arange(self.lens[b] if n is None else n)
        return self.table[b, pos // self.page], pos % self.page

    def _fields(self, which):
        P, H, page, Dh = self.num_pages, self.Hkv, self.page, self.Dh
        r = self.bytes.reshape(P, H, -1)
        half, sc = page * Dh // 2, page * Dh // 32
        c, s = r[:, :, which * half:][:, :, :half], r[:, :, 2 * half + which * sc:][:, :, :sc]
        if which == 0:
            return c.reshape(P, H, page, Dh // 2), s.reshape(P, H, page, Dh // 32)
        return c.reshape(P, H, page // 4, Dh // 8, 4, 4), s.reshape(P, H, page // 4, Dh // 32, 4)

    def put(self, b, which, codes, scales, pos):
        """Vectorised write(): codes [n, Hkv, Dh], scales [n, Hkv, Dh/32] at positions pos."""
        c, s = self._fields(which)
        assert np.shares_memory(c, self.bytes) and np.shares_memory(s, self.bytes)
        pid, off = self.table[b, pos // self.page], pos % self.page
        data = codes[..., 0::2] | codes[..., 1::2] << 4
        if which == 0:
            c[pid, :, off], s[pid, :, off] = data, scales
        else:
            c[pid, :, off // 4, :, off % 4] = data.reshape(*data.shape[:-1], self.Dh // 8, 4)
            s[pid, :, off // 4, :, off % 4] = scales

    def fill(self, seed, lo=123, hi=128):
        g = np.random.default_rng(seed)
        self.k, self.v = [], []
        for b, n in enumerate(self.lens):
            for which, out in ((0, self.k), (1, self.v)):
                codes = g.integers(0, 16, (n, self.Hkv, self.Dh)).astype(np.uint8)
                scales = g.integers(lo, hi, (n, self.Hkv, self.Dh // 32)).astype(np.uint8)
                self.put(b, which, codes, scales, np.arange(n))
                out.append(values(codes, scales))
        return self

    def device(self):
        """(pages, max_pages, page, num_pages, kv) on the GPU."""
        return (torch.from_numpy(self.table).cuda(), self.max_pages, self.page, self.num_pages,
                torch.from_numpy(self.bytes).cuda())

    def lens_device(self):
        return torch.tensor(self.lens, dtype=torch.int32, device="cuda")


def attend(q, k, v, scale, window, hidden=None):
    """float64 torch: q [Lq, H, Dh] at the end of k, v [Lk, Hkv, Dh].  Returns y [Lq, H, Dh], the sums
    sum_j p_j |v_j| of the same shape, and [Lq, H, 1] the largest scale * sum |q k| of a visible key.
    hidden: bool [Lk], keys that nothing sees."""
    Lq, H, Dh = q.shape
    Lk, Hkv = k.shape[:2]
    y, a = torch.zeros_like(q), torch.zeros_like(q)
    big = torch.zeros(Lq, H, 1, dtype=q.dtype, device=q.device)
    if Lk == 0 or Lq == 0:
        return y, a, big
    pos = Lk - Lq + torch.arange(Lq, device=q.device)[:, None]
    j = torch.arange(Lk, device=q.device)[None]
    seen = j <= pos
    if window:
        seen &= j > pos - window
    if hidden is not None:
        seen &= ~hidden[None]
    for h in range(H):
        kk, vv = k[:, h // (H // Hkv)].contiguous(), v[:, h // (H // Hkv)].contiguous()
        s = scale * (q[:, h] @ kk.t().contiguous())
        mag = abs(scale) * (q[:, h].abs() @ kk.abs().t().contiguous())
        s = s.masked_fill(~seen, -math.inf)
        w = torch.exp(s - s.amax(1, keepdim=True).clamp(min=-1e300))
        w = torch.where(seen, w, 0.0)
        p = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        y[:, h], a[:, h] = p @ vv, p @ vv.abs()
        big[:, h] = torch.where(seen, mag, 0.0).amax(1, keepdim=True)
    return y, a, big


def decode_tolerance(a, big, L, Dh):
    """Largest error of an fp32 output.  A score is a sum of Dh products of up to three exact parts of q with exact keys: each of
    the 3 Dh additions is off by at most 2^-24 of sum |q k|, the parts themselves by 2^-24, the scaling and the two
    roundings of the exponent's argument by 4 * 2^-24 of |s|, exp by 2^-22; p depends on a score in numerator
    and sum: twice.  A weight is carried in two bf16 parts: 2^-18.  A sum over L keys goes 32 at a time through
    the matrix cores: L/32 + 32 additions for each part, and up to 80 in joining."""
    return (2 * (3 * Dh + 8) * 2.0**-24 * big + 2.0**-21 + 2.0**-18 + (L / 16 + 144) * 2.0**-24) * a + 1e-37


def prefill_tolerance(y, a, big, v_max, L, Dh, dtype):
    """As above for 16-bit outputs: q, k, v exact; each weight is rounded to the type (half a step of it, or half the least
    subnormal, against a sum of at least one) and so is y."""
    u = torch.finfo(dtype).eps / 2
    least = 2.0**-25 if dtype == torch.float16 else 0.0
    return (u * y.abs() + least + (2 * (Dh + 8) * 2.0**-24 * big + 2.0**-21 + u + (L / 16 + 144) * 2.0**-24) * a * (1 + u)
            + L * least * v_max)


def rows_with_gap(x, gap):
    """x [n, heads, Dh] as a part of wider rows: gap elements (NaN) lie before and behind each row's."""
    n, heads, Dh = x.shape
    wide = torch.full((n, heads * Dh + 2 * gap), math.nan, dtype=x.dtype, device=x.device)
    wide[:, gap:gap + heads * Dh] = x.reshape(n, -1)
    return wide[:, gap:gap + heads * Dh].unflatten(1, (heads, Dh))


def cumulative(lens, first=0):
    return torch.tensor(np.cumsum([first] + list(lens)), dtype=torch.int32, device="cuda")
