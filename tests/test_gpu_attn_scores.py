"""Attention at scores of any size: from fractions to 2^35, both signs, where the rounding of scale * q . k alone is many powers of
two.  A single visible key's weight is 1, equal scores have equal weights, and the largest score wins, whatever its size."""
import numpy as np
import pytest
import torch

from tests import attn_helpers as ah
from tests.gpu_util import progress
from tests.test_gpu_attn import decode, normal, prefill

pytestmark = pytest.mark.gpu

# scale * q . k; from 2^16 on another form of the weights is taken
SCORES = [3.0, 2.0**15, 2.0**17, 2.0**20, 2.0**24, 2.0**25, 2.0**27, 1e10, 1.2345e10]
# heads and sequences for four, two and one wave per 32 queries
SHARES = [(1, 1), (64, 1), (264, 2)]


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


def prefill_limit(ref, a, dtype):
    """y is rounded once, u of it; a weight is rounded to the type, u of it and of its part of sum p |v|; fp32 sums and
    exponentials as below, 2^-16; 310 weights under fp16's least, 2^-36 of the largest, with |v| < 6 are under 2^-25."""
    u = torch.finfo(dtype).eps / 2
    return u * ref.abs() + (u + 2.0**-16) * (1 + u) * a + (2.0**-25 if dtype == torch.float16 else 0.0)


def decode_limit(a):
    """With exact q . k, a weight's exponent is off by the roundings of scale, of log2(e), of their product and of the
    difference, each 2^-24 of it; below -26 (base 2) a weight no longer counts in fp32.  So it is off by 26 * 4 * 2^-24 of
    ln 2 of itself and the exponential's own 2^-22; twice, in the sum and in what divides it; and the sums, a few hundred
    additions of 2^-24: less than 2^-16."""
    return 2.0**-16 * a + 1e-37


@pytest.mark.parametrize("type", [1, 2])
@pytest.mark.parametrize("H,B", SHARES)
@pytest.mark.parametrize("score", SCORES)
def test_prefill_one_and_equal_keys(qg, score, H, B, type):
    """Window 1: y is v.  Without: every query sees equal keys, y is their mean."""
    progress("prefill equal scores %g H %d type %d" % (score, H, type))
    dt, n = ah.TYPES[type], 300
    for Dh in (64, 128, 256):
        q, k = (torch.full((B * n, heads, Dh), 4.0, dtype=dt, device="cuda") for heads in (H, 1))
        v = normal(7, (B * n, 1, Dh), dt)
        for window in (1, 0):
            for sign in (1.0, -1.0):
                y, st = prefill(qg, q, k, v, [n] * B, [n] * B, type, H, 1, Dh, sign * score / (16 * Dh), window)
                assert int(st) == 0
                for b in range(B):
                    vv = v[b * n:(b + 1) * n].double()
                    count = torch.arange(1, n + 1, device="cuda")[:, None, None]
                    ref, a = (vv, vv.abs()) if window else (vv.cumsum(0) / count, vv.abs().cumsum(0) / count)
                    err = (y[b * n:(b + 1) * n].double() - ref).abs()
                    assert bool((err <= prefill_limit(ref, a, dt)).all()), (Dh, window, sign, float(err.nan_to_num(9e9).max()))


@pytest.mark.parametrize("type", [1, 2])
@pytest.mark.parametrize("scale", [1.0, -1.0])
def test_prefill_large_products(qg, scale, type):
    """q = k = 1024 in every channel: the products themselves are 2^26 to 2^28."""
    progress("prefill products of 2^27 type %d" % type)
    dt, n = ah.TYPES[type], 90
    for Dh in (64, 128, 256):
        q = torch.full((n, 2, Dh), 1024.0, dtype=dt, device="cuda")
        k, v = q[:, :1].contiguous(), normal(8, (n, 1, Dh), dt)
        v[:, :, ::3] = 0.0
        y, _ = prefill(qg, q, k, v, [n], [n], type, 2, 1, Dh, scale, 1)
        err, vv = (y.double() - v.double()).abs(), v.double()
        assert bool((err <= prefill_limit(vv, vv.abs(), dt)).all())


def exact_scores(rows, keys, Dh, order, seed):
    """q [rows, 1, Dh] and k [keys, 1, Dh] whose products are exact: one channel, powers of two from 2^-6 to 2^24 (in turn over the
    rows) times whole numbers of at most 6."""
    g = np.random.default_rng(seed)
    q, k = np.zeros((rows, 1, Dh)), np.zeros((keys, 1, Dh))
    q[:, 0, 3] = np.exp2(np.arange(rows) % 31 - 6.0) * np.where(np.arange(rows) % 2, -1.0, 1.0)
    vals = g.choice([-6.0, -4.0, -3.0, -2.0, -1.0, 0.0, 1.0, 2.0, 3.0, 4.0, 6.0], keys)
    k[:, 0, 3] = vals if order == "any" else np.sort(vals) if order == "rising" else np.sort(vals)[::-1]
    return torch.from_numpy(q).cuda(), torch.from_numpy(k).cuda()


@pytest.mark.parametrize("type", [1, 2])
@pytest.mark.parametrize("H,B", SHARES)
@pytest.mark.parametrize("order", ["any", "rising", "falling"])
def test_prefill_far_and_near_rows(qg, order, H, B, type):
    """Rows whose scores are fractions beside rows whose scores are 2^33 or so, and rows that pass from one to the other."""
    progress("prefill scores of all sizes %s H %d type %d" % (order, H, type))
    dt, n = ah.TYPES[type], 310
    for Dh, window in ((64, 0), (128, 70), (256, 0)):
        q, k = exact_scores(n, n, Dh, order, 3)
        up = 2.0**10 if type == 1 else 1.0  # fp16's largest power of two is 2^15
        q = (q / up).to(dt).repeat(B, H, 1)
        k, v = k.to(dt).repeat(B, 1, 1), normal(9, (B * n, 1, Dh), dt)
        y, st = prefill(qg, q, k, v, [n] * B, [n] * B, type, H, 1, Dh, 64.0 * up, window)
        assert int(st) == 0
        for b in range(B):
            at = slice(b * n, (b + 1) * n)
            ref, a, _ = ah.attend(q[at, :1].double(), k[at].double(), v[at].double(), 64.0 * up, window)
            err = (y[at].double() - ref).abs()
            assert bool((err <= prefill_limit(ref, a, dt)).all()), (Dh, b, float(err.nan_to_num(9e9).max()))


def cache_with_keys(c, keys):
    """Cache c with keys [positions, Dh] (E2M1 values, scale 1) for every sequence and head, in place of its own."""
    for b, n in enumerate(c.lens):
        x = np.broadcast_to(keys[:n, None], (n, c.Hkv, c.Dh))
        scales = np.full((n, c.Hkv, c.Dh // 32), 127, np.uint8)
        codes = np.searchsorted(ah.E2M1[:8], np.abs(x)).astype(np.uint8) | np.signbit(x).astype(np.uint8) << 3
        c.put(b, 0, codes, scales, np.arange(n))
        c.k[b] = ah.values(codes, scales)
        assert np.array_equal(c.k[b], x)
    return c


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("score", SCORES)
def test_decode_one_and_equal_keys(qg, score, type):
    progress("decode equal scores %g type %d" % (score, type))
    lens = [1, 40, 700, 5000]
    for Dh, G, Tq in ((64, 1, 1), (128, 4, 2), (256, 16, 1)):
        c = ah.Cache(lens, 2, Dh, 16, 21).fill(22)
        cache_with_keys(c, np.full((max(lens), Dh), 4.0))
        q = torch.full((len(lens) * Tq, 2 * G, Dh), 4.0, dtype=ah.TYPES[type], device="cuda")
        for window in (1, 0):
            for sign in (1.0, -1.0):
                y, st = decode(qg, c, q, type, Tq, 2 * G, sign * score / (16 * Dh), window)
                assert int(st) == 0
                for b, n in enumerate(lens):
                    at = slice(b * Tq, (b + 1) * Tq)
                    k, v = (torch.from_numpy(x[b]).cuda() for x in (c.k, c.v))
                    ref, a, _ = ah.attend(q[at].double(), k, v, 0.0, window)  # equal scores
                    err = (y[at].double() - ref).abs()
                    assert bool((err <= decode_limit(a)).all()), (Dh, window, sign, n, float(err.nan_to_num(9e9).max()))


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("order", ["any", "rising", "falling"])
def test_decode_far_and_near_rows(qg, order, type):
    """As for prompts; several chunks and the join among them."""
    progress("decode scores of all sizes %s type %d" % (order, type))
    lens = [33, 640, 2500, 9001]
    for Dh, G, Tq, window in ((64, 31, 1, 0), (128, 8, 1, 0), (128, 16, 2, 1700), (256, 5, 7, 0)):
        q, k = exact_scores(G * Tq, max(lens), Dh, order, 5)
        c = ah.Cache(lens, 1, Dh, 32, 23).fill(24)
        cache_with_keys(c, k[:, 0].cpu().numpy())
        up = 2.0**10 if type == 1 else 1.0
        q = (q / up).to(ah.TYPES[type]).view(Tq, G, Dh).repeat(len(lens), 1, 1)
        y, st = decode(qg, c, q, type, Tq, G, 64.0 * up, window)
        assert int(st) == 0
        for b, n in enumerate(lens):
            at = slice(b * Tq, (b + 1) * Tq)
            kk, vv = (torch.from_numpy(x[b]).cuda() for x in (c.k, c.v))
            ref, a, _ = ah.attend(q[at].double(), kk, vv, 64.0 * up, window)
            err = (y[at].double() - ref).abs()
            assert bool((err <= decode_limit(a)).all()), (Dh, G, Tq, n, float(err.nan_to_num(9e9).max()))


def test_decode_products_of_real_numbers(qg):
    """fp32 queries of about 1e10 in every channel: one visible key, and one key above all others."""
    progress("decode products of 1e10")
    for Dh in (64, 128, 256):
        c = ah.Cache([1, 700], 1, Dh, 16, 25).fill(26)
        q = normal(27, (2, 4, Dh), torch.float32, 1e10)
        y, _ = decode(qg, c, q, 0, 1, 4, 1.0, 0)
        for b in range(2):
            k, v = (torch.from_numpy(x[b]).cuda() for x in (c.k, c.v))
            s = torch.matmul(q[b].double(), k[:, 0].t().contiguous())
            best = s.topk(min(2, s.shape[1]), dim=1)
            if s.shape[1] > 1:  # more apart than the scores' own roundings
                assert float((best.values[:, 0] - best.values[:, 1]).min()) > 1e6
            ref = v[best.indices[:, 0], 0]
            assert bool(((y[b].double() - ref).abs() <= decode_limit(ref.abs())).all()), (Dh, b)


@pytest.mark.parametrize("Dh,G", [(64, 1), (128, 8), (256, 16)])
def test_decode_largest_queries(qg, Dh, G):
    """fp32 queries up to the largest finite value, at the keys of the least scales; each score is moderate.  The limit is
    attn_helpers' own."""
    progress("decode queries of 3.4e38, Dh %d G %d" % (Dh, G))
    c = ah.Cache([300, 40], 1, Dh, 16, 31).fill(32, 7, 8)
    for b, n in enumerate(c.lens):  # values of ordinary size
        codes = np.random.default_rng(b).integers(0, 16, (n, 1, Dh)).astype(np.uint8)
        scales = np.full((n, 1, Dh // 32), 126, np.uint8)
        c.put(b, 1, codes, scales, np.arange(n))
        c.v[b] = ah.values(codes, scales)
    q = normal(34, (2, G, Dh), torch.float32, 1e37)
    top = torch.finfo(torch.float32).max
    q[:, :, 0], q[:, :, 1], q[:, 0, 2] = top, -top, torch.nextafter(torch.tensor(top), torch.tensor(0.0)).item()
    y, st = decode(qg, c, q, 0, 1, G, 0.01, 0)
    assert int(st) == 0
    for b, n in enumerate(c.lens):
        k, v = (torch.from_numpy(x[b]).cuda() for x in (c.k, c.v))
        ref, a, big = ah.attend(q[b:b + 1].double(), k, v, 0.01, 0)
        assert bool(((y[b:b + 1].double() - ref).abs() <= ah.decode_tolerance(a, big, n, Dh)).all()), b
