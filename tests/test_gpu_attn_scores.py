"""Attention at scores of any size: from fractions to 2^35, both signs, where the rounding of scale * q . k alone is many powers of
two.  A single visible key's weight is 1, equal scores have equal weights, and the largest score wins, whatever its size."""
import numpy as np
import pytest
import torch

from tests import attn_helpers as ah
from tests.gpu_util import progress
from tests.test_gpu_attn import normal, prefill

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
    exponentials, less than 2^-16: with exact q . k, a weight's exponent is off by the roundings of scale, of log2(e), of
    their product and of the difference, each 2^-24 of it; below -26 (base 2) a weight no longer counts in fp32.  So it is off
    by 26 * 4 * 2^-24 of ln 2 of itself and the exponential's own 2^-22; twice, in the sum and in what divides it; and the
    sums, a few hundred additions of 2^-24.  310 weights under fp16's least, 2^-36 of the largest, with |v| < 6 are under 2^-25."""
    u = torch.finfo(dtype).eps / 2
    return u * ref.abs() + (u + 2.0**-16) * (1 + u) * a + (2.0**-25 if dtype == torch.float16 else 0.0)


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
