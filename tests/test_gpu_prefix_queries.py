"""attn_decode_kv4_prefix with shared rows and fp32 queries whose elements lie far apart: what is small beside the row's
largest element keeps the bits that the header says, 2^-23 of itself, where the keys hide the large one."""
import numpy as np
import pytest
import torch

from tests import attn_helpers as ah
from tests import sinks_helpers as sh
from tests.gpu_util import progress
from tests.test_gpu_prefix import Shared
from tests.test_gpu_prefix_shared import CASES, lengths, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


def one_channel_a_block(prefix, B, Hkv, Dh, page, channel):
    """Keys that are zero but for one channel of each 32, `channel` among them: no block is zero, whose scale would be 2^-120."""
    s = Shared(prefix, lengths(prefix, B), Hkv, Dh, page, 121)
    g = np.random.default_rng(122)
    skip, held = prefix // page, []
    for b, n in enumerate(s.c.lens):
        codes = np.zeros((n, Hkv, Dh), np.uint8)
        codes[..., channel % 32::32] = g.integers(1, 8, (n, Hkv, Dh // 32)) + 8 * g.integers(0, 2, (n, Hkv, Dh // 32))
        scales = g.integers(125, 129, (n, Hkv, Dh // 32)).astype(np.uint8)
        own = np.arange(n) if b == 0 else np.arange(min(prefix - skip * page, n), n)
        s.c.put(b, 0, codes[own], scales[own], own)
        held.append(ah.values(codes, scales))
    s.k = [np.concatenate([held[0], held[b + 1][min(prefix - skip * page, s.c.lens[b + 1]):]])[:n] for b, n in enumerate(s.lens)]
    return s


def check(y, q, s, Tq, scale):
    """As sinks_helpers.check_decode, but of scores that are one product each: a query's element is off by 2^-23 of itself and
    its two parts' products are rounded, 2^-22 of the score; the factor, its product with the score and the largest score, and
    the argument of exp are rounded, and so are the differences that joins take: 5 * 2^-24 of the largest score.  Twice, in
    numerator and sum, with exp's 2^-22 each time.  A weight is two fp16 or three bf16 parts: 2^-24, or 2^-36."""
    for b, n in enumerate(s.lens):
        kk, vv = (torch.from_numpy(np.ascontiguousarray(x[b])).cuda() for x in (s.k, s.v))
        rows = slice(b * Tq, (b + 1) * Tq)
        seen = sh.sees(n - Tq + torch.arange(Tq, device="cuda"), n, 0, 0)
        ref, a, big = sh.attend(q[rows].double(), kk, vv, scale, seen)
        lim = (2 * 9 * 2.0**-24 * big + 2.0**-21 + 2.0**-24 + (n / 16 + 144) * 2.0**-24) * a + 1e-37
        lim = lim + 2.0**-36 * vv[:s.prefix].abs().sum(0).repeat_interleave(q.shape[1] // kk.shape[1], 0)
        err = (y[rows].double() - ref).abs()
        assert bool((err <= lim).all()), "sequence %d (%d positions): %.3g of the tolerance" % (b, n, float((err / lim).max()))


@pytest.mark.parametrize("most,channel", [(15, 1), (20, -1), (25, 32), (30, 40)])
@pytest.mark.parametrize("prefix,B,Tq,G,Hkv,Dh,page", [CASES[i] for i in (0, 1, 2, 3, 4, 5, 7, 8)])
def test_small_elements_of_a_row(qg, prefix, B, Tq, G, Hkv, Dh, page, channel, most):
    """One element of every row up to 2^most times the others, where the keys are zero; 24 bits of what they meet count."""
    channel %= Dh
    progress("shared prefix queries 2^%d apart, channel %d of %d, prefix %d" % (most, channel, Dh, prefix))
    s = one_channel_a_block(prefix, B, Hkv, Dh, page, channel)
    q = torch.zeros(B * Tq, G * Hkv, Dh, device="cuda")
    size = 1 + sh.normal(123, q.shape[:2], torch.float32).abs().fmod(1.0)
    q[..., channel] = size * sh.normal(124, q.shape[:2], torch.float32).sign()
    assert bool((q[..., channel] != 0).all())
    large = (channel + 2) % Dh  # not a channel of any key
    apart = torch.arange(q.shape[0] * q.shape[1], device="cuda").view(q.shape[:2]) % (most + 1)
    q[..., large] = torch.exp2((most - apart // 2).float())
    y, st = run(qg, s, q, 0, Tq, G * Hkv, 1.0)
    assert int(st) == 0
    check(y, q, s, Tq, 1.0)


@pytest.mark.parametrize("unit", [2.0**-70, 2.0**-50, 2.0**-20, 2.0**40, 2.0**70])
def test_rows_of_any_size(qg, unit):
    """The same with all elements larger or smaller: rows beyond 2^60 either way are taken otherwise."""
    prefix, B, Tq, G, Hkv, Dh, page = CASES[3]
    progress("shared prefix queries around %g" % unit)
    s = one_channel_a_block(prefix, B, Hkv, Dh, page, 7)
    q = torch.zeros(B, G * Hkv, Dh, device="cuda")
    q[..., 7] = unit * (1 + sh.normal(125, q.shape[:2], torch.float32).abs().fmod(1.0))
    q[..., 9] = unit * 2.0**25
    q[::7, :, 9] = 0
    y, st = run(qg, s, q, 0, 1, G * Hkv, 1.0 / unit)
    assert int(st) == 0
    check(y, q, s, 1, 1.0 / unit)
