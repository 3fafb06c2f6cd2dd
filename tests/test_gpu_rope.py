"""qk_norm_rope against the formula in 64 bits, at tolerances derived in sinks_helpers."""
import math

import numpy as np
import pytest
import torch

from tests import attn_helpers as ah
from tests import sinks_helpers as sh
from tests.gpu_util import progress

pytestmark = pytest.mark.gpu
TYPES = ah.TYPES


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


def freqs(R, base=10000.0):
    return torch.tensor([base ** (-2 * i / R) for i in range(R // 2)], dtype=torch.float32, device="cuda")


def call(qg, q, k, lens, news, R, neighbours, out, freq=None, wq=None, wk=None, eps=1e-6, first=0, into=None, stream=None,
         lens_d=None, cu=None):
    n, H, Dh = q.shape
    Hkv, t = k.shape[1], [i for i in TYPES if TYPES[i] == q.dtype][0]
    yq, yk = into or (torch.full((n, h, Dh), 77.0, dtype=TYPES[out], device="cuda") for h in (H, Hkv))
    st = sh.status()
    freq = freqs(R) if freq is None and R else freq
    qg.qk_norm_rope(t, q, q.stride(0), k, k.stride(0), n, ah.cumulative(news, first) if cu is None else cu,
                    torch.tensor(lens, dtype=torch.int32, device="cuda") if lens_d is None else lens_d, len(lens), H, Hkv,
                    Dh, wq, wk, eps, R, qg.ROPE_NEIGHBOURS if neighbours else qg.ROPE_HALVES, freq, out, yq, yq.stride(0),
                    yk, yk.stride(0), st, stream=stream)
    return yq, yk, st


def check(got, x, w, lens, news, freq, eps, neighbours, first=0, skip=()):
    """got, x [n, heads, Dh]; rows of no sequence, and of those in skip, keep 77."""
    pos = torch.full((x.shape[0],), -1.0, dtype=torch.float64)
    at = first
    for b, (n, m) in enumerate(zip(lens, news)):
        if b not in skip:
            pos[at:at + m] = torch.arange(n - m, n, dtype=torch.float64)
        at += m
    there = (pos >= 0).cuda()
    assert bool((got[~there] == 77.0).all())
    y, pair, angle = sh.rope(x[there].double(), None if w is None else w.double(), pos.cuda()[there], freq.double(), eps,
                             neighbours)
    err, lim = (got[there].double() - y).abs(), sh.rope_tolerance(y, pair, angle, got.dtype)
    assert bool((err <= lim).all()), "%.3g of the tolerance" % float((err / lim).max())


CASES = [
    # lens, new, H, Hkv, Dh, R
    ([1], [1], 1, 1, 64, 64),
    ([1, 0, 9], [1, 0, 1], 4, 2, 128, 128),
    ([5, 1, 129, 1000], [5, 1, 100, 3], 3, 1, 256, 256),
    ([40, 0, 0, 7], [33, 0, 0, 7], 5, 5, 64, 16),
    ([70000, 3], [65, 3], 32, 8, 128, 64),
    ([1 << 20, (1 << 30) - 1], [3, 2], 2, 1, 128, 128),
    ([77], [77], 7, 3, 256, 64),
    ([12], [12], 3, 2, 128, 0),
    ([8, 9], [2, 2], 16, 1, 64, 48),
    ([2] * 70, [1] * 70, 40, 8, 128, 128),
    ([1 + i % 5 for i in range(4200)], [(i % 7) % (1 + i % 5) for i in range(4200)], 1, 1, 64, 32),
    ([3001], [3001], 24, 8, 128, 128),
    ([2100, 300], [2100, 300], 9, 4, 256, 256),
    ([9000], [9000], 12, 4, 64, 64),
]


@pytest.mark.parametrize("type,out", [(0, 0), (1, 1), (2, 2), (0, 1), (0, 2)])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("lens,news,H,Hkv,Dh,R", CASES)
def test_values(qg, lens, news, H, Hkv, Dh, R, neighbours, type, out):
    progress("rope %s H %d Hkv %d Dh %d R %d %s type %d to %d" % (lens[:5], H, Hkv, Dh, R, neighbours, type, out))
    n = sum(news)
    qkv = sh.normal(7, (n, H + 2 * Hkv, Dh), TYPES[type])
    q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    wq, wk = (1 + 0.3 * sh.normal(8 + i, (Dh,), torch.float32) for i in range(2))
    yq, yk, st = call(qg, q, k, lens, news, R, neighbours, out, wq=wq, wk=wk)
    freq = freqs(R) if R else torch.zeros(0, device="cuda")
    check(yq, q, wq, lens, news, freq, 1e-6, neighbours)
    check(yk, k, wk, lens, news, freq, 1e-6, neighbours)
    assert int(st) == 0


@pytest.mark.parametrize("neighbours", [False, True])
def test_angles(qg, neighbours):
    """Every eighth of a turn and what lies next to it, angles of many turns, negative and zero frequencies, at far
    positions; heads of one channel that is not zero show sine and cosine by themselves."""
    progress("rope angles")
    f = [0.0, math.pi / 4, -math.pi / 4, math.pi / 2, math.pi, 3 * math.pi / 4, -1.5 * math.pi, 2 * math.pi, 1.9999999, 1e-9,
         -1e-30, 1e-42, 0.7853981, 0.78539824, 1.0, 0.5]
    freq = torch.tensor(f + [-x for x in f], dtype=torch.float32, device="cuda")
    lens, news = [1, 2, 9, 1000, 123456, (1 << 30) - 1], [1, 2, 8, 5, 5, 5]
    x = torch.zeros(sum(news), 64, 64, device="cuda")
    x[:, torch.arange(64), torch.arange(64)] = 1.0
    yq, yk, st = call(qg, x, x[:, :1], lens, news, 64, neighbours, 0, freq=freq)
    check(yq, x, None, lens, news, freq, 1e-6, neighbours)
    assert int(st) == 0


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("spread", [0.0, 1e-38, 1e-20, 1e-4, 200.0, 1e10, 1e19, 2.0**66, 8e36])
@pytest.mark.parametrize("eps", [2.0**-100, 1e-6, 2.0**100])
def test_magnitudes(qg, type, spread, eps):
    """Squares that vanish and squares beyond fp32; a zero head gives zeros."""
    if type == 1 and spread > 200:
        spread = 16000.0
    progress("rope spread %g eps %g type %d" % (spread, eps, type))
    x = sh.normal(3, (5, 6, 128), TYPES[0], 1.0)
    x = (x.clamp(-4, 4) * spread).to(TYPES[type])
    x[:, 1] = 0
    x[0, 2, 1:] = 0
    x[1, 3, ::3] *= 2.0**-20
    yq, yk, st = call(qg, x, x[:, 2:4], [5], [5], 128, False, type, eps=eps)
    check(yq, x, None, [5], [5], freqs(128), float(np.float32(eps)), False)
    check(yk, x[:, 2:4], None, [5], [5], freqs(128), float(np.float32(eps)), False)
    assert not yq[:, 1].any() and int(st) == 0


def test_weights_of_one_side_only(qg):
    q, k = sh.normal(1, (9, 4, 64), torch.bfloat16), sh.normal(2, (9, 2, 64), torch.bfloat16)
    w = sh.normal(3, (64,), torch.float32)
    for wq, wk in ((w, None), (None, w)):
        yq, yk, _ = call(qg, q, k, [9], [9], 64, True, 2, wq=wq, wk=wk)
        check(yq, q, wq, [9], [9], freqs(64), 1e-6, True)
        check(yk, k, wk, [9], [9], freqs(64), 1e-6, True)


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("neighbours", [False, True])
def test_in_place_rows_apart_and_tokens_of_no_sequence(qg, type, neighbours):
    """In the rows of a fused projection: the values and what lies beside the heads stay; rows of no sequence may be NaN."""
    progress("rope in place type %d" % type)
    lens, news, first, H, Hkv, Dh = [40, 3, 200], [40, 3, 17], 3, 6, 2, 128
    n = first + sum(news) + 2
    qkv = sh.normal(4, (n, H + 2 * Hkv, Dh), TYPES[type])
    qkv[:first] = math.nan
    qkv[-2:] = math.nan
    before, (q, k) = qkv.clone(), (qkv[:, :H], qkv[:, H:H + Hkv])
    apart = [torch.full((n, h * Dh + 16), 77.0, dtype=TYPES[type], device="cuda") for h in (H, Hkv)]
    into = [x[:, 8:-8].unflatten(1, (-1, Dh)) for x in apart]
    yq, yk, st = call(qg, q, k, lens, news, 96, neighbours, type, first=first, into=into)
    check(yq, q, None, lens, news, freqs(96), 1e-6, neighbours, first=first)
    check(yk, k, None, lens, news, freqs(96), 1e-6, neighbours, first=first)
    for x in apart:
        assert bool((x[:, :8] == 77.0).all()) and bool((x[:, -8:] == 77.0).all())
    assert torch.equal(qkv.nan_to_num(9.0), before.nan_to_num(9.0)) and int(st) == 0
    call(qg, q, k, lens, news, 96, neighbours, type, first=first, into=(q, k))
    want = before.clone()
    want[first:-2, :H], want[first:-2, H:H + Hkv] = yq[first:-2], yk[first:-2]
    assert torch.equal(qkv.nan_to_num(9.0), want.nan_to_num(9.0))


def test_infinities_and_nan_stay_in_their_head(qg):
    x = sh.normal(5, (3, 4, 64), torch.float32)
    want, _, _ = call(qg, x, x[:, :1], [3], [3], 64, False, 0)
    x[1, 2, 5], x[2, 0, 9] = math.inf, math.nan
    got, _, _ = call(qg, x, x[:, :1], [3], [3], 64, False, 0)
    assert bool(got[2, 0].isnan().all()) and bool(got[1, 2, 5].isnan()) and bool(got[1, 2, 37].isnan())
    rest = torch.ones(3, 4, dtype=torch.bool, device="cuda")
    rest[1, 2] = rest[2, 0] = False
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("type", [0, 1, 2])
def test_channels_that_do_not_turn_are_by_themselves(qg, type, neighbours):
    """y_c = u_c there: an infinity makes its own channel NaN (Inf * 0) and the others of its head 0, and a weight that is
    none its own channel only."""
    progress("rope apart type %d" % type)
    for Dh, R in ((64, 16), (128, 0), (128, 96), (256, 64)):
        for c in (R, R + 1, Dh - 9, Dh - 1):
            x = sh.normal(6, (2, 3, Dh), TYPES[type])
            x[1, 1, c] = math.inf
            got, _, _ = call(qg, x, x[:, :1], [2], [2], R, neighbours, type)
            want = torch.zeros(Dh, device="cuda")
            want[c] = math.nan
            assert torch.equal(got[1, 1].float().nan_to_num(9.0), want.nan_to_num(9.0)), (Dh, R, c)
            x = sh.normal(6, (2, 3, Dh), TYPES[type])
            w = torch.ones(Dh, device="cuda")
            plain, _, _ = call(qg, x, x[:, :1], [2], [2], R, neighbours, type, wq=w)
            w[c] = math.nan
            got, _, _ = call(qg, x, x[:, :1], [2], [2], R, neighbours, type, wq=w)
            assert bool(got[..., c].isnan().all())
            plain[..., c] = got[..., c] = 0
            assert torch.equal(got, plain), (Dh, R, c)


def test_data_errors(qg):
    """The faulty sequence is left out and reported, the others are computed."""
    progress("rope data errors")
    lens, news = [20, 37, 18], [20, 30, 18]
    q, k = sh.normal(1, (68, 4, 64), torch.float32), sh.normal(2, (68, 2, 64), torch.float32)
    for bad in (29, -1, 1 << 30, (1 << 31) - 1, -(1 << 31)):
        yq, yk, st = call(qg, q, k, [20, bad, 18], news, 64, False, 0)
        assert int(st) == qg.DEV_BAD_LENGTH
        check(yq, q, None, lens, news, freqs(64), 1e-6, False, skip=(1,))
        check(yk, k, None, lens, news, freqs(64), 1e-6, False, skip=(1,))
    cu = torch.tensor([0, 20, 69, 68], dtype=torch.int32, device="cuda")  # past the tokens, then backwards
    yq, yk, st = call(qg, q, k, lens, news, 64, False, 0, cu=cu)
    assert int(st) == qg.DEV_BAD_LENGTH
    check(yq, q, None, lens, news, freqs(64), 1e-6, False, skip=(1, 2))


def test_far_rows(qg):
    """Rows whose bytes begin past 32-bit offsets."""
    progress("rope far rows")
    n, ld = 300, 1 << 23
    wide = torch.empty(n, ld, dtype=torch.float16, device="cuda")  # 4.7 GiB
    q, k = wide[:, :256].unflatten(1, (4, 64)), wide[:, 512:640].unflatten(1, (2, 64))
    q.copy_(sh.normal(1, (n, 4, 64), torch.float16))
    k.copy_(sh.normal(2, (n, 2, 64), torch.float16))
    yq, yk, _ = call(qg, q, k, [n], [n], 64, False, 1)
    check(yq, q, None, [n], [n], freqs(64), 1e-6, False)
    check(yk, k, None, [n], [n], freqs(64), 1e-6, False)
    call(qg, q, k, [n], [n], 64, False, 1, into=(q, k))
    assert torch.equal(q, yq) and torch.equal(k, yk)


def test_captured_and_on_another_stream(qg):
    progress("rope graph")
    q, k = sh.normal(1, (6, 8, 128), torch.float32), sh.normal(2, (6, 2, 128), torch.float32)
    cu, lens = ah.cumulative([1] * 6), torch.tensor([3, 9, 1, 77, 1000, 5], dtype=torch.int32, device="cuda")
    freq = freqs(128)
    yq, yk, st = torch.empty_like(q), torch.empty_like(k), sh.status()

    def go(q_out, k_out, **more):
        qg.qk_norm_rope(0, q, 1024, k, 256, 6, cu, lens, 6, 8, 2, 128, None, None, 1e-5, 128, qg.ROPE_HALVES, freq, 0, q_out,
                        1024, k_out, 256, st, **more)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(yq, yk)
    for rep in range(3):
        lens.add_(1 + rep)
        q.copy_(sh.normal(10 + rep, q.shape, torch.float32))
        graph.replay()
        eq, ek = torch.empty_like(q), torch.empty_like(k)
        go(eq, ek)
        torch.cuda.synchronize()
        assert torch.equal(eq, yq) and torch.equal(ek, yk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    go(oq, ok, stream=s)
    s.synchronize()
    assert torch.equal(oq, yq) and torch.equal(ok, yk) and int(st) == 0
