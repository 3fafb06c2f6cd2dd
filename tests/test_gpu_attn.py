"""The FP4 key/value cache and attention over it and over prompts, against plain implementations in 64 bits
(attn_helpers).  Cache bytes and gathered values must be equal; attention is held to tolerances derived there."""
import math

import numpy as np
import pytest
import torch

import synth
from tests import attn_helpers as ah
from tests.gpu_util import assert_within_bound, dev, empty, host, progress, sentinel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def normal(seed, shape, dtype, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * spread).to(dtype)


# ---- the cache -------------------------------------------------------------------------------------------------

def append_case(qg, lens, news, Hkv, Dh, page, type, seed, spread=1.0, gap=0, first=0, behind=0):
    """Appends the last `news` positions of `lens`; every byte of the cache must be the reference's."""
    c = ah.Cache(lens, Hkv, Dh, page, seed)
    before = c.bytes.copy()
    n = first + sum(news) + behind
    k, v = (normal(seed + i, (n, Hkv, Dh), ah.TYPES[type], spread) for i in (1, 2))
    for x in (k, v):  # ties, the borders of the steps, zero blocks, signed zeros
        if n > first:
            x[first, 0, :8] = torch.tensor([6, 5, -5, 3.5, 2.5, -1.75, 0.25, -0.0], device="cuda").to(x.dtype)
            x[first, 0, 8:32] = 0.75
            x[first, -1, 32:64] = 0.0
    pages, mp, pg, np_, kv = c.device()
    k2, v2 = (ah.rows_with_gap(x, gap) if gap else x for x in (k, v))
    st = status()
    qg.kv4_append(type, k2, k2.stride(0), v2, v2.stride(0), n, ah.cumulative(news, first), c.lens_device(), len(lens),
                  Hkv, Dh, pages, mp, pg, np_, kv, st)
    for which, x in ((0, k), (1, v)):
        codes, scales = ah.quantize(x.double().cpu().numpy())
        at = first
        for b, m in enumerate(news):
            c.put(b, which, codes[at:at + m], scales[at:at + m], np.arange(lens[b] - m, lens[b]))
            at += m
    assert np.array_equal(host(kv), c.bytes) and int(st) == 0
    return c, before


APPEND_CASES = [
    # lens, new, Hkv, Dh, page
    ([1], [1], 1, 64, 16),
    ([5, 0, 33, 16, 17], [5, 0, 33, 16, 17], 2, 128, 16),
    ([5, 1, 33, 16, 18, 200], [1, 1, 1, 1, 1, 1], 8, 128, 32),
    ([7, 300, 64, 65], [3, 299, 0, 2], 3, 256, 64),
    ([1000], [999], 5, 64, 128),
    ([2] * 130, [1] * 130, 1, 64, 16),
    ([1 + i % 5 for i in range(4200)], [(i % 7) % (1 + i % 5) for i in range(4200)], 1, 64, 16),
    ([3000, 1700], [3000, 1700], 16, 64, 32),   # two pieces, and two groups, a wave
    ([9000], [9000], 8, 128, 64),
]


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("lens,news,Hkv,Dh,page", APPEND_CASES)
def test_append_bytes(qg, lens, news, Hkv, Dh, page, type):
    progress("append %s type %d" % ((lens[:6], Hkv, Dh, page), type))
    append_case(qg, lens, news, Hkv, Dh, page, type, 11 + Hkv)


@pytest.mark.parametrize("spread", [2.0**-135, 1e-30, 1e-6, 1e30, 5e37])
def test_append_magnitudes(qg, spread):
    """Blocks near the least scale (and below it, subnormal ones too) and near the largest of fp32."""
    progress("append spread %g" % spread)
    append_case(qg, [70, 3], [70, 3], 2, 64, 16, 0, 5, spread)


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("e", [-130, -119, -14, 0, 9, 126])
def test_append_borders(qg, type, e):
    """Every border between two codes, both signs, and its neighbours in the type on either side."""
    progress("append borders e %d type %d" % (e, type))
    dt = ah.TYPES[type]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.99, 0.0, 0.5, 1.0, 3.0], dtype=torch.float64)
    vals = (mids * 2.0 ** max(e, -149)).to(dt)
    up = torch.nextafter(vals.float(), torch.tensor(math.inf)) if type == 0 else (vals.view(torch.int16) + 1).view(dt)
    down = torch.nextafter(vals.float(), torch.tensor(0.0)) if type == 0 else (
        torch.where(vals.view(torch.int16) > 0, vals.view(torch.int16) - 1, vals.view(torch.int16)).view(dt))
    x = torch.cat([vals, up.to(dt), down.to(dt)])
    x = torch.cat([x, -x])
    x = x[torch.isfinite(x) & (x.double().abs() <= 6 * 2.0**e)]
    g = np.random.default_rng(1)
    rows = torch.zeros(48, 1, 64, dtype=dt)
    for r in range(48):
        rows[r, 0] = x[torch.from_numpy(g.integers(0, len(x), 64))]
        rows[r, 0, ::32] = torch.tensor(6 * 2.0**e).to(dt) if 6 * 2.0**e <= torch.finfo(dt).max else x.abs().max()
    c = ah.Cache([48], 1, 64, 16, 3)
    pages, mp, pg, np_, kv = c.device()
    k = rows.cuda()
    v = k.flip(0).contiguous()
    st = status()
    qg.kv4_append(type, k, 64, v, 64, 48, ah.cumulative([48]), c.lens_device(), 1, 1, 64, pages, mp, pg, np_, kv, st)
    for which, t in ((0, k), (1, v)):
        c.put(0, which, *ah.quantize(t.double().cpu().numpy()), np.arange(48))
    assert np.array_equal(host(kv), c.bytes) and int(st) == 0


def test_append_rows_apart_and_tokens_of_no_sequence(qg):
    progress("append with gaps")
    append_case(qg, [40, 9], [40, 7], 2, 128, 16, 2, 6, gap=8, first=3, behind=2)


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("lens,news,Hkv,Dh,page", APPEND_CASES)
def test_gather_values(qg, lens, news, Hkv, Dh, page, type):
    progress("gather %s type %d" % ((lens[:6], Hkv, Dh, page), type))
    c = ah.Cache(lens, Hkv, Dh, page, 3).fill(4, 110, 135)
    n, w = 2 + sum(news) + 1, Hkv * Dh
    out = [torch.full((n, w + 16), 77.0, dtype=ah.TYPES[type], device="cuda") for _ in range(2)]
    k, v = (x[:, 8:8 + w].unflatten(1, (Hkv, Dh)) for x in out)
    st = status()
    qg.kv4_gather(type, k, w + 16, v, w + 16, n, ah.cumulative(news, 2), c.lens_device(), len(lens), Hkv, Dh,
                  *c.device(), st)
    for x, full, held in ((k, out[0], c.k), (v, out[1], c.v)):
        ref = torch.full((n, w + 16), 77.0, dtype=torch.float64)
        want = np.concatenate([held[b][lens[b] - m:] for b, m in enumerate(news)])
        ref[2:n - 1, 8:8 + w] = torch.from_numpy(want.reshape(-1, w))
        assert torch.equal(full.cpu(), ref.to(ah.TYPES[type]))
    assert int(st) == 0


def test_gather_float16_rounds_and_overflows_as_the_type(qg):
    c = ah.Cache([40], 1, 64, 16, 3).fill(9, 95, 160)
    k, v = (empty((40, 1, 64), torch.float16) for _ in range(2))
    qg.kv4_gather(1, k, 64, v, 64, 40, ah.cumulative([40]), c.lens_device(), 1, 1, 64, *c.device(), status())
    assert torch.equal(k.cpu(), torch.from_numpy(c.k[0]).half()) and torch.equal(v.cpu(), torch.from_numpy(c.v[0]).half())
    assert torch.isinf(k).any() and (k == 0).any()


@pytest.mark.parametrize("what", ["length", "more new than held", "offsets", "page low", "page high"])
def test_cache_data_errors(qg, what):
    """The faulty sequence (or page) is left out and reported; the others are written."""
    progress("cache data error: " + what)
    Hkv, Dh, page, lens = 2, 64, 16, [20, 37, 18]
    c = ah.Cache(lens, Hkv, Dh, page, 8).fill(1)
    pages, mp, pg, np_, kv = c.device()
    given, cu = list(lens), [0, 20, 57, 75]
    skip = {1: range(37)}
    code = qg.DEV_BAD_LENGTH
    if what == "length":
        given[1] = mp * page + 1
    elif what == "more new than held":
        given[1] = 36
    elif what == "offsets":
        cu = [0, 20, 76, 75]  # the second ends past the tokens, the third runs backwards
        skip = {1: range(37), 2: range(18)}
    else:
        pages[1, 1] = -1 if what == "page low" else np_
        skip, code = {1: range(16, 32)}, qg.DEV_BAD_PAGE
    lens_d = torch.tensor(given, dtype=torch.int32, device="cuda")
    cu_d = torch.tensor(cu, dtype=torch.int32, device="cuda")
    k, v = (torch.full((75, Hkv, Dh), 9.0, device="cuda") for _ in range(2))
    st = status()
    qg.kv4_gather(0, k, Hkv * Dh, v, Hkv * Dh, 75, cu_d, lens_d, 3, Hkv, Dh, pages, mp, pg, np_, kv, st)
    assert int(st) == code
    for x, held in ((k, c.k), (v, c.v)):
        want = np.concatenate(held)
        for b, gone in skip.items():
            want[[sum(lens[:b]) + j for j in gone]] = 9.0
        assert np.array_equal(host(x), want.astype(np.float32))
    st = status()
    before = host(kv).copy()
    k, v = (normal(i, (75, Hkv, Dh), torch.float32) for i in (1, 2))
    qg.kv4_append(0, k, Hkv * Dh, v, Hkv * Dh, 75, cu_d, lens_d, 3, Hkv, Dh, pages, mp, pg, np_, kv, st)
    assert int(st) == code
    for which, x in ((0, k), (1, v)):
        codes, scales = ah.quantize(x.double().cpu().numpy())
        for b, n in enumerate(lens):
            pos = np.array([j for j in range(n) if j not in skip.get(b, ())], dtype=np.int64)
            c.put(b, which, codes[sum(lens[:b]) + pos], scales[sum(lens[:b]) + pos], pos)
    assert np.array_equal(host(kv), c.bytes) and not np.array_equal(before, c.bytes)


# ---- attention of new tokens over the cache --------------------------------------------------------------------

def decode(qg, c, q, type, Tq, H, scale, window, max_len=None, stream=None, ldq=None, lens=None, cache=None, y=None):
    B, Dh = len(c.lens), c.Dh
    max_len = max_len or max(max(c.lens), 1)
    y = sentinel((B * Tq, H, Dh), torch.float32, 77.0) if y is None else y
    nb = qg.attn_decode_workspace_bytes(B, Tq, H, c.Hkv, Dh, max_len, window)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    st = status()
    qg.attn_decode_kv4(type, q, ldq or H * Dh, c.lens_device() if lens is None else lens, B, Tq, H, c.Hkv, Dh, scale,
                       window, max_len, *(cache or c.device()), y, ws, nb, st, stream=stream)
    return y, st


def check_decode(y, c, q, Tq, scale, window, hidden=None):
    for b, n in enumerate(c.lens):
        k, v = (torch.from_numpy(x[b]).cuda() for x in (c.k, c.v))
        ref, a, big = ah.attend(q[b * Tq:(b + 1) * Tq].double(), k, v, scale, window,
                                None if hidden is None or b not in hidden else hidden[b])
        err = (y[b * Tq:(b + 1) * Tq].double() - ref).abs()
        lim = ah.decode_tolerance(a, big, n, c.Dh)
        assert bool((err <= lim).all()), "sequence %d (%d positions): %.3g of the tolerance" % (
            b, n, float((err / lim).max()))


DECODE_CASES = [
    # lens, Tq, G, Hkv, Dh, page, window
    ([1], 1, 1, 1, 64, 16, 0),
    ([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65], 1, 4, 2, 128, 16, 0),
    ([127, 128, 129, 255, 256, 257, 500], 1, 5, 3, 64, 32, 0),
    ([300, 0, 1023, 1025], 1, 8, 2, 256, 64, 0),
    ([2047, 2049, 7], 1, 16, 1, 128, 128, 0),
    ([1, 2, 3, 40, 530], 4, 3, 2, 128, 16, 0),       # queries before the first position
    ([5, 77, 300], 16, 1, 2, 64, 16, 0),
    ([600, 18], 3, 17, 1, 64, 64, 0),                # rows past two tiles of 16
    ([90, 260], 1, 40, 2, 128, 32, 0),
    ([700, 33, 2, 129], 1, 4, 2, 128, 16, 1),        # the window is the query's own key
    ([700, 33, 2, 129], 2, 4, 2, 64, 16, 33),
    ([1500, 1499, 64], 5, 2, 1, 256, 256, 100),
    ([9001, 8191], 1, 4, 1, 128, 64, 0),
    ([20011], 2, 2, 1, 64, 64, 5000),
]


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("lens,Tq,G,Hkv,Dh,page,window", DECODE_CASES)
def test_decode(qg, lens, Tq, G, Hkv, Dh, page, window, type):
    progress("decode %s Tq %d G %d Hkv %d Dh %d page %d window %d type %d" % (lens, Tq, G, Hkv, Dh, page, window, type))
    c = ah.Cache(lens, Hkv, Dh, page, 21).fill(22)
    H = G * Hkv
    q = normal(23, (len(lens) * Tq, H, Dh), ah.TYPES[type])
    scale = 0.7 * Dh**-0.5
    y, st = decode(qg, c, q, type, Tq, H, scale, window)
    assert int(st) == 0
    check_decode(y, c, q, Tq, scale, window)


@pytest.mark.parametrize("Dh,n", [(64, 1280), (128, 640), (256, 320)])
def test_decode_one_chunk_and_several(qg, Dh, n):
    """Lengths on both sides of the longest single chunk, in one call; each alone gives the same bits."""
    progress("decode one chunk Dh %d" % Dh)
    lens = [n - 1, n, n + 1, 2 * n]
    c = ah.Cache(lens, 2, Dh, 64, 81).fill(82)
    q = normal(83, (4, 8, Dh), torch.float32)
    y, st = decode(qg, c, q, 0, 1, 8, 0.1, 0)
    assert int(st) == 0
    check_decode(y, c, q, 1, 0.1, 0)
    for b in range(4):
        pages, kv = c.device()[0], c.device()[4]
        nb = qg.attn_decode_workspace_bytes(1, 1, 8, 2, Dh, lens[b], 0)
        ws, one, st = torch.empty(nb, dtype=torch.uint8, device="cuda"), torch.empty_like(y[:1]), status()
        qg.attn_decode_kv4(0, q[b], 8 * Dh, c.lens_device()[b:b + 1], 1, 1, 8, 2, Dh, 0.1, 0, lens[b], pages[b:b + 1],
                           c.max_pages, 64, c.num_pages, kv, one, ws, nb, st)
        assert int(st) == 0 and torch.equal(one, y[b:b + 1])


@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 1, 450, 449])
def test_decode_windows_as_long_as_the_sequence(qg, window):
    c = ah.Cache([450, 0, 3], 1, 64, 16, 31).fill(32)
    q = normal(33, (3 * 16, 2, 64), torch.float32)
    y, _ = decode(qg, c, q, 0, 16, 2, 0.1, window)
    check_decode(y, c, q, 16, 0.1, window)


@pytest.mark.parametrize("scale", [0.0, -0.05, 8.0])
def test_decode_scales(qg, scale):
    """Equal weights, the order turned round, and scores of thousands (one key takes all)."""
    progress("decode scale %g" % scale)
    c = ah.Cache([450, 33], 2, 128, 16, 31).fill(32)
    q = normal(33, (2, 8, 128), torch.float32)
    y, _ = decode(qg, c, q, 0, 1, 8, scale, 0)
    check_decode(y, c, q, 1, scale, 0)


@pytest.mark.parametrize("lo,hi,spread", [(7, 9, 1.0), (60, 66, 2.0**60), (185, 190, 2.0**-62)])
def test_decode_far_scales(qg, lo, hi, spread):
    """Caches of tiny and huge values: exponents far outside 16-bit floating point."""
    progress("decode cache scales %d..%d" % (lo, hi))
    c = ah.Cache([300, 40], 1, 64, 16, 31).fill(32, lo, hi)
    q = normal(33, (2, 4, 64), torch.float32, spread)
    y, _ = decode(qg, c, q, 0, 1, 4, 0.1, 0)
    check_decode(y, c, q, 1, 0.1, 0)


def test_decode_is_the_same_alone_and_in_a_batch(qg):
    """A sequence's result does not depend on its batch, on max_len's slack or on the run."""
    progress("decode batch invariance")
    lens = [3, 5000, 260, 1, 1024, 9000]
    c = ah.Cache(lens, 2, 128, 16, 41).fill(42)
    q = normal(43, (6, 8, 128), torch.float32)
    y, _ = decode(qg, c, q, 0, 1, 8, 0.09, 0)
    again, _ = decode(qg, c, q, 0, 1, 8, 0.09, 0, max_len=c.max_pages * 16)
    assert torch.equal(y, again)
    pages, mp, pg, np_, kv = c.device()
    for b, n in enumerate(lens):
        one = ah.Cache([n], 2, 128, 16, 0)
        alone, _ = decode(qg, one, q[b:b + 1].contiguous(), 0, 1, 8, 0.09, 0, max_len=max(n, 700),
                          cache=(pages[b:b + 1].contiguous(), mp, pg, np_, kv))
        assert torch.equal(alone[0], y[b]), (b, n)


@pytest.mark.parametrize("Tq,Dh,window", [(1, 64, 100), (3, 128, 37), (2, 256, 1), (1, 128, 640)])
def test_decode_what_lies_before_every_window(qg, Tq, Dh, window):
    """Positions that no query sees any more: their pages are gone from the table, and in the first page that is still
    needed they may hold anything."""
    progress("decode before the window %d Dh %d" % (window, Dh))
    c = ah.Cache([777, 130, 2000, 33], 2, Dh, 32, 71).fill(72)
    q = normal(73, (4 * Tq, 6, Dh), torch.float32)
    first = [max(n - Tq - window + 1, 0) for n in c.lens]
    hidden = {}
    for b, at in enumerate(first):
        gone = torch.arange(c.lens[b], device="cuda") < at
        hidden[b] = gone
        for pos in range(at // 32 * 32, at):
            for which in (0, 1):
                ah.write(c.bytes, 32, 2, Dh, c.table[b, pos // 32], pos % 32, which, np.full((2, Dh), 15, np.uint8),
                         np.full((2, Dh // 32), 255, np.uint8))
        c.table[b, :at // 32] = -1
    y, st = decode(qg, c, q, 0, Tq, 6, 0.1, window)
    assert int(st) == 0
    check_decode(y, c, q, Tq, 0.1, window, hidden)


def test_decode_rows_apart(qg):
    c = ah.Cache([100, 7], 2, 64, 16, 51).fill(52)
    q = normal(53, (2, 4, 64), torch.bfloat16)
    wide = ah.rows_with_gap(q, 8)
    y, _ = decode(qg, c, wide, 2, 1, 4, 0.1, 0, ldq=wide.stride(0))
    assert torch.equal(y, decode(qg, c, q, 2, 1, 4, 0.1, 0)[0])


def test_decode_data_errors(qg):
    """Lengths out of range give zeros, a bad page is left out of the softmax, both are reported."""
    progress("decode data errors")
    lens = [100, 70, 50, 1200]
    c = ah.Cache(lens, 2, 128, 16, 61).fill(62)
    q = normal(63, (4, 8, 128), torch.float32)
    good, _ = decode(qg, c, q, 0, 1, 8, 0.09, 0)
    for bad in (-1, 1201, 1 << 30, -(1 << 31)):
        given = torch.tensor([100, bad, 50, 1200], dtype=torch.int32, device="cuda")
        y, st = decode(qg, c, q, 0, 1, 8, 0.09, 0, lens=given)
        assert int(st) == qg.DEV_BAD_LENGTH
        assert not y[1].any() and torch.equal(y[[0, 2, 3]], good[[0, 2, 3]])
    for bad in (-1, c.num_pages, 1 << 30, -(1 << 31)):
        cache = c.device()
        cache[0][0, 2] = bad
        cache[0][2, :] = bad  # nothing left to see
        cache[0][3, 40:44] = bad
        y, st = decode(qg, c, q, 0, 1, 8, 0.09, 0, cache=cache)
        assert int(st) == qg.DEV_BAD_PAGE and not y[2].any()
        hidden = {0: torch.zeros(100, dtype=torch.bool, device="cuda"),
                  2: torch.ones(50, dtype=torch.bool, device="cuda"),
                  3: torch.zeros(1200, dtype=torch.bool, device="cuda")}
        hidden[0][32:48] = True
        hidden[3][640:704] = True
        check_decode(y, c, q, 1, 0.09, 0, hidden)


def test_decode_captured_twice_on_one_workspace(qg):
    """Two graphs that share a workspace, replayed in turn with other work between, against the eager calls."""
    progress("decode graphs")
    c = ah.Cache([3000, 17, 0, 900], 2, 128, 64, 71).fill(72)
    cache, lens = c.device(), c.lens_device()
    nb = qg.attn_decode_workspace_bytes(4, 1, 8, 2, 128, 4000, 0)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    st = status()
    qs = [normal(73 + i, (4, 8, 128), torch.float32) for i in range(2)]
    ys = [sentinel((4, 8, 128), torch.float32, 5.0) for _ in range(2)]

    def call(i):
        qg.attn_decode_kv4(0, qs[i], 1024, lens, 4, 1, 8, 2, 128, 0.1, 0, 3000, *cache, ys[i], ws, nb, st)

    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for rep in range(3):
        for i in range(2):
            qs[i].copy_(normal(100 + 10 * rep + i, (4, 8, 128), torch.float32))
        for i in (0, 1):
            graphs[i].replay()
        torch.cuda.synchronize()
        got = [y.clone() for y in ys]
        for i in range(2):
            ys[i].fill_(3.0)
            call(i)
            assert torch.equal(ys[i], got[i]), (rep, i)
            check_decode(got[i], c, qs[i], 1, 0.1, 0)


def test_decode_on_another_stream(qg):
    c = ah.Cache([700, 17], 2, 128, 64, 81).fill(82)
    q = normal(83, (2, 8, 128), torch.float16)
    want, _ = decode(qg, c, q, 1, 1, 8, 0.1, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, _ = decode(qg, c, q, 1, 1, 8, 0.1, 0)
    y2, _ = decode(qg, c, q, 1, 1, 8, 0.1, 0, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(y2, want)


def test_far_offsets(qg):
    """A cache of more than 4 GiB: pages whose bytes begin past 32-bit offsets are written, read and attended to."""
    progress("far offsets")
    Hkv, Dh, page, lens = 2, 128, 256, [700, 300]
    each = ah.page_bytes(page, Hkv, Dh)
    num = (1 << 32) // each + 400
    kv = torch.zeros(num, each, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[num - 1, 5, num - 300], [num - 301, 9, 0]], dtype=torch.int32, device="cuda")
    cache = (table, 3, page, num, kv)
    k, v = (normal(90 + i, (1000, Hkv, Dh), torch.bfloat16) for i in range(2))
    cu, lens_d, st = ah.cumulative(lens), torch.tensor(lens, dtype=torch.int32, device="cuda"), status()
    qg.kv4_append(2, k, 256, v, 256, 1000, cu, lens_d, 2, Hkv, Dh, *cache, st)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    qg.kv4_gather(2, k2, 256, v2, 256, 1000, cu, lens_d, 2, Hkv, Dh, *cache, st)
    c = ah.Cache(lens, Hkv, Dh, page, 1)
    c.k, c.v = [], []
    for x, x2, out in ((k, k2, c.k), (v, v2, c.v)):
        want = ah.values(*ah.quantize(x.double().cpu().numpy()))
        assert np.array_equal(x2.double().cpu().numpy(), want)
        out += [want[:700], want[700:]]
    q = normal(95, (2, 4, Dh), torch.float32)
    y, st2 = decode(qg, c, q, 0, 1, 4, 0.1, 0, cache=cache)
    check_decode(y, c, q, 1, 0.1, 0)
    assert int(st) == 0 and int(st2) == 0


def test_far_rows(qg):
    """Rows of k, v and q whose bytes begin past 32-bit offsets."""
    progress("far rows")
    n, Hkv, Dh, ld = 300, 2, 64, 1 << 23
    wide = torch.empty(n, ld, dtype=torch.float16, device="cuda")  # 4.7 GiB
    k, v, q = (wide[:, i * 512:i * 512 + 128].unflatten(1, (2, 64)) for i in range(3))
    for i, x in enumerate((k, v, q)):
        x.copy_(normal(30 + i, (n, Hkv, Dh), torch.float16))
    c = ah.Cache([n], Hkv, Dh, 64, 33)
    cache, cu, lens, st = c.device(), ah.cumulative([n]), c.lens_device(), status()
    qg.kv4_append(1, k, ld, v, ld, n, cu, lens, 1, Hkv, Dh, *cache, st)
    c.k, c.v = ([ah.values(*ah.quantize(x.double().cpu().numpy()))] for x in (k, v))
    y, st2 = decode(qg, c, q[n - 3:], 1, 3, Hkv, 0.1, 0, ldq=ld, cache=cache)
    check_decode(y, c, q[n - 3:].contiguous(), 3, 0.1, 0)
    y, st3 = prefill(qg, q, k, v, [n], [n], 1, Hkv, Hkv, Dh, 0.1, 0)
    check_prefill(y, q.contiguous(), k.contiguous(), v.contiguous(), [n], [n], 0.1, 0)
    qg.kv4_gather(1, k, ld, v, ld, n, cu, lens, 1, Hkv, Dh, *cache, st)
    assert np.array_equal(k.double().cpu().numpy(), c.k[0]) and np.array_equal(v.double().cpu().numpy(), c.v[0])
    assert int(st) == int(st2) == int(st3) == 0


def test_steps_captured_as_one_graph(qg):
    """Lengths that grow on the device, the new tokens into the cache and attention over it, captured once: every replay
    is the next step, and gives what eager calls give."""
    progress("captured steps")
    B, H, Hkv, Dh, page, mp, steps = 3, 8, 2, 128, 16, 8, 6
    start = [0, 14, 61]
    w, i32 = Hkv * Dh, dict(dtype=torch.int32, device="cuda")
    pages = torch.randperm(B * mp, generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda().view(B, mp)
    cu, st = ah.cumulative([1] * B), status()
    new = [[normal(200 + 3 * s + i, (B, h, Dh), torch.bfloat16) for i, h in enumerate((H, Hkv, Hkv))] for s in range(steps)]
    q, k, v = (torch.empty_like(x) for x in new[0])
    nb = qg.attn_decode_workspace_bytes(B, 1, H, Hkv, Dh, mp * page, 0)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def state():
        return (torch.tensor(start, **i32), torch.zeros(B * mp, ah.page_bytes(page, Hkv, Dh), dtype=torch.uint8, device="cuda"),
                torch.empty(B, H, Dh, device="cuda"))

    def step(lens, kv, y):
        lens.add_(1)
        qg.kv4_append(2, k, w, v, w, B, cu, lens, B, Hkv, Dh, pages, mp, page, B * mp, kv, st)
        qg.attn_decode_kv4(2, q, H * Dh, lens, B, 1, H, Hkv, Dh, 0.1, 0, mp * page, pages, mp, page, B * mp, kv, y, ws, nb, st)

    eager, captured = state(), state()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(*captured)
    for s in range(steps):
        for x, given in zip((q, k, v), new[s]):
            x.copy_(given)
        graph.replay()
        step(*eager)
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b), s
    assert int(st) == 0 and eager[0].tolist() == [n + steps for n in start]


# ---- attention of packed prompts -------------------------------------------------------------------------------

def prefill(qg, q, k, v, lq, lk, type, H, Hkv, Dh, scale, window, first=(0, 0), stream=None):
    y = torch.full((q.shape[0], H, Dh), 77.0, dtype=q.dtype, device="cuda")
    st = status()
    qg.attn_prefill(type, q, q.stride(0), k, k.stride(0), v, v.stride(0), q.shape[0], k.shape[0],
                    ah.cumulative(lq, first[0]), ah.cumulative(lk, first[1]), len(lq), H, Hkv, Dh, scale, window, y, st,
                    stream=stream)
    return y, st


def check_prefill(y, q, k, v, lq, lk, scale, window, first=(0, 0)):
    at, kat = first
    assert bool((y[:at] == 77.0).all())
    for b, (n, m) in enumerate(zip(lq, lk)):
        kk, vv = k[kat:kat + m].double(), v[kat:kat + m].double()
        ref, a, big = ah.attend(q[at:at + n].double(), kk, vv, scale, window)
        err = (y[at:at + n].double() - ref).abs()
        vm = float(vv.abs().max()) if m else 0.0
        lim = ah.prefill_tolerance(ref, a, big, vm, m, q.shape[2], q.dtype)
        assert bool((err <= lim).all()), "sequence %d (%d of %d): %.3g of the tolerance" % (
            b, n, m, float((err / lim.clamp(min=1e-300)).max()))
        at, kat = at + n, kat + m
    assert bool((y[at:] == 77.0).all())


PREFILL_CASES = [
    # queries, keys, G, Hkv, Dh, window
    ([1], [1], 1, 1, 64, 0),
    ([5, 1, 129], [5, 1, 129], 4, 2, 64, 0),
    ([0, 17, 0, 31, 32, 33], [0, 17, 5, 31, 32, 33], 2, 2, 128, 0),
    ([63, 64, 65, 127, 128], [63, 64, 65, 127, 128], 1, 3, 128, 0),
    ([255, 257, 300], [255, 257, 300], 3, 1, 256, 0),
    ([1, 7, 100], [1000, 333, 100], 4, 1, 128, 0),          # the last chunk of longer prompts
    ([40, 200, 9], [3, 64, 0], 2, 1, 64, 0),                # queries before the first key: empty rows
    ([700], [700], 8, 1, 64, 0),
    ([515, 64], [1030, 64], 5, 2, 128, 0),
    ([300, 70], [300, 70], 2, 2, 64, 1),
    ([300, 70, 9], [310, 70, 400], 2, 1, 128, 65),
    ([260], [520], 1, 2, 256, 130),
    ([1500], [1500], 2, 1, 128, 0),
    # enough tiles for one wave per 32 queries, and for two (the cases above: four)
    ([300, 0, 129, 1, 64], [300, 7, 129, 1, 200], 8, 8, 64, 0),
    ([300, 0, 129, 1, 64], [300, 7, 129, 1, 200], 4, 16, 128, 0),
    ([130, 257, 5], [700, 257, 5], 8, 8, 128, 90),
    ([300, 129, 40], [300, 129, 3], 8, 8, 256, 0),
    ([511], [900], 4, 8, 64, 0),
    ([500], [500], 4, 8, 128, 0),
    ([64, 500], [128, 530], 2, 8, 128, 200),
    ([330], [331], 4, 8, 256, 0),
    # 64 sequences and more: the two ways to find a tile
    ([(7 * i) % 40 for i in range(64)], [(7 * i) % 40 + i % 3 for i in range(64)], 2, 1, 64, 0),
    ([(11 * i) % 150 for i in range(70)], [(11 * i) % 150 for i in range(70)], 2, 2, 128, 0),
    ([0] * 64 + [3] + [0] * 100 + [140], [9] * 64 + [5] + [0] * 100 + [200], 8, 4, 64, 17),
]


@pytest.mark.parametrize("type", [1, 2])
@pytest.mark.parametrize("lq,lk,G,Hkv,Dh,window", PREFILL_CASES)
def test_prefill(qg, lq, lk, G, Hkv, Dh, window, type):
    progress("prefill %s/%s G %d Hkv %d Dh %d window %d type %d" % (lq[:6], lk[:6], G, Hkv, Dh, window, type))
    H, dt = G * Hkv, ah.TYPES[type]
    q = normal(1, (max(1, sum(lq)), H, Dh), dt)
    k, v = (normal(i, (max(1, sum(lk)), Hkv, Dh), dt) for i in (2, 3))
    scale = Dh**-0.5
    y, st = prefill(qg, q, k, v, lq, lk, type, H, Hkv, Dh, scale, window)
    assert int(st) == 0
    check_prefill(y, q, k, v, lq, lk, scale, window)


@pytest.mark.parametrize("type", [1, 2])
@pytest.mark.parametrize("lq,lk,G,Hkv,Dh,window", [
    ([300, 0, 129, 1, 64], [300, 7, 129, 1, 200], 8, 16, 64, 0),
    ([300, 0, 129, 1, 64], [300, 7, 129, 1, 200], 8, 16, 128, 0),
    ([130, 257, 5, 290], [700, 257, 5, 300], 9, 15, 128, 90),
    ([310, 257, 128], [200, 300, 900], 9, 15, 64, 129),
    ([300, 129, 140], [300, 129, 3], 8, 8, 256, 0),
    ([127, 1, 385], [500, 1, 385], 5, 13, 256, 200),
    ([(11 * i) % 150 for i in range(70)], [(11 * i) % 150 for i in range(70)], 4, 4, 128, 0),
    ([(11 * i) % 150 for i in range(64)], [(13 * i) % 150 for i in range(64)], 4, 5, 64, 0),
])
def test_prefill_tiles_of_128_queries(qg, lq, lk, G, Hkv, Dh, window, type):
    """Heads and tokens enough for more than one round of full tiles."""
    test_prefill(qg, lq, lk, G, Hkv, Dh, window, type)


@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_prefill_parts_of_a_fused_projection(qg, Dh):
    """q, k and v as parts of one matrix whose other columns are NaN; packed rows that belong to no sequence are NaN in q, k and v
    and stay as they were in y."""
    progress("prefill strided Dh %d" % Dh)
    H, Hkv, lens = 4, 2, [37, 100, 1, 64]
    n = 3 + sum(lens) + 70
    wide = torch.full((n, (H + 2 * Hkv + 1) * Dh), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[3:3 + sum(lens), :(H + 2 * Hkv) * Dh] = normal(5, (sum(lens), (H + 2 * Hkv) * Dh), torch.bfloat16)
    q, k, v, _ = wide.unflatten(1, (-1, Dh)).split([H, Hkv, Hkv, 1], dim=1)
    y, st = prefill(qg, q, k, v, lens, lens, 2, H, Hkv, Dh, 0.1, 0, first=(3, 3))
    check_prefill(y, q, k, v, lens, lens, 0.1, 0, first=(3, 3))
    assert int(st) == 0


@pytest.mark.parametrize("scale,spread", [(0.0, 1.0), (-0.2, 1.0), (4.0, 1.0), (0.05, 50.0)])
def test_prefill_scales(qg, scale, spread):
    progress("prefill scale %g spread %g" % (scale, spread))
    lens = [333, 90]
    q, k, v = (normal(i, (423, 2, 128), torch.float16, spread) for i in (1, 2, 3))
    y, _ = prefill(qg, q, k, v, lens, lens, 1, 2, 2, 128, scale, 0)
    check_prefill(y, q, k, v, lens, lens, scale, 0)


@pytest.mark.parametrize("window", [(1 << 31) - 1, 200, 199])
def test_prefill_windows_as_long_as_the_sequence(qg, window):
    q, k, v = (normal(i, (203, 2, 64), torch.float16) for i in (1, 2, 3))
    y, _ = prefill(qg, q, k, v, [200, 3], [200, 3], 1, 2, 2, 64, 0.1, window)
    check_prefill(y, q, k, v, [200, 3], [200, 3], 0.1, window)


@pytest.mark.parametrize("lq,lk,H,window", [(5, 300, 2, 40), (200, 700, 16, 129), (1, 100, 1, 1), (700, 1000, 64, 77)])
def test_prefill_keys_that_no_query_sees(qg, lq, lk, H, window):
    """They come before the first query's window and may be NaN."""
    progress("prefill unseen keys %d %d window %d" % (lq, lk, window))
    q, k, v = (normal(i, (n, H, 128), torch.bfloat16) for i, n in ((1, lq), (2, lk), (3, lk)))
    k[:lk - lq - window + 1] = v[:lk - lq - window + 1] = math.nan
    y, st = prefill(qg, q, k, v, [lq], [lk], 2, H, H, 128, 0.1, window)
    assert int(st) == 0
    clean = [torch.nan_to_num(x) for x in (k, v)]
    check_prefill(y, q, *clean, [lq], [lk], 0.1, window)


@pytest.mark.parametrize("type", [1, 2])
@pytest.mark.parametrize("H", [1, 64, 256])
def test_prefill_many_small_weights(qg, H, type):
    """One key of score 0 and value 0, 4000 of score -17 (a weight of 2^-24.5, between 0 and the type's least in fp16) and
    value 1.  The rounding of the weights is the same for all 4000, at most half a step, and so is y's: eps / 2 each;
    fp32 sums of 4001 terms are off by less than 4001 * 2^-24 each, in numerator and denominator."""
    progress("prefill small weights H %d type %d" % (H, type))
    n, dt = 4001, ah.TYPES[type]
    q = torch.zeros(1, H, 64, dtype=dt, device="cuda")
    k, v = torch.zeros(n, 1, 64, dtype=dt, device="cuda"), torch.ones(n, 1, 64, dtype=dt, device="cuda")
    q[..., 0], k[1:, :, 0], v[0] = 4.0, -4.25, 0.0
    y, _ = prefill(qg, q, k, v, [1], [n], type, H, 1, 64, 1.0, 0)
    w = (n - 1) * math.exp(-17.0)
    ref = w / (1.0 + w)
    assert float((y.double() / ref - 1).abs().max()) <= torch.finfo(dt).eps * 1.01 + 2 * n * 2.0**-24


def test_prefill_rising_scores(qg):
    """Every later key outweighs all before it by far: the running maximum moves at every step."""
    progress("prefill rising scores")
    n = 600
    q = torch.ones(n, 1, 64, device="cuda").bfloat16()
    k = (torch.arange(n, device="cuda").float()[:, None, None] * torch.ones(1, 1, 64, device="cuda")).bfloat16()
    v = normal(3, (n, 1, 64), torch.bfloat16)
    for kk in (k, k.flip(0).contiguous()):
        y, _ = prefill(qg, q, kk, v, [n], [n], 2, 1, 1, 64, 0.5, 0)
        check_prefill(y, q, kk, v, [n], [n], 0.5, 0)


def test_prefill_largest_sum_of_queries(qg):
    """Many heads and tokens at once: every tile of a launch of thousands of workgroups is found and written."""
    progress("prefill many tiles")
    lens = [1000, 1, 3, 2500, 128, 127, 700]
    n = sum(lens)
    q, k, v = (normal(i, (n, h, 64), torch.bfloat16) for i, h in ((1, 24), (2, 3), (3, 3)))
    y, st = prefill(qg, q, k, v, lens, lens, 2, 24, 3, 64, 0.125, 0)
    assert int(st) == 0
    check_prefill(y, q, k, v, lens, lens, 0.125, 0)


def test_prefill_data_errors(qg):
    """A sequence whose offsets make no sense is left out, reported, and the others are computed."""
    progress("prefill data errors")
    H, Hkv, Dh, lens = 2, 1, 64, [70, 40, 90]
    q, k, v = (normal(i, (200, h, Dh), torch.bfloat16) for i, h in ((1, H), (2, Hkv), (3, Hkv)))
    good, _ = prefill(qg, q, k, v, lens, lens, 2, H, Hkv, Dh, 0.1, 0)
    for which in (0, 1):
        for cu in ([0, 70, 110, 201], [0, 70, 110, 1 << 30], [0, 70, 110, -5], [-3, 70, 110, 200], [0, 70, 60, 200]):
            off = [[0, 70, 110, 200], [0, 70, 110, 200]]
            off[which] = cu
            bad = {b for b in range(3) if cu[b] < 0 or cu[b + 1] < cu[b] or cu[b + 1] > 200}
            y = torch.full((200, H, Dh), 77.0, dtype=torch.bfloat16, device="cuda")
            st = status()
            dc = [torch.tensor(o, dtype=torch.int32, device="cuda") for o in off]
            qg.attn_prefill(2, q, H * Dh, k, Dh, v, Dh, 200, 200, dc[0], dc[1], 3, H, Hkv, Dh, 0.1, 0, y, st)
            assert int(st) == qg.DEV_BAD_LENGTH, cu
            if cu[2] < cu[1]:  # rows of two sequences at once: nothing is said of them
                continue
            for b in range(3):
                rows = slice(off[0][b], off[0][b + 1])
                if b in bad:
                    if which == 1:
                        assert bool((y[rows] == 77.0).all()), (cu, b)
                elif off[0][b:b + 2] == [0, 70, 110, 200][b:b + 2] and off[1][b:b + 2] == [0, 70, 110, 200][b:b + 2]:
                    assert torch.equal(y[rows], good[rows]), (cu, b)


def test_prefill_captured_and_on_another_stream(qg):
    progress("prefill graph")
    H, Hkv, Dh, lens = 4, 2, 128, [200, 77]
    q, k, v = (normal(i, (277, h, Dh), torch.bfloat16) for i, h in ((1, H), (2, Hkv), (3, Hkv)))
    cu, st = ah.cumulative(lens), status()
    y = torch.zeros(277, H, Dh, dtype=torch.bfloat16, device="cuda")

    def call(stream=None):
        qg.attn_prefill(2, q, H * Dh, k, Hkv * Dh, v, Hkv * Dh, 277, 277, cu, cu, 2, H, Hkv, Dh, 0.1, 0, y, st,
                        stream=stream)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(3):
        q.copy_(normal(50 + rep, (277, H, Dh), torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y.zero_()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        call(s)
        s.synchronize()
        assert torch.equal(y, got)
        check_prefill(y, q, k, v, lens, lens, 0.1, 0)


def test_binding_refuses_what_does_not_fit(qg):
    """Tensors too small for the sizes given, wrong strides and types are refused before any launch."""
    x = torch.zeros(8, 2, 64, device="cuda")
    h = x.half()
    i = torch.zeros(8, dtype=torch.int32, device="cuda")
    kv = torch.zeros(qg.kv4_page_bytes(16, 2, 64), dtype=torch.uint8, device="cuda")
    ok = dict(type=0, k=x, ldk=128, v=x, ldv=128, n=8, cu=i, lens=i, B=1, Hkv=2, Dh=64, pages=i, max_pages=1, page=16,
              num_pages=1, kv=kv, d_status=i)
    for bad, err in [(dict(n=9), ValueError), (dict(ldk=256), ValueError), (dict(k=h), TypeError),
                     (dict(B=8), ValueError), (dict(num_pages=2), ValueError), (dict(max_pages=9), ValueError),
                     (dict(lens=i.long()), TypeError), (dict(v=x.transpose(1, 2)), ValueError),
                     (dict(v=x[:, :, ::2], Hkv=1), ValueError), (dict(k=x[::2], n=4), ValueError),
                     (dict(n=0), qg.QGError), (dict(page=17), qg.QGError)]:
        with pytest.raises(err):
            qg.kv4_append(**{**ok, **bad})
    with pytest.raises(ValueError):
        qg.attn_prefill(1, h, 128, h, 128, h, 128, 8, 8, i, i, 1, 2, 2, 64, 0.1, 0, h[:7], i)
    with pytest.raises(ValueError):
        qg.attn_decode_kv4(0, x, 128, i, 8, 1, 2, 2, 64, 0.1, 0, 16, i, 1, 16, 1, kv, x[:4], kv, 256, i)
    torch.cuda.synchronize()


# ---- together --------------------------------------------------------------------------------------------------

def test_prompt_then_decode_through_the_projections(qg, orc):
    """A prompt in two chunks and three decode steps as a model runs them: q, k, v of a step from the Q8_0 mat-vec,
    append, attention, the activation quantizer and the grouped output projection.  Each stage is checked on the
    inputs that the stage before left."""
    progress("prompt, then decode steps")
    K, H, Hkv, Dh, page, G, N = 512, 16, 4, 64, 16, 4, 96
    B, lens = 2, [70, 33]
    g = synth.rng(7)
    W = synth.q8_0_weight(g, (H + 2 * Hkv) * Dh, K)
    Wo = np.concatenate([synth.q8_0_weight(g, N, H * Dh // G) for _ in range(G)])
    Wd, Wod = dev(W), dev(Wo)
    c = ah.Cache([n + 8 for n in lens], Hkv, Dh, page, 9)
    cache = c.device()
    scale = Dh**-0.5 * 0.02
    # first chunk: all but 20 tokens of each prompt go in, then the rest attends to what the cache gives back
    k, v = (normal(i, (sum(lens), Hkv, Dh), torch.bfloat16) for i in (1, 2))
    cu, st = ah.cumulative(lens), status()
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    args = (B, Hkv, Dh, *cache)
    qg.kv4_append(2, k, Hkv * Dh, v, Hkv * Dh, sum(lens), cu, lens_d, *args, st)
    kc, vc = torch.empty_like(k), torch.empty_like(v)
    qg.kv4_gather(2, kc, Hkv * Dh, vc, Hkv * Dh, sum(lens), cu, lens_d, *args, st)
    q = normal(3, (40, H, Dh), torch.bfloat16)
    y, st2 = prefill(qg, q, kc, vc, [20, 20], lens, 2, H, Hkv, Dh, scale, 0)
    check_prefill(y, q, kc, vc, [20, 20], lens, scale, 0)
    held = [[list(x[:70]), list(x[70:])] for x in (kc.double().cpu().numpy(), vc.double().cpu().numpy())]
    one = ah.cumulative([1, 1])
    nb = qg.attn_decode_workspace_bytes(B, 1, H, Hkv, Dh, 78, 0)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    for step in range(3):
        x = dev(synth.activations(g, B, K))
        qkv = empty((B, H + 2 * Hkv, Dh), torch.float32)
        qg.qgemv_q8_0_f32(Wd, (H + 2 * Hkv) * Dh, K, x, B, qkv)
        lens_d += 1
        qs, ks, vs = qkv.split([H, Hkv, Hkv], dim=1)
        ld = (H + 2 * Hkv) * Dh
        qg.kv4_append(0, ks, ld, vs, ld, B, one, lens_d, *args, st)
        y = empty((B, H, Dh), torch.float32)
        qg.attn_decode_kv4(0, qs, ld, lens_d, B, 1, H, Hkv, Dh, scale, 0, 78, *cache, y, ws, nb, st)
        for part, src in ((0, ks), (1, vs)):
            new = ah.values(*ah.quantize(src.double().cpu().numpy()))
            for b in range(B):
                held[part][b].append(new[b])
        c.k, c.v = ([np.stack(s) for s in held[p]] for p in (0, 1))
        c.lens = [len(s) for s in c.k]
        check_decode(y, c, qs, 1, scale, 0)
        qx, dx, sx = (empty((B, H * Dh), torch.int8), empty((B, H * Dh // 32), torch.float32),
                      empty((B, H * Dh // 32), torch.int32))
        qg.quantize_act_q8(y, B, H * Dh, qx, dx, sx)
        out = empty((B, G * N), torch.float32)
        qg.qgemv_grouped(0, Wod, G, N, H * Dh // G, qx, dx, sx, B, out)
        rq, rd, _ = orc.quantize_act_q8(host(y).reshape(B, -1))
        for j in range(G):
            w = H * Dh // G
            ref, bnd = orc.gemv(0, Wo[j * N:(j + 1) * N], N, w, np.ascontiguousarray(rq[:, j * w:(j + 1) * w]),
                                np.ascontiguousarray(rd[:, j * w // 32:(j + 1) * w // 32]))
            assert_within_bound(host(out)[:, j * N:(j + 1) * N], ref, bnd, what="output group %d" % j)
    assert int(st) == 0 and int(st2) == 0
