"""Attention with a window and first positions that stay visible (attn_decode_kv4_sinks, attn_prefill_sinks), against the
formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

from tests import attn_helpers as ah
from tests import sinks_helpers as sh
from tests.gpu_util import progress

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


def decode(qg, c, q, type, Tq, H, scale, window, sinks, max_len=None, lens=None, cache=None, stream=None, ldq=None):
    B, max_len = len(c.lens), max_len or max(max(c.lens), 1)
    y = torch.full((B * Tq, H, c.Dh), 77.0, device="cuda")
    nb = qg.attn_decode_sinks_workspace_bytes(B, Tq, H, c.Hkv, c.Dh, max_len, window, sinks)
    ws, st = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda"), sh.status()
    qg.attn_decode_kv4_sinks(type, q, ldq or H * c.Dh, c.lens_device() if lens is None else lens, B, Tq, H, c.Hkv, c.Dh,
                             scale, window, sinks, max_len, *(cache or c.device()), y, ws, nb, st, stream=stream)
    return y, st


def hide(c, Tq, window, sinks):
    """What no query sees: whole pages leave the table, the rest of the others holds NaN scales.  Returns the masks."""
    masks, page, Dh, Hkv = {}, c.page, c.Dh, c.Hkv
    for b, n in enumerate(c.lens):
        seen = sh.sees(n - Tq + torch.arange(Tq), n, window, sinks).any(0).numpy()
        masks[b] = torch.from_numpy(~seen).cuda()
        for p in range(-(-n // page)):
            here = seen[p * page:(p + 1) * page]
            if not here.any():
                c.table[b, p] = -1
                continue
            pos = p * page + np.nonzero(~here)[0]
            for which in (0, 1):
                c.put(b, which, np.full((len(pos), Hkv, Dh), 15, np.uint8), np.full((len(pos), Hkv, Dh // 32), 255, np.uint8), pos)
    return masks


DECODE_CASES = [
    # lens, Tq, G, Hkv, Dh, page, window, sinks
    ([1], 1, 1, 1, 64, 16, 1, 1),
    ([0, 1, 2, 3, 4, 5, 6, 17, 20, 21], 1, 4, 2, 128, 16, 1, 4),
    ([15, 16, 17, 31, 32, 33, 34, 47, 48, 49, 50], 1, 2, 2, 128, 16, 16, 16),     # begins next to the sinks
    ([18, 33, 36, 52, 65, 80, 100], 1, 3, 1, 64, 16, 17, 1),
    ([200, 36, 37, 38, 51, 52, 53], 1, 4, 2, 256, 32, 20, 17),
    ([700, 33, 2, 129], 3, 4, 2, 64, 64, 33, 5),
    ([1, 2, 3, 40, 530], 4, 3, 2, 128, 16, 9, 4),                                 # queries before the first position
    ([300, 20], 16, 1, 2, 64, 16, 3, 31),
    ([1500, 1499, 64], 5, 2, 1, 256, 256, 100, 300),                              # sinks inside one page, window in others
    ([5000, 900, 640], 1, 4, 1, 128, 16, 700, 650),                               # several chunks, one across the gap
    ([5000, 4097], 1, 8, 2, 256, 64, 2000, 1000),
    ([20011, 9000], 2, 2, 1, 64, 64, 5000, 4100),
    ([20011], 1, 17, 1, 128, 128, 257, 2049),                                     # more sinks than window
    ([9001], 1, 4, 1, 128, 32, 8000, 1000),                                       # one position is hidden
    ([9001], 1, 4, 1, 128, 32, 8000, 1001),                                       # none is
    ([4000, 77], 1, 40, 2, 128, 64, 1024, 4),
]


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("lens,Tq,G,Hkv,Dh,page,window,sinks", DECODE_CASES)
def test_decode(qg, lens, Tq, G, Hkv, Dh, page, window, sinks, type):
    progress("sinks decode %s Tq %d G %d Hkv %d Dh %d page %d window %d sinks %d type %d" % (
        lens[:5], Tq, G, Hkv, Dh, page, window, sinks, type))
    c = ah.Cache(lens, Hkv, Dh, page, 21).fill(22)
    hide(c, Tq, window, sinks)
    q = sh.normal(23, (len(lens) * Tq, G * Hkv, Dh), ah.TYPES[type])
    y, st = decode(qg, c, q, type, Tq, G * Hkv, 0.7 * Dh**-0.5, window, sinks)
    assert int(st) == 0
    sh.check_decode(y, q, c.k, c.v, lens, Tq, 0.7 * Dh**-0.5, window, sinks)


@pytest.mark.parametrize("Tq,Dh,window", [(1, 128, 700), (3, 64, 33), (2, 256, 0), (1, 128, 1 << 30)])
def test_without_sinks_or_window_as_the_plain_call(qg, Tq, Dh, window):
    """sinks = 0: bit for bit attn_decode_kv4; window = 0 and windows over everything: whatever the sinks are."""
    c = ah.Cache([3000, 17, 900], 2, Dh, 16, 31).fill(32)
    q = sh.normal(33, (3 * Tq, 8, Dh), torch.float32)
    nb = qg.attn_decode_workspace_bytes(3, Tq, 8, 2, Dh, 3000, window)
    ws, y, st = torch.empty(nb, dtype=torch.uint8, device="cuda"), torch.empty(3 * Tq, 8, Dh, device="cuda"), sh.status()
    qg.attn_decode_kv4(0, q, 8 * Dh, c.lens_device(), 3, Tq, 8, 2, Dh, 0.1, window, 3000, *c.device(), y, ws, nb, st)
    for sinks in (0,) if 0 < window < 3000 else (0, 5, 3000, (1 << 31) - 1):
        got, _ = decode(qg, c, q, 0, Tq, 8, 0.1, window, sinks)
        assert torch.equal(got, y), sinks


def test_decode_is_the_same_alone_and_in_a_batch(qg):
    """Also where max_len says that nothing can be hidden, and where it does not."""
    lens = [3, 5000, 260, 1, 1024, 9000]
    c = ah.Cache(lens, 2, 128, 16, 41).fill(42)
    q = sh.normal(43, (6, 8, 128), torch.float32)
    y, _ = decode(qg, c, q, 0, 1, 8, 0.09, 900, 70)
    pages, mp, pg, np_, kv = c.device()
    for b, n in enumerate(lens):
        one = ah.Cache([n], 2, 128, 16, 0)
        for most in (n, 16 * c.max_pages):
            alone, _ = decode(qg, one, q[b:b + 1].contiguous(), 0, 1, 8, 0.09, 900, 70, max_len=most,
                              cache=(pages[b:b + 1].contiguous(), mp, pg, np_, kv))
            assert torch.equal(alone[0], y[b]), (b, n, most)


@pytest.mark.parametrize("scale", [0.0, -0.05, 8.0])
def test_decode_scales_and_rows_apart(qg, scale):
    c = ah.Cache([450, 33], 2, 128, 16, 31).fill(32)
    q = sh.normal(33, (2, 8, 128), torch.bfloat16)
    wide = ah.rows_with_gap(q, 8)
    y, _ = decode(qg, c, wide, 2, 1, 8, scale, 100, 7, ldq=wide.stride(0))
    sh.check_decode(y, q, c.k, c.v, c.lens, 1, scale, 100, 7)


def test_decode_data_errors(qg):
    """A length out of range gives zeros; bad pages, of the sinks or the window, are left out; all are reported."""
    lens = [300, 70, 1200]
    c = ah.Cache(lens, 2, 128, 16, 61).fill(62)
    q = sh.normal(63, (3, 8, 128), torch.float32)
    good, _ = decode(qg, c, q, 0, 1, 8, 0.09, 100, 40)
    for bad in (-1, 1201, 1 << 30, -(1 << 31)):
        y, st = decode(qg, c, q, 0, 1, 8, 0.09, 100, 40, lens=torch.tensor([300, bad, 1200], dtype=torch.int32, device="cuda"))
        assert int(st) == qg.DEV_BAD_LENGTH and not y[1].any() and torch.equal(y[[0, 2]], good[[0, 2]])
    for bad in (-1, c.num_pages, 1 << 30):
        cache = c.device()
        cache[0][0, 1] = cache[0][0, 13] = bad  # positions 16..31 and 208..223
        cache[0][2, :] = bad  # nothing left to see
        y, st = decode(qg, c, q, 0, 1, 8, 0.09, 100, 40, cache=cache)
        assert int(st) == qg.DEV_BAD_PAGE and not y[2].any() and torch.equal(y[1], good[1])
        gone = torch.zeros(300, dtype=torch.bool, device="cuda")
        gone[16:32] = gone[208:224] = True
        sh.check_decode(y, q, c.k, c.v, lens, 1, 0.09, 100, 40,
                        {0: gone, 2: torch.ones(1200, dtype=torch.bool, device="cuda")})


def test_decode_captured_twice_on_one_workspace(qg):
    """Two graphs of a growing sequence that share a workspace, replayed in turn, against eager calls."""
    progress("sinks decode graphs")
    c = ah.Cache([3000, 17, 0, 900], 2, 128, 64, 71).fill(72)
    cache, lens, st = c.device(), c.lens_device(), sh.status()
    lens.sub_(torch.tensor([12, 12, 0, 12], dtype=torch.int32, device="cuda"))
    nb = qg.attn_decode_sinks_workspace_bytes(4, 1, 8, 2, 128, 3000, 1500, 130)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    qs = [sh.normal(73 + i, (4, 8, 128), torch.float32) for i in range(2)]
    ys = [torch.empty(4, 8, 128, device="cuda") for _ in range(2)]

    def call(i):
        qg.attn_decode_kv4_sinks(0, qs[i], 1024, lens, 4, 1, 8, 2, 128, 0.1, 1500, 130, 3000, *cache, ys[i], ws, nb, st)

    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for rep in range(3):
        lens.add_(torch.tensor([4, 4, 0, 4], dtype=torch.int32, device="cuda"))
        for i in range(2):
            qs[i].copy_(sh.normal(100 + 10 * rep + i, (4, 8, 128), torch.float32))
            graphs[i].replay()
        torch.cuda.synchronize()
        got = [y.clone() for y in ys]
        now = lens.tolist()
        for i in range(2):
            call(i)
            assert torch.equal(ys[i], got[i]), (rep, i)
            sh.check_decode(got[i], qs[i], [k[:n] for k, n in zip(c.k, now)], [v[:n] for v, n in zip(c.v, now)], now, 1, 0.1,
                            1500, 130)
    assert int(st) == 0


def test_decode_on_another_stream(qg):
    c = ah.Cache([700, 17], 2, 128, 64, 81).fill(82)
    q = sh.normal(83, (2, 8, 128), torch.float16)
    want, _ = decode(qg, c, q, 1, 1, 8, 0.1, 90, 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, _ = decode(qg, c, q, 1, 1, 8, 0.1, 90, 3, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


# ---- prompts ---------------------------------------------------------------------------------------------------

def prefill(qg, q, k, v, lq, lk, type, H, Hkv, Dh, scale, window, sinks, first=(0, 0), stream=None):
    y = torch.full((q.shape[0], H, Dh), 77.0, dtype=q.dtype, device="cuda")
    st = sh.status()
    qg.attn_prefill_sinks(type, q, q.stride(0), k, k.stride(0), v, v.stride(0), q.shape[0], k.shape[0],
                          ah.cumulative(lq, first[0]), ah.cumulative(lk, first[1]), len(lq), H, Hkv, Dh, scale, window,
                          sinks, y, st, stream=stream)
    return y, st


def check_prefill(y, q, k, v, lq, lk, scale, window, sinks, first=(0, 0)):
    at, kat = first
    assert bool((y[:at] == 77.0).all())
    for b, (n, m) in enumerate(zip(lq, lk)):
        seen = sh.sees(m - n + torch.arange(n, device="cuda"), m, window, sinks)
        kk, vv = k[kat:kat + m].double(), v[kat:kat + m].double()
        vv = torch.where(seen.any(0)[:, None, None], vv, 0.0) if n else vv
        ref, a, big = sh.attend(q[at:at + n].double(), kk, vv, scale, seen)
        err = (y[at:at + n].double() - ref).abs()
        vm = float(vv.abs().max()) if n and m else 0.0
        lim = ah.prefill_tolerance(ref, a, big, vm, m, q.shape[2], q.dtype)
        assert bool((err <= lim).all()), "sequence %d (%d of %d): %.3g of the tolerance" % (
            b, n, m, float((err / lim.clamp(min=1e-300)).max()))
        at, kat = at + n, kat + m
    assert bool((y[at:] == 77.0).all())


PREFILL_CASES = [
    # queries, keys, G, Hkv, Dh, window, sinks
    ([1], [1], 1, 1, 64, 1, 1),
    ([5, 1, 129], [5, 1, 129], 4, 2, 64, 2, 3),
    ([0, 17, 0, 31, 32, 33, 200], [0, 17, 5, 31, 32, 33, 200], 2, 2, 128, 16, 16),
    ([63, 64, 65, 127, 128, 333], [63, 64, 65, 127, 128, 333], 1, 3, 128, 64, 1),
    ([255, 257, 300], [255, 257, 300], 3, 1, 256, 33, 40),
    ([1, 7, 100], [1000, 333, 100], 4, 1, 128, 50, 4),          # the last chunk of longer prompts
    ([40, 200, 9], [3, 64, 0], 2, 1, 64, 7, 2),                 # queries before the first key: empty rows
    ([700], [700], 8, 1, 64, 128, 128),
    ([515, 64], [1030, 64], 5, 2, 128, 300, 70),
    ([300, 70], [300, 70], 2, 2, 64, 1, 300),                   # all keys are sinks
    ([300, 70, 9], [310, 70, 400], 2, 1, 128, 65, 129),         # more than a tile of sinks
    ([260], [520], 1, 2, 256, 130, 31),
    ([1500], [1500], 2, 1, 128, 200, 64),
    ([130, 257, 5], [700, 257, 5], 8, 8, 128, 90, 5),
    ([300, 129, 40], [300, 129, 3], 8, 8, 256, 60, 60),
    ([300, 0, 129, 1, 64], [300, 7, 129, 1, 200], 8, 8, 64, 40, 65),
    ([2000], [3000], 4, 8, 64, 700, 100),
    ([1800], [2500], 4, 8, 128, 400, 200),
    ([(11 * i) % 150 for i in range(70)], [(11 * i) % 150 for i in range(70)], 2, 2, 128, 20, 3),
    ([0] * 64 + [3] + [0] * 100 + [140], [9] * 64 + [5] + [0] * 100 + [200], 8, 4, 64, 17, 6),
]


@pytest.mark.parametrize("type", [1, 2])
@pytest.mark.parametrize("lq,lk,G,Hkv,Dh,window,sinks", PREFILL_CASES)
def test_prefill(qg, lq, lk, G, Hkv, Dh, window, sinks, type):
    progress("sinks prefill %s of %s G %d Hkv %d Dh %d window %d sinks %d type %d" % (
        lq[:5], lk[:5], G, Hkv, Dh, window, sinks, type))
    H, dt = G * Hkv, ah.TYPES[type]
    q = sh.normal(1, (3 + sum(lq) + 2, H, Dh), dt)
    kv = sh.normal(2, (5 + sum(lk) + 1, 2 * Hkv, Dh), dt)
    at = 5  # rows that no query sees, between the sinks and the first window too, hold NaN
    kv[:5] = kv[-1:] = math.nan
    for n, m in zip(lq, lk):
        gone = ~sh.sees(m - n + torch.arange(n, device="cuda"), m, window, sinks).any(0) if n else torch.ones(m, dtype=torch.bool, device="cuda")
        kv[at:at + m][gone] = math.nan
        at += m
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    y, st = prefill(qg, q, k, v, lq, lk, type, H, Hkv, Dh, 0.7 * Dh**-0.5, window, sinks, (3, 5))
    assert int(st) == 0
    check_prefill(y, q, k, v, lq, lk, 0.7 * Dh**-0.5, window, sinks, (3, 5))


@pytest.mark.parametrize("window", [0, 40, 5000])
def test_prefill_without_sinks_or_window_as_the_plain_call(qg, window):
    q, k, v = (sh.normal(i, (400, 4, 64), torch.float16) for i in range(3))
    cu, st, y = ah.cumulative([300, 100]), sh.status(), torch.empty_like(q)
    qg.attn_prefill(1, q, 256, k, 256, v, 256, 400, 400, cu, cu, 2, 4, 4, 64, 0.1, window, y, st)
    for sinks in (0,) if window == 40 else (0, 7, (1 << 31) - 1):
        got, _ = prefill(qg, q, k, v, [300, 100], [300, 100], 1, 4, 4, 64, 0.1, window, sinks)
        assert torch.equal(got, y)


@pytest.mark.parametrize("scale", [0.0, -0.05, 8.0])
def test_prefill_scales(qg, scale):
    q, k, v = (sh.normal(i, (333, 4, 128), torch.bfloat16) for i in range(3))
    y, _ = prefill(qg, q, k, v, [333], [333], 2, 4, 4, 128, scale, 50, 9)
    check_prefill(y, q, k, v, [333], [333], scale, 50, 9)


def test_prefill_data_errors(qg):
    q, k, v = (sh.normal(i, (200, 2, 64), torch.bfloat16) for i in range(3))
    cu, bad = ah.cumulative([100, 60, 40]), torch.tensor([0, 100, 201, 200], dtype=torch.int32, device="cuda")
    want, _ = prefill(qg, q, k, v, [100, 60, 40], [100, 60, 40], 2, 2, 2, 64, 0.1, 20, 4)
    y, st = torch.full_like(q, 77.0), sh.status()
    qg.attn_prefill_sinks(2, q, 128, k, 128, v, 128, 200, 200, cu, bad, 3, 2, 2, 64, 0.1, 20, 4, y, st)
    assert int(st) == qg.DEV_BAD_LENGTH and torch.equal(y[:100], want[:100]) and bool((y[100:160] == 77.0).all())


def test_prefill_captured_and_on_another_stream(qg):
    q, k, v = (sh.normal(i, (333, 4, 128), torch.bfloat16) for i in range(3))
    cu, st = ah.cumulative([300, 33]), sh.status()
    y = torch.empty_like(q)

    def go(out, **more):
        qg.attn_prefill_sinks(2, q, 512, k, 512, v, 512, 333, 333, cu, cu, 2, 4, 4, 128, 0.1, 60, 5, out, st, **more)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(y)
    for rep in range(3):
        q.copy_(sh.normal(20 + rep, q.shape, q.dtype))
        graph.replay()
        eager = torch.empty_like(q)
        go(eager)
        torch.cuda.synchronize()
        assert torch.equal(eager, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(q)
    go(other, stream=s)
    s.synchronize()
    assert torch.equal(other, y) and int(st) == 0
