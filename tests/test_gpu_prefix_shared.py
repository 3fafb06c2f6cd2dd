"""attn_decode_kv4_prefix where workgroups take the rows of many sequences against the shared positions: enough rows and
positions that the call does not let each sequence walk the prefix by itself, which every test here makes sure of."""
import functools

import numpy as np
import pytest
import torch

from tests import attn_helpers as ah
from tests import sinks_helpers as sh
from tests.gpu_util import progress
from tests.test_gpu_prefix import Shared, decode

pytestmark = pytest.mark.gpu

CASES = [
    # prefix, sequences, Tq, G, Hkv, Dh, page; rows of a workgroup
    (2501, 150, 1, 1, 1, 64, 16),    # 32
    (4099, 40, 1, 17, 3, 64, 64),    # 64
    (4099, 64, 2, 17, 3, 64, 32),    # 128
    (1499, 150, 1, 1, 1, 128, 16),   # 32
    (4099, 40, 1, 17, 2, 128, 64),   # 64
    (2501, 64, 2, 17, 3, 128, 128),  # 128
    (700, 150, 1, 17, 3, 128, 16),   # 32, one chunk
    (4099, 24, 1, 1, 2, 256, 64),    # 64, the least there
    (2501, 64, 2, 17, 3, 256, 256),  # 128
]
SMALL = CASES[3]


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


def lengths(prefix, B):
    """Sequences behind the prefix, at its end, inside it, of a few positions and of none."""
    lens = [prefix + 1 + 7 * i % 50 for i in range(B)]
    lens[1:7] = prefix, prefix - 5, 0, 100, prefix + 300, 3
    return lens


@functools.lru_cache(maxsize=1)
def cached(prefix, B, Hkv, Dh, page):
    return Shared(prefix, lengths(prefix, B), Hkv, Dh, page, 21)


def shared(qg, s, Tq, H, max_len):
    """Each sequence by itself would need the workspace of a plain call, over a tile more."""
    args = (len(s.lens), Tq, H, s.Hkv, s.Dh)
    nb = qg.attn_decode_prefix_workspace_bytes(*args, max_len, s.prefix)
    return nb > 256 and nb != qg.attn_decode_workspace_bytes(*args, max_len + 16, 0)


def run(qg, s, q, type, Tq, H, scale, max_len=None, **more):
    assert shared(qg, s, Tq, H, max_len or max(max(s.lens), s.prefix))
    return decode(qg, s, q, type, Tq, H, scale, max_len, **more)


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("prefix,B,Tq,G,Hkv,Dh,page", CASES)
def test_values(qg, prefix, B, Tq, G, Hkv, Dh, page, type):
    progress("shared prefix %d B %d Tq %d G %d Hkv %d Dh %d page %d type %d" % (prefix, B, Tq, G, Hkv, Dh, page, type))
    s = cached(prefix, B, Hkv, Dh, page)
    q = sh.normal(23, (B * Tq, G * Hkv, Dh), ah.TYPES[type])
    y, st = run(qg, s, q, type, Tq, G * Hkv, 0.7 * Dh**-0.5)
    assert int(st) == 0
    sh.check_decode(y, q, s.k, s.v, s.lens, Tq, 0.7 * Dh**-0.5, 0, 0, prefix=prefix)


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("lo,hi", [(100, 137), (100, 138), (7, 44), (199, 236), (30, 200)])
def test_scales_far_apart(qg, lo, hi, type):
    """Scales over 36 binades (all that fp16 operands hold) and over more, in one chunk, at the ends of the range too."""
    progress("shared prefix scales %d..%d type %d" % (lo, hi - 1, type))
    prefix, B, Tq, G, Hkv, Dh, page = SMALL
    s = Shared(prefix, lengths(prefix, B), Hkv, Dh, page, 91, lo, hi)
    q = sh.normal(93, (B, G, Dh), ah.TYPES[type], 2.0 ** (min(127 - (hi - 1), 0) if type else 127 - (hi - 1)))
    y, st = run(qg, s, q, type, 1, G, 0.5)
    assert int(st) == 0 and bool(y.isfinite().all())
    sh.check_decode(y, q, s.k, s.v, s.lens, 1, 0.5, 0, 0, prefix=prefix)


@pytest.mark.parametrize("scale", [0.0, -0.05, 8.0])
def test_scales_of_scores_and_queries_far_apart(qg, scale):
    """Elements of a row 2^-40 of its largest, or that and zeros: such rows do not fit two fp16 parts."""
    prefix, B, Tq, G, Hkv, Dh, page = SMALL
    s = cached(prefix, B, Hkv, Dh, page)
    for far in (False, True):
        q = sh.normal(33, (B, G, Dh), torch.float32)
        if far:
            q[::40, :, 5] *= 2.0**-40
            q[1] = 0
        y, _ = run(qg, s, q, 0, 1, G, scale)
        sh.check_decode(y, q, s.k, s.v, s.lens, 1, scale, 0, 0, prefix=prefix)


@pytest.mark.parametrize("type", [0, 1, 2])
def test_scores_of_any_size(qg, type):
    prefix, B, Tq, G, Hkv, Dh, page = SMALL
    s = cached(prefix, B, Hkv, Dh, page)
    q = sh.normal(43, (B, G, Dh), ah.TYPES[type])
    q[::3] *= 1e4 if type == 1 else 1e28
    q[1] = 0
    y, st = run(qg, s, q, type, 1, G, 1.0)
    assert int(st) == 0 and bool(y.isfinite().all())
    sh.check_decode(y, q, s.k, s.v, s.lens, 1, 1.0, 0, 0, prefix=prefix)


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("most", [5, 130, 701])
@pytest.mark.parametrize("prefix,B,Tq,G,Hkv,Dh,page", [CASES[0], SMALL, CASES[7]])
def test_places_that_nothing_sees_may_hold_anything(qg, prefix, B, Tq, G, Hkv, Dh, page, most, type):
    """All sequences end inside the prefix; behind the longest its places hold scales that are NaN or infinite."""
    progress("shared prefix unseen from %d Dh %d type %d" % (most, Dh, type))
    lens = [most - i % min(most, 90) for i in range(B)]
    s = Shared(prefix, lens, Hkv, Dh, page, 25)
    s.max_pages = -(-prefix // page)  # max_len is the prefix at least
    s.table = np.full((B, s.max_pages), -1, np.int32)
    over = np.arange(most, prefix)
    for which in (0, 1):
        s.c.put(0, which, np.full((len(over), Hkv, Dh), 15, np.uint8), np.full((len(over), Hkv, Dh // 32), 255, np.uint8), over)
    q = sh.normal(27, (B, G * Hkv, Dh), ah.TYPES[type])
    y, st = run(qg, s, q, type, 1, G * Hkv, 0.1)
    assert int(st) == 0
    sh.check_decode(y, q, s.k, s.v, lens, 1, 0.1, 0, 0, prefix=most)


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("prefix,most,Dh", [(300, 5, 128), (300, 130, 64), (2500, 701, 128), (700, 260, 256)])
def test_the_same_where_each_sequence_walks_by_itself(qg, prefix, most, Dh, type):
    progress("prefix unseen from %d Dh %d type %d" % (most, Dh, type))
    lens = [most, most - 1, 0, 3]
    s = Shared(prefix, lens, 2, Dh, 16, 35)
    s.max_pages = -(-prefix // 16)
    s.table = np.full((4, s.max_pages), -1, np.int32)
    over = np.arange(most, prefix)
    for which in (0, 1):
        s.c.put(0, which, np.full((len(over), 2, Dh), 15, np.uint8), np.full((len(over), 2, Dh // 32), 255, np.uint8), over)
    q = sh.normal(37, (4, 8, Dh), ah.TYPES[type])
    assert not shared(qg, s, 1, 8, prefix)
    y, st = decode(qg, s, q, type, 1, 8, 0.1)
    assert int(st) == 0
    sh.check_decode(y, q, s.k, s.v, lens, 1, 0.1, 0, 0, prefix=most)


def test_data_errors(qg):
    """A length out of range gives zeros; bad pages are left out, the prefix's for all; all are reported."""
    prefix, B, Tq, G, Hkv, Dh, page = SMALL
    s = cached(prefix, B, Hkv, Dh, page)
    q = sh.normal(73, (B, G, Dh), torch.float32)
    good, _ = run(qg, s, q, 0, 1, G, 0.1)
    rest = torch.ones(B, dtype=torch.bool, device="cuda")
    rest[9] = False
    for bad in (-1, max(s.lens) + 1, 1 << 30, -(1 << 31)):
        lens = torch.tensor(s.lens, dtype=torch.int32, device="cuda")
        lens[9] = bad
        y, st = run(qg, s, q, 0, 1, G, 0.1, lens=lens)
        assert int(st) == qg.DEV_BAD_LENGTH and not y[9].any() and torch.equal(y[rest], good[rest])
    for bad in (-1, s.c.num_pages, 1 << 30):
        for type in (0, 2):
            cache, qt = s.device(), q.to(ah.TYPES[type])
            cache[0][2] = cache[0][50] = bad  # positions 32..47 and 800..815 of all
            y, st = run(qg, s, qt, type, 1, G, 0.1, cache=cache)
            assert int(st) == qg.DEV_BAD_PAGE
            hidden = {b: torch.zeros(n, dtype=torch.bool, device="cuda") for b, n in enumerate(s.lens)}
            for gone in hidden.values():
                gone[32:48] = True
                gone[800:816] = True
            sh.check_decode(y, qt, s.k, s.v, s.lens, 1, 0.1, 0, 0, hidden, prefix)
    cache = s.device()
    cache[0][:] = -1
    cache[1][:] = -1
    y, st = run(qg, s, q, 0, 1, G, 0.1, cache=cache)
    assert int(st) == qg.DEV_BAD_PAGE and not y.any()


def test_captured_twice_on_one_workspace_on_another_stream_and_with_longer_max_len(qg):
    progress("shared prefix graphs")
    prefix, B, Tq, G, Hkv, Dh, page = SMALL
    s = cached(prefix, B, Hkv, Dh, page)
    qs = [sh.normal(63 + i, (B, G, Dh), torch.float32) for i in range(2)]
    want = [run(qg, s, q, 0, 1, G, 0.1)[0] for q in qs]
    most = s.max_pages * page
    assert all(torch.equal(run(qg, s, q, 0, 1, G, 0.1, max_len=most)[0], w) for q, w in zip(qs, want))
    cache, lens, st = s.device(), torch.tensor(s.lens, dtype=torch.int32, device="cuda"), sh.status()
    nb = qg.attn_decode_prefix_workspace_bytes(B, 1, G, Hkv, Dh, most, prefix)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    ys, now = [torch.empty(B, G, Dh, device="cuda") for _ in range(2)], torch.empty(B, G, Dh, device="cuda")

    def call(i, y, **more):
        qg.attn_decode_kv4_prefix(0, now if i is None else qs[i], G * Dh, lens, B, 1, G, Hkv, Dh, 0.1, most, prefix, *cache,
                                  y, ws, nb, st, **more)

    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, ys[i])
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(3):
        for i in range(2):
            ys[i].fill_(5.0)
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(ys, want))
        now.copy_(qs[1])
        out = torch.full_like(now, 7.0)
        side.wait_stream(torch.cuda.current_stream())
        call(None, out, stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(out, want[1]) and int(st) == 0
