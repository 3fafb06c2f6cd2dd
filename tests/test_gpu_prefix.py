"""Decode over a prefix that the sequences of a batch share (attn_decode_kv4_prefix), against the formula in 64 bits."""
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


class Shared:
    """A prefix and sequences that go on from it.  Table entries that are not needed name no page; places of a sequence's
    first page that the prefix covers hold NaN scales."""

    def __init__(self, prefix, lens, Hkv, Dh, page, seed, lo=123, hi=128):
        self.prefix, self.lens, self.Hkv, self.Dh, self.page = prefix, list(lens), Hkv, Dh, page
        skip = prefix // page
        own = [n - skip * page if n > prefix else 0 for n in lens]
        self.c = c = ah.Cache([prefix] + own, Hkv, Dh, page, seed).fill(seed + 1, lo, hi)
        self.max_pages = max(-(-max(list(lens) + [1]) // page), 1) + 1
        self.table = np.full((len(lens), self.max_pages), -1, np.int32)
        self.k, self.v = [], []
        for b, n in enumerate(lens):
            m = -(-own[b] // page)
            self.table[b, skip:skip + m] = c.table[b + 1, :m]
            over = np.arange(min(prefix - skip * page, own[b]))
            for which, held, out in ((0, c.k, self.k), (1, c.v, self.v)):
                c.put(b + 1, which, np.full((len(over), Hkv, Dh), 15, np.uint8),
                      np.full((len(over), Hkv, Dh // 32), 255, np.uint8), over)
                out.append(np.concatenate([held[0], held[b + 1][len(over):]])[:max(n, 0)])
        self.prefix_pages = c.table[0, :-(-prefix // page)].copy()

    def device(self):
        return (torch.from_numpy(self.prefix_pages).cuda(), torch.from_numpy(self.table).cuda(), self.max_pages, self.page,
                self.c.num_pages, torch.from_numpy(self.c.bytes).cuda())


def decode(qg, s, q, type, Tq, H, scale, max_len=None, lens=None, cache=None, stream=None, ldq=None):
    B, max_len = len(s.lens), max_len or max(max(s.lens), s.prefix, 1)
    y = torch.full((B * Tq, H, s.Dh), 77.0, device="cuda")
    nb = qg.attn_decode_prefix_workspace_bytes(B, Tq, H, s.Hkv, s.Dh, max_len, s.prefix)
    ws, st = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda"), sh.status()
    lens = torch.tensor(s.lens, dtype=torch.int32, device="cuda") if lens is None else lens
    prefix_pages, *rest = cache or s.device()
    qg.attn_decode_kv4_prefix(type, q, ldq or H * s.Dh, lens, B, Tq, H, s.Hkv, s.Dh, scale, max_len, s.prefix, prefix_pages,
                              *rest, y, ws, nb, st, stream=stream)
    return y, st


CASES = [
    # prefix, lens, Tq, G, Hkv, Dh, page
    (1, [1], 1, 1, 1, 64, 16),
    (1, [2, 1, 0, 17], 1, 4, 2, 128, 16),
    (16, [17, 16, 15, 33, 0, 5], 1, 3, 2, 64, 16),          # sequences that end inside the prefix
    (17, [18, 40, 17, 33], 1, 8, 1, 256, 32),
    (300, [301, 350, 320, 431], 1, 4, 2, 128, 16),
    (300, [301, 350, 298, 0, 299, 3], 4, 2, 2, 128, 64),      # queries on both sides of the prefix's end
    (63, [64, 65, 70], 16, 1, 2, 64, 16),
    (640, [640 + i for i in range(33)], 1, 1, 3, 128, 128),
    (1000, [1000, 2900, 1001], 2, 5, 1, 128, 64),             # a tail of several chunks
    (4099, [4100 + 7 * i for i in range(20)], 1, 8, 2, 128, 64),
    (2500, [2600 + i for i in range(40)], 1, 16, 1, 256, 256),
    (3001, [3002 + i for i in range(70)], 3, 1, 2, 64, 32),
    (9000, [9100, 9001], 1, 17, 1, 128, 128),
    (5000, [5001], 1, 2, 2, 64, 16),
    (20000, [20050 + 3 * i for i in range(9)], 1, 4, 1, 256, 64),
    (33, [34 + i % 50 for i in range(300)], 1, 2, 1, 64, 16),
]


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("prefix,lens,Tq,G,Hkv,Dh,page", CASES)
def test_values(qg, prefix, lens, Tq, G, Hkv, Dh, page, type):
    progress("prefix %d lens %s Tq %d G %d Hkv %d Dh %d page %d type %d" % (prefix, lens[:5], Tq, G, Hkv, Dh, page, type))
    s = Shared(prefix, lens, Hkv, Dh, page, 21)
    q = sh.normal(23, (len(lens) * Tq, G * Hkv, Dh), ah.TYPES[type])
    y, st = decode(qg, s, q, type, Tq, G * Hkv, 0.7 * Dh**-0.5)
    assert int(st) == 0
    sh.check_decode(y, q, s.k, s.v, lens, Tq, 0.7 * Dh**-0.5, 0, 0, prefix=prefix)


@pytest.mark.parametrize("scale", [0.0, -0.05, 8.0])
def test_scales_and_rows_apart(qg, scale):
    s = Shared(450, [500, 451, 33], 2, 128, 16, 31)
    q = sh.normal(33, (3, 8, 128), torch.bfloat16)
    wide = ah.rows_with_gap(q, 8)
    y, _ = decode(qg, s, wide, 2, 1, 8, scale, ldq=wide.stride(0))
    sh.check_decode(y, q, s.k, s.v, s.lens, 1, scale, 0, 0, prefix=s.prefix)


@pytest.mark.parametrize("lo,hi,spread", [(7, 9, 1.0), (60, 66, 2.0**60), (185, 190, 2.0**-62)])
@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_far_scales(qg, lo, hi, spread, Dh):
    """Caches of tiny and huge values: exponents far outside 16-bit floating point."""
    s = Shared(300, [340, 301], 1, Dh, 16, 31, lo, hi)
    for type in (0, 2):
        q = sh.normal(33, (2, 20, Dh), ah.TYPES[type], spread)
        y, _ = decode(qg, s, q, type, 1, 20, 0.1)
        sh.check_decode(y, q, s.k, s.v, s.lens, 1, 0.1, 0, 0, prefix=s.prefix)


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("lo,hi", [(100, 137), (100, 138), (7, 44), (199, 236), (30, 200)])
def test_scales_far_apart(qg, lo, hi, type):
    """Scales over 36 binades (all that fp16 operands hold) and over more, in one chunk, at the ends of the range too."""
    progress("prefix scales %d..%d type %d" % (lo, hi - 1, type))
    s = Shared(260, [280, 261, 100], 1, 128, 16, 91, lo, hi)
    q = sh.normal(93, (3, 16, 128), ah.TYPES[type], 2.0 ** (min(127 - (hi - 1), 0) if type else 127 - (hi - 1)))
    y, st = decode(qg, s, q, type, 1, 16, 0.5)
    assert int(st) == 0 and bool(y.isfinite().all())
    sh.check_decode(y, q, s.k, s.v, s.lens, 1, 0.5, 0, 0, prefix=s.prefix)


def test_queries_far_apart(qg):
    """Elements of one fp32 row over 60 binades: the small ones count where the keys hide the large ones."""
    s = Shared(200, [210, 201], 1, 64, 16, 95)
    q = sh.normal(96, (2, 12, 64), torch.float32)
    q[:, :4, :32] *= 2.0**60
    q[:, 4:6, 5] *= 2.0**25
    q[:, 6, 9] = 0
    for keys in (s.c.k[0], s.c.k[1], s.c.k[2]):  # channels whose keys are all zero
        keys[..., :6] = 0
    for b, n in enumerate([200] + [m - 192 for m in s.lens]):
        codes = np.zeros((n, 1, 64), np.uint8)
        scales = np.full((n, 1, 2), 127, np.uint8)
        g = np.random.default_rng(b)
        codes[..., 6:] = g.integers(0, 16, (n, 1, 58))
        own = np.arange(n) if b == 0 else np.arange(8, n)
        s.c.put(b, 0, codes[own], scales[own], own)
        kv = ah.values(codes, scales)
        if b == 0:
            shared = kv
        else:
            s.k[b - 1] = np.concatenate([shared, kv[8:]])
    q[:, :4, 6:32] = 0  # what is left of the large ones meets zeros only
    y, _ = decode(qg, s, q, 0, 1, 12, 0.3)
    sh.check_decode(y, q, s.k, s.v, s.lens, 1, 0.3, 0, 0, prefix=200)


@pytest.mark.parametrize("type", [0, 1, 2])
def test_scores_of_any_size(qg, type):
    """Scores up to 1e30 of either sign beside small ones: each row's greatest key takes all, the rest nothing."""
    progress("prefix scores type %d" % type)
    s = Shared(700, [720, 705, 760], 2, 128, 16, 41)
    q = sh.normal(43, (3, 8, 128), ah.TYPES[type])
    q[:, ::3] *= 1e4 if type == 1 else 1e28
    q[1, 1] = 0
    y, st = decode(qg, s, q, type, 1, 8, 1.0)
    assert int(st) == 0 and bool(y.isfinite().all())
    sh.check_decode(y, q, s.k, s.v, s.lens, 1, 1.0, 0, 0, prefix=s.prefix)


def test_without_a_prefix_as_the_plain_call(qg):
    c = ah.Cache([3000, 17, 0], 2, 128, 16, 31).fill(32)
    q, st = sh.normal(33, (3, 8, 128), torch.float32), sh.status()
    nb = qg.attn_decode_workspace_bytes(3, 1, 8, 2, 128, 3000, 0)
    assert qg.attn_decode_prefix_workspace_bytes(3, 1, 8, 2, 128, 3000, 0) == nb
    ws, y, z = torch.empty(nb, dtype=torch.uint8, device="cuda"), torch.empty_like(q), torch.empty_like(q)
    qg.attn_decode_kv4(0, q, 1024, c.lens_device(), 3, 1, 8, 2, 128, 0.1, 0, 3000, *c.device(), y, ws, nb, st)
    qg.attn_decode_kv4_prefix(0, q, 1024, c.lens_device(), 3, 1, 8, 2, 128, 0.1, 3000, 0, None, *c.device(), z, ws, nb, st)
    assert torch.equal(y, z)


def test_same_as_tables_that_share_pages(qg):
    """The plain call over tables whose first blocks are the prefix's pages, within the two calls' tolerances."""
    s = Shared(640, [700, 641, 1300], 2, 128, 64, 51)
    q = sh.normal(53, (3, 8, 128), torch.float32)
    y, _ = decode(qg, s, q, 0, 1, 8, 0.1)
    table = s.table.copy()
    table[:, :10] = s.prefix_pages
    nb = qg.attn_decode_workspace_bytes(3, 1, 8, 2, 128, 1300, 0)
    ws, z, st = torch.empty(nb, dtype=torch.uint8, device="cuda"), torch.empty_like(q), sh.status()
    _, _, mp, page, num, kv = s.device()
    qg.attn_decode_kv4(0, q, 1024, torch.tensor(s.lens, dtype=torch.int32, device="cuda"), 3, 1, 8, 2, 128, 0.1, 0, 1300,
                       torch.from_numpy(table).cuda(), mp, page, num, kv, z, ws, nb, st)
    for out in (y, z):
        sh.check_decode(out, q, s.k, s.v, s.lens, 1, 0.1, 0, 0, prefix=s.prefix)


def test_runs_are_alike_and_max_len_has_no_effect(qg):
    s = Shared(2000, [2100, 2001, 3900, 7] * 5, 2, 128, 64, 61)
    q = sh.normal(63, (20, 8, 128), torch.float32)
    y, _ = decode(qg, s, q, 0, 1, 8, 0.1)
    for max_len in (None, s.max_pages * 64):
        assert torch.equal(decode(qg, s, q, 0, 1, 8, 0.1, max_len=max_len)[0], y)


def test_data_errors(qg):
    """A length out of range gives zeros; bad pages are left out, the prefix's for all; all are reported."""
    s = Shared(100, [150, 130, 300], 2, 128, 16, 71)
    q = sh.normal(73, (3, 8, 128), torch.float32)
    good, _ = decode(qg, s, q, 0, 1, 8, 0.1)
    for bad in (-1, 301, 1 << 30, -(1 << 31)):
        y, st = decode(qg, s, q, 0, 1, 8, 0.1, lens=torch.tensor([150, bad, 300], dtype=torch.int32, device="cuda"))
        assert int(st) == qg.DEV_BAD_LENGTH and not y[1].any() and torch.equal(y[[0, 2]], good[[0, 2]])
    for bad in (-1, s.c.num_pages, 1 << 30):
        cache = s.device()
        cache[0][2] = bad      # positions 32..47 of all
        cache[1][2, 10] = bad  # positions 160..175 of the last
        y, st = decode(qg, s, q, 0, 1, 8, 0.1, cache=cache)
        assert int(st) == qg.DEV_BAD_PAGE
        hidden = {b: torch.zeros(n, dtype=torch.bool, device="cuda") for b, n in enumerate(s.lens)}
        for b in range(3):
            hidden[b][32:48] = True
        hidden[2][160:176] = True
        sh.check_decode(y, q, s.k, s.v, s.lens, 1, 0.1, 0, 0, hidden, s.prefix)
    cache = s.device()
    cache[0][:] = -1
    cache[1][:] = -1
    y, st = decode(qg, s, q, 0, 1, 8, 0.1, cache=cache)
    assert int(st) == qg.DEV_BAD_PAGE and not y.any()


def test_captured_twice_on_one_workspace_and_on_another_stream(qg):
    progress("prefix graphs")
    s = Shared(900, [1000, 960, 930, 5], 2, 128, 64, 81)
    cache, lens, st = s.device(), torch.tensor([988, 948, 918, 5], dtype=torch.int32, device="cuda"), sh.status()
    nb = qg.attn_decode_prefix_workspace_bytes(4, 1, 8, 2, 128, 1000, 900)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    qs = [sh.normal(83 + i, (4, 8, 128), torch.float32) for i in range(2)]
    ys = [torch.empty(4, 8, 128, device="cuda") for _ in range(2)]

    def call(i, out=None, **more):
        qg.attn_decode_kv4_prefix(0, qs[i], 1024, lens, 4, 1, 8, 2, 128, 0.1, 1000, 900, *cache, ys[i] if out is None else out,
                                  ws, nb, st, **more)

    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for rep in range(3):
        lens.add_(torch.tensor([4, 4, 4, 0], dtype=torch.int32, device="cuda"))
        for i in range(2):
            qs[i].copy_(sh.normal(100 + 10 * rep + i, (4, 8, 128), torch.float32))
            graphs[i].replay()
        torch.cuda.synchronize()
        got = [y.clone() for y in ys]
        now = lens.tolist()
        for i in range(2):
            call(i)
            assert torch.equal(ys[i], got[i]), (rep, i)
            sh.check_decode(got[i], qs[i], [k[:n] for k, n in zip(s.k, now)], [v[:n] for v, n in zip(s.v, now)], now, 1, 0.1, 0, 0,
                            prefix=900)
    stream, other = torch.cuda.Stream(), torch.empty_like(ys[0])
    stream.wait_stream(torch.cuda.current_stream())
    call(0, other, stream=stream)
    stream.synchronize()
    assert torch.equal(other, ys[0]) and int(st) == 0
