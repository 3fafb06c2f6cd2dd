"""The cache and attention calls at the ends of what they take: the most sequences and heads, the largest page, the longest chunks; pages that
sequences share; two calls at once."""
import numpy as np
import pytest
import torch

from tests import attn_helpers as ah
from tests.gpu_util import host, progress
from tests.test_gpu_attn import check_decode, decode, normal, prefill, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


@pytest.mark.parametrize("Tq", [1, 16])
def test_most_sequences(qg, Tq):
    """65535 sequences of 0 to 18 positions: appended, read back, attended to.  Distinct lengths are few, so the reference takes
    each length's sequences at once."""
    progress("65535 sequences Tq %d" % Tq)
    B, Dh, page = 65535, 64, 16
    lens = np.arange(B) * 7 % 19
    n = int(lens.sum())
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), **i32)
    lens_d = torch.tensor(lens, **i32)
    pages = torch.randperm(2 * B, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda().view(B, 2)
    kv = torch.full((2 * B, qg.kv4_page_bytes(page, 1, Dh)), 255, dtype=torch.uint8, device="cuda")
    cache, st = (pages, 2, page, 2 * B, kv), status()
    k, v = (normal(i, (n, 1, Dh), torch.bfloat16) for i in (1, 2))
    qg.kv4_append(2, k, Dh, v, Dh, n, cu, lens_d, B, 1, Dh, *cache, st)
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    qg.kv4_gather(2, k2, Dh, v2, Dh, n, cu, lens_d, B, 1, Dh, *cache, st)
    some = np.random.default_rng(2).integers(0, n, 3000)
    for x, x2 in ((k, k2), (v, v2)):
        want = ah.values(*ah.quantize(x[some].double().cpu().numpy()))
        assert np.array_equal(x2[some].double().cpu().numpy(), want)
    q = normal(3, (B * Tq, 2, Dh), torch.float32)
    nb = qg.attn_decode_workspace_bytes(B, Tq, 2, 1, Dh, 2 * page, 0)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    y = torch.full((B * Tq, 2, Dh), 7.0, device="cuda")
    qg.attn_decode_kv4(0, q, 2 * Dh, lens_d, B, Tq, 2, 1, Dh, 0.125, 0, 2 * page, *cache, y, ws, nb, st)
    yp, st2 = prefill(qg, normal(4, (n, 2, Dh), torch.bfloat16), k2, v2, list(lens), list(lens), 2, 2, 1, Dh, 0.125, 0)
    qp = normal(4, (n, 2, Dh), torch.bfloat16)
    assert int(st) == 0 and int(st2) == 0
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)])[:-1], device="cuda")
    for m in range(19):
        of = torch.tensor(np.nonzero(lens == m)[0], device="cuda")
        rows = y.view(B, Tq, 2, Dh)[of].double()
        if m == 0:
            assert not rows.any()
            continue
        at = starts[of][:, None] + torch.arange(m, device="cuda")
        kk, vv = k2[at][:, :, 0].double(), v2[at][:, :, 0].double()  # [sequences, m, Dh]
        for out, qq in ((rows, q.view(B, Tq, 2, Dh)[of]), (yp[at].double(), qp[at])):
            L = qq.shape[1]
            x = qq.double().flatten(1, 2)
            s, mag = (torch.matmul(f(x), f(kk).transpose(1, 2).contiguous()).view(len(of), L, 2, m) * 0.125
                      for f in (lambda t: t, torch.abs))
            seen = torch.arange(m, device="cuda") <= (m - L + torch.arange(L, device="cuda"))[:, None]
            s = s.masked_fill(~seen[:, None], -1e30)
            w = torch.exp(s - s.amax(-1, keepdim=True)) * seen[:, None]
            p = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
            ref = torch.matmul(p.flatten(1, 2), vv).view_as(out)
            a = torch.matmul(p.flatten(1, 2), vv.abs()).view_as(out)
            big = (mag * seen[:, None]).amax(-1, keepdim=True)
            lim = ah.decode_tolerance(a, big, m, Dh) if out is rows else ah.prefill_tolerance(
                ref, a, big, float(vv.abs().max()), m, Dh, torch.bfloat16)
            assert bool(((out - ref).abs() <= lim).all()), (m, L)


@pytest.mark.parametrize("Tq,Dh", [(1, 64), (16, 128)])
def test_most_heads(qg, Tq, Dh):
    """1024 query heads on one key head: up to 16384 rows."""
    progress("1024 heads Tq %d Dh %d" % (Tq, Dh))
    c = ah.Cache([300, 1, 2100], 1, Dh, 64, 5).fill(6)
    q = normal(7, (3 * Tq, 1024, Dh), torch.bfloat16)
    y, st = decode(qg, c, q, 2, Tq, 1024, 0.1, 0)
    assert int(st) == 0
    check_decode(y, c, q, Tq, 0.1, 0)


@pytest.mark.parametrize("Dh", [64, 256])
def test_largest_page(qg, Dh):
    progress("page of 65536 Dh %d" % Dh)
    lens, Hkv = [65536 + 40, 70], 2
    c = ah.Cache(lens, Hkv, Dh, 65536, 8, spare=1)
    k, v = (normal(i, (sum(lens), Hkv, Dh), torch.bfloat16) for i in (9, 10))
    cache, st, cu, w = c.device(), status(), ah.cumulative(lens), Hkv * Dh
    qg.kv4_append(2, k, w, v, w, sum(lens), cu, c.lens_device(), 2, Hkv, Dh, *cache, st)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    qg.kv4_gather(2, k2, w, v2, w, sum(lens), cu, c.lens_device(), 2, Hkv, Dh, *cache, st)
    for which, (x, x2) in enumerate(((k, k2), (v, v2))):
        codes, scales = ah.quantize(x.double().cpu().numpy())
        assert np.array_equal(x2.double().cpu().numpy(), ah.values(codes, scales))
        for b, at in ((0, 0), (1, lens[0])):
            c.put(b, which, codes[at:at + lens[b]], scales[at:at + lens[b]], np.arange(lens[b]))
    assert np.array_equal(host(cache[4]), c.bytes)
    c.k, c.v = ([x[:lens[0]].double().cpu().numpy(), x[lens[0]:].double().cpu().numpy()] for x in (k2, v2))
    q = normal(11, (2, 4, Dh), torch.float32)
    y, st2 = decode(qg, c, q, 0, 1, 4, 0.1, 0, cache=cache)
    assert int(st) == 0 and int(st2) == 0
    check_decode(y, c, q, 1, 0.1, 0)


@pytest.mark.parametrize("page,window", [(16, 0), (32, 1 << 20)])
def test_longest_chunks(qg, page, window):
    """More than 2^20 positions: chunks of 8192 positions, 512 pages or, begun inside a page, 257; the pages of the last
    chunk end with the table."""
    progress("longest chunks page %d window %d" % (page, window))
    n = (1 << 20) + 8192 + 21
    c = ah.Cache([n, 5], 1, 64, page, 12, spare=0, max_pages=-(-n // page)).fill(13)
    q = normal(14, (2, 3, 64), torch.float32)
    y, st = decode(qg, c, q, 0, 1, 3, 0.2, window)
    assert int(st) == 0
    check_decode(y, c, q, 1, 0.2, window)


def test_shared_pages(qg):
    """Sequences that begin with the same pages, and two that are the same altogether."""
    progress("shared pages")
    lens = [200, 137, 137, 64]
    c = ah.Cache(lens, 2, 128, 16, 15).fill(16)
    q = normal(17, (4, 8, 128), torch.float32)
    q[2] = q[1]
    for b in range(1, 4):  # all of the first 128 (or 64) positions are sequence 0's
        m = min(lens[b] // 16, 8)
        c.table[b, :m] = c.table[0, :m]
        for x in (c.k, c.v):
            x[b][:16 * m] = x[0][:16 * m]
    c.table[2], c.k[2], c.v[2] = c.table[1], c.k[1], c.v[1]
    y, st = decode(qg, c, q, 0, 1, 8, 0.1, 0)
    assert int(st) == 0 and torch.equal(y[1], y[2])
    check_decode(y, c, q, 1, 0.1, 0)
    k, v = (torch.empty(sum(lens), 2, 128, device="cuda") for _ in range(2))
    qg.kv4_gather(0, k, 256, v, 256, sum(lens), ah.cumulative(lens), c.lens_device(), 4, 2, 128, *c.device(), st)
    assert np.array_equal(host(k), np.concatenate(c.k)) and np.array_equal(host(v), np.concatenate(c.v)) and int(st) == 0


def test_two_calls_at_once(qg):
    """Decode steps and prompts on two streams, with a workspace each and one status word."""
    progress("two streams")
    c = ah.Cache([5000, 900, 17], 2, 128, 64, 18).fill(19)
    cache, lens, st = c.device(), c.lens_device(), status()
    qs = [normal(20 + i, (3, 8, 128), torch.float32) for i in range(2)]
    nb = qg.attn_decode_workspace_bytes(3, 1, 8, 2, 128, 5000, 0)
    wss = [torch.empty(nb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    n = 700
    ps = [[normal(30 + 3 * i + j, (n, h, 128), torch.float16) for j, h in enumerate((8, 2, 2))] for i in range(2)]
    cu = ah.cumulative([n])
    ys = [[torch.zeros(3, 8, 128, device="cuda") for _ in range(2)] for _ in range(2)]
    yps = [[torch.zeros(n, 8, 128, dtype=torch.float16, device="cuda") for _ in range(2)] for _ in range(2)]

    def call(i, turn, stream=None):
        for _ in range(5):
            qg.attn_decode_kv4(0, qs[i], 1024, lens, 3, 1, 8, 2, 128, 0.1, 0, 5000, *cache, ys[turn][i], wss[i], nb, st,
                               stream=stream)
            qg.attn_prefill(1, ps[i][0], 1024, ps[i][1], 256, ps[i][2], 256, n, n, cu, cu, 1, 8, 2, 128, 0.1, 0,
                            yps[turn][i], st, stream=stream)

    for i in range(2):
        call(i, 0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        call(i, 1, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(ys[0][i], ys[1][i]) and torch.equal(yps[0][i], yps[1][i])
    assert int(st) == 0
