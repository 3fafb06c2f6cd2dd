"""The operators between projections and attention as a serving loop runs them, each stage checked on the inputs that the
stage before left: norm and rotation, the FP4 cache, attention with sinks over a prompt and over steps, and steps of
several answers to one prompt.  The step is captured once; every replay is the next step, and gives what eager calls give."""
import numpy as np
import pytest
import torch

from tests import attn_helpers as ah
from tests import sinks_helpers as sh
from tests.gpu_util import progress
from tests.test_gpu_rope import check as check_rope, freqs
from tests.test_gpu_sinks import check_prefill

pytestmark = pytest.mark.gpu
H, HKV, EPS = 8, 2, 1e-6


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


def held(x):
    """What the cache holds of x [n, Hkv, Dh]."""
    return ah.values(*ah.quantize(x.double().cpu().numpy()))


@pytest.mark.parametrize("Dh,R", [(64, 64), (128, 32)])
def test_prompt_and_steps_with_sinks(qg, Dh, R):
    progress("chain with sinks Dh %d" % Dh)
    page, mp, window, sinks, steps = 16, 20, 40, 5, 12
    start = [30, 0, 210]
    B, n, w = 3, sum(start), HKV * Dh
    i32 = dict(dtype=torch.int32, device="cuda")
    order = torch.randperm(B * mp, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    pages, st = order.cuda().view(B, mp), sh.status()
    freq, scale = freqs(R), Dh**-0.5
    wq, wk = (1 + 0.2 * sh.normal(i, (Dh,), torch.float32) for i in (1, 2))

    def rope(qkv, cu, lens, out_type, q_out, k_out):
        q, k = qkv[:, :H], qkv[:, H:H + HKV]
        qg.qk_norm_rope(qg.TYPE_F32, q, q.stride(0), k, k.stride(0), qkv.shape[0], cu, lens, B, H, HKV, Dh, wq, wk, EPS, R,
                        qg.ROPE_HALVES, freq, out_type, q_out, q_out.stride(0), k_out, k_out.stride(0), st)

    # the prompt: fp32 projections to 16-bit rows, attention over them, and the keys and values into the cache
    kv = torch.zeros(B * mp, ah.page_bytes(page, HKV, Dh), dtype=torch.uint8, device="cuda")
    qkv = sh.normal(3, (n, H + 2 * HKV, Dh), torch.float32)
    q, k = (torch.full((n, h, Dh), 77.0, dtype=torch.bfloat16, device="cuda") for h in (H, HKV))
    cu, lens = ah.cumulative(start), torch.tensor(start, **i32)
    rope(qkv, cu, lens, qg.TYPE_BF16, q, k)
    check_rope(q, qkv[:, :H], wq, start, start, freq, EPS, False)
    check_rope(k, qkv[:, H:H + HKV], wk, start, start, freq, EPS, False)
    v, y = qkv[:, H + HKV:].bfloat16(), torch.empty_like(q)
    qg.attn_prefill_sinks(qg.TYPE_BF16, q, H * Dh, k, w, v, w, n, n, cu, cu, B, H, HKV, Dh, scale, window, sinks, y, st)
    check_prefill(y, q, k, v, start, start, scale, window, sinks)
    qg.kv4_append(qg.TYPE_BF16, k, w, v, w, n, cu, lens, B, HKV, Dh, pages, mp, page, B * mp, kv, st)
    ks, vs = ([np.split(held(x), np.cumsum(start)[:-1])] for x in (k, v))
    ks, vs = list(ks[0]), list(vs[0])

    # steps: norm and rotation in place, into the cache, attention; a captured step beside an eager one
    one, max_len = ah.cumulative([1] * B), mp * page
    nb = qg.attn_decode_sinks_workspace_bytes(B, 1, H, HKV, Dh, max_len, window, sinks)
    new = torch.empty(B, H + 2 * HKV, Dh, device="cuda")

    def state():
        return dict(lens=lens.clone(), kv=kv.clone(), qkv=torch.empty_like(new), y=torch.empty(B, H, Dh, device="cuda"),
                    ws=torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda"))

    def step(s):
        s["lens"].add_(1)
        s["qkv"].copy_(new)
        q, k, v = s["qkv"].split([H, HKV, HKV], dim=1)
        ld = s["qkv"].stride(0)
        rope(s["qkv"], one, s["lens"], qg.TYPE_F32, q, k)
        qg.kv4_append(qg.TYPE_F32, k, ld, v, ld, B, one, s["lens"], B, HKV, Dh, pages, mp, page, B * mp, s["kv"], st)
        qg.attn_decode_kv4_sinks(qg.TYPE_F32, q, ld, s["lens"], B, 1, H, HKV, Dh, scale, window, sinks, max_len, pages, mp,
                                 page, B * mp, s["kv"], s["y"], s["ws"], nb, st)

    eager, captured = state(), state()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(captured)
    now = list(start)
    for i in range(steps):
        new.copy_(sh.normal(100 + i, new.shape, torch.float32))
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for name in ("lens", "kv", "qkv", "y"):
            assert torch.equal(eager[name], captured[name]), (i, name)
        now = [m + 1 for m in now]
        q, k, v = eager["qkv"].split([H, HKV, HKV], dim=1)
        check_rope(q, new[:, :H], wq, now, [1] * B, freq, EPS, False)
        check_rope(k, new[:, H:H + HKV], wk, now, [1] * B, freq, EPS, False)
        for b in range(B):
            ks[b] = np.concatenate([ks[b], held(k[b:b + 1])])
            vs[b] = np.concatenate([vs[b], held(v[b:b + 1])])
        sh.check_decode(eager["y"], q.contiguous(), ks, vs, now, 1, scale, window, sinks)
    assert int(st) == 0


@pytest.mark.parametrize("prefix", [37, 700])
def test_answers_to_one_prompt(qg, prefix):
    """One prompt into pages that all answers read; each answer's tokens into pages of its own.  700: enough for the
    shared walk with 24 answers."""
    progress("chain over a shared prefix of %d" % prefix)
    B, Dh, page, steps, R = 24 if prefix > 100 else 3, 128, 16, 5, 128
    skip, w = prefix // page, HKV * Dh
    first = -(-prefix // page)
    mp = skip + 2
    num = first + 2 * B
    order = torch.randperm(num, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    prefix_pages = order[:first].contiguous()
    pages = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    pages[:, skip:] = order[first:].view(B, 2)
    st, freq, scale = sh.status(), freqs(R), Dh**-0.5
    kv = torch.full((num, ah.page_bytes(page, HKV, Dh)), 0xFF, dtype=torch.uint8, device="cuda")

    def rope(qkv, cu, lens, count):
        q, k, v = qkv.split([H, HKV, HKV], dim=1)
        ld = qkv.stride(0)
        qg.qk_norm_rope(qg.TYPE_F32, q, ld, k, ld, qkv.shape[0], cu, lens, count, H, HKV, Dh, None, None, EPS, R,
                        qg.ROPE_NEIGHBOURS, freq, qg.TYPE_F32, q, ld, k, ld, st)
        return q, k, v, ld

    # the prompt, as one sequence of its own
    qkv = sh.normal(5, (prefix, H + 2 * HKV, Dh), torch.float32)
    one_len, one_cu = torch.tensor([prefix], dtype=torch.int32, device="cuda"), ah.cumulative([prefix])
    _, k, v, ld = rope(qkv, one_cu, one_len, 1)
    qg.kv4_append(qg.TYPE_F32, k, ld, v, ld, prefix, one_cu, one_len, 1, HKV, Dh, prefix_pages.view(1, -1), first, page, num, kv, st)
    ks, vs = [held(k)] * B, [held(v)] * B

    lens, cu, max_len = torch.full((B,), prefix, dtype=torch.int32, device="cuda"), ah.cumulative([1] * B), mp * page
    nb = qg.attn_decode_prefix_workspace_bytes(B, 1, H, HKV, Dh, max_len, prefix)
    ws, y = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda"), torch.empty(B, H, Dh, device="cuda")
    new = torch.empty(B, H + 2 * HKV, Dh, device="cuda")

    def step():
        lens.add_(1)
        q, k, v, ld = rope(new, cu, lens, B)
        qg.kv4_append(qg.TYPE_F32, k, ld, v, ld, B, cu, lens, B, HKV, Dh, pages, mp, page, num, kv, st)
        qg.attn_decode_kv4_prefix(qg.TYPE_F32, q, ld, lens, B, 1, H, HKV, Dh, scale, max_len, prefix, prefix_pages, pages, mp,
                                  page, num, kv, y, ws, nb, st)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        raw = sh.normal(200 + i, new.shape, torch.float32)
        new.copy_(raw)
        if i % 2:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        q, k, v = new.split([H, HKV, HKV], dim=1)
        check_rope(q, raw[:, :H], None, [prefix + i + 1] * B, [1] * B, freq, EPS, True)
        ks = [np.concatenate([ks[b], held(k[b:b + 1])]) for b in range(B)]
        vs = [np.concatenate([vs[b], held(v[b:b + 1])]) for b in range(B)]
        sh.check_decode(y, q.contiguous(), ks, vs, [prefix + i + 1] * B, 1, scale, 0, 0, prefix=prefix)
    assert int(st) == 0
