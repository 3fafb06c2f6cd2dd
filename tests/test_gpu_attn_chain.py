"""A prompt as a model runs it, in two chunks: q, k, v from the prompt's GEMM, into the FP4 cache, attention over the chunk itself and
then over what the cache gives back, the activation quantizer and the output projection.  Each stage is checked on the
inputs that the stage before left."""
import numpy as np
import pytest
import torch

import synth
from tests import attn_helpers as ah
from tests.gpu_util import assert_within_bound, dev, empty, host, oracle_threads, progress
from tests.test_gpu_attn import prefill

pytestmark = pytest.mark.gpu


def check(y, q, k, v, lq, lk, scale):
    """attn_helpers' tolerance, which knows no underflow, and what that can take: scores lie hundreds apart here, and where the key that
    takes all has the value 0, others of weights about 2^-130 are all there is.  A weight below 2^-126 is 0 in fp32, and so is
    the factor of that size that a new maximum gives the sums before it, of m weights up to 2^8: at most m 2^-118 of the
    largest value."""
    at = kat = 0
    for n, m in zip(lq, lk):
        vv = v[kat:kat + m].double()
        ref, a, big = ah.attend(q[at:at + n].double(), k[kat:kat + m].double(), vv, scale, 0)
        most = float(vv.abs().max()) if m else 0.0
        lim = ah.prefill_tolerance(ref, a, big, most, m, q.shape[2], q.dtype) + m * 2.0**-118 * most
        assert bool(((y[at:at + n].double() - ref).abs() <= lim).all()), (n, m)
        at, kat = at + n, kat + m
    assert at == len(y)


@pytest.mark.parametrize("Dh", [64, 128])
def test_prompt_through_the_projections(orc, Dh):
    import routed_moe_matvec_amd as qg
    progress("prompt through the projections Dh %d" % Dh)
    K, H, Hkv, page, N = 512, 512 // Dh, 2, 16, 96
    first, second = [45, 0, 130], [20, 33, 1]
    lens, B = [a + b for a, b in zip(first, second)], 3
    width, w = (H + 2 * Hkv) * Dh, Hkv * Dh
    g = synth.rng(11)
    W, Wo = synth.q4k_weight(g, width, K), synth.q8_0_weight(g, N, H * Dh)
    Wd, Wod = dev(W), dev(Wo)
    c = ah.Cache(lens, Hkv, Dh, page, 12)
    cache, st = c.device(), torch.zeros(1, dtype=torch.int32, device="cuda")
    held = [[np.zeros((0, Hkv, Dh)) for _ in range(B)] for _ in (0, 1)]
    done = [0] * B
    for news in (first, second):
        n = sum(news)
        xb = synth.bf16_activations(g, n, K)
        qkv = empty((n, H + 2 * Hkv, Dh), torch.float32)
        qg.qgemm_prefill(qg.FMT_Q4K, Wd, width, K, dev(xb.view(np.int16)), n, qkv)
        ref, bound = orc.prefill(orc.FMT_Q4K, W, width, K, xb, nthreads=oracle_threads())
        assert_within_bound(host(qkv).reshape(n, -1), ref, bound, what="q, k, v")
        done = [a + b for a, b in zip(done, news)]
        cu, lens_d = ah.cumulative(news), torch.tensor(done, dtype=torch.int32, device="cuda")
        _, ks, vs = qkv.split([H, Hkv, Hkv], dim=1)
        qg.kv4_append(qg.TYPE_F32, ks, width, vs, width, n, cu, lens_d, B, Hkv, Dh, *cache, st)
        for part, src in ((0, ks), (1, vs)):
            x = ah.values(*ah.quantize(src.double().cpu().numpy()))
            at = 0
            for b, m in enumerate(news):
                held[part][b] = np.concatenate([held[part][b], x[at:at + m]])
                at += m
        q, k, v = qkv.bfloat16().split([H, Hkv, Hkv], dim=1)
        lk = news
        if done != news:  # the second chunk sees the first through the cache
            k, v = (empty((sum(done), Hkv, Dh), torch.bfloat16) for _ in range(2))
            qg.kv4_gather(qg.TYPE_BF16, k, w, v, w, sum(done), ah.cumulative(done), lens_d, B, Hkv, Dh, *cache, st)
            for part, x in ((0, k), (1, v)):
                assert np.array_equal(x.double().cpu().numpy(), np.concatenate(held[part]))
            lk = done
        scale = Dh**-0.5 * 0.05
        y, st2 = prefill(qg, q, k, v, news, lk, qg.TYPE_BF16, H, Hkv, Dh, scale, 0)
        check(y, q, k, v, news, lk, scale)
        qx, dx, sx = (empty((n, H * Dh), torch.int8), empty((n, H * Dh // 32), torch.float32),
                      empty((n, H * Dh // 32), torch.int32))
        qg.quantize_act_q8(y.float(), n, H * Dh, qx, dx, sx)
        out = empty((n, N), torch.float32)
        qg.qgemm_q8_0(Wod, N, H * Dh, qx, dx, n, out)
        rq, rd, _ = orc.quantize_act_q8(host(y.float()).reshape(n, -1))
        ref, bound = orc.gemv(orc.FMT_Q8_0, Wo, N, H * Dh, rq, rd)
        assert_within_bound(host(out), ref, bound, what="output projection")
        assert int(st) == 0 and int(st2) == 0
