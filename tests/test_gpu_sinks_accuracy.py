"""attn_prefill_sinks over whole sequences, against the norm of the output: its two roundings and no more, and the same bits
in every run, alone and beside another call."""
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


@pytest.mark.parametrize("Dh", [64, 128, 256])
@pytest.mark.parametrize("H,lens,window,sinks", [
    (1, [700, 90], 64, 3),               # few queries a workgroup, the keys split
    (32, [600, 31, 257], 128, 4),
    (64, [1500, 300, 1], 200, 70),
    (64, [2100, 1999], 512, 4),
])
@pytest.mark.parametrize("type", [1, 2])
def test_error_of_the_norm_and_every_run_the_same(qg, type, H, lens, window, sinks, Dh):
    """Weights and outputs are each rounded to the type once: an error of at most eps / 2 of each, spread evenly, is eps / 2 /
    sqrt(3) in the mean square, and both together less than eps / 2 of the norm."""
    progress("sinks prefill error of the norm H %d lens %s window %d Dh %d type %d" % (H, lens, window, Dh, type))
    dt, n, scale = ah.TYPES[type], sum(lens), 2 * Dh**-0.5
    q, k, v = (sh.normal(151 + i, (n, heads, Dh), dt) for i, heads in enumerate((H, 1, 1)))
    cu, st = ah.cumulative(lens), sh.status()
    ys = [torch.full((n, H, Dh), 7.0, dtype=dt, device="cuda") for _ in range(6)]
    streams = [None, None, torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for y, stream in zip(ys, streams):  # the last four may run at once
        qg.attn_prefill_sinks(type, q, H * Dh, k, Dh, v, Dh, n, n, cu, cu, len(lens), H, 1, Dh, scale, window, sinks, y, st,
                              stream=stream)
    torch.cuda.synchronize()
    assert int(st) == 0 and all(torch.equal(y, ys[0]) for y in ys[1:])
    at = 0
    for m in lens:
        rows = slice(at, at + m)
        seen = sh.sees(torch.arange(m, device="cuda"), m, window, sinks)
        ref = sh.attend(q[rows].double(), k[rows].double(), v[rows].double(), scale, seen)[0]
        err = float((ys[0][rows].double() - ref).norm() / ref.norm())
        assert err < torch.finfo(dt).eps / 2, (m, err)
        at += m
