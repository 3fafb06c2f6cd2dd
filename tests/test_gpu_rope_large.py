"""qk_norm_rope over heads whose squares are far beyond fp32, up to all elements at the type's largest: the formula in 64
bits.  The tolerances are sinks_helpers': the powers of two on elements and on their root are exact."""
import math

import pytest
import torch

from tests import attn_helpers as ah
from tests import sinks_helpers as sh
from tests.gpu_util import progress
from tests.test_gpu_rope import call, check, freqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


def signs(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return 1.0 - 2.0 * torch.randint(0, 2, shape, generator=g, device="cuda")


@pytest.mark.parametrize("type,out", [(0, 0), (2, 2), (0, 1), (0, 2)])
@pytest.mark.parametrize("eps", [2.0**-100, 1e-6, 2.0**100])
@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_heads_of_the_largest_numbers(qg, Dh, eps, type, out):
    """A head of equal magnitudes becomes +-w, turned: from where the squares' sum leaves fp32 to the type's largest."""
    progress("rope largest Dh %d eps %g type %d to %d" % (Dh, eps, type, out))
    dtype = ah.TYPES[type]
    sizes = [2.0**58, 2.0**59, 2.0**62, 2.0**63, 1.3e20, 1e30, 1e37, 2.1e37, 3.1e37, 4.4e37, 1e38, 2.0**127,
             torch.finfo(dtype).max]
    n = len(sizes)
    x = (signs((n, 4, Dh), 1).double() * torch.tensor(sizes, dtype=torch.float64, device="cuda")[:, None, None]).to(dtype)
    assert bool(x.isfinite().all())
    w = 1 + 0.3 * sh.normal(2, (Dh,), torch.float32)
    for R, neighbours in ((Dh, False), (Dh // 2, True)):
        yq, yk, st = call(qg, x, x[:, 1:3], [n + 5], [n], R, neighbours, out, wq=w, eps=eps)
        check(yq, x, w, [n + 5], [n], freqs(R), eps, neighbours)
        check(yk, x[:, 1:3], None, [n + 5], [n], freqs(R), eps, neighbours)
        assert bool(yq.float().abs().amax(2).min() > 0.1) and int(st) == 0


@pytest.mark.parametrize("type", [0, 2])
@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_large_and_small_elements_in_one_head(qg, Dh, type):
    """One, some and all but one element large, the others ordinary, tiny or zero: pairs of small elements keep their bits."""
    progress("rope large beside small Dh %d type %d" % (Dh, type))
    dtype = ah.TYPES[type]
    large = torch.finfo(dtype).max
    x = sh.normal(3, (8, 6, Dh), torch.float32)
    for i, most in enumerate((large, 2.0**64, 2.0**100, 3.1e37)):
        x[2 * i, 0, 5] = most
        x[2 * i, 1, ::3] = -most
        x[2 * i, 2, 1:] = most
        x[2 * i, 3] *= 2.0**-50
        x[2 * i, 3, Dh // 2] = most
        x[2 * i, 4] = 0
        x[2 * i, 4, -1] = -most
        x[2 * i + 1, 1] = 0  # and rows between them that need no such care
    x = x.to(dtype)
    assert bool(x.isfinite().all())
    for R, neighbours in ((Dh, False), (Dh, True), (Dh // 4, False), (0, False)):
        yq, yk, _ = call(qg, x, x[:, :2], [40], [8], R, neighbours, type)
        freq = freqs(R) if R else torch.zeros(0, device="cuda")
        check(yq, x, None, [40], [8], freq, 1e-6, neighbours)
        check(yk, x[:, :2], None, [40], [8], freq, 1e-6, neighbours)
        for i in range(4):  # one element alone is the head: sqrt(Dh) is left, of both outputs of its pair
            off = abs(float(yq[2 * i, 4].double().square().sum().sqrt()) / math.sqrt(Dh) - 1)
            assert off < math.sqrt(2) * (20 * 2.0**-24 + torch.finfo(dtype).eps / 2)
