"""attn_decode_kv4_prefix gives a sequence the same bits for any max_len, as the call without a prefix does: lengths of a
few hundred, and bounds on both sides of what one workgroup walks."""
import numpy as np
import pytest
import torch

from tests import attn_helpers as ah
from tests import sinks_helpers as sh
from tests.gpu_util import progress
from tests.test_gpu_prefix import Shared, decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("prefix,lens,Tq,G,Hkv,Dh,page", [
    (300, [301, 431, 350, 300, 17, 0], 1, 4, 2, 128, 16),
    (300, [420, 301, 305], 3, 4, 2, 128, 64),
    (17, [18, 900, 600], 1, 17, 1, 128, 16),
    (300, [301, 431, 350, 8], 1, 8, 1, 64, 16),
    (300, [301, 431, 350, 8], 2, 2, 2, 256, 32),
    (1499, [1500 + i % 50 for i in range(150)], 1, 1, 1, 128, 16),  # rows of all sequences together
])
def test_results_do_not_depend_on_max_len(qg, prefix, lens, Tq, G, Hkv, Dh, page, type):
    progress("prefix %d max_len Dh %d Tq %d type %d" % (prefix, Dh, Tq, type))
    s = Shared(prefix, lens, Hkv, Dh, page, 131)
    most = 70000 // page * page
    s.table = np.pad(s.table, ((0, 0), (0, most // page - s.max_pages)), constant_values=-1)
    s.max_pages = most // page
    q = sh.normal(133, (len(lens) * Tq, G * Hkv, Dh), ah.TYPES[type])
    y, st = decode(qg, s, q, type, Tq, G * Hkv, 0.1)
    sh.check_decode(y, q, s.k, s.v, lens, Tq, 0.1, 0, 0, prefix=prefix)
    for max_len in (624, 625, 640, 641, 1264, 1265, 1280, 1281, 2544, 2545, 5104, 8176, 8192, most):
        if max_len >= max(lens):
            assert torch.equal(decode(qg, s, q, type, Tq, G * Hkv, 0.1, max_len=max_len)[0], y), max_len
    assert int(st) == 0
