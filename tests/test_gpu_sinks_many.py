"""attn_decode_kv4_sinks at the most workgroups that a call may need: more than one launch of eight waves holds."""
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


def test_more_workgroups_than_one_launch_holds(qg):
    """13 million of 2^24: the sequences of both ends and of the middle against calls of their own, and in 64 bits."""
    B, H, Dh, window, sinks, page = 65535, 200, 64, 16, 4, 16
    progress("sinks, %d sequences of %d key heads" % (B, H))
    c = ah.Cache([64] * 8, H, Dh, page, 141, max_pages=4).fill(142)
    pages, max_pages, _, num_pages, kv = c.device()
    which = torch.arange(B, device="cuda") % 8  # eight caches that the sequences share
    table = pages[which].contiguous()
    lens = (torch.arange(B, device="cuda") * 7 % 65).to(torch.int32)
    lens[40000] = 65  # out of range
    q = torch.empty(B, H, Dh, dtype=torch.float16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(143)
    for b in range(0, B, 8192):
        q[b:b + 8192] = torch.randn(q[b:b + 8192].shape, generator=g, device="cuda")
    y, st = torch.full((B, H, Dh), 77.0, device="cuda"), sh.status()
    nb = qg.attn_decode_sinks_workspace_bytes(B, 1, H, H, Dh, 64, window, sinks)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def call(at, n, out, status):
        qg.attn_decode_kv4_sinks(1, q[at:at + n], H * Dh, lens[at:at + n], n, 1, H, H, Dh, 0.2, window, sinks, 64,
                                 table[at:at + n], max_pages, page, num_pages, kv, out, ws, nb, status)

    call(0, B, y, st)
    torch.cuda.synchronize()
    assert int(st) == qg.DEV_BAD_LENGTH and not y[40000].any() and not bool((y == 77.0).any())
    halves = ((1 << 23) - 1) // H  # the sequences of a launch
    for at, n in ((0, 40), (halves - 20, 40), (halves + 1000, 8), (B - 40, 40)):
        part, ok = torch.empty(n, H, Dh, device="cuda"), sh.status()
        call(at, n, part, ok)
        assert torch.equal(part, y[at:at + n]) and int(ok) == 0
        now, own = lens[at:at + n].tolist(), which[at:at + n].tolist()
        sh.check_decode(part[:8], q[at:at + 8], [c.k[i][:m] for i, m in zip(own[:8], now[:8])],
                        [c.v[i][:m] for i, m in zip(own[:8], now[:8])], now[:8], 1, 0.2, window, sinks)
