"""The binding's compiled half gives, for tensors on the GPU, what its checked half gives: the address, or the same error."""
import itertools

import pytest
import torch

from tests import sinks_helpers as sh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


def outcome(f, *args):
    try:
        return f(*args)
    except Exception as e:  # noqa: BLE001: its kind and words are what is compared
        return type(e), str(e)


def test_rows(qg):
    base = {t: torch.zeros(6, 10, 64, dtype=d, device="cuda") for t, d in ((0, torch.float32), (1, torch.float16), (2, torch.bfloat16))}
    x = base[2]
    tensors = [x, x[:, :2], x[:, 2:6], x[1:], x.view(60, 64), x.view(-1), x[:, :, :32], x[::2], x.transpose(0, 1), x[:1, :2],
               x[:, :2].unflatten(2, (2, 32)), x[0, 0, 0], x.expand(2, 6, 10, 64), base[0], base[1], x.cpu(), None, 4096,
               torch.nn.Parameter(x.float()), torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")]
    for t, type, rows, (width, ld) in itertools.product(
            tensors, (0, 1, 2, 7), (1, 5, 6, 7, 60), ((128, 640), (640, 640), (128, 128), (64, 64), (256, 640), (128, 1280))):
        args = (t, "x", 0, type, rows, width, ld)
        assert outcome(qg._rows_ptr, *args) == outcome(qg._checked_rows_ptr, *args), args
    for device in (1, None):
        args = (x, "x", device, 2, 6, 640, 640)
        assert outcome(qg._rows_ptr, *args) == outcome(qg._checked_rows_ptr, *args)


def test_arrays(qg):
    i = torch.zeros(9, 4, dtype=torch.int32, device="cuda")
    for t, dtype, count, device in itertools.product(
            (i, i[:, :2], i.t(), i.float(), i.long(), i.cpu(), None, 64, i[0, 0]),
            (torch.int32, torch.float32, None), (0, 1, 36, 37, 144, 145, -3), (0, 1, None)):
        args = (t, "i", device, dtype, count)
        assert outcome(qg._array_ptr, *args) == outcome(qg._checked_array_ptr, *args), args


def test_arguments_that_do_not_fit_are_refused(qg):
    q, k = sh.normal(1, (3, 2, 64), torch.float32), sh.normal(2, (3, 2, 64), torch.float32)
    cu, lens = torch.tensor([0, 3], dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda")
    good = [0, q, 128, k, 128, 3, cu, lens, 1, 2, 2, 64, None, None, 1e-6, 0, 0, None, 0, q, 128, k, 128, sh.status()]
    qg.qk_norm_rope(*good)
    for at, x, error in ((15, 1 << 32, OverflowError), (16, -(1 << 40), OverflowError), (15, "16", TypeError),
                         (14, "x", TypeError), (15, 8, qg.QGError), (14, float("nan"), qg.QGError)):
        with pytest.raises(error):
            qg.qk_norm_rope(*good[:at], x, *good[at + 1:])
