"""Tensors that have no memory of their own: what vmap and grad wrap others in, and sparse ones.  Both halves of the binding
raise the same error for them, and the calls pass it on."""
import pytest
import torch

from tests import attn_helpers as ah
from tests import sinks_helpers as sh
from tests.test_gpu_binding import outcome

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import routed_moe_matvec_amd as qg
    return qg


def wrapped(f):
    """f of a tensor that is [3, 2, 64] inside vmap, vmap of vmap, grad, jvp and functionalize."""
    x = sh.normal(1, (3, 2, 64), torch.float32)

    def loss(y):
        f(y)
        return y.sum()

    torch.vmap(loss)(x.expand(2, 3, 2, 64).contiguous())
    torch.vmap(loss, in_dims=1)(x[:, None].repeat(1, 2, 1, 1))
    torch.vmap(torch.vmap(loss))(x.expand(2, 2, 3, 2, 64).contiguous())
    torch.func.grad(loss)(x)
    torch.func.jvp(loss, (x,), (x,))
    torch.func.functionalize(loss)(x)


def test_halves_agree(qg):
    seen = []

    def f(y):
        args = (y, "y", 0, 0, 3, 128, 128)
        want = outcome(qg._checked_rows_ptr, *args)
        assert outcome(qg._rows_ptr, *args) == want
        seen.append(want)
        for dtype, count in ((torch.float32, 100), (None, 100), (torch.int32, 1), (torch.float32, 1000)):
            args = (y, "y", 0, dtype, count)
            assert outcome(qg._array_ptr, *args) == outcome(qg._checked_array_ptr, *args), args

    wrapped(f)
    assert len(seen) == 6 and any(isinstance(w, tuple) and w[0] is RuntimeError for w in seen)


def test_halves_agree_on_sparse_tensors(qg):
    x = sh.normal(1, (6, 64), torch.float32)
    for y in (x.to_sparse(), x.to_sparse_csr()):
        for args in ((y, "y", 0, 0, 6, 64, 64), (y, "y", 0, 0, 6, 32, 64), (y, "y", 0, 2, 6, 64, 64)):
            assert outcome(qg._rows_ptr, *args) == outcome(qg._checked_rows_ptr, *args), args
        for args in ((y, "y", 0, torch.float32, 100), (y, "y", 0, None, 100), (y, "y", 0, torch.int32, 1)):
            assert outcome(qg._array_ptr, *args) == outcome(qg._checked_array_ptr, *args), args


def test_calls_raise(qg):
    """The error that a tensor without storage gives, from the first argument and from others, and the call after it works."""
    cu, lens = ah.cumulative([3]), torch.tensor([3], dtype=torch.int32, device="cuda")
    k, st = sh.normal(2, (3, 2, 64), torch.float32), sh.status()
    q_out, k_out = torch.empty_like(k), torch.empty_like(k)
    pages, kv = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(qg.kv4_page_bytes(16, 2, 64), dtype=torch.uint8, device="cuda")

    def rope(q, k):
        qg.qk_norm_rope(0, q, 128, k, 128, 3, cu, lens, 1, 2, 2, 64, None, None, 1e-6, 64, 0,
                        torch.ones(32, device="cuda"), 0, q_out, 128, k_out, 128, st)

    def append(x, k):
        qg.kv4_append(0, x, 128, k, 128, 3, cu, lens, 1, 2, 64, pages, 1, 16, 1, kv, st)

    def f(y):
        for args in ((y, k), (k, y), (y, y)):
            for call in (rope, append):
                with pytest.raises(RuntimeError, match="storage"):
                    call(*args)

    x = sh.normal(1, (3, 2, 64), torch.float32)
    torch.vmap(lambda y: (f(y), y.sum())[1])(x.expand(2, 3, 2, 64).contiguous())
    torch.func.grad(lambda y: (f(y), y.sum())[1])(x)
    rope(x, k)
    append(x, k)
    assert int(st) == 0 and bool(q_out.isfinite().all())
