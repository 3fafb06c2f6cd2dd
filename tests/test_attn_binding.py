"""The binding of the cache and attention calls, without a GPU: tensors of two devices are refused before any launch, whose kernels
would otherwise read one device's addresses on the other."""
import pytest
import torch

import routed_moe_matvec_amd as qg


class On(torch.Tensor):
    """A tensor that says that it lies on a GPU."""

    @staticmethod
    def make(t, index):
        x = torch.Tensor._make_subclass(On, t)
        x.index = index
        return x

    is_cuda = True

    def get_device(self):
        return self.index


def calls(on):
    """Calls whose tensors lie where on(name) says."""
    def rows(name, dtype):
        return On.make(torch.zeros(4, 2, 64, dtype=dtype), on(name))

    def ints(name):
        return On.make(torch.zeros(8, dtype=torch.int32), on(name))

    def raw(name, n):
        return On.make(torch.zeros(n, dtype=torch.uint8), on(name))

    size = qg.kv4_page_bytes(16, 2, 64)
    def cache():
        return ints("pages"), 1, 16, 1, raw("kv", size)

    f32, f16 = torch.float32, torch.float16
    for move in (qg.kv4_append, qg.kv4_gather):
        yield "k v cu lens pages kv d_status", lambda move=move: move(
            0, rows("k", f32), 128, rows("v", f32), 128, 4, ints("cu"), ints("lens"), 1, 2, 64, *cache(), ints("d_status"))
    yield "q lens pages kv y ws d_status", lambda: qg.attn_decode_kv4(
        0, rows("q", f32), 128, ints("lens"), 4, 1, 2, 2, 64, 0.1, 0, 16, On.make(torch.zeros(4, 1, dtype=torch.int32),
        on("pages")), 1, 16, 1, raw("kv", size), rows("y", f32), raw("ws", 256), 256, ints("d_status"))
    yield "q k v cu_q cu_k y d_status", lambda: qg.attn_prefill(
        1, rows("q", f16), 128, rows("k", f16), 128, rows("v", f16), 128, 4, 4, ints("cu_q"), ints("cu_k"), 1, 2, 2, 64,
        0.1, 0, rows("y", f16), ints("d_status"))


@pytest.mark.parametrize("which", range(4))
def test_tensors_of_two_devices_are_refused(which):
    names = [n for n, _ in calls(lambda name: 0)][which].split()
    for odd in names[1:]:  # the first says where the call runs
        for here, there in ((0, 1), (1, 0)):
            call = [c for _, c in calls(lambda name: there if name == odd else here)][which]
            with pytest.raises(ValueError, match="^%s is on device %d, the call's first tensor on device %d$" % (odd, there, here)):
                call()
    for odd in names:
        call = [c for _, c in calls(lambda name: -1 if name == odd else 0)][which]
        with pytest.raises(TypeError):
            call()
