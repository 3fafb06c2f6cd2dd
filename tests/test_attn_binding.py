"""The binding of the cache and attention calls, without a GPU: tensors of two devices are refused before any launch, whose kernels
would otherwise read one device's addresses on the other."""
import ctypes

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


def test_launches_too_large_for_their_tokens_are_refused():
    """2^24 workgroups and more from the tokens, not from the sequences; a call below is refused for another reason."""
    from tests.test_attn_host import AT, DECODE, DECODE_T, MOVE, MOVE_T, PREFILL, PREFILL_T, _call
    lib = ctypes.CDLL(qg.library_path())
    long = dict(n=1 << 24, Dh=256, B=1)
    for name in ("kv4_append", "kv4_gather"):
        for Hkv, code in ((32, -2), (28, -3)):  # 16 and 14 pieces of a row; the cache 8 bytes off
            assert _call(lib, name, MOVE_T, {**MOVE, **long, "Hkv": Hkv,
                                              "ldk": 256 * Hkv, "ldv": 256 * Hkv, "kv": AT + 8}) == code
    assert _call(lib, "attn_prefill", PREFILL_T, {**PREFILL, "nq": 1 << 24, "nk": 1 << 24, "B": 1, "H": 128, "ldq": 1 << 14}) == -2
    rows = dict(B=65535, H=512, Hkv=2, ldq=1 << 16, max_len=128)
    assert _call(lib, "attn_decode_kv4", DECODE_T, {**DECODE, **rows, "ws_bytes": 1 << 62}) == -2
    chunks = dict(B=2048, H=8, Hkv=8, ldq=1 << 10, max_len=1 << 22, page=65536, max_pages=64)
    nb = qg.attn_decode_workspace_bytes(2048, 1, 8, 8, 128, 1 << 22, 0)
    assert nb == 2048 * 8 * 130 * 4 * 1024  # 1024 chunks: 2^24 workgroups
    assert _call(lib, "attn_decode_kv4", DECODE_T, {**DECODE, **chunks, "ws_bytes": nb}) == -2
