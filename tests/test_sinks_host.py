"""qk_norm_rope and the attention calls with sinks and with a shared prefix, without a GPU: what they and their binding refuse,
their workspaces, and the test references' own pins.  No call here reaches a kernel launch."""
import ctypes
import math

import pytest
import torch

import routed_moe_matvec_amd as qg
from tests import sinks_helpers as sh
from tests.test_attn_binding import On
from tests.test_attn_host import (AT, BAD_DECODE, BAD_PREFILL, DECODE, DECODE_T, F, I, PREFILL, PREFILL_T, VP, _call)


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(qg.library_path())


def put(args, types, after, **more):
    """The arguments with more of them behind `after`, and their types (int, or a pointer where the value is AT)."""
    names, out, t = list(args), {}, []
    for name, kind in zip(names, types):
        out[name] = args[name]
        t.append(kind)
        if name == after:
            out.update(more)
            t += [VP if v == AT else I for v in more.values()]
    return out, t


SINKS, SINKS_T = put(DECODE, DECODE_T, "window", sinks=4)
PRE_SINKS, PRE_SINKS_T = put(PREFILL, PREFILL_T, "window", sinks=4)
PREFIX, PREFIX_T = put({n: v for n, v in DECODE.items() if n != "window"},
                       [t for n, t in zip(DECODE, DECODE_T) if n != "window"], "max_len", prefix=40, prefix_pages=AT)
ROPE = dict(type=0, q=AT, ldq=512, k=AT, ldk=256, n=5, cu=AT, lens=AT, B=3, H=4, Hkv=2, Dh=128, wq=AT, wk=AT, eps=1e-6,
            R=128, style=0, freq=AT, out_type=2, q_out=AT, ldq_out=512, k_out=AT, ldk_out=256, d_status=AT, stream=None)
ROPE_T = [I, VP, I, VP, I, I, VP, VP, I, I, I, I, VP, VP, F, I, I, VP, I, VP, I, VP, I, VP, VP]
BAD_ROPE = [(dict(type=3), -4), (dict(type=-1), -4), (dict(type=1), -4), (dict(type=2, out_type=0), -4),
            (dict(out_type=4), -4), (dict(style=2), -4), (dict(style=-1), -4)] + [
    ({n: None}, -1) for n in "q k cu lens freq q_out k_out d_status".split()] + [
    (change, -2) for change in (
        dict(n=0), dict(n=(1 << 24) + 1), dict(B=0), dict(B=65536), dict(H=0), dict(Hkv=0), dict(H=1025, ldq=1 << 18),
        dict(Hkv=1025, ldk=1 << 18), dict(Dh=96), dict(Dh=512), dict(R=-16), dict(R=144), dict(R=24), dict(eps=0.0),
        dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-31), dict(ldq=511), dict(ldq=514),
        dict(ldk=255), dict(ldq_out=508), dict(ldk_out=252), dict(ldk_out=260), dict(n=1 << 24, H=64, ldq=1 << 14, ldq_out=1 << 14))] + [
    ({n: AT + 8}, -3) for n in "q k wq wk q_out k_out".split()] + [
    ({n: AT + 2}, -3) for n in "cu lens freq d_status".split()]


def test_rope_refuses(lib):
    for change, code in BAD_ROPE:
        assert _call(lib, "qk_norm_rope", ROPE_T, {**ROPE, **change}) == code, change
    # where nothing turns no frequencies are needed: refused for another reason only
    assert _call(lib, "qk_norm_rope", ROPE_T, {**ROPE, "R": 0, "freq": None, "cu": AT + 1}) == -3
    # the most tokens of one launch: 24 heads of 128 are three groups, 32 are four
    for H, code in ((20, -3), (28, -2)):
        rows = dict(H=H, Hkv=4, ldq=4096, ldk=512, ldq_out=4096, ldk_out=512)
        assert _call(lib, "qk_norm_rope", ROPE_T, {**ROPE, **rows, "n": 1 << 24, "cu": AT + 1}) == code


def test_rope_in_place_refuses_other_types_and_strides(lib):
    """A row of another type or stride would be written over heads that other waves still read."""
    apart = dict(q_out=AT + (1 << 20), k_out=AT + (1 << 21))
    for change in (dict(q_out=AT), dict(k_out=AT), dict(out_type=0, q_out=AT, ldq_out=1024),
                   dict(out_type=0, k_out=AT, ldk_out=512)):
        assert _call(lib, "qk_norm_rope", ROPE_T, {**ROPE, **apart, **change}) == -2, change


@pytest.mark.parametrize("change,code", BAD_DECODE + [(dict(sinks=-1), -2)])
def test_sinks_decode_refuses(lib, change, code):
    assert _call(lib, "attn_decode_kv4_sinks", SINKS_T, {**SINKS, **change}) == code


@pytest.mark.parametrize("change,code", BAD_PREFILL + [(dict(sinks=-1), -2)])
def test_sinks_prefill_refuses(lib, change, code):
    assert _call(lib, "attn_prefill_sinks", PRE_SINKS_T, {**PRE_SINKS, **change}) == code


@pytest.mark.parametrize("change,code", [b for b in BAD_DECODE if "window" not in b[0]] + [
    (dict(prefix=-1), -2), (dict(prefix=129), -2), (dict(prefix_pages=None), -1), (dict(prefix_pages=AT + 2), -3)])
def test_prefix_decode_refuses(lib, change, code):
    assert _call(lib, "attn_decode_kv4_prefix", PREFIX_T, {**PREFIX, **change}) == code


def test_workspaces():
    """Exactly what is asked for is enough: one byte less is refused."""
    lib = ctypes.CDLL(qg.library_path())
    for sinks, window in ((0, 0), (4, 100), (300, 1), (1 << 30, 1 << 30), ((1 << 31) - 1, (1 << 31) - 1)):
        nb = qg.attn_decode_sinks_workspace_bytes(3, 1, 4, 2, 128, 128, window, sinks)
        assert nb > 0
        assert _call(lib, "attn_decode_kv4_sinks", SINKS_T, {**SINKS, "window": window, "sinks": sinks, "ws_bytes": nb - 1}) == -5
    long = dict(max_len=1 << 22, page=4096, max_pages=1024)
    assert qg.attn_decode_sinks_workspace_bytes(3, 1, 4, 2, 128, 1 << 22, 0, 4) == qg.attn_decode_workspace_bytes(
        3, 1, 4, 2, 128, 1 << 22, 0)
    assert qg.attn_decode_sinks_workspace_bytes(3, 1, 4, 2, 128, 1 << 22, 100, 4) < 1 << 10
    for prefix in (0, 1, 17, 128):
        nb = qg.attn_decode_prefix_workspace_bytes(3, 1, 4, 2, 128, 128, prefix)
        assert nb > 0
        assert _call(lib, "attn_decode_kv4_prefix", PREFIX_T, {**PREFIX, "prefix": prefix, "ws_bytes": nb - 1}) == -5
    nb = qg.attn_decode_prefix_workspace_bytes(3, 1, 4, 2, 128, 1 << 22, 1 << 21)
    assert _call(lib, "attn_decode_kv4_prefix", PREFIX_T, {**PREFIX, **long, "prefix": 1 << 21, "ws_bytes": nb - 1}) == -5
    for bad in [(0, 1, 4, 2, 128, 128, 1, 1), (3, 1, 4, 2, 128, 128, -1, 1), (3, 1, 4, 2, 128, 128, 1, -1)]:
        assert qg.attn_decode_sinks_workspace_bytes(*bad) == 0
    for bad in [(3, 17, 4, 2, 128, 128, 1), (3, 1, 4, 2, 128, 128, -1), (3, 1, 4, 2, 128, 128, 129)]:
        assert qg.attn_decode_prefix_workspace_bytes(*bad) == 0


def test_launches_too_large_are_refused(lib):
    assert _call(lib, "attn_decode_kv4_sinks", SINKS_T, {**SINKS, "B": 65535, "H": 512, "Hkv": 512, "ldq": 1 << 16,
                                                         "ws_bytes": 1 << 62}) == -2
    assert _call(lib, "attn_decode_kv4_prefix", PREFIX_T, {**PREFIX, "B": 65535, "H": 512, "Hkv": 512, "ldq": 1 << 16,
                                                           "ws_bytes": 1 << 62}) == -2
    assert _call(lib, "attn_prefill_sinks", PRE_SINKS_T, {**PRE_SINKS, "nq": 1 << 24, "nk": 1 << 24, "B": 1, "H": 128,
                                                          "ldq": 1 << 14}) == -2


# ---- the binding -----------------------------------------------------------------------------------------------

def calls(on):
    """Calls whose tensors lie where on(name) says."""
    def rows(name, dtype, heads=2):
        return On.make(torch.zeros(4, heads, 64, dtype=dtype), on(name))

    def flat(name, n, dtype=torch.int32):
        return On.make(torch.zeros(n, dtype=dtype), on(name))

    f32, f16, size = torch.float32, torch.float16, qg.kv4_page_bytes(16, 2, 64)
    yield "q k cu lens wq wk freq q_out k_out d_status", lambda: qg.qk_norm_rope(
        0, rows("q", f32), 128, rows("k", f32), 128, 4, flat("cu", 2), flat("lens", 1), 1, 2, 2, 64, flat("wq", 64, f32),
        flat("wk", 64, f32), 1e-6, 64, 0, flat("freq", 32, f32), 1, rows("q_out", f16), 128, rows("k_out", f16), 128,
        flat("d_status", 1))
    yield "q lens pages kv y ws d_status", lambda: qg.attn_decode_kv4_sinks(
        0, rows("q", f32), 128, flat("lens", 4), 4, 1, 2, 2, 64, 0.1, 3, 2, 16, flat("pages", 4), 1, 16, 1,
        flat("kv", size, torch.uint8), rows("y", f32), flat("ws", 256, torch.uint8), 256, flat("d_status", 1))
    yield "q k v cu_q cu_k y d_status", lambda: qg.attn_prefill_sinks(
        1, rows("q", f16), 128, rows("k", f16), 128, rows("v", f16), 128, 4, 4, flat("cu_q", 2), flat("cu_k", 2), 1, 2, 2, 64,
        0.1, 2, 1, rows("y", f16), flat("d_status", 1))
    yield "q lens prefix_pages pages kv y ws d_status", lambda: qg.attn_decode_kv4_prefix(
        0, rows("q", f32), 128, flat("lens", 4), 4, 1, 2, 2, 64, 0.1, 16, 9, flat("prefix_pages", 1), flat("pages", 4), 1, 16, 1,
        flat("kv", size, torch.uint8), rows("y", f32), flat("ws", 256, torch.uint8), 256, flat("d_status", 1))


@pytest.mark.parametrize("which", range(4))
def test_tensors_of_two_devices_or_of_the_host_are_refused(which):
    names = [n for n, _ in calls(lambda name: 0)][which].split()
    for odd in names:
        if odd != names[0]:  # the first says where the call runs
            with pytest.raises(ValueError, match="^%s is on device 1, the call's first tensor on device 0$" % odd):
                [c for _, c in calls(lambda name: 1 if name == odd else 0)][which]()
        with pytest.raises(TypeError):
            [c for _, c in calls(lambda name: -1 if name == odd else 0)][which]()


def test_small_tensors_and_wrong_types_are_refused():
    good = dict(type=0, q=torch.zeros(4, 2, 64), ldq=128, k=torch.zeros(4, 2, 64), ldk=128, n=4,
                cu=torch.zeros(2, dtype=torch.int32), lens=torch.zeros(1, dtype=torch.int32), B=1, H=2, Hkv=2, Dh=64,
                wq=torch.zeros(64), wk=torch.zeros(64), eps=1e-6, R=64, style=0, freq=torch.zeros(32), out_type=2,
                q_out=torch.zeros(4, 2, 64, dtype=torch.bfloat16), ldq_out=128,
                k_out=torch.zeros(4, 2, 64, dtype=torch.bfloat16), ldk_out=128, d_status=torch.zeros(1, dtype=torch.int32))
    for name, x, error in [("q", torch.zeros(3, 2, 64), ValueError), ("k", torch.zeros(4, 2, 32), ValueError),
                           ("q", torch.zeros(4, 2, 64, dtype=torch.float16), TypeError), ("wq", torch.zeros(63), ValueError),
                           ("wk", torch.zeros(64, dtype=torch.float64), TypeError), ("freq", torch.zeros(31), ValueError),
                           ("cu", torch.zeros(1, dtype=torch.int32), ValueError), ("lens", torch.zeros(1), TypeError),
                           ("q_out", torch.zeros(4, 2, 64), TypeError),
                           ("k_out", torch.zeros(4, 1, 64, dtype=torch.bfloat16), ValueError)]:
        args = {n: On.make(v, 0) if isinstance(v, torch.Tensor) else v for n, v in {**good, name: x}.items()}
        with pytest.raises(error, match=name):
            qg.qk_norm_rope(*args.values())
    x, i = On.make(torch.zeros(4, 2, 64), 0), On.make(torch.zeros(8, dtype=torch.int32), 0)
    with pytest.raises(ValueError, match="prefix_pages"):  # 145 positions are ten pages of 16
        qg.attn_decode_kv4_prefix(0, x, 128, i, 4, 1, 2, 2, 64, 0.1, 160, 145, i, i, 1, 16, 1, x, x, x, 0, i)


# ---- the references --------------------------------------------------------------------------------------------

def test_reference_mask_by_hand():
    seen = sh.sees(torch.tensor([-1, 0, 3, 5]), 6, 2, 1)
    assert seen.int().tolist() == [[0] * 6, [1, 0, 0, 0, 0, 0], [1, 0, 1, 1, 0, 0], [1, 0, 0, 0, 1, 1]]
    assert torch.equal(sh.sees(torch.tensor([4]), 6, 0, 3), torch.tensor([[True] * 5 + [False]]))


def test_reference_attention_agrees_with_the_plain_one():
    from tests import attn_helpers as ah
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(n, h, 8, generator=g, dtype=torch.float64) for n, h in ((5, 4), (9, 2), (9, 2)))
    for window in (0, 3):
        got = sh.attend(q, k, v, 0.3, sh.sees(torch.arange(4, 9), 9, window, 0))
        for x, y in zip(got, ah.attend(q, k, v, 0.3, window)):
            assert torch.allclose(x, y, rtol=1e-14, atol=0)


@pytest.mark.parametrize("neighbours", [False, True])
def test_reference_rotation_by_hand(neighbours):
    x = torch.tensor([[[3.0, 4.0, 0.0, 0.0, 5.0]]], dtype=torch.float64)  # mean square 10
    quarter = torch.tensor([math.pi / 2, 0.0], dtype=torch.float64)
    y, pair, angle = sh.rope(x, torch.tensor([1.0, 1, 1, 1, 2], dtype=torch.float64), torch.tensor([1.0]).double(), quarter, 0.0,
                             neighbours)
    want = [-4.0, 3, 0, 0, 10] if neighbours else [0.0, 4, 3, 0, 10]  # (0, 1) or (0, 2) a quarter turn
    assert torch.allclose(y[0, 0] * math.sqrt(10), torch.tensor(want, dtype=torch.float64), atol=1e-12)
    y, _, _ = sh.rope(x, None, torch.tensor([0.0]).double(), quarter, 0.0, neighbours)
    assert torch.allclose(y * math.sqrt(10), x, atol=1e-12)
