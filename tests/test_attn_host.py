"""The cache and attention calls without a GPU: what they refuse, their sizes, and the test references' own pins.
No call here reaches a kernel launch: every one fails validation first."""
import ctypes

import numpy as np
import pytest

from tests import attn_helpers as ah

VP, I, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
AT = 1 << 40  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import routed_moe_matvec_amd as qg
    return ctypes.CDLL(qg.library_path())


CACHE = dict(pages=AT, max_pages=8, page=16, num_pages=9, kv=AT)
MOVE = dict(type=2, k=AT, ldk=256, v=AT, ldv=256, n=5, cu=AT, lens=AT, B=3, Hkv=2, Dh=128, **CACHE, d_status=AT,
            stream=None)
MOVE_T = [I, VP, I, VP, I, I, VP, VP, I, I, I, VP, I, I, I, VP, VP, VP]
DECODE = dict(type=0, q=AT, ldq=512, lens=AT, B=3, Tq=1, H=4, Hkv=2, Dh=128, scale=0.1, window=0, max_len=128, **CACHE,
              y=AT, ws=AT, ws_bytes=1 << 40, d_status=AT, stream=None)
DECODE_T = [I, VP, I, VP, I, I, I, I, I, F, I, I, VP, I, I, I, VP, VP, VP, SZ, VP, VP]
PREFILL = dict(type=1, q=AT, ldq=512, k=AT, ldk=256, v=AT, ldv=256, nq=7, nk=9, cu_q=AT, cu_k=AT, B=2, H=4, Hkv=2,
               Dh=128, scale=0.1, window=0, y=AT, d_status=AT, stream=None)
PREFILL_T = [I, VP, I, VP, I, VP, I, I, I, VP, VP, I, I, I, I, F, I, VP, VP, VP]

BAD_CACHE = [(dict(Hkv=0), -2), (dict(Dh=96), -2), (dict(Dh=0), -2), (dict(page=24), -2), (dict(page=8), -2),
             (dict(page=131072), -2), (dict(max_pages=0), -2), (dict(num_pages=0), -2), (dict(B=0), -2),
             (dict(B=65536), -2), (dict(pages=None), -1), (dict(kv=None), -1), (dict(lens=None), -1),
             (dict(d_status=None), -1), (dict(kv=AT + 8), -3), (dict(lens=AT + 2), -3), (dict(pages=AT + 1), -3),
             (dict(d_status=AT + 2), -3), (dict(max_pages=1 << 20, page=4096), -2)]
BAD_MOVE = BAD_CACHE + [(dict(type=3), -4), (dict(type=-1), -4), (dict(k=None), -1), (dict(v=None), -1),
                        (dict(cu=None), -1), (dict(n=0), -2), (dict(n=(1 << 24) + 1), -2), (dict(ldk=255), -2),
                        (dict(ldv=248), -2), (dict(ldk=260), -2), (dict(k=AT + 8), -3), (dict(v=AT + 2), -3),
                        (dict(cu=AT + 1), -3), (dict(Hkv=1025, ldk=1 << 20, ldv=1 << 20), -2)]
BAD_DECODE = BAD_CACHE + [(dict(type=5), -4), (dict(q=None), -1), (dict(y=None), -1), (dict(ws=None), -1),
                          (dict(Tq=0), -2), (dict(Tq=17), -2), (dict(H=5), -2), (dict(H=0), -2),
                          (dict(H=1026, ldq=1 << 18), -2), (dict(window=-1), -2), (dict(max_len=0), -2),
                          (dict(max_len=129), -2), (dict(ldq=511), -2), (dict(ldq=514), -2),
                          (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2), (dict(ws_bytes=0), -5),
                          (dict(q=AT + 4), -3), (dict(y=AT + 8), -3), (dict(ws=AT + 8), -3)]
BAD_PREFILL = [(dict(type=0), -4), (dict(type=3), -4)] + [({n: None}, -1) for n in "q k v cu_q cu_k y d_status".split()] + [
    (dict(B=0), -2), (dict(H=3), -2), (dict(Dh=32), -2), (dict(nq=0), -2), (dict(nk=0), -2), (dict(nk=(1 << 24) + 1), -2),
    (dict(window=-2), -2), (dict(scale=float("inf")), -2), (dict(ldq=504), -2), (dict(ldk=252), -2), (dict(ldv=260), -2),
    (dict(Hkv=0), -2), (dict(q=AT + 8), -3), (dict(v=AT + 4), -3), (dict(y=AT + 2), -3), (dict(cu_q=AT + 2), -3)]


def _call(lib, name, types, args):
    f = getattr(lib, name)
    f.restype, f.argtypes = I, types
    return f(*args.values())


@pytest.mark.parametrize("name", ["kv4_append", "kv4_gather"])
def test_cache_moves_refuse(lib, name):
    for change, code in BAD_MOVE:
        assert _call(lib, name, MOVE_T, {**MOVE, **change}) == code, change


def test_decode_refuses(lib):
    for change, code in BAD_DECODE:
        assert _call(lib, "attn_decode_kv4", DECODE_T, {**DECODE, **change}) == code, change


def test_prefill_refuses(lib):
    for change, code in BAD_PREFILL:
        assert _call(lib, "attn_prefill", PREFILL_T, {**PREFILL, **change}) == code, change


def test_launches_too_large_are_refused(lib):
    """2^24 workgroups of 256 threads and more."""
    many = dict(B=65535, Hkv=1024, Dh=256, ldk=1 << 18, ldv=1 << 18)
    for name in ("kv4_append", "kv4_gather"):
        assert _call(lib, name, MOVE_T, {**MOVE, **many, "n": 100}) == -2
    assert _call(lib, "attn_decode_kv4", DECODE_T, {**DECODE, "B": 65535, "H": 512, "Hkv": 512, "ldq": 1 << 16}) == -2
    long = dict(B=64, max_len=1 << 29, page=65536, max_pages=1 << 13, Tq=16, H=512, Hkv=8, ldq=1 << 16)
    assert _call(lib, "attn_decode_kv4", DECODE_T, {**DECODE, **long, "ws_bytes": 1 << 62}) == -2
    assert _call(lib, "attn_prefill", PREFILL_T, {**PREFILL, "B": 65535, "H": 1024, "Hkv": 1024, "ldq": 1 << 17,
                                                  "ldk": 1 << 17, "ldv": 1 << 17, "nq": 70000, "nk": 70000}) == -2


def test_sizes():
    import routed_moe_matvec_amd as qg
    for page, Hkv, Dh in [(16, 1, 64), (64, 8, 128), (65536, 3, 256)]:
        assert qg.kv4_page_bytes(page, Hkv, Dh) == ah.page_bytes(page, Hkv, Dh)
        assert qg.kv4_page_bytes(page, Hkv, Dh) % 16 == 0
    for bad in [(15, 1, 64), (16, 0, 64), (16, 1, 80), (48, 1, 64), (16, 1025, 64)]:
        assert qg.kv4_page_bytes(*bad) == 0
    assert qg.attn_decode_workspace_bytes(3, 1, 4, 2, 128, 128, 0) > 0
    for bad in [(0, 1, 4, 2, 128, 128, 0), (3, 17, 4, 2, 128, 128, 0), (3, 1, 4, 3, 128, 128, 0),
                (3, 1, 4, 2, 100, 128, 0), (3, 1, 4, 2, 128, 0, 0), (3, 1, 4, 2, 128, 128, -1)]:
        assert qg.attn_decode_workspace_bytes(*bad) == 0, bad
    for code in (qg.DEV_BAD_LENGTH, qg.DEV_BAD_PAGE):
        assert qg.qg_status_string(code) not in ("", "unknown status")


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    import routed_moe_matvec_amd as qg
    x = torch.zeros(4, 2, 64)
    i = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(TypeError):
        qg.kv4_append(0, x, 128, x, 128, 4, i, i, 1, 2, 64, i, 1, 16, 1, x, i)
    with pytest.raises(TypeError):
        qg.attn_prefill(1, x, 128, x, 128, x, 128, 4, 4, i, i, 1, 2, 2, 64, 1.0, 0, x, i)


def test_reference_quantizer_by_hand():
    x = np.zeros((1, 64))
    x[0, :12] = [6, 5, -5, 3.5, 2.5, 1.75, 1.25, .75, .25, -.25, 0.2, -0.0]
    x[0, 32] = 6.001
    x[0, 33] = 1.0
    codes, scales = ah.quantize(x)
    assert scales[0].tolist() == [127, 128]
    # 5 between 4 (code 6) and 6 (7), 3.5 between 3 (5) and 4 (6), 2.5: 2 (4) | 3 (5), 1.75: 1.5 (3) | 2 (4), 1.25: 1 (2) | 1.5,
    # .75: .5 (1) | 1 (2), .25: 0 | .5
    assert codes[0, :12].tolist() == [7, 6, 14, 6, 4, 4, 2, 2, 0, 8, 0, 8]
    assert codes[0, 32:34].tolist() == [5, 1]  # 3.0005 and .5 steps of 2
    assert ah.values(codes, scales)[0, :4].tolist() == [6, 4, -4, 4]
    tiny, s = ah.quantize(np.full((1, 32), 2.0**-140))
    assert s[0, 0] == 7 and not tiny.any()


def test_reference_layouts_agree():
    """The vectorised cache writer and the byte-by-byte one."""
    c = ah.Cache([37, 0, 5], 2, 64, 16, 1).fill(2)
    other = np.full_like(c.bytes, 0xFF)
    g = np.random.default_rng(2)
    for b, n in enumerate(c.lens):
        for which in (0, 1):
            codes = g.integers(0, 16, (n, 2, 64)).astype(np.uint8)
            scales = g.integers(123, 128, (n, 2, 2)).astype(np.uint8)
            for t in range(n):
                ah.write(other, 16, 2, 64, c.table[b, t // 16], t % 16, which, codes[t], scales[t])
    assert np.array_equal(other, c.bytes)


def test_reference_attention_by_hand():
    import torch
    q = torch.tensor([[[1.0, 0.0]], [[0.0, 2.0]]], dtype=torch.float64)
    k = torch.tensor([[[0.0, 0.0]], [[np.log(3.0), 0.0]], [[0.0, np.log(2.0) / 2]]], dtype=torch.float64)
    v = torch.tensor([[[1.0, 0.0]], [[5.0, 4.0]], [[0.0, 9.0]]], dtype=torch.float64)
    y, a, big = ah.attend(q, k, v, 1.0, 0)
    assert torch.allclose(y[0, 0], torch.tensor([4.0, 3.0], dtype=torch.float64))          # weights 1/4, 3/4
    assert torch.allclose(y[1, 0], torch.tensor([1.5, 5.5], dtype=torch.float64))          # 1/4, 1/4, 1/2
    y, _, _ = ah.attend(q, k, v, 1.0, 1)
    assert torch.equal(y[:, 0], v[1:, 0])                                                   # each its own key only
    y, _, _ = ah.attend(q, k[:1], v[:1], 1.0, 0)
    assert torch.equal(y[:, 0], torch.tensor([[0.0, 0.0], [1.0, 0.0]], dtype=torch.float64))  # position -1 sees nothing
