"""Errors over whole sequences, against the norm of the output: attn_decode_kv4 as fp32 arithmetic, with a model of the kernel's
operands that shows what its error would be with one part of the queries or weights less, and attn_prefill's two roundings.

The limit of the former.  A score of size s is the sum of at most 24 products of 32 channels, whose roundings are independent: sqrt(24) * 2^-24 of
the largest partial sum, which is below 4 here: 1.2e-6.  An output is the sum of 3 products for each 32 positions, in up to 128
steps: sqrt(384) * 2^-24, 1.2e-6.  The exponential is off by 2^-23.  Together 1.7e-6, and half as much again: 2.5e-6."""
import numpy as np
import pytest
import torch

from tests import attn_helpers as ah
from tests.gpu_util import progress

LIMIT = 2.5e-6
LENS = [300, 640, 2500, 9001]
SHAPES = [(Dh, G) for Dh in (64, 128, 256) for G in (1, 4, 16)]
Q_PARTS = {0: 3, 1: 2, 2: 1}


def problem(Dh, G, type):
    """A cache of ordinary values and queries [sequences, G, Dh] (CPU)."""
    c = ah.Cache(LENS, 1, Dh, 64, 51).fill(52)
    g = torch.Generator().manual_seed(53)
    return c, torch.randn(len(LENS), G, Dh, generator=g).to(ah.TYPES[type])


def error(y, c, q, b):
    """Relative error of sequence b's output y [G, Dh], over its norm."""
    k, v = (torch.from_numpy(x[b]) for x in (c.k, c.v))
    ref = ah.attend(q[b:b + 1].double(), k, v, c.Dh**-0.5, 0)[0][0]
    return float((y.double() - ref).norm() / ref.norm())


def nearest_parts(x, n):
    """The sum of n bf16 numbers that each take the nearest to what is left of x."""
    total = torch.zeros_like(x)
    for _ in range(n):
        total = total + (x - total).float().bfloat16().double()
    return total


def cut_parts(x, n):
    """The sum of n bf16 numbers that each take the next eight bits of x (fp32), cut off."""
    total = torch.zeros_like(x)
    for _ in range(n):
        left = (x - total).float().view(torch.int32) & -65536
        total = total + left.view(torch.float32).double()
    return total


def model(c, q, b, q_parts, w_parts):
    """The output with operands in parts and everything else in 64 bits."""
    k, v = (torch.from_numpy(x[b])[:, 0] for x in (c.k, c.v))
    s = nearest_parts(q[b].double(), q_parts) @ k.t() * c.Dh**-0.5
    w = torch.exp(s - s.amax(1, keepdim=True)).float().double()
    return cut_parts(w, w_parts) @ v / w.sum(1, keepdim=True)


@pytest.mark.parametrize("Dh,G", SHAPES)
@pytest.mark.parametrize("type", [0, 1, 2])
def test_a_part_less_passes_the_limit(Dh, G, type):
    c, q = problem(Dh, G, type)

    def worst(q_parts, w_parts):
        return max(error(model(c, q, b, q_parts, w_parts), c, q, b) for b in range(len(LENS)))

    assert worst(Q_PARTS[type], 3) < LIMIT / 10
    assert worst(Q_PARTS[type], 2) > LIMIT
    if type != 2:
        assert worst(Q_PARTS[type] - 1, 3) > LIMIT


@pytest.mark.gpu
@pytest.mark.parametrize("Dh,G", SHAPES)
@pytest.mark.parametrize("type", [0, 1, 2])
def test_decode_error_of_the_norm(Dh, G, type):
    import routed_moe_matvec_amd as qg
    progress("decode error of the norm Dh %d G %d type %d" % (Dh, G, type))
    c, q = problem(Dh, G, type)
    i32 = dict(dtype=torch.int32, device="cuda")
    nb = qg.attn_decode_workspace_bytes(len(LENS), 1, G, 1, Dh, max(LENS), 0)
    ws, st = torch.empty(nb, dtype=torch.uint8, device="cuda"), torch.zeros(1, **i32)
    y = torch.empty(len(LENS), G, Dh, device="cuda")
    qg.attn_decode_kv4(type, q.cuda(), G * Dh, torch.tensor(LENS, **i32), len(LENS), 1, G, 1, Dh, Dh**-0.5, 0, max(LENS),
                       *c.device(), y, ws, nb, st)
    assert int(st) == 0
    y = y.cpu()
    errs = [error(y[b], c, q, b) for b in range(len(LENS))]
    assert np.max(errs) < LIMIT, errs


@pytest.mark.gpu
@pytest.mark.parametrize("Dh", [64, 128, 256])
@pytest.mark.parametrize("H,lens", [(1, [700, 90]), (32, [600, 31, 257]), (64, [1500, 300, 1])])
@pytest.mark.parametrize("type", [1, 2])
def test_prefill_error_of_the_norm(type, H, lens, Dh):
    """Weights and outputs are each rounded to the type once: an error of at most eps / 2 of each, spread evenly, is eps / 2 / sqrt(3)
    in the mean square, and both together less than eps / 2 of the norm.  Every run gives the same bits."""
    import routed_moe_matvec_amd as qg
    progress("prefill error of the norm H %d lens %s Dh %d type %d" % (H, lens, Dh, type))
    dt, n = ah.TYPES[type], sum(lens)
    g = torch.Generator(device="cuda")
    g.manual_seed(54)
    q, k, v = (torch.randn(n, heads, Dh, generator=g, device="cuda").to(dt) for heads in (H, 1, 1))
    cu, st = ah.cumulative(lens), torch.zeros(1, dtype=torch.int32, device="cuda")
    ys = []
    for _ in range(3):
        ys.append(torch.full((n, H, Dh), 7.0, dtype=dt, device="cuda"))
        qg.attn_prefill(type, q, H * Dh, k, Dh, v, Dh, n, n, cu, cu, len(lens), H, 1, Dh, 2 * Dh**-0.5, 0, ys[-1], st)
    assert int(st) == 0 and torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
    at = 0
    for m in lens:
        rows = slice(at, at + m)
        ref = ah.attend(q[rows].double(), k[rows].double(), v[rows].double(), 2 * Dh**-0.5, 0)[0]
        err = float((ys[0][rows].double() - ref).norm() / ref.norm())
        assert err < torch.finfo(dt).eps / 2, (m, err)
        at += m
