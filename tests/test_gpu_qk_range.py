"""The gradient of the query/key norm where a gradient times a weight leaves
fp32's range, or its normal numbers, and the result does not. Tolerances are
those of tests/test_gpu_qk.py (derived there); columns are held to 2^-50 of what
their head's largest gradient and largest weight give besides, which is far
below them in all cases but the one that says so."""
import pytest
import torch

import lora_adapter_batching_amd as L
from tests import qk_ref as R
from tests.test_gpu_qk import BF, E, LEAST, Case, held

pytestmark = pytest.mark.gpu


def check_dweight(c, dw):
    """As in Case.check_backward, where fp32 holds the sum: a partial sum of any order is at most
    mag = sum (|g_i| + |g_j|) r |x|, so below 2^127 none leaves the range. Past that a
    partial sum can, and the column is not compared (gradients near 2^127: the true sum itself is
    then above 2^128)."""
    for kind in (0, 1):
        v, w, g = c.v64(c.x, kind), c.w[kind].double(), c.v64(c.gr, kind)
        _, ref = R.backward(v, w, c.pos, c.freqs, c.eps, c.nb, g)
        a = (v / torch.sqrt((v * v).mean(-1, keepdim=True) + c.eps)).abs()
        G = g.abs() + R.other(g.abs(), c.rot, c.nb)
        mag = (G * a).sum((0, 1))
        steps = (c.T / 256 + 2) * (c.H[kind] * max(32, c.D) / 512 + 1) + 56
        # (2^-149: a sum of subnormal numbers is rounded at half of it each step)
        tol = (26 + steps) * E * mag + (c.slip() * G * a).sum((0, 1)) + c.T * c.H[kind] * 2.0 ** -149
        ok = mag < 2.0 ** 127
        held(dw[kind].double()[ok], ref[ok], tol[ok], f"dw {kind}")


def check_dx(c, big, apart=0.0):
    """As in Case.check_backward; results past bf16's range (from halfway between its largest number
    and 2^128 on) are infinities. apart: what a column is held to besides, of its head's largest
    gradient times the largest weight times r."""
    for kind in (0, 1):
        v, w, g = c.v64(c.x, kind), c.w[kind].double(), c.v64(c.gr, kind)
        dx, _ = R.backward(v, w, c.pos, c.freqs, c.eps, c.nb, g)
        r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + c.eps)
        G, a = g.abs() + R.other(g.abs(), c.rot, c.nb), (v * r).abs()
        S = (G * w.abs() * a).mean(-1, keepdim=True)
        err = r * ((32 * E + c.slip()) * G * w.abs() + (64 * E + c.slip().amax(-1, keepdim=True)) * a * S)
        err = err + apart * r * g.abs().amax(-1, keepdim=True) * w.abs().max()
        got, top = c.v64(big, kind), 2.0 ** 128 - 2.0 ** 119
        over, under = dx.abs() - err >= top, dx.abs() + err < top
        assert torch.equal(got[over], torch.copysign(torch.full_like(dx, float("inf")), dx)[over])
        held(got[under], dx[under], (BF * (dx.abs() + err) + err + LEAST)[under], f"dx {kind}")
    c.untouched(big)


def scaled(T, hq, hk, D, nb, w, eps):
    c = Case(T, hq, hk, D, D - D % 16, nb, eps=eps)
    c.w = tuple((v.double() * 2.0 ** w).to(torch.bfloat16) for v in c.w)
    c.heads = L.QKHeads(hq, hk, D, *c.w, c.freqs, eps=eps, neighbours=nb)
    return c


# powers of two of values, weights and gradients. Weights within 2^-32 .. 2^32
# reach the kernels as they are: their products with the gradients passed 2^128 (the
# first four) or fell below 2^-126.
@pytest.mark.parametrize("T", [12, 2050])
@pytest.mark.parametrize("x,w,g,eps", [(60, 20, 110, 1e-6), (60, -20, 125, 1e-6), (10, 31, 90, 1e-6), (40, 31, 100, 1e-6), (-40, -31, -115, 1e-30),
                                       (-40, -20, -120, 1e-30), (-55, 20, -130, 1e-33), (0, 0, -64, 1e-6), (0, 0, 63, 1e-6)])
@pytest.mark.parametrize("nb", [False, True])
def test_gradients_and_weights_of_any_size(T, x, w, g, eps, nb):
    c = scaled(T, 4, 1, 64, nb, w, eps)
    c.x = (c.x.double() * 2.0 ** x).to(torch.bfloat16)
    gr = c.gr.double()
    if g > 120:                                                      # (keeps the values themselves in range)
        gr = gr.clamp(-4, 4)
    c.gr = (gr * 2.0 ** g).to(torch.bfloat16)
    c.check_forward(c.forward())
    dw = torch.empty((2, 64), device="cuda")
    back = c.backward(dw, ws=L.new_workspace_qk(c.heads, T))
    c.check_backward(back)
    check_dweight(c, dw)
    assert torch.equal(back, c.backward())


@pytest.mark.parametrize("T", [9, 2049])
@pytest.mark.parametrize("w", [-31, 0, 31, 60])
@pytest.mark.parametrize("D", [24, 64, 128, 256])
def test_heads_of_different_sizes_side_by_side(T, w, D):
    """Heads that share a wave, each at a size of its own, some without any gradient."""
    c = scaled(T, 8, 2, D, False, w, 1e-6)
    powers = torch.tensor([-125, 70, 0, -64, -65, 63, 64, -20, 100, -100], dtype=torch.float64, device="cuda")
    big = c.gr[:, 8:8 + 10 * D].double().view(-1, 10, D)
    big = big * torch.exp2(powers)[None, :, None]
    big[::3, 2] = 0
    c.gr[:, 8:8 + 10 * D] = big.to(torch.bfloat16).view(-1, 10 * D)
    x = c.x[:, 8:8 + 10 * D].double().view(-1, 10, D)                # r keeps dx in range
    x[:, [1, 6, 8]] *= 2.0 ** 50
    c.x[:, 8:8 + 10 * D] = x.to(torch.bfloat16).view(-1, 10 * D)
    check_dx(c, c.backward())


@pytest.mark.parametrize("T", [5, 2050])
@pytest.mark.parametrize("nb", [False, True])
def test_largest_gradients(T, nb):
    """Gradients at the end of the type: turned, they are up to 1.4 times as large."""
    c = scaled(T, 4, 1, 64, nb, -20, 1e-6)
    c.gr = torch.copysign(torch.full_like(c.gr, torch.finfo(torch.bfloat16).max), c.gr)
    c.check_backward(c.backward())


@pytest.mark.parametrize("T", [7, 2050])
@pytest.mark.parametrize("flip", [False, True])
def test_columns_apart(T, flip):
    """One head's gradients and weights over the whole of the type: each column is right to its
    rounding and to 2^-50 of the largest gradient times the largest weight times r."""
    c = Case(T, 4, 1, 64, 64, eps=1e-6)
    spread = torch.linspace(-100, 20, 64, dtype=torch.float64, device="cuda").round()
    c.w = tuple((v.double() * torch.exp2(spread)).to(torch.bfloat16) for v in c.w)
    c.heads = L.QKHeads(4, 1, 64, *c.w, c.freqs, eps=c.eps)
    p = spread.flip(0) if flip else spread
    for kind in (0, 1):
        c.cols(c.gr, kind).copy_((c.v64(c.gr, kind) * torch.exp2(p)).reshape(T, -1))
    check_dx(c, c.backward(), 2.0 ** -50)
