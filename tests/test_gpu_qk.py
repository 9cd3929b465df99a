"""The query/key norm with rotation, and its gradient, on the GPU against
plain 64-bit forms (tests/qk_ref.py).

Tolerances, derived before any run, in units of e = 2^-24 (half a step of fp32;
H = 2^-8 half a step of bf16). A head's sum of squares: 8 terms in a lane and up
to five sums over lanes, each e, halved by the root; eps, mean, square root and
reciprocal (one whole step): together r is off by at most 10 e of itself. cos
and sin: the argument is rounded once to half turns (pi e / 2 absolute), the
64-bit product before it loses |p f| 2^-52, and the functions are off by at most
4 steps: 10 e + |p f| 2^-52, absolute. A weight times them one e more, and two
products, their sum and r four. So
    out: (10 + 10 + 1 + 4) e, taken as 32 e + |p f| 2^-52, of r (|w_i x_i| + |w_j x_j|).
The gradient, with G = |g_i| + |g_j|, a = r |x|, S = mean(G |w| a):
    m off by 13 e G; g = m w by 14 e; x r by 12 e of a; their mean's sum of 8 and up
    to five more by 14 e, so mean(g x r) by 41 e of S; dx by
    r (32 e G |w| + 64 e a S), the rotation's |p f| 2^-52 in either;
    dw: 26 e of G a each and its sum: a lane's own tokens in turn (at most T / 256 + 2 of
    them times the head groups), 4 lanes' steps, 2 waves' and up to 48 of workgroups.
Rounding to bf16 is half a step: H of the value, and 2^-134 below 2^-126, where bf16's
step stays 2^-133 (heads near 2^122 have gradients there).
"""
import numpy as np
import pytest
import torch

import lora_adapter_batching_amd as L
from lora_adapter_batching_amd import binding as B
from tests import qk_ref as R

pytestmark = pytest.mark.gpu

BF, E, LEAST = 2.0 ** -8, 2.0 ** -24, 2.0 ** -134


class Case:
    def __init__(self, T, hq, hk, D, rot, nb=False, seed=0, eps=1e-6, far=131072, base=1e6):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + T * 1000 + D)
        self.T, self.H, self.D, self.rot, self.nb, self.eps, self.g = T, (hq, hk), D, rot, nb, eps, g
        # queries, keys and values of a token side by side, behind other columns
        ld = 8 + (hq + 2 * hk) * D
        mk = lambda: torch.randn((T + 1, ld), generator=g, device="cuda") * torch.exp(torch.randn((T + 1, 1), generator=g, device="cuda"))  # noqa: E731
        self.x, self.gr = mk().to(torch.bfloat16), mk().to(torch.bfloat16)
        w = lambda: (1 + 0.3 * torch.randn((D,), generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
        self.w = (w(), w())
        self.freqs = base ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / max(1, rot // 2))
        self.pos = torch.randint(-far, far + 1, (T,), generator=g, device="cuda").int()
        if T > 2:
            self.pos[0], self.pos[1] = 0, far
        self.heads = L.QKHeads(hq, hk, D, self.w[0] if hq else None, self.w[1] if hk else None, self.freqs, eps=eps, neighbours=nb)

    def cols(self, t, kind):
        a = 8 + (0 if kind == 0 else self.H[0] * self.D)
        return t[:self.T, a:a + self.H[kind] * self.D] if self.H[kind] else None

    def wide(self, fill=7.0):
        return torch.full_like(self.x, fill)

    def v64(self, t, kind):
        return self.cols(t, kind).double().view(self.T, self.H[kind], self.D)

    def slip(self):
        """|p f| 2^-52 of every column (0 where nothing turns)."""
        a = (self.pos.double().abs()[:, None, None] * self.freqs) * 2.0 ** -52
        one = torch.zeros((self.T, 1, self.D), dtype=torch.float64, device="cuda")
        i, j = (t.cuda() for t in R.pairs(self.D, self.rot, self.nb))
        one[..., i], one[..., j] = a, a
        return one

    def forward(self, out=None, ko=None):
        big = self.wide() if out is None else out
        L.qk_norm_rope(self.cols(self.x, 0), self.cols(self.x, 1), self.heads, self.pos, self.cols(big, 0), self.cols(big, 1))
        return big

    def check_forward(self, big, x=None):
        x = self.x if x is None else x
        for kind in (0, 1):
            if not self.H[kind]:
                continue
            v, w = self.v64(x, kind), self.w[kind].double()
            ref = R.forward(v, w, self.pos, self.freqs, self.eps, self.nb)
            r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + self.eps)
            n = (v * r * w).abs()
            err = (32 * E + self.slip()) * (n + R.other(n, self.rot, self.nb))
            held(self.v64(big, kind), ref, BF * (ref.abs() + err) + err + LEAST, f"out {kind}")
        self.untouched(big)

    def untouched(self, big):
        n = 8 + sum(self.H) * self.D
        assert torch.all(big[self.T] == 7) and torch.all(big[:, :8] == 7) and torch.all(big[:, n:] == 7)

    def backward(self, dw=None, flags=0, ws=None):
        big = self.wide()
        L.qk_norm_rope_backward(self.cols(self.x, 0), self.cols(self.x, 1), self.heads, self.pos, self.cols(self.gr, 0), self.cols(self.gr, 1),
                                self.cols(big, 0), self.cols(big, 1), dweight=dw, flags=flags, ws=ws)
        return big

    def check_backward(self, big, dw=None, dw0=0.0):
        for kind in (0, 1):
            if not self.H[kind]:
                if dw is not None:
                    assert torch.all(dw[kind] == dw0)
                continue
            v, w, g = self.v64(self.x, kind), self.w[kind].double(), self.v64(self.gr, kind)
            dx, dref = R.backward(v, w, self.pos, self.freqs, self.eps, self.nb, g)
            r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + self.eps)
            G, a = g.abs() + R.other(g.abs(), self.rot, self.nb), (v * r).abs()
            S = (G * w.abs() * a).mean(-1, keepdim=True)
            err = r * ((32 * E + self.slip()) * G * w.abs() + (64 * E + self.slip().amax(-1, keepdim=True)) * a * S)
            held(self.v64(big, kind), dx, BF * (dx.abs() + err) + err + LEAST, f"dx {kind}")
            if dw is not None:
                mag = (G * a).sum((0, 1)) + abs(dw0)
                steps = (self.T / 256 + 2) * (self.H[kind] * max(32, self.D) / 512 + 1) + 56
                held(dw[kind].double(), dref + dw0, (26 + steps) * E * mag + (self.slip() * G * a).sum((0, 1)), f"dw {kind}")
        self.untouched(big)


def held(got, ref, tol, what):
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref)), what
    ok = torch.isfinite(ref)
    bad = ((got - ref).abs() > tol) & ok
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((got - ref).abs()[bad].max())}"


# tokens around the borders between the kernels' forms, every number of lanes a
# head takes, heads that do not fill a wave's groups, one kind alone, part turned
SHAPES = [(1, 1, 1, 8, 0), (1, 32, 8, 128, 128), (2, 3, 1, 16, 16), (3, 5, 2, 24, 16), (5, 9, 9, 32, 32), (17, 0, 3, 40, 32), (50, 5, 0, 48, 48),
          (64, 32, 8, 128, 128), (33, 17, 1, 64, 64), (100, 7, 3, 72, 64), (333, 12, 3, 64, 32), (511, 6, 2, 80, 80), (513, 4, 4, 96, 48),
          (700, 2, 1, 120, 112), (300, 8, 1, 136, 128), (257, 3, 2, 192, 64), (1000, 2, 2, 200, 192), (129, 4, 1, 256, 256), (40, 70, 33, 64, 16),
          (2047, 4, 1, 64, 64), (2048, 4, 1, 64, 64), (2049, 5, 3, 128, 128), (3075, 3, 1, 256, 128), (5000, 16, 2, 32, 32), (4099, 0, 1, 8, 0)]


@pytest.mark.parametrize("nb", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,rot", SHAPES)
def test_forward_and_gradient(T, hq, hk, D, rot, nb):
    c = Case(T, hq, hk, D, rot, nb)
    big = c.forward()
    c.check_forward(big)
    assert torch.equal(big, c.forward())
    ws = L.new_workspace_qk(c.heads, T)
    ws.fill_(255)                                                    # in any state
    dw = torch.full((2, D), float("nan"), device="cuda")
    back = c.backward(dw, ws=ws)
    c.check_backward(back, dw)
    alone = c.backward()                                             # without the weights' gradient
    assert torch.equal(back, alone)
    more, dw2 = torch.full((2, D), 3.0, device="cuda"), torch.empty((2, D), device="cuda")
    c.backward(more, flags=L.GRAD_ACCUMULATE, ws=ws)
    c.check_backward(back, more, 3.0)
    c.backward(dw2, ws=ws)
    assert torch.equal(dw, dw2)                                      # the same bits again


@pytest.mark.parametrize("T,hq,hk,D", [(16384, 32, 8, 128), (12000, 16, 16, 256), (30000, 20, 4, 64)])
def test_large_batches(T, hq, hk, D):
    """Batches past the caches."""
    c = Case(T, hq, hk, D, D)
    c.check_forward(c.forward())
    dw = torch.empty((2, D), device="cuda")
    c.check_backward(c.backward(dw, ws=L.new_workspace_qk(c.heads, T)), dw)


@pytest.mark.parametrize("T", [60, 2100])
def test_far_positions_and_long_waves(T):
    """Angles of 2^31 radians and frequencies from 1 down to 1e-6 of it."""
    c = Case(T, 3, 2, 64, 64, far=2 ** 31 - 1)
    c.pos[2:4] = torch.tensor([-2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("T", [40, 2100])
@pytest.mark.parametrize("nb", [False, True])
def test_in_place(T, nb):
    c = Case(T, 6, 2, 128, 96, nb)
    want, x0 = c.forward(), c.x.clone()
    L.qk_norm_rope(c.cols(c.x, 0), c.cols(c.x, 1), c.heads, c.pos, c.cols(c.x, 0), c.cols(c.x, 1))
    for kind in (0, 1):
        assert torch.equal(c.cols(c.x, kind), c.cols(want, kind))
    n = 8 + 8 * 128
    assert torch.equal(c.x[:, :8], x0[:, :8]) and torch.equal(c.x[:, n:], x0[:, n:]) and torch.equal(c.x[T], x0[T])


@pytest.mark.parametrize("T", [12, 2050])
@pytest.mark.parametrize("nb", [False, True])
def test_sizes_at_the_ends_of_the_type(T, nb):
    """Heads whose squares leave fp32's range either way, heads of zeros, one
    value alone: the norm is that of the 64-bit form."""
    c = Case(T, 4, 1, 64, 64, nb, eps=1e-12)
    x = c.v64(c.x, 0)
    for t, f in [(0, 2.0 ** 100), (1, 2.0 ** 63), (2, 2.0 ** -60), (3, 0.0), (4, 2.0 ** -126), (5, 2.0 ** 122)]:
        c.cols(c.x, 0)[t] = (x[t] * f / max(1e-30, float(x[t].abs().max()))).reshape(-1).to(torch.bfloat16)
    c.cols(c.x, 0)[6] = 0
    c.cols(c.x, 0)[6, 70] = 3e38
    c.cols(c.x, 0)[7, :64] = torch.finfo(torch.bfloat16).max
    # (an x smaller than 2^-126 of its unit has no digits to lose: subnormal products round at 2^-149)
    c.check_forward(c.forward())
    assert not c.cols(c.forward(), 0)[3].any()
    g = c.v64(c.gr, 0)
    for t in (2, 4):                                                 # r is up to 1e6 there: gradients that stay in range
        c.cols(c.gr, 0)[t] = (g[t] * 2.0 ** -20).reshape(-1).to(torch.bfloat16)
    dw = torch.empty((2, 64), device="cuda")
    c.check_backward(c.backward(dw, ws=L.new_workspace_qk(c.heads, T)), dw)


@pytest.mark.parametrize("T", [12, 2050])
@pytest.mark.parametrize("x,w,g,eps", [(50, 100, 60, 1e-6), (50, 100, -80, 1e30), (60, -60, 100, 1e-6), (-40, 110, -50, 1e-30)])
@pytest.mark.parametrize("nb", [False, True])
def test_products_past_the_type_on_the_way(T, x, w, g, eps, nb):
    """Values, weights and gradients (powers of two) of which two multiplied leave
    fp32's range where the results do not; the largest eps."""
    c = Case(T, 4, 1, 64, 64, nb, eps=eps)
    c.x, c.gr = ((t.double() * 2.0 ** f).to(torch.bfloat16) for t, f in ((c.x, x), (c.gr, g)))
    c.w = tuple((v.double() * 2.0 ** w).to(torch.bfloat16) for v in c.w)
    c.heads = L.QKHeads(4, 1, 64, *c.w, c.freqs, eps=eps, neighbours=nb)
    c.check_forward(c.forward())
    dw = torch.empty((2, 64), device="cuda")
    c.check_backward(c.backward(dw, ws=L.new_workspace_qk(c.heads, T)), dw)


@pytest.mark.parametrize("T", [30, 2050])
def test_not_finite_stays_in_its_head(T):
    c = Case(T, 5, 2, 64, 32)
    clean, back = c.forward(), c.backward()
    c.cols(c.x, 0)[1, 64 + 3], c.cols(c.x, 1)[2, 64 + 60], c.cols(c.x, 0)[T - 1, 0] = float("nan"), float("inf"), float("-inf")
    # (the formula: 1 / inf is 0, so an infinity leaves zeros and, at itself and its pair, 0 * inf)
    exact = lambda k, fwd: (R.forward(c.v64(c.x, k), c.w[k].double(), c.pos, c.freqs, c.eps, False) if fwd else  # noqa: E731
                            R.backward(c.v64(c.x, k), c.w[k].double(), c.pos, c.freqs, c.eps, False, c.v64(c.gr, k))[0])
    for fwd, big, ref in ((True, c.forward(), clean), (False, c.backward(), back)):
        for kind, marks in ((0, [(1, 1), (T - 1, 0)]), (1, [(2, 1)])):
            got, want = (c.cols(t, kind).view(T, c.H[kind], 64).clone() for t in (big, ref))
            formula = exact(kind, fwd)
            for t, h in marks:
                assert torch.isnan(formula[t, h]).any()
                assert torch.equal(torch.isnan(got[t, h]), torch.isnan(formula[t, h]))
                assert not got[t, h][~torch.isnan(got[t, h])].any()
                got[t, h] = want[t, h] = 0
            assert torch.equal(got, want)
    # the weights' gradients take it where the kind's sums hold it
    c.cols(c.x, 1)[2, 64 + 60] = 0
    dw = torch.empty((2, 64), device="cuda")
    c.backward(dw, ws=L.new_workspace_qk(c.heads, T))
    assert torch.isnan(dw[0]).all() and torch.isfinite(dw[1]).all()


def test_no_tokens():
    c = Case(3, 2, 1, 64, 64)
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    e = lambda h: torch.empty((0, h * 64), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    L.qk_norm_rope(e(2), e(1), c.heads, none, e(2), e(1))
    dw = torch.full((2, 64), 5.0, device="cuda")
    args = (e(2), e(1), c.heads, none, e(2), e(1), e(2), e(1))
    L.qk_norm_rope_backward(*args, dweight=dw, flags=L.GRAD_ACCUMULATE)
    assert torch.all(dw == 5)
    L.qk_norm_rope_backward(*args, dweight=dw)
    assert not dw.any()


def test_gradient_against_differences_of_the_kernel():
    """The forward's own outputs, at steps whose rounding they show: sum(out * g)
    moves by dx * step and dw * step, off by the outputs' roundings."""
    c = Case(4, 2, 1, 32, 32, eps=1e-3)
    g = c.v64(c.gr, 0)
    dw = torch.empty((2, 32), device="cuda")
    dx = c.v64(c.backward(dw, ws=L.new_workspace_qk(c.heads, 4)), 0)
    loss = lambda: (c.v64(c.forward(), 0) * g).sum((1, 2))  # noqa: E731
    lim = lambda: 2 * BF * (c.v64(c.forward(), 0).abs() * g.abs()).sum((1, 2)).max()  # noqa: E731
    for t, h, d in [(0, 0, 3), (2, 1, 31)]:
        col, x0 = h * 32 + d, float(c.cols(c.x, 0)[t, h * 32 + d])
        step = 2.0 ** np.floor(np.log2(abs(x0) + 2.0 ** -6)) / 4       # x0 +- step are bf16 numbers
        vals = []
        for s in (step, -step):
            c.cols(c.x, 0)[t, col] = x0 + s
            vals.append((float(c.cols(c.x, 0)[t, col]), float(loss()[t])))
        v = c.v64(c.x, 0)[t:t + 1]
        c.cols(c.x, 0)[t, col] = x0
        (a, la), (b, lb) = vals
        # the formula between the two points: its own differences in 64 bits
        ref = []
        for at in (a, b):
            v[0, h, d] = at
            ref.append(float((R.forward(v, c.w[0].double(), c.pos[t:t + 1], c.freqs, c.eps, False) * g[t:t + 1]).sum()))
        assert abs((la - lb) - (ref[0] - ref[1])) <= float(lim())
        # and the gradient is their slope up to the second difference
        mid = c.v64(c.x, 0)[t:t + 1]
        slope = (ref[0] - ref[1]) / (a - b)
        curve = abs(ref[0] + ref[1] - 2 * float((R.forward(mid, c.w[0].double(), c.pos[t:t + 1], c.freqs, c.eps, False) * g[t:t + 1]).sum()))
        assert abs(float(dx[t, h, d]) - slope) <= 2 * BF * abs(slope) + 4 * curve / abs(a - b) + 1e-3


def test_calls_on_two_streams_and_shared_weights():
    jobs = [(Case(300, 8, 2, 128, 128, seed=1), torch.cuda.Stream()), (Case(2500, 4, 4, 64, 64, seed=2), torch.cuda.Stream())]
    out = []
    for c, _ in jobs:
        out.append([c.wide(), c.wide(), torch.zeros((2, c.D), device="cuda"), L.new_workspace_qk(c.heads, c.T)])
    torch.cuda.synchronize()
    for _ in range(4):
        for (c, s), (y, b, dw, ws) in zip(jobs, out):
            L.qk_norm_rope(c.cols(c.x, 0), c.cols(c.x, 1), c.heads, c.pos, c.cols(y, 0), c.cols(y, 1), stream=s)
            L.qk_norm_rope_backward(c.cols(c.x, 0), c.cols(c.x, 1), c.heads, c.pos, c.cols(c.gr, 0), c.cols(c.gr, 1), c.cols(b, 0), c.cols(b, 1),
                                    dweight=dw, ws=ws, stream=s)
    torch.cuda.synchronize()
    for (c, _), (y, b, dw, _) in zip(jobs, out):
        c.check_forward(y)
        c.check_backward(b, dw)


@pytest.mark.parametrize("T", [90, 2100])
def test_captured_and_replayed(T):
    c = Case(T, 6, 2, 128, 128)
    y, b, dw, ws = c.wide(), c.wide(), torch.zeros((2, 128), device="cuda"), L.new_workspace_qk(c.heads, T)

    def step():
        L.qk_norm_rope(c.cols(c.x, 0), c.cols(c.x, 1), c.heads, c.pos, c.cols(y, 0), c.cols(y, 1))
        L.qk_norm_rope_backward(c.cols(c.x, 0), c.cols(c.x, 1), c.heads, c.pos, c.cols(c.gr, 0), c.cols(c.gr, 1), c.cols(b, 0), c.cols(b, 1),
                                dweight=dw, ws=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        c.x.copy_(torch.randn(c.x.shape, generator=c.g, device="cuda"))
        c.pos.add_(17 * k)
        c.w[0].mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, b, dw)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, (y, b, dw)))
    c.check_forward(y)
    c.check_backward(b, dw)


def test_workspace_too_small_is_refused():
    c = Case(40, 2, 1, 64, 64)
    dw = torch.zeros((2, 64), device="cuda")
    for ws, status in ((L.new_workspace_qk(c.heads, 39), B.LORA_WORKSPACE_TOO_SMALL), (None, B.LORA_INVALID_ARGUMENT)):
        with pytest.raises(B.LoraError) as e:
            c.backward(dw, ws=ws)
        assert e.value.status == status
    assert not dw.any()


def test_rows_past_2_to_32_elements():
    """Row offsets above 2^32 elements: the last tokens of a matrix of 4.4e9."""
    T, ld = 270_000, 16384
    x = torch.zeros((T, ld), dtype=torch.bfloat16, device="cuda")
    c = Case(6, 1, 1, 128, 128)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[-6:] = c.pos
    x[-6:, :128], x[-6:, 128:256] = c.cols(c.x, 0), c.cols(c.x, 1)
    out = torch.zeros((T, 256), dtype=torch.bfloat16, device="cuda")
    L.qk_norm_rope(x[:, :128], x[:, 128:256], c.heads, pos, out[:, :128], out[:, 128:])
    big = c.wide()
    c.cols(big, 0)[:], c.cols(big, 1)[:] = out[-6:, :128], out[-6:, 128:]
    c.check_forward(big)
    assert not out[:-6].any()
