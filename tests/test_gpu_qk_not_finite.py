"""Infinities and NaN in the columns that the rotation leaves as they are: by the
formula they stay in their own column of n = x r w and of the weights'
gradient, and reach no pair."""
import pytest
import torch

import lora_adapter_batching_amd as L
from tests import qk_ref as R
from tests.test_gpu_qk import Case

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
FORMS = [(nb, rot, T) for nb in (False, True) for rot in (0, 32, 48) for T in (12, 2050)]


def same(got, want, rel):
    """Infinities and NaN in the same places, the rest as near as two roundings."""
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    bad = torch.isinf(want)
    assert torch.equal(torch.isinf(got), bad) and torch.equal(got[bad], want[bad])
    ok = torch.isfinite(want)
    assert bool(((got[ok] - want[ok]).abs() <= rel * want[ok].abs() + rel).all())


@pytest.mark.parametrize("nb,rot,T", FORMS)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_value(nb, rot, T, value):
    c = Case(T, 3, 1, 64, rot, nb)
    for t, col in ((5, 50), (8, 63)):                                # neighbours 51 and 62 stay as they are
        c.cols(c.x, 0)[t, 64 + col] = value
    out, back = c.forward(), c.backward()
    for kind in (0, 1):
        v, w = c.v64(c.x, kind), c.w[kind].double()
        same(c.v64(out, kind), R.forward(v, w, c.pos, c.freqs, c.eps, nb), 2.0 ** -6)
        dx, _ = R.backward(v, w, c.pos, c.freqs, c.eps, nb, c.v64(c.gr, kind))
        assert torch.equal(torch.isnan(c.v64(back, kind)), torch.isnan(dx))


@pytest.mark.parametrize("nb,rot,T", FORMS)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_weight(nb, rot, T, value):
    c = Case(T, 3, 1, 64, rot, nb)
    c.w[0][50] = value
    c.cols(c.x, 0)[3, 50] = 0                                        # 0 times an infinity is NaN
    out = c.forward()
    for kind in (0, 1):
        same(c.v64(out, kind), R.forward(c.v64(c.x, kind), c.w[kind].double(), c.pos, c.freqs, c.eps, nb), 2.0 ** -6)


@pytest.mark.parametrize("nb,rot,T", FORMS)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_gradient(nb, rot, T, value):
    c = Case(T, 3, 1, 64, rot, nb)
    c.cols(c.gr, 0)[5, 64 + 50] = value
    dw = torch.empty((2, 64), device="cuda")
    back = c.backward(dw, ws=L.new_workspace_qk(c.heads, T))
    for kind in (0, 1):
        dx, dref = R.backward(c.v64(c.x, kind), c.w[kind].double(), c.pos, c.freqs, c.eps, nb, c.v64(c.gr, kind))
        assert torch.equal(torch.isfinite(c.v64(back, kind)), torch.isfinite(dx))
        got = dw[kind].double()
        assert torch.equal(torch.isnan(got), torch.isnan(dref)) and torch.equal(torch.isinf(got), torch.isinf(dref))
        assert int((~torch.isfinite(got)).sum()) == (1 if kind == 0 else 0)
        ok = torch.isfinite(dref)
        assert bool(((got - dref).abs()[ok] <= 1e-3 * T).all())
