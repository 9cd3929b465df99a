"""The query/key norm's forms for batches past the caches (all rows of a call
256 MB and more): every number of lanes a head takes, both pairings, the
gradient with dweight and without."""
import pytest
import torch

import lora_adapter_batching_amd as L
from tests.test_gpu_qk import Case

pytestmark = pytest.mark.gpu

PAST = 256 << 20


@pytest.mark.parametrize("nb", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,rot", [(33001, 52, 13, 32, 32), (36003, 20, 11, 64, 48), (16385, 32, 8, 128, 128), (10007, 16, 11, 256, 64)])
def test_batches_past_the_caches(T, hq, hk, D, rot, nb):
    matrix = 2 * T * (hq + hk) * D
    assert 2 * matrix >= PAST and T >= 2048                          # read and written; with the gradients' rows half as much again
    c = Case(T, hq, hk, D, rot, nb)
    out = c.forward()
    c.check_forward(out)
    del out
    dw = torch.empty((2, D), device="cuda")
    back = c.backward(dw, ws=L.new_workspace_qk(c.heads, T))
    c.check_backward(back, dw)
    assert torch.equal(back, c.backward())


def test_one_token_in_place_of_many_rows():
    """A single token's row has no stride: an output of one row takes the place of the first of several."""
    c = Case(1, 3, 2, 64, 64)
    want = c.forward()
    q, k = c.x[:, 8:8 + 192], c.x[:, 200:200 + 128]
    assert q.shape[0] == 2
    rest = c.x[1].clone()
    L.qk_norm_rope(q, k, c.heads, c.pos, q[:1], k[:1])
    assert torch.equal(q[:1], c.cols(want, 0)) and torch.equal(k[:1], c.cols(want, 1)) and torch.equal(c.x[1], rest)
