"""Products whose sum does not divide into the groups of waves that share it:
some groups multiply stages that no row fills. Every second row (and with 8-bit
weights every second column) is NaN throughout, and so are the bytes behind the
last one; the rows between them are whole numbers, whose products are exact.
One block read past a row's end would be a neighbour's NaN."""
import pytest
import torch

import lora_adapter_batching_amd as L
from lora_adapter_batching_amd import binding as B
from tests.test_gpu_q4 import exact_case as exact_case4
from tests.test_gpu_q8_products import exact_case as exact_case8

pytestmark = pytest.mark.gpu

NAN8 = 0x7F  # e4m3's NaN


def between_nan(x, cls):
    """x in 8 bits, the last of its rows and every second one before it finite,
    the others and the rows behind it NaN, each row right behind the other."""
    T, K = x.shape
    assert T % 2
    blocks = -(-K // 128)
    v = torch.full((T + 3, 128 * blocks), NAN8, dtype=torch.uint8, device="cuda")
    e = torch.full((T + 3, -(-blocks // 4) * 4), 130, dtype=torch.uint8, device="cuda")
    q = cls(v, e, K, rows=T)
    L.q8_quantize(x, q)
    v[1:T:2] = NAN8
    return q


# (tokens, sum, columns, groups): 2, 6, 10 and 14 blocks in four groups, 17 in two
SPLIT4 = [(35, 136, 40, 4), (33, 648, 40, 4), (37, 1160, 72, 4), (35, 1160, 4168, 4), (65, 1672, 6040, 4), (65, 2056, 8296, 2)]


@pytest.mark.parametrize("T,K,N,groups", SPLIT4)
def test_product_on_four_bit_weights(T, K, N, groups):
    k = B.inspect_matmul4(8, T, K, N)
    assert k.groups == groups and -(-K // 128) % groups
    x, w, y0, ref, y064 = exact_case4(8, T, K, N, T + K)
    q, p = between_nan(x, L.Q8Rows), L.new_q4(N, K)
    L.q4_quantize(w, p)
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    for add in (False, True):
        if add:
            y.copy_(y0)
        L.q4_matmul(q, p, y, accumulate=add)
        assert torch.equal(y[::2], (ref + y064 if add else ref).float().to(torch.bfloat16)[::2])
        assert torch.isnan(y[1::2]).all()


@pytest.mark.parametrize("T,K,N", [(129, 640, 11344), (257, 616, 11344)])
def test_empty_loads_of_whole_sums(T, K, N):
    """Stages behind the last block are filled, and not multiplied; a tile of 160 columns has loads of no row."""
    x, w, _, ref, _ = exact_case4(8, T, K, N, T)
    q, p = between_nan(x, L.Q8Rows), L.new_q4(N, K)
    L.q4_quantize(w, p)
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    L.q4_matmul(q, p, y)
    assert torch.equal(y[::2], ref.float().to(torch.bfloat16)[::2]) and torch.isnan(y[1::2]).all()


@pytest.mark.parametrize("T,K,N", [(35, 136, 40), (33, 648, 40), (37, 1160, 72), (35, 1160, 4168)])
def test_product_on_eight_bit_weights(T, K, N):
    k = B.inspect_matmul(T, K, N)
    assert k.groups > 1 and -(-K // 128) % k.groups
    x, w, _, ref, _ = exact_case8(T, K, N, T + K)
    q, p = between_nan(x, L.Q8Rows), L.new_q8_weights(N, K)
    L.q8_quantize(w, p)
    p.values[1::2] = NAN8
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    L.q8_matmul(q, p, y)
    assert torch.equal(y[::2, ::2], ref.float().to(torch.bfloat16)[::2, ::2])
    assert torch.isnan(y[1::2]).all() and torch.isnan(y[:, 1::2]).all()
