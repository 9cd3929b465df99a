"""The longest sums of the product on 4-bit weights, on whole numbers (exact at
every step, see exact_case): one panel, block or exponent too many, too few or
in the wrong place shows, which the bound on random values of that length
cannot say."""
import pytest
import torch

import lora_adapter_batching_amd as L
from tests.q4_products import LONG_SUMS
from tests.test_gpu_q4 import LONG, exact_case, strided, wide_q4
from tests.test_gpu_q8 import wide_q8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,T,K,N", LONG + LONG_SUMS)
def test_long_sums_are_exact(bits, T, K, N):
    x, w, y0, ref, y064 = exact_case(bits, T, K, N, T + K + N)
    q, p = (wide_q4 if bits == 4 else wide_q8)(T, K), wide_q4(N, K)
    (L.q4_quantize if bits == 4 else L.q8_quantize)(x, q)
    L.q4_quantize(w, p)
    big, y = strided(torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda"))
    L.q4_matmul(q, p, y)
    assert torch.equal(y, ref.float().to(torch.bfloat16))
    y.copy_(y0)
    L.q4_matmul(q, p, y, accumulate=True)
    assert torch.equal(y, (ref + y064).float().to(torch.bfloat16))
    assert torch.all(big[T] == 7) and torch.all(big[:, N:] == 7)


@pytest.mark.parametrize("bits,T,K,N", [(8, 100, 31000, 2560), (4, 40, 46592, 2560)])
def test_a_panel_left_out_shows(bits, T, K, N):
    """The comparison itself: without any one of the sum's panels most rows differ."""
    x, w, _, ref, _ = exact_case(bits, T, K, N, T + K + N)
    x, w, ref = x.cpu().double(), w.cpu().double(), ref.cpu()
    want = ref.float().to(torch.bfloat16)
    for panel in (0, 1, -(-K // 128) // 2, -(-K // 128) - 1):
        a, b = 128 * panel, min(K, 128 * panel + 128)
        less = ref - x[:, a:b] @ w[:, a:b].t().contiguous()
        assert float((less.float().to(torch.bfloat16) != want).any(1).float().mean()) > 0.5
