"""Every kernel of the 8-bit product, stored and added to, every column of y.

Whole numbers under power-of-two scales. x and w hold small whole numbers, few
enough that a sum stays far below 2^24; row t of x, block b of the sum and
128-row block c of w are scaled by powers of two of their own, block b by
2^p(b) in x and 2^-p(b) in w. The product is then 2^(a(t) + c(j)) times a whole
number, and exact at every step: e4m3 holds the values, the matrix unit's
groups hold products of 1, 2 and 4, fp32 holds the sums. So y is the bf16
rounding of the exact sum, whatever the order, and one value, exponent or
block too many, too few or in the wrong place shows.

The blocks' exponents differ, so a store's exponent bytes say which block they
belong to; random values (last test) meet the tolerance of test_gpu_q8.py."""
import numpy as np
import pytest
import torch

import lora_adapter_batching_amd as L
from tests import q8_ref as R
from tests.q8_products import PRODUCTS
from tests.test_gpu_q8 import LONG, strided, wide_q8

pytestmark = pytest.mark.gpu

BF, F32 = 2.0 ** -8, 2.0 ** -23


def whole(g, rows, width, top, keep):
    """Whole numbers of [-top, top], the others 0."""
    v = torch.randint(-top, top + 1, (rows, width), generator=g, device=g.device, dtype=torch.int8)
    return v * (torch.rand((rows, width), generator=g, device=g.device) < keep)


def per_block(p, width):
    """2^p of each column's block, float64."""
    return torch.ldexp(torch.ones((), dtype=torch.float64, device=p.device), p).repeat_interleave(128)[:width]


def exact_case(T, K, N, seed, device="cuda"):
    """(x, w, y0 in bf16; the exact product and y0 in float64)."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    pick = lambda n, lo, hi: torch.randint(lo, hi + 1, (n,), generator=g, device=device)  # noqa: E731
    # about 1500 / K of the products are not 0: sums of some tens
    x, w = whole(g, T, K, 2, min(1.0, 1500 / K)), whole(g, N, K, 1, 1.0)
    p, a, c = per_block(pick(-(-K // 128), -20, 20), K), pick(T, -10, 10), pick(-(-N // 128), -10, 10)
    sx = torch.ldexp(torch.ones((), dtype=torch.float64, device=device), a)[:, None]
    sw = per_block(c, N)
    xs, ws = (x.double() * sx * p).to(torch.bfloat16), (w.double() * sw[:, None] / p).to(torch.bfloat16)
    scale = sx * sw[None, :]
    y0 = torch.randint(-64, 65, (T, N), generator=g, device=device).double() * scale
    ref = x.double() @ w.double().t().contiguous()
    assert float(ref.abs().max()) < 2 ** 12
    return xs, ws, y0.to(torch.bfloat16), ref * scale, y0


@pytest.mark.parametrize("T,K,N", PRODUCTS)
def test_every_kernel_is_exact_on_whole_numbers(T, K, N):
    x, w, y0, ref, y064 = exact_case(T, K, N, T + K + N)
    q, p = wide_q8(T, K), wide_q8(N, K, weights=True)
    L.q8_quantize(x, q)
    L.q8_quantize(w, p)
    big, y = strided(torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda"))

    def guards():
        assert torch.all(big[T] == 7) and torch.all(big[:, N:] == 7)

    L.q8_matmul(q, p, y)
    assert torch.equal(y, ref.float().to(torch.bfloat16))
    guards()
    y.copy_(y0)
    L.q8_matmul(q, p, y, accumulate=True)
    assert torch.equal(y, (ref + y064).float().to(torch.bfloat16))
    guards()


TABLE = R.TABLE


def values64(q):
    """(values, powers of two of their exponents) of a store, float64 on the GPU, from its bytes and the definition of e4m3."""
    b = q.values.view(torch.uint8)[:q.rows, :q.width].long()
    e = q.exps[:-(-q.rows // q.block_rows), :-(-q.width // 128)].long()
    e = e.repeat_interleave(q.block_rows, 0)[:q.rows].repeat_interleave(128, 1)[:, :q.width] - 127
    one = torch.ones((), dtype=torch.float64, device="cuda")
    v = torch.ldexp(torch.from_numpy(TABLE).cuda()[b], e)
    top = torch.ldexp(one, e + ((b >> 3) & 15).clamp(min=1) - 7)
    return v, torch.where(v == 0, torch.zeros((), dtype=torch.float64, device="cuda"), top)


# The tolerance of test_gpu_q8.py's check_matmul, over every column; also of the
# sizes that its test of long sums compares in some columns and in row sums,
# whose limit a tile of zeros stays below.
@pytest.mark.parametrize("T,K,N", PRODUCTS + LONG)
def test_every_kernel_on_random_values(T, K, N):
    g = torch.Generator(device="cuda")
    g.manual_seed(T * K + N)
    x = torch.randn((T, K), generator=g, device="cuda") * torch.exp(torch.randn((T, 1), generator=g, device="cuda"))
    x[:, torch.rand(K, generator=g, device="cuda") < 0.02] *= 30
    w = torch.randn((N, K), generator=g, device="cuda")
    y0 = torch.randn((T, N), generator=g, device="cuda").to(torch.bfloat16) * 8
    q, p = wide_q8(T, K), wide_q8(N, K, weights=True)
    L.q8_quantize(x.to(torch.bfloat16), q)
    L.q8_quantize(w.to(torch.bfloat16), p)
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    added = y0.clone()
    L.q8_matmul(q, p, y)
    L.q8_matmul(q, p, added, accumulate=True)
    (a, ta), (b, tb) = values64(q), values64(p)
    ref, mag = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
    tb = tb.t().contiguous()
    grouped = torch.zeros_like(ref)
    for k in range(0, K, 8):
        top = ta[:, k, None] * tb[None, k]
        for i in range(k + 1, k + 8):
            torch.maximum(top, ta[:, i, None] * tb[None, i], out=top)
        grouped += top
    for got, base in ((y, None), (added, y0.double())):
        want, size = (ref, mag) if base is None else (ref + base, mag + base.abs())
        err = 7 * 2.0 ** -13 * grouped + (R.padded(K) + 2) * F32 * size
        bad = (got.double() - want).abs() > BF * (want.abs() + err) + err
        assert torch.isfinite(got).all() and not bad.any(), int(bad.sum())
