"""Plain 64-bit forms of the 8-bit operators and of the gated activation
(numpy, from the definitions), shared by their tests."""
from __future__ import annotations

import numpy as np

BLOCK = 128


def e4m3_table() -> np.ndarray:
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        mag = np.nan if (e == 15 and m == 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = -mag if b & 128 else mag
    return v


TABLE = e4m3_table()


def padded(n: int) -> int:
    return -(-n // BLOCK) * BLOCK


def block_exponents(x: np.ndarray, block_rows: int) -> np.ndarray:
    """Biased exponent per block: the smallest e >= 1 with max|x| <= 448 *
    2^(e - 127) over the block's finite values."""
    rows, width = x.shape
    nr, nb = -(-rows // block_rows), padded(width) // BLOCK
    p = np.zeros((nr * block_rows, nb * BLOCK))
    p[:rows, :width] = np.where(np.isfinite(x), np.abs(x), 0.0)
    top = p.reshape(nr, block_rows, nb, BLOCK).max(axis=(1, 3))
    m, ex = np.frexp(top)                       # top = m 2^ex, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = ex - 9 + (m > 0.875) + 127
    return np.where(top > 0, np.maximum(e, 1), 1).astype(np.int64)


def spread(e: np.ndarray, rows: int, width: int, block_rows: int) -> np.ndarray:
    """The scale of every element."""
    s = np.ldexp(1.0, e - 127)
    return np.repeat(np.repeat(s, block_rows, 0)[:rows], BLOCK, 1)[:, :width]


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to even, of |v| <= 448; NaN for anything not finite."""
    a = np.abs(np.where(np.isfinite(v), v, 1.0))
    step = np.ldexp(1.0, np.maximum(np.frexp(a)[1] - 1, -6) - 3)
    q = np.copysign(np.rint(a / step) * step, v)
    return np.where(np.isfinite(v), q, np.nan)


def quantize(x: np.ndarray, block_rows: int = 1):
    """(values in units of their scale, biased exponents)."""
    x = np.asarray(x, np.float64)
    e = block_exponents(x, block_rows)
    with np.errstate(invalid="ignore"):
        return round_e4m3(x / spread(e, *x.shape, block_rows)), e


def restore(values: np.ndarray, e: np.ndarray, block_rows: int = 1) -> np.ndarray:
    return values * spread(e, *values.shape, block_rows)


def read_store(q) -> np.ndarray:
    """float64 values of a Q8Rows / Q8Weights on the GPU (decoded on the host from its bytes)."""
    import torch
    b = q.values.view(torch.uint8)[:q.rows, :q.width].cpu().numpy()
    e = q.exps.cpu().numpy()[:-(-q.rows // q.block_rows), :padded(q.width) // BLOCK].astype(np.int64)
    return TABLE[b] * spread(e, q.rows, q.width, q.block_rows)


def swiglu(gate_up: np.ndarray):
    F = gate_up.shape[1] // 2
    g, u = gate_up[:, :F], gate_up[:, F:]
    s = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
    return g, u, s, g * s * u


def swiglu_grad(gate_up: np.ndarray, dh: np.ndarray) -> np.ndarray:
    g, u, s, _ = swiglu(gate_up)
    return np.concatenate([dh * u * s * (1 + g * (1 - s)), dh * g * s], axis=1)
