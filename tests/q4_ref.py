"""Plain 64-bit forms of the 4-bit operators (numpy, from the definitions),
shared by their tests."""
from __future__ import annotations

import numpy as np

PANEL, GROUP = 128, 32
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
TABLE = np.concatenate([GRID, -GRID])


def panels(width: int) -> int:
    return -(-width // PANEL)


def block_exponents(x: np.ndarray, block_rows: int = 1) -> np.ndarray:
    """Biased exponent of every row and 32 columns, whole panels: the smallest
    e >= 1 with max|x| <= 6 * 2^(e - 127) over the block; 255 where it holds
    anything that is not finite."""
    rows, width = x.shape
    nr, nb = -(-rows // block_rows), 4 * panels(width)
    p = np.zeros((nr * block_rows, nb * GROUP))
    p[:rows, :width] = np.where(np.isnan(x), np.inf, np.abs(x))
    top = p.reshape(nr, block_rows, nb, GROUP).max(axis=(1, 3))
    m, ex = np.frexp(np.where(np.isfinite(top), top, 1.0))  # top = m 2^ex, 0.5 <= m < 1; 6 = 0.75 * 2^3
    e = np.where(top > 0, np.maximum(ex - 3 + (m > 0.75) + 127, 1), 1)
    return np.repeat(np.where(np.isfinite(top), e, 255), block_rows, 0)[:rows].astype(np.int64)


def spread(e: np.ndarray, width: int) -> np.ndarray:
    """The scale of every element (NaN for the exponent 255)."""
    s = np.where(e == 255, np.nan, np.ldexp(1.0, e - 127))
    return np.repeat(s, GROUP, 1)[:, :width]


def round_e2m1(v: np.ndarray) -> np.ndarray:
    """Nearest e2m1 value, ties to the even code, of |v| <= 6."""
    a = np.abs(v)
    step = np.ldexp(1.0, np.maximum(np.frexp(a)[1] - 1, 0) - 1)
    return np.copysign(np.rint(a / step) * step, v)


def quantize(x: np.ndarray, block_rows: int = 1):
    """(values in units of their scale, biased exponents); 0 in blocks without a scale."""
    x = np.asarray(x, np.float64)
    e = block_exponents(x, block_rows)
    s = spread(e, x.shape[1])
    with np.errstate(invalid="ignore"):
        v = round_e2m1(np.where(np.isnan(s), 0.0, x / np.where(np.isnan(s), 1.0, s)))
    return np.where(np.isnan(s), 0.0, v), e


def restore(values: np.ndarray, e: np.ndarray) -> np.ndarray:
    return values * spread(e, values.shape[1])


def codes(q) -> np.ndarray:
    """The codes of a Q4, whole panels: [rows, panels * 128]."""
    b = q.values[:panels(q.width), :q.rows].cpu().numpy().transpose(1, 0, 2)
    return np.stack([b & 15, b >> 4], axis=3).reshape(q.rows, -1)


def exponents(q) -> np.ndarray:
    """Biased exponents of every row and 32 columns, whole panels."""
    e = q.exps[:panels(q.width), :q.rows].cpu().numpy().transpose(1, 0, 2)
    return e.reshape(q.rows, -1).astype(np.int64)


def read_store(q) -> np.ndarray:
    """float64 values of a Q4 (decoded on the host from its bytes)."""
    return TABLE[codes(q)[:, :q.width]] * spread(exponents(q), q.width)
