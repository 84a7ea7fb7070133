"""Float64 restatement of the paged cache: the e4m3 rows, their write and
read-back, and causal attention with a window and first tokens (numpy only;
imports nothing from the product path)."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def e4m3_grid() -> np.ndarray:
    """The finite non-negative values of e4m3, by code 0 .. 126."""
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def e4m3_value(code: np.ndarray) -> np.ndarray:
    code = np.asarray(code, dtype=np.uint8)
    v = np.append(e4m3_grid(), np.nan)[code & 127]
    return np.where(code & 128, -v, v)


def e4m3_code(x: np.ndarray) -> np.ndarray:
    """Nearest code, ties to the even one, saturating at 448."""
    grid = e4m3_grid()
    a = np.minimum(np.abs(x), E4M3_MAX)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def row_exponent(amax: float) -> int:
    """min { k : amax <= 448 * 2^k }, clipped to [-124, 119]"""
    k = -124
    while k < 119 and amax > E4M3_MAX * 2.0 ** k:
        k += 1
    return k


def quantise_row(x: np.ndarray) -> tuple[np.ndarray, int]:
    """(codes, scale byte) of one row."""
    k = row_exponent(float(np.abs(x).max()))
    return e4m3_code(x * 2.0 ** -k), k + 127


def dequantise_row(code: np.ndarray, scale: int) -> np.ndarray:
    return e4m3_value(code) * 2.0 ** (int(scale) - 127)


def visible(p: int, t: np.ndarray, window: int, sinks: int) -> np.ndarray:
    """Which tokens t the row at position p sees."""
    return (t <= p) & ((window == 0) | (t > p - window) | (t < sinks))


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, see: np.ndarray, scale: float):
    """out [D], lse of one query over the tokens `see` marks; k, v [N][D]."""
    if not see.any():
        return np.zeros(v.shape[1]), -np.inf
    z = scale * (k[see] @ q)
    top = z.max()
    e = np.exp(z - top)
    return (e @ v[see]) / e.sum(), top + np.log(e.sum())


def attend_rows(q: np.ndarray, k: np.ndarray, v: np.ndarray, positions, valid: np.ndarray, window: int,
                sinks: int, scale: float):
    """q [R][G][D] at `positions` [R], one KV head's k, v [N][D], valid [N]
    (False: a token whose page is bad) -> out [R][G][D], lse [R][G]"""
    R, G, D = q.shape
    out, lse = np.zeros((R, G, D)), np.full((R, G), -np.inf)
    t = np.arange(k.shape[0])
    for r in range(R):
        see = visible(int(positions[r]), t, window, sinks) & valid
        if not see.any():
            continue
        z = scale * (q[r] @ k[see].T)
        top = z.max(axis=1, keepdims=True)
        e = np.exp(z - top)
        s = e.sum(axis=1, keepdims=True)
        out[r] = (e @ v[see]) / s
        lse[r] = (top + np.log(s))[:, 0]
    return out, lse
