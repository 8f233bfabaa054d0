"""Oracle for the operators around the K/V cache -- TEST INFRASTRUCTURE ONLY.

Everything is float64 NumPy, row by row from the definitions, and shares nothing with the library:

* :func:`norm_rope` -- RMS norm of each (token, head) row and the rotation by position;
* :class:`Fp8Cache` -- the FP8 cache: e4m3 codes and one power-of-two scale per (16 tokens, head),
  appended to block by block; rows of a block that are live and not part of the append stay;
* :func:`attention` -- softmax attention of query segments, each with its own number of visible
  keys, K/V heads shared by groups of query heads; a row that sees no key is 0 with lse -inf.
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_decode, e4m3_values

BLOCK = 16
E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -100, 119
_VALS = e4m3_values()


def norm_rope(x, weight=None, norm=True, eps=1e-6, table=None, positions=None, axis_pairs=(),
              interleaved=False) -> np.ndarray:
    """x [L, H, D]; weight [D] or [H, D]; table [rows, pairs, 2]; positions [L, axes]."""
    y = np.array(x, dtype=np.float64)
    L, H, D = y.shape
    if norm:
        for t in range(L):
            for h in range(H):
                y[t, h] /= np.sqrt(np.mean(y[t, h] ** 2) + eps)
        if weight is not None:
            y *= np.asarray(weight, np.float64)
    if table is None:
        return y
    table = np.asarray(table, np.float64)
    pairs = sum(axis_pairs)
    axis = [a for a, n in enumerate(axis_pairs) for _ in range(n)]
    out = y.copy()
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, pairs + i)
        cs = table[np.asarray(positions)[:, axis[i]], i]          # [L, 2]
        c, s = cs[:, 0, None], cs[:, 1, None]
        out[:, :, a] = y[:, :, a] * c - y[:, :, b] * s
        out[:, :, b] = y[:, :, a] * s + y[:, :, b] * c
    return out


def scale_exponent(top: float) -> int:
    """The least e with top / 2^e <= 448, kept in [EXP_MIN, EXP_MAX]."""
    if top <= 0:
        return EXP_MIN
    m, e = np.frexp(top)                        # top = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    return int(min(EXP_MAX, max(EXP_MIN, e - 9 + (1 if m > 0.875 else 0))))


def encode(y) -> np.ndarray:
    """float64 -> e4m3 codes: nearest, ties to the even code, saturated at 448, NaN for NaN."""
    y = np.asarray(y, np.float64)
    a = np.abs(np.nan_to_num(y, nan=0.0))
    hi = np.clip(np.searchsorted(_VALS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - _VALS[lo], _VALS[hi] - a
    code = np.where((d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0)), hi, lo)
    code = np.where(a >= E4M3_MAX, 126, code)
    code = code | (np.signbit(y).astype(np.int64) << 7)
    return np.where(np.isnan(y), 0x7F, code).astype(np.uint8)


class Fp8Cache:
    """codes [pages, page_size, H, D] and scale bytes [pages, page_size / 16, H] of one tensor."""

    def __init__(self, pages: int, page_size: int, heads: int, head_dim: int):
        self.codes = np.zeros((pages, page_size, heads, head_dim), np.uint8)
        self.scale = np.zeros((pages, page_size // BLOCK, heads), np.uint8)
        self.page_size = page_size

    def append(self, rows, token0: int, live: int, page_row) -> None:
        """rows: float64 [L, H, D] of logical tokens token0.., `live` tokens in the sequence."""
        rows = np.asarray(rows, np.float64)
        L, H, _ = rows.shape
        for b in range(token0 // BLOCK, (token0 + L - 1) // BLOCK + 1):
            t0 = b * BLOCK
            page = int(page_row[t0 // self.page_size])
            r0 = t0 % self.page_size
            for h in range(H):
                e_old = int(self.scale[page, r0 // BLOCK, h]) - 127
                value, alive = {}, []
                for r in range(BLOCK):
                    t = t0 + r
                    if token0 <= t < token0 + L:
                        value[r] = rows[t - token0, h]
                    elif t < live:
                        value[r] = e4m3_decode(self.codes[page, r0 + r, h]).astype(np.float64) * \
                            2.0 ** e_old
                    else:
                        continue
                    value[r] = np.where(np.isfinite(value[r]), value[r], np.nan)
                    alive.append(r)
                top = max(np.max(np.abs(np.nan_to_num(value[r], nan=0.0))) for r in alive)
                e = scale_exponent(float(top))
                for r in alive:
                    self.codes[page, r0 + r, h] = encode(value[r] * 2.0 ** -e)
                self.scale[page, r0 // BLOCK, h] = e + 127

    def values(self, page_row, tokens: int) -> np.ndarray:
        """The values the cache holds for logical tokens [0, tokens): float64 [tokens, H, D]."""
        return decode_rows(self.codes, self.scale, page_row, tokens)


def decode_rows(codes, scale, page_row, tokens: int) -> np.ndarray:
    ps = codes.shape[1]
    out = np.empty((tokens,) + codes.shape[2:], np.float64)
    for t in range(tokens):
        page, r = int(page_row[t // ps]), t % ps
        e = scale[page, r // BLOCK].astype(np.float64) - 127
        out[t] = e4m3_decode(codes[page, r]).astype(np.float64) * (2.0 ** e)[:, None]
    return out


def attention(q, k, v, rows_end, kv_end, scale: float):
    """q [T, Hq, D], k, v [N, Hkv, D]: out [T, Hq, D] and lse [Hq, T] (natural log)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    T, Hq, _ = q.shape
    group = Hq // k.shape[1]
    out, lse = np.zeros_like(q), np.full((Hq, T), -np.inf)
    lo = 0
    for hi, n in zip(rows_end, kv_end):
        if n > 0:
            for h in range(Hq):
                t = q[lo:hi, h] @ k[:n, h // group].T * scale
                top = t.max(axis=1, keepdims=True) if hi > lo else t
                p = np.exp(t - top)
                total = p.sum(axis=1, keepdims=True)
                out[lo:hi, h] = p @ v[:n, h // group] / total
                lse[h, lo:hi] = (top + np.log(total))[:, 0]
        lo = hi
    return out, lse
