"""Shared by the tests of the operators around the K/V cache: rotation tables, seeded rows, and the
tolerances, which are derived here."""
from __future__ import annotations

import numpy as np
import torch

# fp32 arithmetic of one row: 128 squares summed (relative error below 12 half-ulps along any lane
# and shuffle tree of depth 11), a reciprocal square root (2 ulp), two products, and a rotation of
# two products and a sum whose terms are at most |a| + |b|: under 2^-19 of |a| + |b| with room.
FP32_REL = 2.0 ** -19
BF16_HALF = 2.0 ** -8          # rounding to bf16: at most half a step, relative to the value


def table_of(rows: int, pairs: int, seed: int = 0) -> np.ndarray:
    """fp32 [rows, pairs, 2]: cos and sin of position times a falling frequency."""
    ang = np.arange(rows)[:, None] * 1000.0 ** (-np.arange(pairs) / pairs)
    return np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


def positions_of(L: int, axes: int, rows: int, seed: int) -> np.ndarray:
    return np.random.default_rng(seed).integers(0, rows, size=(L, axes)).astype(np.int32)


def bf16_rows(L: int, H: int, D: int, seed: int, scale: float = 1.0) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(L, H, D, generator=g) * scale
    return (x * torch.exp(0.5 * torch.randn(L, H, 1, generator=g))).to(torch.bfloat16)


def bf16_weight(shape, seed: int) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(*shape, generator=g)).to(torch.bfloat16)


def pair_size(y: np.ndarray, pairs: int, interleaved: bool) -> np.ndarray:
    """|a| + |b| of the pair each channel belongs to (|y| for channels that are not turned): what
    the fp32 error of a rotated value is relative to.  A rotation keeps sqrt(a^2 + b^2), so the
    rotated values' own |a| + |b| is within sqrt 2 of it; times 2 covers that."""
    size = np.abs(y)
    if pairs:
        first = np.arange(pairs) * (2 if interleaved else 1)
        second = first + (1 if interleaved else pairs)
        s = 2 * (np.abs(y[..., first]) + np.abs(y[..., second]))
        size[..., first] = s
        size[..., second] = s
    return size


def assert_bf16_rows(got: torch.Tensor, want: np.ndarray, pairs: int, interleaved: bool, what=""):
    tol = BF16_HALF * np.abs(want) + FP32_REL * pair_size(want, pairs, interleaved) + 1e-38
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.isfinite(err).all(), f"{what}: non-finite rows"
    worst = (err / tol).max() if err.size else 0.0
    assert worst <= 1, f"{what}: {worst:.3f} of the tolerance"
