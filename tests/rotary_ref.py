"""float64 reference of the rotation by positions, on the CPU."""

from __future__ import annotations

import torch

from tests import cache_ref as R


def token_positions(positions, T, parents=None):
    """[B, T] int64: the positions that a step's tokens have by themselves."""
    B = positions.shape[0]
    at = torch.zeros((B, T), dtype=torch.int64)
    for b in range(B):
        for t in range(T):
            depth = t if parents is None else len(R.path_of(parents[b], t)) - 1
            at[b, t] = int(positions[b]) + depth
    return at


def rotate(x, freqs, interleaved, ids, axes=None):
    """x [B, T, heads, D] by ids [A, B, T]: the result in float64, and what bounds a float32 evaluation's error.

    Cosine and sine are rounded to float32 (2^-24 relative to at most 1), each product (2^-24 of it) and the sum
    (2^-24 of at most |a| + |b|): the value is off by at most 3 * 2^-24 (|a| + |b|), and then rounded to bf16 (2^-8 of
    it).
    """
    x = x.double()
    half = freqs.shape[0]
    axes = torch.zeros(half, dtype=torch.long) if axes is None else axes.long().clamp(0, ids.shape[0] - 1)
    angle = ids.double()[axes].permute(1, 2, 0) * freqs.double()
    cos, sin = angle.cos()[:, :, None], angle.sin()[:, :, None]
    first = torch.arange(half) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    a, b = x[..., first], x[..., second]
    y, off = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    off[..., first] = off[..., second] = 3 * 2.0 ** -24 * (a.abs() + b.abs())
    # a bf16 has steps of 2^-133 at least
    return y, off + 2.0 ** -8 * (y.abs() + off) * (off > 0) + 2.0 ** -134
