"""Oracle: rotary positions in fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Pair p of a head is features (2p, 2p + 1) (interleaved) or (p, p + R) (half),
R pairs in all, the first dim_t / 2 of them on the t axis, then h, then w. The
pair is one complex number, multiplied by amplitude * e^(i pos f).

Parity: pinned by complex rotation in closed form, by the invariance of
rotated dot products under a common shift of positions, and, for the
transpose, by central differences (tests/test_oracle_rules.py).
"""

from __future__ import annotations

import math

import numpy as np


def frequencies(dims, base=10000.0, scaling="none", factor=(1.0, 1.0, 1.0), original=(1.0, 1.0, 1.0), slow=1.0,
                fast=32.0):
    """(angle per unit of position, axis) of every pair."""
    f, axis = [], []
    for a in range(3):
        d, s = dims[a], factor[a]
        for i in range(d // 2):
            b = base * s ** (d / (d - 2)) if scaling == "ntk" and d > 2 else base
            x = b ** (-2.0 * i / d)
            if scaling == "linear":
                x /= s
            elif scaling == "by_parts":
                turns = original[a] * x / (2 * math.pi)
                g = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
                x *= g + (1 - g) / s
            f.append(x)
            axis.append(a)
    return np.array(f), np.array(axis, dtype=np.int64)


def grid_positions(T, H, W, offset=(0, 0, 0)):
    """[L, 3] (t, h, w) of every natural token, plus the offset."""
    n = np.arange(T * H * W)
    return np.stack((n // (H * W), n // W % H, n % W), -1) + np.asarray(offset, dtype=np.int64)


def rotate(x, pos, f, axis, layout="interleaved", amplitude=1.0, transpose=False):
    """x [B, L, heads, D], pos [L, 3] or [B, L, 3] -> fp64 [B, L, heads, D]."""
    x = x.astype(np.float64).copy()
    R = f.size
    first = np.arange(R) * (2 if layout == "interleaved" else 1)
    second = first + (1 if layout == "interleaved" else R)
    pos = np.broadcast_to(pos, x.shape[:2] + (3,))
    ang = pos[..., axis].astype(np.float64) * f
    turn = amplitude * np.exp((-1j if transpose else 1j) * ang)[:, :, None]
    z = (x[..., first] + 1j * x[..., second]) * turn
    x[..., first], x[..., second] = z.real, z.imag
    return x
