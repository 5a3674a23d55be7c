"""fp64 reference of the rotary positions (test infrastructure only).

Every pair is a complex number, multiplied by e^(i sign p_a base^(-2 i / d_a)).
Parity status: pinned by a two-channel hand value, by the transpose giving the input back, and
by scores that depend on position differences only.
"""

from __future__ import annotations

import numpy as np


def grid_positions(grid, start, N):
    """[min(N, cells), axes] positions of the grid's cells, last axis fastest."""
    cells = int(np.prod(grid, dtype=object))
    n = np.arange(min(N, cells))
    pos = np.zeros((len(n), len(grid)))
    for a in range(len(grid) - 1, -1, -1):
        pos[:, a] = n % grid[a] + start[a]
        n = n // grid[a]
    return pos


def rotate(x, axes, positions, base, pairing, sign=1.0):
    """x [B, H, N, D] (array), positions [n, axes] or [B, n, axes] of the first n tokens."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    B = x.shape[0]
    positions = np.asarray(positions, dtype=np.float64)
    positions = np.broadcast_to(positions, (B,) + positions.shape[-2:])
    n = positions.shape[1]
    first = 0
    for a, d in enumerate(axes):
        i = np.arange(d // 2)
        c1, c2 = (first + 2 * i, first + 2 * i + 1) if pairing == 0 else (first + i, first + i + d // 2)
        phi = positions[:, None, :, a:a + 1] * base ** (-2.0 * i / d)
        z = (x[:, :, :n, c1] + 1j * x[:, :, :n, c2]) * np.exp(1j * sign * phi)
        y[:, :, :n, c1], y[:, :, :n, c2] = z.real, z.imag
        first += d
    return y
