"""CPU oracle of the head norms, the position rotation and the append into packed pages ("vLLM
Usage", TQ Packed Page Contract: the rows that write_tq4_kv encodes; Slot Mapping).

fp64 over the definitions, pair by pair.  Pins live in ``tests/test_append_host.py``.
"""

from __future__ import annotations

import math

import numpy as np

from oracle import tq_oracle as o


def rope_table(rot_dim: int, num_positions: int, base: float = 10000.0, inv_freq=None) -> np.ndarray:
    """cos then sin of position * frequency, fp64 [num_positions, rot_dim]."""
    out = np.empty((num_positions, rot_dim))
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim) if inv_freq is None else float(inv_freq[i])
        for p in range(num_positions):
            out[p, i], out[p, rot_dim // 2 + i] = math.cos(p * f), math.sin(p * f)
    return out


def norm_heads(x, weight, eps):
    """x[T, H, D] w / sqrt(mean x^2 + eps)."""
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def rotate(x, positions, table, interleaved):
    """Rotated rows, and for every channel the sum of the magnitudes of its pair (what the
    rounding of a channel is measured against)."""
    x = np.asarray(x, dtype=np.float64)
    y, size = x.copy(), np.abs(x)
    if table is None:
        return y, size
    table = np.asarray(table, dtype=np.float64)
    half = table.shape[1] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = table[positions, i][:, None], table[positions, half + i][:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
        size[:, :, a] = size[:, :, b] = np.abs(x[:, :, a]) + np.abs(x[:, :, b])
    return y, size


def norm_rope(x, positions, table, interleaved=False, weight=None, eps=1e-6):
    return rotate(norm_heads(x, weight, eps), positions, table, interleaved)


def encode(x, signs, centroids32):
    """(index [N, D], norm [N], distance of each coordinate to the nearest decision point) of rows
    x[N, D], whatever their scale."""
    return o.encode_rows(np.asarray(x, dtype=np.float64), o.rotation_matrix(signs), centroids32)
