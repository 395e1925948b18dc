"""RMS norm of query and key heads and the position rotation, fp64 on the CPU.

The pages take queries and keys "with their position encoding applied"; this
is the encoding of the models they name (rotation of pairs by position), with
the per-head norm that some of them put before it:

  y = x / sqrt(mean(x^2) + eps) * weight
  (a, b) -> (a cos - b sin, b cos + a sin),  angle = position * inv_freq[j]

for the pairs (j, j + rot/2), or (2j, 2j + 1) interleaved.  The rotation is
written as a product of complex numbers.
"""
from __future__ import annotations

import numpy as np


def oracle_norm_rope(x, weight, positions, inv_freq, interleaved=False, eps=1e-6):
    """x [rows, heads, D] -> fp64; rows of negative positions are zero."""
    x = np.array(x, dtype=np.float64)
    positions = np.asarray(positions, dtype=np.float64)
    if weight is not None:
        rms = np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        x = x / rms * np.asarray(weight, dtype=np.float64)
    half = len(inv_freq)
    if half:
        turn = np.exp(1j * positions[:, None, None] * np.asarray(inv_freq, dtype=np.float64))
        first, second = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                         else (slice(0, half), slice(half, 2 * half)))
        z = (x[..., first] + 1j * x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
    x[positions < 0] = 0.0
    return x
