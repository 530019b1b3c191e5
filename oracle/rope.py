"""Head norms and rotary positions, float64 (test infrastructure only; see the
package docstring)."""
from __future__ import annotations

import numpy as np

from .attention import bf16_bits_to_f64


def norm(x, weight, eps):
    """Rows [.., D] over their root mean square, times ``weight`` (None: as they are)."""
    if weight is None:
        return np.array(x, dtype=np.float64)
    x = np.asarray(x, np.float64)
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def rotate(y, positions, inv_freq, freq_axis=None, interleaved=False):
    """Turn the first ``2 * len(inv_freq)`` values of the rows y [n, H, D]:
    pair i by ``positions[axis, t] * inv_freq[i]``.  Returns (rotated, size):
    ``size`` holds |a| + |b| of each value's pair (|y| where none turns)."""
    y = np.asarray(y, np.float64)
    out, size = y.copy(), np.abs(y)
    pos = np.atleast_2d(np.asarray(positions, np.int64))
    nf = len(inv_freq)
    for i in range(nf):
        a_i, b_i = (2 * i, 2 * i + 1) if interleaved else (i, i + nf)
        axis = 0 if freq_axis is None else int(freq_axis[i])
        ang = pos[axis].astype(np.float64) * float(np.float32(inv_freq[i]))
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = y[:, :, a_i], y[:, :, b_i]
        out[:, :, a_i], out[:, :, b_i] = a * c - b * s, b * c + a * s
        size[:, :, a_i] = size[:, :, b_i] = np.abs(a) + np.abs(b)
    return out, size


def qk_norm_rope(bits, weight_bits, eps, positions, inv_freq, freq_axis=None, interleaved=False):
    """bf16 rows [n, H, D] (bit patterns) -> (finished rows, pair sizes)."""
    w = None if weight_bits is None else bf16_bits_to_f64(weight_bits)
    return rotate(norm(bf16_bits_to_f64(bits), w, eps), positions, inv_freq, freq_axis, interleaved)
