"""Per-head RMS norm and position rotation in float64.

Test infrastructure only (see ``oracle/__init__.py``).  The pages leave
positions to the model; this is the definition ``duo.h`` states: pair j of the
first rot_dim channels, (j, j + rot_dim/2) or interleaved (2j, 2j+1), turns by
position * inv_freq[j], times mscale; later channels pass.
"""

import numpy as np

__all__ = ["norm", "rotate", "pair_size"]


def norm(x, weight, eps):
    """x [..., d] / rms(x) * weight."""
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def _pairs(rot, interleaved):
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def rotate(y, pos, inv_freq, interleaved=False, mscale=1.0):
    """y [tokens, heads, d] at integer pos [tokens]."""
    inv_freq = np.asarray(inv_freq, np.float64)
    a, b = _pairs(2 * len(inv_freq), interleaved)
    ang = np.asarray(pos, np.float64)[:, None] * inv_freq
    turn = mscale * np.exp(1j * ang)[:, None, :]
    z = (y[..., a] + 1j * y[..., b]) * turn
    out = np.array(y, np.float64)
    out[..., a], out[..., b] = z.real, z.imag
    return out


def pair_size(y, rot, interleaved=False, mscale=1.0):
    """|y_a| + |y_b| of each channel's pair times mscale (|y| past rot): what
    an error of the rotation is relative to."""
    a, b = _pairs(rot, interleaved)
    out = np.abs(np.array(y, np.float64))
    s = (out[..., a] + out[..., b]) * mscale
    out[..., a], out[..., b] = s, s
    return out
