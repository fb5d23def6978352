"""Float64 statement of the per-head norm with position rotation and its gradient."""

import numpy as np


def _pairs(x, interleaved):
    if interleaved:
        return x[..., 0::2], x[..., 1::2]
    h = x.shape[-1] // 2
    return x[..., :h], x[..., h:]


def _unpair(a, b, interleaved):
    out = np.empty(a.shape[:-1] + (2 * a.shape[-1],))
    if interleaved:
        out[..., 0::2], out[..., 1::2] = a, b
    else:
        h = a.shape[-1]
        out[..., :h], out[..., h:] = a, b
    return out


def rotate(y, cos, sin, interleaved):
    """Rotates the pairs of y (..., S, D) by the angles of cos, sin (S, D/2)."""
    a, b = _pairs(y, interleaved)
    return _unpair(a * cos - b * sin, a * sin + b * cos, interleaved)


def norm_rotation(x, w, cos, sin, eps=1e-6, interleaved=True):
    """x (..., S, D): x / rms(x) * w, then rotated."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(x * r * w, cos, sin, interleaved)


def norm_rotation_backward(dout, x, w, cos, sin, eps=1e-6, interleaved=True):
    """(dx, dw); dw summed over every leading axis."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    z = rotate(dout, cos, -sin, interleaved)
    g = z * w
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdims=True))
    return dx, (z * x * r).reshape(-1, x.shape[-1]).sum(0)
