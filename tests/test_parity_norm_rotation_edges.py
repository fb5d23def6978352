"""GPU parity of the per-head norms at their edges, vs the float64 oracle (tolerances as derived
in test_parity_norm_rotation.py)."""

import numpy as np
import pytest
import torch

from oracle import norm_rotation as nr
from test_parity_norm_rotation import E, TYPES, _bsa, _check_forward, _inputs, _np, _tensor, _u

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("D,inter", [(64, True), (128, False)])
@pytest.mark.parametrize("Hq,Hkv,S", [(1, 1, 1), (6, 3, 37), (9, 5, 130)])
def test_without_eps(dt, D, inter, Hq, Hkv, S):
    """eps = 0, heads that are no multiple of a step: the rows that fill up the last step count
    neither in the rows' gradients nor in the weights'."""
    q, k, qw, kw, cos, sin = _inputs(2, Hq, Hkv, S, D, TYPES[dt], "fused", seed=8)
    g = torch.Generator().manual_seed(9)
    dq, dk = (_tensor(g, 2, h, S, D, TYPES[dt], "heads") for h in (Hq, Hkv))
    bsa = _bsa()
    qo, ko = bsa.qk_norm_rotation(q, k, qw, kw, cos, sin, eps=0.0, interleaved=inter)
    _check_forward(qo, q, qw, cos, sin, 0.0, inter)
    _check_forward(ko, k, kw, cos, sin, 0.0, inter)
    got = bsa.qk_norm_rotation_backward(dq, dk, q, k, qw, kw, cos, sin, eps=0.0, interleaved=inter)
    for x, w, d, dx, dw in ((q, qw, dq, got[0], got[2]), (k, kw, dk, got[1], got[3])):
        xd, wd, dd = _np(x), _np(w), _np(d)
        rx, rw = nr.norm_rotation_backward(dd, xd, wd, _np(cos), _np(sin), 0.0, inter)
        r = 1 / np.sqrt((xd * xd).mean(-1, keepdims=True))
        a, b = nr._pairs(np.abs(dd), inter)
        z = nr._unpair(a + b, a + b, inter)
        size = r * z * np.abs(wd) + r ** 3 * np.abs(xd) * (z * np.abs(wd * xd)).mean(-1, keepdims=True)
        u = _u(x.dtype)
        tol = u * np.abs(rx) + (1 + u) * 40 * E * size + (6e-8 if dt == "f16" else 0)
        assert (np.abs(_np(dx) - rx) <= tol).all()
        tw = (2 * S * x.shape[1] + 40) * E * (z * np.abs(xd) * r).reshape(-1, D).sum(0)
        assert (np.abs(_np(dw) - rw) <= tw).all()
