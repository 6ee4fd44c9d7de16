"""fp64 CPU oracle of the q/k normalisation and rotation (test infrastructure).

Only the test suite may import this module; it shares no code with the GPU library.  Written
from the definition: every row as x / sqrt(mean x^2 + eps) * gamma, the rotation as one
complex multiplication per pair; the backward as the transpose of each step.  Pinned by
``tests/test_oracle_kv8.py`` (finite differences, torch autograd, a rotation by hand).
"""
from __future__ import annotations

import numpy as np

from .proj import _f64


def _turn(x, pos, rope_dims, rope_base, sign):
    h = rope_dims // 2
    y = x.copy()
    if h:
        theta = rope_base ** (-2.0 * np.arange(h) / rope_dims)
        z = (x[..., :h] + 1j * x[..., h:2 * h]) * np.exp(sign * 1j * np.asarray(pos, np.float64)[:, None, None] * theta)
        y[..., :h], y[..., h:2 * h] = z.real, z.imag
    return y


def forward(x, gamma, pos, rope_dims=42, rope_base=10000.0, eps=1e-6):
    """x [T, H, D] -> the normalised, rotated rows."""
    x = _f64(x)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * _f64(gamma)
    return _turn(y, _f64(pos), rope_dims, rope_base, 1.0)


def backward(x, gamma, pos, dy, rope_dims=42, rope_base=10000.0, eps=1e-6):
    """(dx, dgamma) of sum(dy * forward(x))."""
    x, gamma = _f64(x), _f64(gamma)
    rms = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = _turn(_f64(dy), _f64(pos), rope_dims, rope_base, -1.0)
    dgamma = (u * x / rms).sum((0, 1))
    u = u * gamma
    return u / rms - x * (u * x).mean(-1, keepdims=True) / rms ** 3, dgamma
