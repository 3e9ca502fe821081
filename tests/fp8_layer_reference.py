"""The layers of 8-bit feed-forward blocks from their definitions, in plain numpy with 64 bits (test infrastructure only).

z = A B^T + bias; y = act(z), or act(gate) * other, + residual; dz from dy and z.
"""
import math

import numpy as np

import fp8_reference as ref

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
_erf = np.vectorize(math.erf, otypes=[np.float64])
_C = math.sqrt(2.0 / math.pi)


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(z, kind):
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "silu":
        return z * _sigmoid(z)
    if kind == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(_C * (z + 0.044715 * z ** 3)))
    return z


def slope(z, kind):
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "silu":
        s = _sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    if kind == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        t = np.tanh(_C * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def forward(z, kind, gated):
    n = z.shape[1] // 2
    return act(z[:, :n], kind) * z[:, n:] if gated else act(z, kind)


def backward(z, dy, kind, gated):
    n = dy.shape[1]

    def through(g, x):
        return np.where(x > 0, g, 0.0) if kind == "relu" else g * slope(x, kind)

    if gated:
        return np.concatenate((through(dy * z[:, n:], z[:, :n]), dy * act(z[:, :n], kind)), axis=1)
    return through(dy, z)


def act_error(z, kind):
    """How far the FP32 evaluation of act may be from 64 bits.

    e^x, the reciprocal that two values share and the products around them are within 2^-20 of the value together;
    gelu's distribution is within 1.5e-7 / 2, so 2e-7 |z| with its roundings.  The exponent u (|u| up to 1.6 |z| (1 +
    0.045 z^2)) is rounded to 2^-22 of itself, which moves s(u) by |u| s (1 - s) 2^-22 <= 2^-22 / 4 and the value by |z|
    times that.  Below its clamp silu is held at 40 s(-40) < 2e-16, and the gelus at less than 1e-14.
    """
    if kind in ("none", "relu"):
        return np.zeros_like(z)
    return 2.0 ** -20 * np.abs(act(z, kind)) + (2e-7 if kind == "gelu" else 2.0 ** -24) * np.minimum(np.abs(z), 60) + 1e-14


def layer(a, sa, b, sb, bias, kind, gated, residual):
    """(z, y, how far FP32 may be from z and from y) of float64 values a [M, K], b [rows, K] (blocks)."""
    z, terms = ref.matmul(a, sa, b, sb, 128)
    K = a.shape[1]
    dz = ref.bound(K, terms)
    if bias is not None:
        z = z + bias
        dz = dz + 2.0 ** -24 * np.abs(z)
    n = z.shape[1] // 2 if gated else z.shape[1]
    g, dg = z[:, :n], dz[:, :n]
    y = act(g, kind)
    # the slopes are at most 1.13 in magnitude
    err = 1.13 * dg + act_error(g, kind)
    if gated:
        u, du = z[:, n:], dz[:, n:]
        err = err * (np.abs(u) + du) + np.abs(y) * du
        y = y * u
        err = err + 2.0 ** -24 * np.abs(y)
    if residual is not None:
        y = y + residual
        err = err + 2.0 ** -24 * np.abs(y)
    return z, y, dz, err
