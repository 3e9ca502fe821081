"""The cross entropy of hidden @ weight^T from its definition, in plain numpy with 64 bits (test infrastructure only)."""
import numpy as np


def forward(hidden, weight, targets, active, eps=0.0, z=0.0, cap=0.0):
    """(loss [T], lse [T], y [T, V]): 0 on inactive rows; inactive targets may hold anything."""
    x = hidden.astype(np.float64) @ weight.astype(np.float64).T
    y = cap * np.tanh(x / cap) if cap else x
    top = y.max(axis=1)
    lse = top + np.log(np.exp(y - top[:, None]).sum(axis=1))
    t = np.where(active, targets, 0)
    loss = lse - (1 - eps) * y[np.arange(len(t)), t] - eps * y.mean(axis=1) + z * lse ** 2
    return np.where(active, loss, 0.0), lse, y


def reduce(loss, active, reduction):
    n = int(active.sum())
    return loss if reduction == "none" else loss.sum() if reduction == "sum" else loss.sum() / n if n else 0.0


def row_gradients(g, active, reduction):
    """The gradient of each row's loss from that of the reduced one."""
    n = int(active.sum())
    if reduction == "mean":
        g = g / n if n else 0.0
    return np.where(active, np.broadcast_to(np.asarray(g, np.float64), active.shape), 0.0)


def logits_gradient(y, lse, targets, active, rows, eps=0.0, z=0.0, cap=0.0):
    """d loss / d logits [T, V], and its parts' magnitudes: the softmax's, the target distribution's, the cap's slope."""
    V = y.shape[1]
    p = np.exp(y - lse[:, None]) * (1 + 2 * z * lse)[:, None]
    want = np.full_like(y, eps / V)
    want[np.arange(len(targets)), np.where(active, targets, 0)] += 1 - eps
    slope = 1 - (y / cap) ** 2 if cap else np.ones_like(y)
    on, r = active[:, None], rows[:, None]
    return np.where(on, r * (p - want) * slope, 0.0), np.where(on, np.abs(r * p), 0.0), np.where(on, np.abs(r * want), 0.0), slope


def backward(hidden, weight, targets, active, rows, eps=0.0, z=0.0, cap=0.0):
    _, lse, y = forward(hidden, weight, targets, active, eps, z, cap)
    d = logits_gradient(y, lse, targets, active, rows, eps, z, cap)[0]
    return d @ weight.astype(np.float64), d.T @ hidden.astype(np.float64)


def logit_bound(hidden, weight, cap=0.0):
    """[T] largest error of a row's FP32 logits: H additions of at most 2^-23 of the terms' magnitudes each; a cap adds
    a few roundings of tanh (each 2^-23 of 1) and of the products around it, times the cap."""
    terms = (np.abs(hidden).astype(np.float64) @ np.abs(weight).astype(np.float64).T).max(axis=1)
    return (hidden.shape[1] + 2) * 2.0 ** -23 * terms + 8 * 2.0 ** -23 * cap


def lse_bound(hidden, weight, y, cap=0.0):
    """The logits' error, the exponentials' (argument and result a few 2^-23 each, relative; the argument's range is
    the logits') and the sum's (V / 256 merges and 256 / 4 additions, relative), and the result's rounding."""
    span = np.abs(y).max(axis=1)
    n = y.shape[1] / 256 + 64 + 16
    return logit_bound(hidden, weight, cap) + 2.0 ** -23 * (4 * span + n + 8)


def loss_bound(hidden, weight, y, lse, eps, z, cap):
    b = lse_bound(hidden, weight, y, cap)
    mean = np.abs(y).mean(axis=1) * 2.0 ** -23 * (y.shape[1] / 256 + 64)  # the sum over the classes
    return b * (2 + 2 * z * np.abs(lse)) + eps * mean + 4 * 2.0 ** -23 * (np.abs(lse) * (1 + z * np.abs(lse)) + np.abs(y).max(axis=1))


def gradient_bounds(hidden, weight, y, lse, targets, active, rows, eps, z, cap, scale):
    """([T, H], [V, H]) how far BF16 gradients may be.

    The softmax has the logits' and lse's errors (relative) and a few roundings of its argument; the cap's slope the
    logits' error over the cap, twice, and a few roundings of its exponential's argument (2 |x| / cap); dx is rounded to BF16, whose unit roundoff is
    2^-8, summed in FP32 (2^-23 an addition), and the result is rounded to BF16.
    """
    h, w = np.abs(hidden).astype(np.float64), np.abs(weight).astype(np.float64)
    d, p, want, slope = logits_gradient(y, lse, targets, active, rows, eps, z, cap)
    u = 2.0 ** -23
    rel = 2 * lse_bound(hidden, weight, y, cap) + 16 * u * (1 + np.abs(lse))
    bent = 4 * logit_bound(hidden, weight, cap) / cap + 8 * u * (2 + 2 * (h @ w.T).max(axis=1) / cap) if cap else 0 * lse
    ad = np.abs(d)
    err = 2.0 ** -8 * ad + slope * (p * rel[:, None] + (p + want) * (bent + 4 * u)[:, None])
    tiny = 1e-30 * max(1.0, abs(scale))
    dh, dw = d @ weight.astype(np.float64), d.T @ hidden.astype(np.float64)
    bh = err @ w + (y.shape[1] + 600) * u * (ad @ w) + 2.0 ** -8 * np.abs(dh) + tiny
    bw = err.T @ h + (len(lse) + 16) * u * (ad.T @ h) + 2.0 ** -8 * np.abs(dw) + tiny
    return bh, bw
