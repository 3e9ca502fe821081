"""The FP8 operators from their definitions, in plain numpy with 64-bit sums (test infrastructure only)."""
import numpy as np

GROUP = 128


def e4m3(v):
    """The nearest E4M3 value of each float64 (ties to even, saturating at 448, NaN stays)."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -6))  # |v| = m 2^e with m in [0.5, 1)
    step = np.exp2(e - 1.0 - 3.0)                      # 8 steps a binade; subnormals share the smallest binade's
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def groups(n):
    return -(-n // GROUP)


def quantize(x, block_rows):
    """(values, scale, dequantised) of x [R, C] (float32 or BF16 values as float32); scale is [groups(C), R / block]."""
    x = np.asarray(x, dtype=np.float32)
    R, C = x.shape
    scale = np.empty((groups(C), -(-R // block_rows)), np.float32)
    q = np.empty((R, C))
    with np.errstate(all="ignore"):
        for g in range(groups(C)):
            for b in range(scale.shape[1]):
                rs, cs = slice(b * block_rows, (b + 1) * block_rows), slice(g * GROUP, (g + 1) * GROUP)
                piece = x[rs, cs]
                amax = np.float32(np.max(np.abs(piece)))  # NaN if any is
                s = np.float32(np.maximum(amax, np.float32(2.0 ** -100)) / np.float32(448.0))
                r = np.float32(np.float32(1.0) / s)
                scale[g, b] = s
                q[rs, cs] = e4m3((piece * r).astype(np.float32))
    return q, scale


def expand(scale, rows, cols, block_rows):
    """The scale of every element [rows, cols], float64."""
    s = np.repeat(scale.T.astype(np.float64), block_rows, axis=0)[:rows]
    return np.repeat(s, GROUP, axis=1)[:, :cols]


def matmul(a, sa, b, sb, b_block_rows):
    """(product, sum of the terms' magnitudes) in 64 bits of float64 values a [M, K], b [N, K]."""
    da = a * expand(sa, a.shape[0], a.shape[1], 1)
    db = b * expand(sb, b.shape[0], b.shape[1], b_block_rows)
    return da @ db.T, np.abs(da) @ np.abs(db).T


def bound(K, terms):
    """How far an FP32 sum of the product may be from 64 bits.

    A group's sum takes at most 128 additions, its scaling and addition to the total 3 roundings, and the total one
    more a group; each is at most 2^-23 of the sum of the terms' magnitudes (2^-24 where it rounds to nearest, 2^-23
    where the tensor core truncates).
    """
    n = min(K, GROUP) + 3 + groups(K)
    return n * 2.0 ** -23 * terms + 1e-37
