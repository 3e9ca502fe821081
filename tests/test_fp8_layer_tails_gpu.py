"""The activations over their whole range, where they vanish too: relative to their own value, not to their argument.

A product of zeros leaves the bias, which is then the activation's argument, exactly.  What FP32 may be off by:
silu and gelu_tanh, an exponent u = z or 2 v of up to 58 in magnitude rounded to 2^-24 of itself moves e^u by 58 * 2^-24 =
2^-18.1 at most; gelu_tanh's takes three roundings (z^2, its polynomial's and the product's), but above -7 it is at
most 36: 3 * 36 * 2^-24 = 2^-17.2; e^x, the sums and the reciprocal that two share are 6 * 2^-23 more.  gelu: Q's fit,
4.1e-5 of Q, and the exponent z^2 / 2 * log2 e of up to 104, two roundings of 2^-24 in a power of two: 8.6e-6, together
with those 6 * 2^-23 below 2^-14; and 3e-7 |z| for either sign (8e-8 of the fit, the rest six terms' roundings).
"""
import math

import numpy as np
import pytest
import torch

import vocab_selected_token_tile_gb300 as rlk

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def exact(z, act):
    if act == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    u = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    e = np.exp(-np.abs(u))
    return z * np.where(u >= 0, 1 / (1 + e), e / (1 + e))


def bound(z, act):
    y = np.abs(exact(z, act))
    if act == "silu":
        return np.where(z >= -40, 2.0 ** -18 + 6 * 2.0 ** -23, 0) * y + np.where(z >= -40, 0, 2e-16)
    if act == "gelu_tanh":
        return np.where(z >= -7, 2.0 ** -17 + 6 * 2.0 ** -23, 0) * y + np.where(z >= -7, 0, 3e-15)
    far = np.where(z >= -12, 2.0 ** -14 * y, 3e-32)
    return np.where(z < 0, np.minimum(far, np.maximum(3e-7 * np.abs(z), 3e-32)), 3e-7 * np.abs(z))


def arguments(low):
    near = np.concatenate([np.linspace(-14, 14, 2500), np.linspace(low, 60, 800)])
    tiny = np.logspace(-30, 0, 400)
    z = np.concatenate([near, tiny, -tiny]).astype(np.float32)
    return np.concatenate([z, np.full(-len(z) % 64, -5.5, np.float32)])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,K", [(2, 128), (2, 2048), (130, 128), (130, 2048), (600, 128)])
@pytest.mark.parametrize("groups", [0, 1])
def test_activations_relative_to_their_value(built, groups, M, K, gated, act):
    z = arguments(-50.0)
    n = len(z)
    rows = 2 * n if gated else n
    a, sa = rlk.fp8_quantize(torch.ones((M, K), dtype=torch.bfloat16, device="cuda"))
    b, sb = rlk.fp8_quantize(torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda"), block_rows=128)
    bias = torch.from_numpy(np.concatenate([z, np.ones(n, np.float32)]) if gated else z).cuda()
    if groups:
        ends = torch.tensor([M], dtype=torch.int32, device="cuda")
        got = rlk.fp8_grouped_matmul(a, sa, b[None], sb[None], ends, bias[None], act, gated, out_dtype=torch.float32)
    else:
        got = rlk.fp8_matmul_act(a, sa, b, sb, bias, act, gated, out_dtype=torch.float32)
    assert (got == got[0]).all()
    z = z.astype(np.float64)
    d = np.abs(got[0].double().cpu().numpy() - exact(z, act))
    worst = np.argmax(d / (bound(z, act) + 1e-37))
    assert np.all(d <= bound(z, act) + 1e-37), (z[worst], d[worst], bound(z, act)[worst])
