"""FP8 layers in training: what autograd's functions give, against the public calls that they stand for."""
import numpy as np
import pytest
import torch

import vocab_selected_token_tile_gb300 as rlk
from vocab_selected_token_tile_gb300 import autograd

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

BF16, F32 = torch.bfloat16, torch.float32


def rand(*shape, seed, sigma=1.0, dtype=BF16):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * np.float32(sigma)
    return torch.from_numpy(x).cuda().to(dtype)


# ------------------------------------------------------------------ residuals that are views

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lead", [(7,), (150,), (3, 50), (2, 1)])
@pytest.mark.parametrize("kind", ["row expanded", "all expanded", "transposed"])
@pytest.mark.parametrize("n", [192, 1])
def test_residual_that_is_a_view(built, kind, lead, n, dtype):
    x, w = rand(*lead, 130, seed=1), rand(n, 130, seed=2, sigma=0.1)
    if kind == "row expanded":  # one row for all tokens, as a broadcast sum gives it
        base = rand(*([1] * len(lead)), n, seed=3, dtype=dtype)
        view = lambda t: t.expand(*lead, n)  # noqa: E731
    elif kind == "all expanded":
        base = rand(1, seed=3, dtype=dtype)
        view = lambda t: t.expand(*lead, n)  # noqa: E731
    else:
        base = rand(n, *lead[::-1], seed=3, dtype=dtype)
        view = lambda t: t.permute(*range(t.dim() - 1, -1, -1))  # noqa: E731
    dy = rand(*lead, n, seed=4)
    plain = view(base).contiguous()
    want = autograd.fp8_linear(x, w, activation="silu", residual=plain)
    assert torch.equal(autograd.fp8_linear(x, w, activation="silu", residual=view(base)), want)
    leaf = base.clone().requires_grad_()
    y = autograd.fp8_linear(x, w, activation="silu", residual=view(leaf))
    assert torch.equal(y.detach(), want)
    got, = torch.autograd.grad(y, leaf, dy)
    leaf = base.clone().requires_grad_()
    want_grad, = torch.autograd.grad(view(leaf), leaf, dy.to(dtype))
    assert torch.equal(got, want_grad)


def test_residual_without_columns(built):
    x, w = rand(2, 3, 64, seed=5), torch.zeros((0, 64), dtype=BF16, device="cuda")
    assert autograd.fp8_linear(x, w, residual=torch.zeros((2, 3, 0), dtype=BF16, device="cuda")).shape == (2, 3, 0)
