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


# ------------------------------------------------------------------ results in FP32

# The same sums, so a BF16 result is the FP32 one, rounded.
@pytest.mark.parametrize("kw", [{}, dict(activation="gelu"), dict(activation="silu", gated=True), dict(bias=True),
                                dict(residual=F32), dict(activation="relu", bias=True, residual=BF16)])
@pytest.mark.parametrize("lead", [(5,), (3, 67), (300,)])
@pytest.mark.parametrize("trained", [False, True])
def test_fp32_results(built, trained, lead, kw):
    kw, n = dict(kw), 192
    rows = 2 * n if kw.get("gated") else n
    x, w = rand(*lead, 200, seed=11), rand(rows, 200, seed=12, sigma=0.07, dtype=F32).requires_grad_(trained)
    if kw.get("bias"):
        kw["bias"] = rand(rows, seed=13, dtype=F32)
    if kw.get("residual"):
        kw["residual"] = rand(*lead, n, seed=14, sigma=30.0, dtype=kw["residual"])
    y = autograd.fp8_linear(x, w, **kw, out_dtype=F32)
    assert y.dtype == F32 and y.shape == (*lead, n) and y.requires_grad == trained
    short = autograd.fp8_linear(x, w, **kw)
    assert short.dtype == BF16 and torch.equal(short, y.to(BF16)) and not torch.equal(short.to(F32), y)
    assert torch.equal(autograd.fp8_linear(x, w, **kw, out_dtype=BF16), short)
    if trained:
        dy = rand(*lead, n, seed=15)
        # a BF16 gradient gives the same bits whichever type it is held in
        got, = torch.autograd.grad(y, w, dy.to(F32))
        want, = torch.autograd.grad(short, w, dy)
        assert torch.equal(got, want)


def test_an_fp32_stream_keeps_its_digits(built):
    x, w = rand(90, 64, seed=21), torch.zeros((128, 64), dtype=BF16, device="cuda")
    stream = rand(90, 128, seed=22, sigma=100.0, dtype=F32)
    assert torch.equal(autograd.fp8_linear(x, w, residual=stream, out_dtype=F32), stream)
    leaf = stream.clone().requires_grad_()
    y = autograd.fp8_linear(x, w, residual=leaf, out_dtype=F32)
    dy = rand(90, 128, seed=23, dtype=F32)
    assert torch.equal(y.detach(), stream) and torch.equal(torch.autograd.grad(y, leaf, dy)[0], dy)


@pytest.mark.parametrize("trained", [False, True])
@pytest.mark.parametrize("act,gated,bias", [(None, False, False), ("silu", True, True), ("gelu", False, False)])
def test_fp32_results_by_groups(built, trained, act, gated, bias):
    ends, M, n = torch.tensor([40, 40, 175], dtype=torch.int32, device="cuda"), 180, 128
    rows = 2 * n if gated else n
    x, w = rand(M, 136, seed=31), rand(3, rows, 136, seed=32, sigma=0.08).requires_grad_(trained)
    b = rand(3, rows, seed=33) if bias else None
    y = autograd.fp8_grouped_linear(x, w, ends, b, act, gated, out_dtype=F32)
    short = autograd.fp8_grouped_linear(x, w, ends, b, act, gated)
    assert y.dtype == F32 and short.dtype == BF16 and torch.equal(short, y.to(BF16)) and (y[175:] == 0).all()
    if trained:
        dy = rand(M, n, seed=34)
        assert torch.equal(torch.autograd.grad(y, w, dy.to(F32))[0], torch.autograd.grad(short, w, dy)[0])


@pytest.mark.parametrize("trained", [False, True])
def test_other_result_types_are_refused(built, trained):
    x, w = rand(4, 64, seed=41), rand(128, 64, seed=42).requires_grad_(trained)
    ends = torch.tensor([4], dtype=torch.int32, device="cuda")
    for call in (lambda: autograd.fp8_linear(x, w, out_dtype=torch.float16),
                 lambda: autograd.fp8_linear(x, w, activation="relu", out_dtype=torch.float64),
                 lambda: autograd.fp8_grouped_linear(x, w[None], ends, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
