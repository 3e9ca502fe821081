"""Layers and losses of a batch without rows (an expert that received no token), on the GPU."""
import pytest
import torch

import vocab_selected_token_tile_gb300 as rlk
from vocab_selected_token_tile_gb300.autograd import fp8_linear, linear_cross_entropy

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("lead", [(0,), (3, 0), (0, 5)])
@pytest.mark.parametrize("need_x,need_w", [(True, True), (True, False), (False, True)])
def test_fp8_linear_of_no_rows(built, lead, need_x, need_w):
    x = torch.empty((*lead, 200), dtype=torch.bfloat16, device="cuda", requires_grad=need_x)
    w = torch.randn((130, 200), device="cuda", requires_grad=need_w)
    y = fp8_linear(x, w)
    assert y.shape == (*lead, 130) and y.dtype == torch.bfloat16
    y.backward(torch.empty_like(y))
    if need_x:
        assert x.grad.shape == x.shape
    if need_w:
        assert w.grad.shape == w.shape and w.grad.dtype == torch.float32 and (w.grad == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_over_no_elements(built, dtype):
    q, s = rlk.fp8_quantize(torch.empty((0, 40), dtype=torch.bfloat16, device="cuda"), transpose=True)
    b, sb = rlk.fp8_quantize(torch.empty((0, 70), dtype=torch.bfloat16, device="cuda"), transpose=True)
    assert q.shape == (40, 0) and b.shape == (70, 0)
    out = rlk.fp8_matmul(q, s, b, sb, b_block_rows=1, out_dtype=dtype)
    assert out.shape == (40, 70) and out.dtype == dtype and (out == 0).all()
    buf = torch.full((40, 80), 5.0, dtype=dtype, device="cuda")
    rlk.fp8_matmul(q, s, b, sb, b_block_rows=1, out=buf[:, :70])
    assert (buf[:, :70] == 0).all() and (buf[:, 70:] == 5).all()
    total = torch.full((40, 70), 2.0, device="cuda")
    assert rlk.fp8_matmul(q, s, b, sb, b_block_rows=1, out=total, accumulate=True) is total and (total == 2).all()


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("need_h,need_w", [(True, True), (True, False), (False, True)])
def test_cross_entropy_of_no_rows(built, reduction, need_h, need_w):
    h = torch.empty((0, 96), dtype=torch.bfloat16, device="cuda", requires_grad=need_h)
    w = torch.randn((50, 96), device="cuda").to(torch.bfloat16).requires_grad_(need_w)
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    loss = linear_cross_entropy(h, w, t, None, reduction=reduction)
    assert loss.shape == ((0,) if reduction == "none" else ()) and (loss == 0).all()
    loss.sum().backward()
    if need_h:
        assert h.grad.shape == (0, 96)
    if need_w:
        assert (w.grad == 0).all()
