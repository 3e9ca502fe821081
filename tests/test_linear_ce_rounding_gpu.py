"""The cross entropy where its roundings or its accepted options could carry a bias, against 64 bits, on the GPU."""
import pytest
import torch

from vocab_selected_token_tile_gb300.autograd import linear_cross_entropy

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("eps", [0.0, 0.05, 0.1, 0.3, 0.6])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_smoothed_targets_rows_have_no_bias(built, reduction, eps):
    # hidden is positive and the targets' logits about -40, so that every row's entry for its target is
    # -(1 - eps) - eps / V to within e^-40, and dweight's rows of targets are sums of hidden times it
    T, V, H, rows = 512, 2048, 64, 32
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = (torch.randn((T, H), generator=gen, device="cuda").abs() + 0.5).to(torch.bfloat16)
    w = (torch.randn((V, H), generator=gen, device="cuda") * 0.02).to(torch.bfloat16)
    w[:rows] = -0.5
    t = torch.arange(T, device="cuda") % rows
    wr = w.clone().requires_grad_()
    loss = linear_cross_entropy(h, wr, t, None, reduction=reduction, label_smoothing=eps)
    loss.sum().mul(0.7).backward()
    y = h.double() @ w.double().t()
    d = torch.softmax(y, dim=1) - eps / V
    d[torch.arange(T, device="cuda"), t] -= 1 - eps
    want = (d.t() @ h.double())[:rows] * 0.7 / (T if reduction == "mean" else 1)
    off = float((wr.grad[:rows].double() / want - 1).mean())
    # each of the 2048 elements is rounded to BF16, by 2^-8 of it at most and evenly to both sides: five standard
    # deviations of their mean; an entry of -1 - eps / (V (1 - eps)) is rounded to -1
    assert abs(off) <= 5 * 2.0 ** -8 / 3 ** 0.5 / (rows * H) ** 0.5 + eps / (V * (1 - eps)) + 1e-6
