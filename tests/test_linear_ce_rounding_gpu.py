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


@pytest.mark.parametrize("cap", [0.01, 3.0, 30.0, 1e3, 1e5, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("sigma", [0.05, 1.0])  # logits up to about 1 and 16
def test_caps_of_any_size(built, cap, sigma):
    T, V, H = 130, 700, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn((V, H), generator=gen, device="cuda") * 0.5 * sigma).to(torch.bfloat16)
    t = torch.randint(0, V, (T,), generator=gen, device="cuda")
    hr, wr = h.clone().requires_grad_(), w.clone().requires_grad_()
    loss, lse = linear_cross_entropy(hr, wr, t, None, reduction="none", softcap=cap, return_lse=True)
    loss.sum().backward()
    h64, w64, u = h.double(), w.double(), 2.0 ** -23
    x = h64 @ w64.t()
    y = cap * torch.tanh(x / cap)
    slope = 1 / torch.cosh(x / cap) ** 2
    want = torch.logsumexp(y, dim=1)
    # a logit: H additions of at most u of the terms' magnitudes each; then of y itself the exponential's form has
    # 6 u at the worst (r = 2 / (e^(2v) + 1) at v >= 1/2: argument 8 v u / 2, result 2 u, division u, of r <= 0.54,
    # against y / cap >= 0.46) and the polynomial 2 u
    x_off = (H + 2) * u * (h64.abs() @ w64.abs().t())
    y_off = (slope * x_off + 8 * u * y.abs()).amax(dim=1)
    # the exponentials' arguments and results, V / 128 and 128 / 4 partial sums, the result's rounding
    lse_off = y_off + u * (4 * y.abs().amax(dim=1) + V / 128 + 64 + 8)
    assert ((lse.double() - want).abs() <= lse_off).all()
    rows = torch.arange(T, device="cuda")
    assert ((loss.double() - (want - y[rows, t])).abs() <= lse_off + y_off + 4 * u * (want.abs() + y.abs().amax(dim=1))).all()
    p = torch.exp(y - want[:, None])
    one = torch.nn.functional.one_hot(t, V)
    d = (p - one) * slope
    # the softmax's relative error; the slope's (x / cap's, twice over, and its exponential's argument); BF16's 2^-8
    rel = (2 * lse_off + 16 * u * (1 + want.abs()))[:, None]
    bent = 4 * x_off / cap + 8 * u * (2 + 2 * (x / cap).abs())
    err = 2.0 ** -8 * d.abs() + slope * (p * rel + (p + one) * (bent + 4 * u))
    for got, exact, e, terms, n in ((hr.grad, d @ w64, err @ w64.abs(), d.abs() @ w64.abs(), V + 600),
                                    (wr.grad, d.t() @ h64, err.t() @ h64.abs(), d.abs().t() @ h64.abs(), T + 16)):
        assert ((got.double() - exact).abs() <= e + n * u * terms + 2.0 ** -8 * exact.abs() + 1e-30).all()


def test_a_large_cap_is_no_cap(built):
    gen = torch.Generator(device="cuda").manual_seed(4)
    h = torch.randn((40, 96), generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.randn((500, 96), generator=gen, device="cuda").to(torch.bfloat16)
    t = torch.randint(0, 500, (40,), generator=gen, device="cuda")
    with torch.no_grad():
        # tanh(x) - x is below x^3 / 3: of no weight in 32 bits here
        assert torch.equal(linear_cross_entropy(h, w, t, None, reduction="none", softcap=1e20),
                           linear_cross_entropy(h, w, t, None, reduction="none"))
