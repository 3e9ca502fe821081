"""Forward-mode derivatives of the FP8 layers are refused, not dropped (no GPU)."""
import pytest
import torch
from torch.autograd import forward_ad

from vocab_selected_token_tile_gb300 import autograd


class Step:
    """The layer's calls without the calls: only whether autograd is asked matters here."""

    def __init__(self, x, weight, *rest):
        self.n = weight.shape[-2]

    def forward(self, x, weight):
        return x.new_zeros((x.shape[0], self.n)), None, None


@pytest.fixture
def stand_ins(monkeypatch):
    monkeypatch.setattr(autograd, "Fp8LayerStep", Step)
    monkeypatch.setattr(autograd, "fp8_quantize", lambda x, block_rows=1: (x, x))
    monkeypatch.setattr(autograd, "fp8_matmul_act", lambda a, s, b, t, *k: a.new_zeros((a.shape[0], b.shape[0])))
    monkeypatch.setattr(autograd, "fp8_grouped_matmul", lambda a, s, b, t, *k: a.new_zeros((a.shape[0], b.shape[1])))


def dense(x, w, b, r):
    return autograd.fp8_linear(x, w, bias=b, activation="gelu", residual=r)


def grouped(x, w, b, r):
    return autograd.fp8_grouped_linear(x, torch.stack((w, w)), torch.tensor([1, 3], dtype=torch.int32), torch.stack((b, b)))


def inputs(grad=False):
    return [torch.ones(s, requires_grad=grad) for s in ((3, 8), (5, 8), (5,), (3, 5))]


@pytest.mark.parametrize("f,which", [(dense, 0), (dense, 1), (dense, 2), (dense, 3), (grouped, 0), (grouped, 1), (grouped, 2)])
@pytest.mark.parametrize("grad", [False, True])
def test_tangents_are_refused(stand_ins, f, which, grad):
    args = inputs(grad)
    with forward_ad.dual_level():
        args[which] = forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError):
            f(*args)
        with torch.no_grad(), pytest.raises(NotImplementedError):
            f(*args)


@pytest.mark.parametrize("f", [dense, grouped])
def test_without_tangents(stand_ins, f):
    assert not f(*inputs()).requires_grad
    for k in range(4 if f is dense else 3):
        args = inputs()
        args[k].requires_grad_()
        assert f(*args).requires_grad
        with torch.no_grad():
            assert not f(*args).requires_grad
