"""Forward-mode derivatives of the functions without a forward-mode rule are refused, not dropped (no GPU)."""
import pytest
import torch
from torch.autograd import forward_ad

from vocab_selected_token_tile_gb300 import autograd


@pytest.fixture
def stand_ins(monkeypatch):
    """The calls' results without the calls: only whether autograd is asked matters here."""
    monkeypatch.setattr(autograd, "linear_ce_contract", lambda *a: None)
    monkeypatch.setattr(autograd, "linear_ce_fwd", lambda c, h, w, t, m: (h.float().sum(1), h.float().sum(1)))
    monkeypatch.setattr(autograd, "fp8_quantize", lambda x, block_rows=1: (x, x))
    monkeypatch.setattr(autograd, "fp8_quantize_both", lambda x, block_rows=1: (x, x, x, x))
    monkeypatch.setattr(autograd, "fp8_matmul", lambda a, s, b, t: a.new_zeros((a.shape[0], b.shape[0])))


def functions():
    t = torch.zeros(3, dtype=torch.int64)
    return {"cross entropy": lambda x, w: autograd.linear_cross_entropy(x, w, t, reduction="none"),
            "linear": autograd.fp8_linear}


@pytest.mark.parametrize("name", ["cross entropy", "linear"])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("grad", [False, True])
def test_tangents_are_refused(stand_ins, name, which, grad):
    x, w = torch.ones(3, 8, requires_grad=grad), torch.ones(5, 8, requires_grad=grad)
    with forward_ad.dual_level():
        args = [x, w]
        args[which] = forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError):
            functions()[name](*args)
        with torch.no_grad(), pytest.raises(NotImplementedError):
            functions()[name](*args)


@pytest.mark.parametrize("name", ["cross entropy", "linear"])
def test_without_tangents_as_before(stand_ins, name):
    f = functions()[name]
    x, w = torch.ones(3, 8), torch.ones(5, 8)
    assert not f(x, w).requires_grad
    assert f(x, w.requires_grad_()).requires_grad
    with torch.no_grad():
        assert not f(x, w).requires_grad
    with forward_ad.dual_level():
        assert f(x, w).requires_grad and not f(x, w.detach()).requires_grad
