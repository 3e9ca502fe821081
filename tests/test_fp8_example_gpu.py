"""The FP8 fine-tuning example runs, learns, and its 8-bit head scores like the BF16 one."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_learns_and_the_8_bit_head_agrees(built):
    import fp8_finetune
    net, losses, after = fp8_finetune.train(steps=80)
    # from about ln(1000) = 6.9; label smoothing keeps a floor of about 0.05 ln(1000) + entropy = 0.55
    assert losses[0] > 5.0 and losses[-1] < 0.5 * losses[0]
    rolled, trained, spread = fp8_finetune.rollout_drift(net, after)
    # E4M3 rounds each factor by at most 2^-4 of itself: products by 2^-3.5 at the worst in either direction at random,
    # a logit (a sum over 192 of them) by no more than 2^-3 of the logits' deviation at five standard errors; the
    # log-sum-exp moves by as much again, and BF16 rounds a logit of up to 32 by 2^-4
    assert torch.isfinite(rolled).all()
    assert float((rolled - trained).abs().max()) <= 2 * spread * 2.0 ** -3 + 2.0 ** -4
