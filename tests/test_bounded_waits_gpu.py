"""Waits of a CTA pair's kernels that run out: a status, and a context that goes on, on the GPU."""
import pytest
import torch

import vocab_selected_token_tile_gb300 as rlk

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def test_expired_waits_are_reported_and_leave_a_usable_context(built):
    # one tile's K range takes 4.4 ms here, and a limit of 1 ns ends a wait at its 512th poll, after about 2 ms
    T, V, H = 8, 512, 1 << 20
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.empty((V, H), dtype=torch.bfloat16, device="cuda").normal_(0.0, 0.001, generator=gen)
    t = torch.randint(0, V, (T,), generator=gen, device="cuda")
    one = torch.ones((), device="cuda")
    c = rlk.linear_ce_contract(h, w, reduction=rlk.REDUCE_SUM, validate=1)
    short = c.replace(wait_timeout_ns=1)
    loss, lse = rlk.linear_ce_fwd(c, h, w, t)
    dh, dw = rlk.linear_ce_bwd(c, h, w, t, None, lse, one)
    for _ in range(3):
        with pytest.raises(rlk.RlkError) as e:
            rlk.linear_ce_fwd(short, h, w, t)
        assert e.value.status == rlk.RLK_ERR_TIMEOUT
        with pytest.raises(rlk.RlkError) as e:
            rlk.linear_ce_bwd(short, h, w, t, None, lse, one)
        assert e.value.status == rlk.RLK_ERR_TIMEOUT
        again, lse2 = rlk.linear_ce_fwd(c, h, w, t)
        assert torch.equal(again, loss) and torch.equal(lse2, lse)
        got = rlk.linear_ce_bwd(c, h, w, t, None, lse, one)
        assert torch.equal(got[0], dh) and torch.equal(got[1], dw)
