"""A layer's backward composed from the public calls, of a batch without rows."""
import pytest
import torch

import vocab_selected_token_tile_gb300 as rlk

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("bias_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act,gated", [(None, False), ("gelu", False), ("silu", True)])
@pytest.mark.parametrize("groups", [0, 3])
@pytest.mark.parametrize("own_stream", [False, True])
def test_act_grad_of_no_rows(built, groups, act, gated, bias_dtype, own_stream):
    N, K = 64, 96
    wide = 2 * N if gated else N
    ends = torch.zeros(groups, dtype=torch.int32, device="cuda") if groups else None
    dy, z = (torch.zeros((0, n), dtype=torch.bfloat16, device="cuda") for n in (N, wide))
    stream = torch.cuda.Stream() if own_stream else None
    q, s, qt, st, db = rlk.fp8_act_grad(dy, z, act, gated, ends=ends, bias_dtype=bias_dtype, stream=stream)
    torch.cuda.synchronize()
    assert q.shape == (0, wide) and s.shape == (-(-wide // 128), 0)
    assert qt.shape == (wide, 0) and st.shape == (0, wide)
    assert db.shape == ((groups, wide) if groups else (wide,)) and db.dtype == bias_dtype and (db == 0).all()
    only = rlk.fp8_act_grad(dy, z, act, gated, ends=ends, transpose=False)
    assert only[2] is None and only[3] is None and only[4] is None and only[0].shape == (0, wide)
    # and what follows takes these
    if groups:
        w, ws = rlk.fp8_quantize(torch.ones((groups, K, wide), dtype=torch.bfloat16, device="cuda"), block_rows=128)
        assert rlk.fp8_grouped_matmul(q, s, w, ws, ends).shape == (0, K)
        xt = rlk.fp8_quantize_grouped(torch.zeros((0, K), dtype=torch.bfloat16, device="cuda"), ends, rowwise=False)
        dw = rlk.fp8_grouped_dweight(qt, st, xt[2], xt[3], ends, 0)
        assert dw.shape == (groups, wide, K) and (dw == 0).all()
    else:
        w, ws = rlk.fp8_quantize(torch.ones((K, wide), dtype=torch.bfloat16, device="cuda"), block_rows=128)
        assert rlk.fp8_matmul(q, s, w, ws).shape == (0, K)
        xt, xts = rlk.fp8_quantize(torch.zeros((0, K), dtype=torch.bfloat16, device="cuda"), transpose=True)
        dw = rlk.fp8_matmul(qt, st, xt, xts, b_block_rows=1)
        assert dw.shape == (wide, K) and (dw == 0).all()


def test_act_grad_of_no_rows_still_checks(built):
    dy = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        rlk.fp8_act_grad(dy, None, "silu")
    with pytest.raises(ValueError):
        rlk.fp8_act_grad(dy, dy, "silu", gated=True)
    with pytest.raises(TypeError):
        rlk.fp8_act_grad(dy, bias_dtype=torch.float16)
