"""The status word of the FP8 product reports an expired wait once, on the GPU."""
import pytest
import torch

import vocab_selected_token_tile_gb300 as rlk

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

TIMEOUT_BIT = 4  # what a kernel sets in the status word when a wait expires


@pytest.mark.parametrize("own_stream", [False, True])
def test_a_time_out_is_reported_once(built, own_stream):
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, s = rlk.fp8_quantize(torch.randn((5, 300), generator=gen, device="cuda"))
    b, t = rlk.fp8_quantize(torch.randn((200, 300), generator=gen, device="cuda"), block_rows=128)
    torch.cuda.synchronize()
    st = torch.cuda.Stream() if own_stream else None
    want = rlk.fp8_matmul(a, s, b, t, validate=True, stream=st)
    raw = (st or torch.cuda.current_stream()).cuda_stream
    word = rlk._fp8_workspaces[(a.device.index, raw)].view(torch.int32)
    word[0] = TIMEOUT_BIT  # as a call before that was not validated leaves it
    torch.cuda.synchronize()
    with pytest.raises(rlk.RlkError) as e:
        rlk.fp8_matmul(a, s, b, t, validate=True, stream=st)
    assert e.value.status == rlk.RLK_ERR_TIMEOUT
    got = rlk.fp8_matmul(a, s, b, t, validate=True, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_a_workspace_of_the_callers_keeps_it(built):
    a, s = rlk.fp8_quantize(torch.ones((5, 300), device="cuda"))
    b, t = rlk.fp8_quantize(torch.ones((200, 300), device="cuda"), block_rows=128)
    ws = torch.zeros(rlk.RLK_FP8_WORKSPACE, dtype=torch.uint8, device="cuda")
    ws.view(torch.int32)[0] = TIMEOUT_BIT
    for _ in range(2):
        with pytest.raises(rlk.RlkError):
            rlk.fp8_matmul(a, s, b, t, validate=True, workspace=ws)
    ws.zero_()
    rlk.fp8_matmul(a, s, b, t, validate=True, workspace=ws)
