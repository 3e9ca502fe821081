"""Calls with a ``stream`` of their own leave the memory alone that the current stream still uses, on the GPU."""
import pytest
import torch

import vocab_selected_token_tile_gb300 as rlk

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

T, V, H = 512, 1024, 1024


def operands():
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn((V, H), generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    return h, w, torch.randint(0, V, (T,), generator=gen, device="cuda")


def calls():
    """(a call on a given stream, the shapes and types of what it allocates) of each kind."""
    h, w, t = operands()
    c = rlk.linear_ce_contract(h, w, reduction=rlk.REDUCE_NONE)
    lse = rlk.linear_ce_fwd(c, h, w, t)[1]
    g = torch.ones(T, device="cuda")
    q, s = rlk.fp8_quantize(h)
    qw, sw = rlk.fp8_quantize(w, block_rows=128)
    f32, bf16, u8 = torch.float32, torch.bfloat16, torch.uint8
    ws = [((rlk.rlk_linear_ce_workspace_size(c, k),), u8) for k in (0, 1)]
    return {
        "quantize": (lambda st: rlk.fp8_quantize_both(h, stream=st), [((T, H), u8), ((H // 128, T), f32),
                                                                     ((H, T), u8), ((T // 128, H), f32)]),
        "matmul": (lambda st: (rlk.fp8_matmul(q, s, qw, sw, stream=st),), [((T, V), bf16)]),
        "ce": (lambda st: rlk.linear_ce_fwd(c, h, w, t, stream=st), [((T,), f32), ((T,), f32), ws[0]]),
        "ce gradients": (lambda st: rlk.linear_ce_bwd(c, h, w, t, None, lse, g, stream=st),
                         [((T, H), bf16), ((V, H), bf16), ws[1]]),
    }


@pytest.mark.parametrize("kind", ["quantize", "matmul", "ce", "ce gradients"])
def test_freed_memory_of_the_current_stream_is_not_written(built, kind):
    call, shapes = calls()[kind]
    want = [r.clone() for r in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # memory of the sizes that the call asks for, in use by copies that are queued here and freed at once
    old = [torch.full(shape, 3, dtype=dtype, device="cuda") for shape, dtype in shapes]
    places = {o.data_ptr() for o in old}
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # some 10 ms: the other stream's work is done before the copies begin
    copies = [o.clone() for o in old]
    del old
    got = call(side)
    assert not places & {r.data_ptr() for r in got}
    side.synchronize()
    torch.cuda.synchronize()
    assert all((c == 3).all() for c in copies)
    assert all(torch.equal(a.float(), b.float()) for a, b in zip(got, want))


def test_results_outlive_work_queued_here(built):
    # a result of the other stream's memory, read here and freed: not handed to that stream before it has been read
    h, _, _ = operands()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    q, s = rlk.fp8_quantize(h, stream=side)
    side.synchronize()
    want = q.view(torch.uint8).clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    copy = q.view(torch.uint8).clone()
    del q, s
    with torch.cuda.stream(side):
        junk = [torch.full((T, H), 9, dtype=torch.uint8, device="cuda") for _ in range(4)]
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(junk) == 4
