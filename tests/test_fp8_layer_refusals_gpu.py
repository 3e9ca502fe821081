"""What the FP8 layers' calls refuse before any launch: host memory, tensors of other shapes, types and layouts."""
import numpy as np
import pytest
import torch

import vocab_selected_token_tile_gb300 as rlk
from vocab_selected_token_tile_gb300 import autograd

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def cuda(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def dense():
    return dict(zip(("a", "a_scale", "b", "b_scale"), (*rlk.fp8_quantize(cuda(10, 256)), *rlk.fp8_quantize(cuda(128, 256), 128))))


def grouped():
    d = dict(zip(("a", "a_scale", "b", "b_scale"), (*rlk.fp8_quantize(cuda(10, 256)), *rlk.fp8_quantize(cuda(3, 128, 256), 128))))
    return {**d, "ends": torch.tensor([2, 5, 9], dtype=torch.int32, device="cuda")}


E4 = torch.float8_e4m3fn


@pytest.mark.parametrize("error,change", [
    (ValueError, dict(a=lambda: cuda(10, 128, dtype=E4))), (TypeError, dict(a=lambda: cuda(10, 256))),
    (ValueError, dict(a=lambda: cuda(10, 256, dtype=E4).cpu())), (ValueError, dict(a_scale=lambda: cuda(2, 11, dtype=torch.float32))),
    (ValueError, dict(a_scale=lambda: cuda(2, 10))), (ValueError, dict(b_scale=lambda: cuda(1, 2, dtype=torch.float32))),
    (ValueError, dict(b_scale=lambda: cuda(2, 1, dtype=torch.float32).cpu())), (ValueError, dict(activation=lambda: "tanh")),
    (ValueError, dict(bias=lambda: cuda(127))), (TypeError, dict(bias=lambda: cuda(128, dtype=torch.float16))),
    (ValueError, dict(bias=lambda: cuda(256)[::2])), (ValueError, dict(residual=lambda: cuda(10, 127))),
    (TypeError, dict(residual=lambda: cuda(10, 128, dtype=torch.float16))), (ValueError, dict(residual=lambda: cuda(128, 10).t())),
    (TypeError, dict(out_dtype=lambda: torch.float16)), (ValueError, dict(out=lambda: cuda(10, 127))),
    (ValueError, dict(out=lambda: cuda(1, 128).expand(10, 128))),
    (ValueError, dict(out=lambda: cuda(10, 128), out_dtype=lambda: torch.float32)),
    (ValueError, dict(b=lambda: cuda(64 * 3, 256, dtype=E4), b_scale=lambda: cuda(2, 2, dtype=torch.float32), gated=lambda: True)),
])
def test_layer_tensors(built, error, change):
    with pytest.raises(error):
        rlk.fp8_matmul_act(**{**dense(), **{k: v() for k, v in change.items()}})


@pytest.mark.parametrize("error,change", [
    (TypeError, dict(ends=lambda: cuda(3, dtype=torch.int64))), (TypeError, dict(ends=lambda: cuda(3, dtype=torch.int32).cpu())),
    (TypeError, dict(ends=lambda: cuda(6, dtype=torch.int32)[::2])), (ValueError, dict(ends=lambda: cuda(4, dtype=torch.int32))),
    (ValueError, dict(b=lambda: cuda(128, 256, dtype=E4))), (ValueError, dict(b_scale=lambda: cuda(2, 1, dtype=torch.float32))),
    (ValueError, dict(bias=lambda: cuda(128))), (ValueError, dict(b=lambda: cuda(1, 128, 256, dtype=E4).expand(3, 128, 256))),
])
def test_group_tensors(built, error, change):
    with pytest.raises(error):
        rlk.fp8_grouped_matmul(**{**grouped(), **{k: v() for k, v in change.items()}})


@pytest.mark.parametrize("n", [0, 1025])
def test_numbers_of_groups(built, n):
    ends, x, w = cuda(n, dtype=torch.int32), cuda(10, 64), cuda(n, 32, 64)
    for call in (lambda: rlk.fp8_quantize_grouped(x, ends), lambda: rlk.fp8_act_grad(x, x, "relu", ends=ends),
                 lambda: autograd.fp8_grouped_linear(x, w, ends),
                 lambda: autograd.fp8_grouped_linear(x, w.requires_grad_(), ends, activation="relu")):
        with pytest.raises(ValueError):
            call()


def test_other_calls_tensors(built):
    ends = cuda(3, dtype=torch.int32)
    for call in (lambda: rlk.fp8_quantize(cuda(2, 128, 128), 1),                      # rows of several matrices
                 lambda: rlk.fp8_quantize(cuda(1, 128, 128).expand(2, 128, 128), 128),  # matrices that overlap
                 lambda: rlk.fp8_act_grad(cuda(5, 64), None, "silu"),
                 lambda: rlk.fp8_act_grad(cuda(5, 64), cuda(5, 64), "silu", gated=True),
                 lambda: rlk.fp8_act_grad(cuda(5, 64), cuda(4, 64), "relu"),
                 lambda: rlk.fp8_grouped_dweight(cuda(8, 128, dtype=E4), cuda(1, 8, dtype=torch.float32),
                                                 cuda(8, 128, dtype=E4), cuda(1, 8, dtype=torch.float32), ends, 10),
                 lambda: rlk.fp8_grouped_dweight(cuda(8, 384, dtype=E4), cuda(3, 8, dtype=torch.float32),
                                                 cuda(8, 384, dtype=E4), cuda(3, 8, dtype=torch.float32), ends, 10, accumulate=True),
                 lambda: autograd.fp8_linear(cuda(4, 64), cuda(32, 64), residual=cuda(32)),  # nothing is broadcast
                 lambda: autograd.fp8_linear(cuda(4, 64), cuda(32, 64).requires_grad_(), bias=cuda(31)),
                 lambda: autograd.fp8_linear(cuda(4, 64), cuda(96, 64).requires_grad_(), gated=True),
                 lambda: autograd.fp8_linear(cuda(4, 64), cuda(32, 60).requires_grad_(), activation="relu"),
                 lambda: autograd.fp8_grouped_linear(cuda(4, 64), cuda(2, 32, 64).requires_grad_(), ends),
                 lambda: autograd.fp8_grouped_linear(cuda(4, 64), cuda(32, 64), ends)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rlk.fp8_act_grad(cuda(5, 64), cuda(5, 64, dtype=torch.float32), "silu"),
                 lambda: rlk.fp8_act_grad(cuda(5, 64), cuda(5, 64), "silu", bias_dtype=torch.float16),
                 lambda: autograd.fp8_grouped_linear(cuda(4, 64), cuda(3, 32, 64).requires_grad_(), ends.long())):
        with pytest.raises(TypeError):
            call()


def test_host_memory(built):
    """Every pointer of the C calls in turn, from host memory: refused by name, and nothing is written."""
    d, g = dense(), grouped()
    host = np.zeros(1 << 16, np.uint8)
    host_at = (host.ctypes.data + 255) & ~255
    out = cuda(10, 128)
    z, bias, res = cuda(10, 128), cuda(128), cuda(10, 128)
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream

    def act(p):
        e = rlk.Fp8Epilogue(bias=p["bias"], residual=p["residual"], z=p["z"], residual_stride=128, z_stride=128)
        return rlk.rlk_fp8_matmul_act(10, 128, 256, p["a"], 256, p["a_scale"], p["b"], 256, p["b_scale"], e, p["c"],
                                      rlk.RLK_BF16, 128, p["workspace"], st)

    def group(p):
        return rlk.rlk_fp8_grouped_matmul(3, 10, 128, 256, p["ends"], p["a"], 256, p["a_scale"], p["b"], 256, 256 * 128,
                                          p["b_scale"], None, p["c"], rlk.RLK_BF16, 128, 1, p["workspace"], st)

    q, s, qt, sq = rlk.fp8_quantize_grouped(cuda(10, 128), g["ends"])
    dw = cuda(3, 128, 128)

    def quantize(p):
        return rlk.rlk_fp8_quantize_grouped(3, 10, 128, p["ends"], p["x"], 0, 128, p["q"], 128, p["scale"], p["qt"], 384,
                                            p["scale_t"], st)

    def dweight(p):
        return rlk.rlk_fp8_grouped_dweight(3, 10, 128, 128, p["ends"], p["a"], 384, p["a_scale"], p["b"], 384, p["b_scale"],
                                           p["c"], rlk.RLK_BF16, 128, 128 * 128, 0, p["workspace"], st)

    def grad(p):
        return rlk.rlk_fp8_act_grad(3, 10, 128, p["ends"], p["dy"], 0, 128, p["z"], 128, 2, 0, p["q"], 128, p["scale"],
                                    p["qt"], 384, p["scale_t"], p["dbias"], 0, p["workspace"], st)

    qt2, sq2, x = cuda(128, 384, dtype=torch.uint8), cuda(3, 128, dtype=torch.float32), cuda(10, 128)
    db = cuda(3, 128)
    calls = [
        (act, dict(a=d["a"], a_scale=d["a_scale"], b=d["b"], b_scale=d["b_scale"], bias=bias, residual=res, z=z, c=out, workspace=ws)),
        (group, dict(ends=g["ends"], a=g["a"], a_scale=g["a_scale"], b=g["b"], b_scale=g["b_scale"], c=out, workspace=ws)),
        (quantize, dict(ends=g["ends"], x=x, q=q, scale=s, qt=qt, scale_t=sq)),
        (dweight, dict(ends=g["ends"], a=qt, a_scale=sq, b=qt2, b_scale=sq2, c=dw, workspace=ws)),
        (grad, dict(ends=g["ends"], dy=x, z=z, q=q, scale=s, qt=qt, scale_t=sq, dbias=db, workspace=ws)),
    ]
    for call, tensors in calls:
        p = {k: v.data_ptr() for k, v in tensors.items()}
        for name in p:
            st_ = call({**p, name: host_at})
            assert st_ == rlk.RLK_ERR_INVALID_ARG, (call.__name__, name)
            message = rlk.rlk_last_error_message()  # the operand that names the device is not named itself
            assert name in message or (name in ("a", "x", "dy") and "device buffers" in message)
        assert call(p) == rlk.RLK_OK, rlk.rlk_last_error_message()
    torch.cuda.synchronize()
    assert not host.any()
