"""FP8 layers in training: what autograd's functions give, against the public calls that they stand for."""
import numpy as np
import pytest
import torch

import vocab_selected_token_tile_gb300 as rlk
from vocab_selected_token_tile_gb300 import autograd

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

BF16, F32 = torch.bfloat16, torch.float32


def rand(*shape, seed, sigma=1.0, dtype=BF16):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * np.float32(sigma)
    return torch.from_numpy(x).cuda().to(dtype)


# ------------------------------------------------------------------ residuals that are views

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lead", [(7,), (150,), (3, 50), (2, 1)])
@pytest.mark.parametrize("kind", ["row expanded", "all expanded", "transposed"])
@pytest.mark.parametrize("n", [192, 1])
def test_residual_that_is_a_view(built, kind, lead, n, dtype):
    x, w = rand(*lead, 130, seed=1), rand(n, 130, seed=2, sigma=0.1)
    if kind == "row expanded":  # one row for all tokens, as a broadcast sum gives it
        base = rand(*([1] * len(lead)), n, seed=3, dtype=dtype)
        view = lambda t: t.expand(*lead, n)  # noqa: E731
    elif kind == "all expanded":
        base = rand(1, seed=3, dtype=dtype)
        view = lambda t: t.expand(*lead, n)  # noqa: E731
    else:
        base = rand(n, *lead[::-1], seed=3, dtype=dtype)
        view = lambda t: t.permute(*range(t.dim() - 1, -1, -1))  # noqa: E731
    dy = rand(*lead, n, seed=4)
    plain = view(base).contiguous()
    want = autograd.fp8_linear(x, w, activation="silu", residual=plain)
    assert torch.equal(autograd.fp8_linear(x, w, activation="silu", residual=view(base)), want)
    leaf = base.clone().requires_grad_()
    y = autograd.fp8_linear(x, w, activation="silu", residual=view(leaf))
    assert torch.equal(y.detach(), want)
    got, = torch.autograd.grad(y, leaf, dy)
    leaf = base.clone().requires_grad_()
    want_grad, = torch.autograd.grad(view(leaf), leaf, dy.to(dtype))
    assert torch.equal(got, want_grad)


def test_residual_without_columns(built):
    x, w = rand(2, 3, 64, seed=5), torch.zeros((0, 64), dtype=BF16, device="cuda")
    assert autograd.fp8_linear(x, w, residual=torch.zeros((2, 3, 0), dtype=BF16, device="cuda")).shape == (2, 3, 0)


# ------------------------------------------------------------------ results in FP32

# The same sums, so a BF16 result is the FP32 one, rounded.
@pytest.mark.parametrize("kw", [{}, dict(activation="gelu"), dict(activation="silu", gated=True), dict(bias=True),
                                dict(residual=F32), dict(activation="relu", bias=True, residual=BF16)])
@pytest.mark.parametrize("lead", [(5,), (3, 67), (300,)])
@pytest.mark.parametrize("trained", [False, True])
def test_fp32_results(built, trained, lead, kw):
    kw, n = dict(kw), 192
    rows = 2 * n if kw.get("gated") else n
    x, w = rand(*lead, 200, seed=11), rand(rows, 200, seed=12, sigma=0.07, dtype=F32).requires_grad_(trained)
    if kw.get("bias"):
        kw["bias"] = rand(rows, seed=13, dtype=F32)
    if kw.get("residual"):
        kw["residual"] = rand(*lead, n, seed=14, sigma=30.0, dtype=kw["residual"])
    y = autograd.fp8_linear(x, w, **kw, out_dtype=F32)
    assert y.dtype == F32 and y.shape == (*lead, n) and y.requires_grad == trained
    short = autograd.fp8_linear(x, w, **kw)
    assert short.dtype == BF16 and torch.equal(short, y.to(BF16)) and not torch.equal(short.to(F32), y)
    assert torch.equal(autograd.fp8_linear(x, w, **kw, out_dtype=BF16), short)
    if trained:
        dy = rand(*lead, n, seed=15)
        # a BF16 gradient gives the same bits whichever type it is held in
        got, = torch.autograd.grad(y, w, dy.to(F32))
        want, = torch.autograd.grad(short, w, dy)
        assert torch.equal(got, want)


def test_an_fp32_stream_keeps_its_digits(built):
    x, w = rand(90, 64, seed=21), torch.zeros((128, 64), dtype=BF16, device="cuda")
    stream = rand(90, 128, seed=22, sigma=100.0, dtype=F32)
    assert torch.equal(autograd.fp8_linear(x, w, residual=stream, out_dtype=F32), stream)
    leaf = stream.clone().requires_grad_()
    y = autograd.fp8_linear(x, w, residual=leaf, out_dtype=F32)
    dy = rand(90, 128, seed=23, dtype=F32)
    assert torch.equal(y.detach(), stream) and torch.equal(torch.autograd.grad(y, leaf, dy)[0], dy)


@pytest.mark.parametrize("trained", [False, True])
@pytest.mark.parametrize("act,gated,bias", [(None, False, False), ("silu", True, True), ("gelu", False, False)])
def test_fp32_results_by_groups(built, trained, act, gated, bias):
    ends, M, n = torch.tensor([40, 40, 175], dtype=torch.int32, device="cuda"), 180, 128
    rows = 2 * n if gated else n
    x, w = rand(M, 136, seed=31), rand(3, rows, 136, seed=32, sigma=0.08).requires_grad_(trained)
    b = rand(3, rows, seed=33) if bias else None
    y = autograd.fp8_grouped_linear(x, w, ends, b, act, gated, out_dtype=F32)
    short = autograd.fp8_grouped_linear(x, w, ends, b, act, gated)
    assert y.dtype == F32 and short.dtype == BF16 and torch.equal(short, y.to(BF16)) and (y[175:] == 0).all()
    if trained:
        dy = rand(M, n, seed=34)
        assert torch.equal(torch.autograd.grad(y, w, dy.to(F32))[0], torch.autograd.grad(short, w, dy)[0])


@pytest.mark.parametrize("trained", [False, True])
def test_other_result_types_are_refused(built, trained):
    x, w = rand(4, 64, seed=41), rand(128, 64, seed=42).requires_grad_(trained)
    ends = torch.tensor([4], dtype=torch.int32, device="cuda")
    for call in (lambda: autograd.fp8_linear(x, w, out_dtype=torch.float16),
                 lambda: autograd.fp8_linear(x, w, activation="relu", out_dtype=torch.float64),
                 lambda: autograd.fp8_grouped_linear(x, w[None], ends, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------ the bits of the calls that the functions stand for

def by_calls(x, w, bias, residual, ends, act, gated, out, dy):
    """(y, dx, dw, dbias) of a layer from the public calls, each with buffers of its own."""
    K = x.shape[1]
    wq, ws, wtq, wts = rlk.fp8_quantize_both(w, block_rows=128)
    z = None
    keep = act is not None or gated
    kind = F32 if bias is None else bias.dtype
    if ends is None:
        xq, xs, xtq, xts = rlk.fp8_quantize_both(x)
        y = rlk.fp8_matmul_act(xq, xs, wq, ws, bias, act, gated, residual, keep, out)
    else:
        xq, xs, xtq, xts = rlk.fp8_quantize_grouped(x, ends)
        y = rlk.fp8_grouped_matmul(xq, xs, wq, ws, ends, bias, act, gated, keep, out)
    if keep:
        y, z = y
    q, s, qt, st, db = rlk.fp8_act_grad(dy, z, act, gated, ends, bias_dtype=kind)
    if ends is None:
        dx = rlk.fp8_matmul(q, s, wtq, wts, out_dtype=x.dtype)
        dw = rlk.fp8_matmul(qt, st, xtq, xts, b_block_rows=1, out_dtype=w.dtype)
    else:
        dx = rlk.fp8_grouped_matmul(q, s, wtq, wts, ends, out_dtype=x.dtype)
        dw = rlk.fp8_grouped_dweight(qt, st, xtq, xts, ends, x.shape[0], out_dtype=w.dtype)
    return y, dx, dw, db


SIZES = [(1, 128, 40), (9, 128, 16), (130, 256, 300), (257, 384, 2056), (300, 2176, 130), (1000, 640, 514)]
LAYERS = [(None, False, True, None), (None, False, False, BF16), ("gelu", False, False, F32), ("silu", True, True, None),
          ("relu", False, True, BF16), ("gelu_tanh", True, False, None), (None, True, True, F32)]


@pytest.mark.parametrize("M,rows,K", SIZES)
@pytest.mark.parametrize("act,gated,bias,residual", LAYERS)
@pytest.mark.parametrize("types", [(BF16, F32, BF16), (F32, BF16, F32)])
def test_a_step_is_its_calls(built, M, rows, K, act, gated, bias, residual, types):
    tx, tw, out = types
    n = rows // 2 if gated else rows
    x, w = rand(M, K, seed=51, dtype=tx), rand(rows, K, seed=52, sigma=0.08, dtype=tw)
    b = rand(rows, seed=53, dtype=tw) if bias else None
    r = rand(M, n, seed=54, dtype=residual) if residual else None
    dy = rand(M, n, seed=55, sigma=1e-3, dtype=out)
    want = by_calls(x, w, b, r, None, act, gated, out, dy)
    leaves = [t.clone().requires_grad_() for t in (x, w, b) if t is not None]
    y = autograd.fp8_linear(*leaves[:2], leaves[2] if bias else None, act, gated, r, out)
    got = (y.detach(), *torch.autograd.grad(y, leaves, dy))
    for g, t in zip(got, want):
        assert g.dtype == t.dtype and torch.equal(g, t)


COUNTS = [[1], [0, 3, 0, 5], [128, 0, 129, 1], [40, 60, 100, 56], [300, 1, 200], [1, 0, 2] * 30]


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("rows,K", [(128, 40), (384, 300), (256, 2056)])
@pytest.mark.parametrize("act,gated,bias", [(None, False, True), (None, False, False), ("gelu", False, False),
                                            ("silu", True, True), ("relu", True, False)])
@pytest.mark.parametrize("types", [(BF16, F32, BF16), (F32, BF16, F32)])
def test_a_step_by_groups_is_its_calls(built, counts, rows, K, act, gated, bias, types):
    tx, tw, out = types
    G, used = len(counts), sum(counts)
    M, n = used + 5, rows // 2 if gated else rows
    ends = torch.tensor(counts, device="cuda").cumsum(0).to(torch.int32)
    x, w = rand(M, K, seed=61, dtype=tx), rand(G, rows, K, seed=62, sigma=0.08, dtype=tw)
    b = rand(G, rows, seed=63, dtype=tw) if bias else None
    dy = rand(M, n, seed=64, sigma=1e-3, dtype=out)
    want = by_calls(x, w, b, None, ends, act, gated, out, dy)
    leaves = [t.clone().requires_grad_() for t in (x, w, b) if t is not None]
    y = autograd.fp8_grouped_linear(*leaves[:2], ends, leaves[2] if bias else None, act, gated, out)
    got = (y.detach(), *torch.autograd.grad(y, leaves, dy))
    for g, t in zip(got, want):
        assert g.dtype == t.dtype and torch.equal(g, t)


def test_only_what_is_asked_for_has_the_same_bits(built):
    """Frozen inputs take other calls (no transposes, no codes along the rows): the same bits."""
    ends = torch.tensor([50, 50, 190], dtype=torch.int32, device="cuda")
    x, w, b, dy = rand(200, 300, seed=71), rand(3, 256, 300, seed=72, sigma=0.08), rand(3, 256, seed=73), rand(200, 256, seed=74)
    for g in (None, ends):
        ww, bb = (w, b) if g is not None else (w[0], b[0])
        for act in (None, "silu"):
            want = by_calls(x, ww, bb, None, g, act, False, BF16, dy)
            for which in range(3):
                args = [t.clone().requires_grad_(k == which) for k, t in enumerate((x, ww, bb))]
                y = autograd.fp8_linear(*args, act) if g is None else autograd.fp8_grouped_linear(args[0], args[1], g, args[2], act)
                assert torch.equal(torch.autograd.grad(y, args[which], dy)[0], want[1 + which]) and torch.equal(y.detach(), want[0])
