"""The layer's formulas against differences, and the refusals of the calls around them, without a GPU.

The C entry points check sizes, types, alignment and overlaps before they look at a device, so made-up addresses do.
"""
import numpy as np
import pytest

import fp8_layer_reference as layer
import vocab_selected_token_tile_gb300 as rlk


@pytest.mark.parametrize("act", layer.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_the_backward_formula_is_the_forward_ones_difference(act, gated):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((7, 12)) * 2
    z += 0.05 * np.sign(z)  # away from relu's corner
    dy = rng.standard_normal((7, 6 if gated else 12))
    dz, h = layer.backward(z, dy, act, gated), 1e-6
    for i in range(7):
        for j in range(12):
            up, down = z.copy(), z.copy()
            up[i, j] += h
            down[i, j] -= h
            diff = ((layer.forward(up, act, gated) - layer.forward(down, act, gated)) * dy).sum() / (2 * h)
            # truncation h^2 f''' / 6, and 2^-52 of the sum's terms over 2 h
            assert abs(diff - dz[i, j]) <= 1e-8 * (1 + np.abs(dy).sum() * 10)


A, B, C, S, T, W, R, Z, E = (0x10000000 * k for k in range(1, 10))  # far apart, 16-byte aligned


def act_call(M=10, N=128, K=256, a=A, lda=256, sa=S, b=B, ldb=256, sb=T, e=None, c=C, ct=rlk.RLK_BF16, ldc=128, w=W):
    return rlk.rlk_fp8_matmul_act(M, N, K, a, lda, sa, b, ldb, sb, e, c, ct, ldc, w, None)


def grouped_call(G=4, M=10, N=128, K=256, ends=E, a=A, lda=256, sa=S, b=B, ldb=256, bg=256 * 128, sb=T, e=None, c=C,
                 ct=rlk.RLK_BF16, ldc=128, rest=0, w=W):
    return rlk.rlk_fp8_grouped_matmul(G, M, N, K, ends, a, lda, sa, b, ldb, bg, sb, e, c, ct, ldc, rest, w, None)


def epi(**k):
    return rlk.Fp8Epilogue(**k)


INVALID, UNSUPPORTED, MISALIGNED = rlk.RLK_ERR_INVALID_ARG, rlk.RLK_ERR_UNSUPPORTED, rlk.RLK_ERR_MISALIGNED


@pytest.mark.parametrize("call", [act_call, grouped_call])
@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(M=-1)), (INVALID, dict(N=-1)), (INVALID, dict(K=0)), (INVALID, dict(a=None)), (INVALID, dict(b=None)),
    (INVALID, dict(sa=None)), (INVALID, dict(sb=None)), (INVALID, dict(c=None)), (INVALID, dict(w=None)),
    (MISALIGNED, dict(a=A + 8)), (MISALIGNED, dict(b=B + 4)), (MISALIGNED, dict(lda=264)), (MISALIGNED, dict(ldb=260)),
    (INVALID, dict(lda=240)), (INVALID, dict(ldb=128)), (INVALID, dict(ldc=127)), (INVALID, dict(ct=7)),
    (MISALIGNED, dict(c=C + 1)), (MISALIGNED, dict(sa=S + 2)), (MISALIGNED, dict(sb=T + 1)), (MISALIGNED, dict(w=W + 8)),
    (UNSUPPORTED, dict(K=1 << 31, lda=1 << 31, ldb=1 << 31)), (UNSUPPORTED, dict(N=1 << 30, ldc=1 << 30)),
    (INVALID, dict(e=dict(activation=5))), (INVALID, dict(e=dict(activation=-1))), (INVALID, dict(e=dict(gated=2))),
    (UNSUPPORTED, dict(N=96, e=dict(gated=1))), (INVALID, dict(e=dict(bias=R, bias_type=3))),
    (MISALIGNED, dict(e=dict(bias=R + 2, bias_type=1))), (MISALIGNED, dict(e=dict(z=Z + 1, z_stride=128))),
    (INVALID, dict(e=dict(z=Z, z_stride=127))), (INVALID, dict(e=dict(z=Z, z_stride=128, gated=1))),
    (INVALID, dict(e=dict(z=C, z_stride=128))), (INVALID, dict(e=dict(bias=C))), (INVALID, dict(c=A)),
    (INVALID, dict(c=W)), (INVALID, dict(e=dict(z=A, z_stride=128))), (INVALID, dict(e=dict(z=W, z_stride=128))),
])
def test_refusals_of_the_layers(built, call, want, kw):
    kw = dict(kw)
    if "e" in kw:
        kw["e"] = epi(**kw["e"])
    assert call(**kw) == want, rlk.rlk_last_error_message()


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(e=dict(residual=R, residual_type=9, residual_stride=128))),
    (INVALID, dict(e=dict(residual=R, residual_stride=100))),
    (MISALIGNED, dict(e=dict(residual=R + 1, residual_stride=128))),
    (INVALID, dict(e=dict(residual=C, residual_stride=136))),                             # in place, another stride
    (INVALID, dict(e=dict(residual=C, residual_type=rlk.RLK_F32, residual_stride=128))),  # and another type
    (INVALID, dict(e=dict(residual=C + 256, residual_stride=128))),                       # a row further
    (INVALID, dict(e=dict(residual=Z, residual_stride=128, z=Z, z_stride=128))),
])
def test_refusals_of_a_residual(built, want, kw):
    assert act_call(e=epi(**kw["e"])) == want, rlk.rlk_last_error_message()


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(G=0)), (INVALID, dict(G=-3)), (UNSUPPORTED, dict(G=1025)), (INVALID, dict(ends=None)),
    (MISALIGNED, dict(ends=E + 2)), (INVALID, dict(bg=256 * 127)), (MISALIGNED, dict(bg=256 * 128 + 8)),
    (INVALID, dict(rest=2)), (UNSUPPORTED, dict(M=(1 << 30) + 1)), (INVALID, dict(c=E)),
    (UNSUPPORTED, dict(e=dict(residual=R, residual_stride=128))),
    (INVALID, dict(b=C - 3 * 256 * 128)),  # the last group's weight lies in c
])
def test_refusals_of_groups(built, want, kw):
    kw = dict(kw)
    if "e" in kw:
        kw["e"] = epi(**kw["e"])
    assert grouped_call(**kw) == want, rlk.rlk_last_error_message()


def test_nothing_to_do(built):
    assert act_call(M=0) == rlk.RLK_OK and act_call(N=0) == rlk.RLK_OK
    assert grouped_call(M=0) == rlk.RLK_OK and grouped_call(N=0) == rlk.RLK_OK
    assert rlk.rlk_fp8_quantize_grouped(3, 0, 5, None, None, 0, 5, None, 0, None, None, 0, None, None) == rlk.RLK_OK
    assert rlk.rlk_fp8_quantize_batch(0, 5, 5, None, 0, 5, 25, None, 0, 0, None, None, 0, 0, None, None) == rlk.RLK_OK


def quantize_call(G=2, rows=100, cols=64, ends=E, x=A, xt=rlk.RLK_BF16, ldx=64, q=B, ldq=64, s=S, qt=C, ldqt=256, st=T):
    return rlk.rlk_fp8_quantize_grouped(G, rows, cols, ends, x, xt, ldx, q, ldq, s, qt, ldqt, st, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(G=0)), (UNSUPPORTED, dict(G=2000)), (INVALID, dict(rows=-1)), (INVALID, dict(xt=4)), (INVALID, dict(x=None)),
    (INVALID, dict(ends=None)), (INVALID, dict(q=None, s=None, qt=None, st=None)), (INVALID, dict(q=None)),
    (INVALID, dict(st=None)), (INVALID, dict(ldx=63)), (MISALIGNED, dict(ldq=72)), (INVALID, dict(ldqt=240)),
    (MISALIGNED, dict(qt=C + 8)), (MISALIGNED, dict(x=A + 1)), (INVALID, dict(q=A)), (INVALID, dict(qt=B)), (INVALID, dict(s=T)),
    (INVALID, dict(st=E))])
def test_refusals_of_the_grouped_quantisation(built, want, kw):
    assert quantize_call(**kw) == want, rlk.rlk_last_error_message()


def batch_call(n=2, rows=100, cols=64, x=A, xt=rlk.RLK_BF16, ldx=64, bx=6400, q=B, ldq=64, bq=6400, s=S, qt=C, ldqt=112,
               bqt=7168, st=T):
    return rlk.rlk_fp8_quantize_batch(n, rows, cols, x, xt, ldx, bx, q, ldq, bq, s, qt, ldqt, bqt, st, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(n=-1)), (INVALID, dict(xt=2)), (INVALID, dict(x=None)), (INVALID, dict(bx=6399)), (INVALID, dict(bq=6384)),
    (MISALIGNED, dict(bq=6408)), (MISALIGNED, dict(bqt=7176)), (INVALID, dict(ldx=60)), (INVALID, dict(q=None, s=None, qt=None, st=None)),
    (INVALID, dict(s=None)), (INVALID, dict(q=A + 12800)), (INVALID, dict(qt=B + 6400)), (UNSUPPORTED, dict(n=(1 << 20) + 1)),
    (UNSUPPORTED, dict(rows=1 << 31))])
def test_refusals_of_several_matrices(built, want, kw):
    assert batch_call(**kw) == want, rlk.rlk_last_error_message()


def dweight_call(G=2, rows=100, M=64, N=32, ends=E, a=A, lda=256, sa=S, b=B, ldb=256, sb=T, c=C, ct=rlk.RLK_F32, ldc=32,
                 cg=2048, acc=0, w=W):
    return rlk.rlk_fp8_grouped_dweight(G, rows, M, N, ends, a, lda, sa, b, ldb, sb, c, ct, ldc, cg, acc, w, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(G=0)), (INVALID, dict(rows=0)), (INVALID, dict(M=-1)), (INVALID, dict(ct=5)), (INVALID, dict(acc=2)),
    (INVALID, dict(acc=1, ct=rlk.RLK_BF16)), (INVALID, dict(lda=240)), (MISALIGNED, dict(ldb=264)), (INVALID, dict(ldc=31)),
    (INVALID, dict(cg=2047)), (INVALID, dict(ends=None)), (INVALID, dict(c=A)), (INVALID, dict(c=W)), (MISALIGNED, dict(c=C + 2)),
    (UNSUPPORTED, dict(M=1 << 26, N=1 << 26, ldc=1 << 26))])
def test_refusals_of_the_groups_weight_gradients(built, want, kw):
    assert dweight_call(**kw) == want, rlk.rlk_last_error_message()


def grad_call(G=0, rows=100, cols=64, ends=E, dy=A, dt=rlk.RLK_BF16, lddy=64, z=Z, ldz=64, act=2, gated=0, q=B, ldq=64,
              s=S, qt=C, ldqt=112, st=T, db=R, bt=rlk.RLK_F32, w=W):
    return rlk.rlk_fp8_act_grad(G, rows, cols, ends, dy, dt, lddy, z, ldz, act, gated, q, ldq, s, qt, ldqt, st, db, bt, w,
                                None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(rows=0)), (INVALID, dict(G=-1)), (UNSUPPORTED, dict(G=1025)), (INVALID, dict(dt=3)), (INVALID, dict(act=9)),
    (INVALID, dict(gated=-1)), (UNSUPPORTED, dict(gated=1, cols=96)), (INVALID, dict(bt=2)), (INVALID, dict(dy=None)),
    (INVALID, dict(z=None)), (INVALID, dict(act=0, gated=1, z=None)), (INVALID, dict(ldz=63)), (INVALID, dict(lddy=63)),
    (INVALID, dict(q=None, s=None, qt=None, st=None, db=None)), (INVALID, dict(w=None)), (MISALIGNED, dict(w=W + 4)),
    (INVALID, dict(G=2, ends=None)), (INVALID, dict(G=2, ldqt=240)), (INVALID, dict(db=W)), (INVALID, dict(q=Z)),
    (INVALID, dict(w=A)), (INVALID, dict(st=R)), (MISALIGNED, dict(db=R + 2)), (INVALID, dict(gated=1, ldz=100, ldq=128))])
def test_refusals_of_the_epilogues_backward(built, want, kw):
    assert grad_call(**kw) == want, rlk.rlk_last_error_message()


def test_workspace_of_the_bias_gradient(built):
    size = rlk.rlk_fp8_act_grad_workspace_size
    assert size(0, 129, 10, 0) == 4 * 2 * 10 and size(0, 129, 64, 1) == 4 * 2 * 128
    assert size(3, 129, 10, 0) == 4 * 4 * 10 and size(500, 2, 10, 0) == 4 * 2 * 10
    assert size(-1, 1, 1, 0) == 0
