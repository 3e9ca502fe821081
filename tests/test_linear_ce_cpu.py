"""The cross-entropy and FP8 references against closed forms and differences, and the calls' refusals (no GPU)."""
import ctypes

import numpy as np
import pytest

import ce_reference as ce
import fp8_reference as f8
import vocab_selected_token_tile_gb300 as rlk


def problem(T=5, V=17, H=6, seed=0):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((T, H)), rng.standard_normal((V, H)), rng.integers(0, V, T), np.arange(T) % 4 != 1)


@pytest.mark.parametrize("eps,z,cap", [(0, 0, 0), (0.1, 0, 0), (0, 1e-2, 0), (0, 0, 2.0), (0.2, 1e-2, 1.5)])
def test_reference_gradients_match_differences(eps, z, cap):
    h, w, t, on = problem()
    rows = ce.row_gradients(np.linspace(-1, 2, len(t)), on, "none")
    dh, dw = ce.backward(h, w, t, on, rows, eps, z, cap)

    def total():
        return float((rows * ce.forward(h, w, t, on, eps, z, cap)[0]).sum())
    for a, d in ((h, dh), (w, dw)):
        for i in np.ndindex(a.shape):
            keep, step = a[i], 1e-6
            a[i] = keep + step
            up = total()
            a[i] = keep - step
            down = total()
            a[i] = keep
            assert abs((up - down) / (2 * step) - d[i]) < 1e-7


def test_reference_closed_forms():
    h, w = np.zeros((3, 4)), np.ones((9, 4))
    t, on = np.array([0, 8, 4]), np.array([True, False, True])
    loss, lse, _ = ce.forward(h, w, t, on, z=0.5)
    assert np.allclose(lse, np.log(9)) and np.allclose(loss, [np.log(9) + 0.5 * np.log(9) ** 2, 0, np.log(9) + 0.5 * np.log(9) ** 2])
    assert ce.reduce(loss, on, "mean") == pytest.approx(loss[0]) and ce.reduce(0 * loss, ~on & on, "mean") == 0.0
    # one smoothing unit spreads the target evenly: a uniform prediction has no gradient
    d = ce.logits_gradient(np.zeros((1, 9)), np.log([9.0]), np.array([2]), np.array([True]), np.ones(1), eps=1.0)[0]
    assert np.allclose(d, 0)


def test_e4m3_reference_rounds_to_the_format():
    # every code: 1 sign, 4 exponent (bias 7), 3 mantissa bits, no infinities, 0x7F NaN
    vals = []
    for code in range(0x7F):
        e, m = code >> 3, code & 7
        vals.append((1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6)
    vals = np.array(vals)
    assert vals[-1] == 448 and np.array_equal(f8.e4m3(vals), vals) and np.array_equal(f8.e4m3(-vals), -vals)
    mid = (vals[1:] + vals[:-1]) / 2  # ties go to the even code
    assert np.array_equal(f8.e4m3(mid), np.where(np.arange(len(mid)) % 2 == 0, vals[:-1], vals[1:]))
    assert np.array_equal(f8.e4m3(mid * (1 + 1e-12)), vals[1:]) and np.array_equal(f8.e4m3(mid * (1 - 1e-12)), vals[:-1])
    assert f8.e4m3(1e9) == 448 and np.isnan(f8.e4m3(np.nan))


def contract(**kw):
    base = dict(T=8, V=1000, H=64)
    base.update(kw)
    return rlk.LinearCeContract(**base)


@pytest.mark.parametrize("kw,status", [
    ({}, rlk.RLK_OK), (dict(T=0), rlk.RLK_OK), (dict(H=7, hidden_stride=8, weight_stride=16, dhidden_stride=8,
                                                    dweight_stride=8), rlk.RLK_OK),
    (dict(T=-1), rlk.RLK_ERR_INVALID_ARG), (dict(V=0), rlk.RLK_ERR_INVALID_ARG), (dict(H=0), rlk.RLK_ERR_INVALID_ARG),
    (dict(T=1 << 31), rlk.RLK_ERR_UNSUPPORTED), (dict(H=1 << 21), rlk.RLK_ERR_UNSUPPORTED),
    (dict(H=7), rlk.RLK_ERR_MISALIGNED), (dict(hidden_stride=68), rlk.RLK_ERR_MISALIGNED),
    (dict(weight_stride=32), rlk.RLK_ERR_INVALID_ARG), (dict(dweight_stride=60), rlk.RLK_ERR_INVALID_ARG),
    (dict(mask_mode=2), rlk.RLK_ERR_INVALID_ARG), (dict(reduction=3), rlk.RLK_ERR_INVALID_ARG),
    (dict(validate=2), rlk.RLK_ERR_INVALID_ARG), (dict(piece=-1), rlk.RLK_ERR_INVALID_ARG),
    (dict(wait_timeout_ns=-1), rlk.RLK_ERR_INVALID_ARG),
    (dict(label_smoothing=-0.1), rlk.RLK_ERR_INVALID_ARG), (dict(label_smoothing=1.5), rlk.RLK_ERR_INVALID_ARG),
    (dict(label_smoothing=float("nan")), rlk.RLK_ERR_INVALID_ARG),
    (dict(z_loss=-1.0), rlk.RLK_ERR_INVALID_ARG), (dict(z_loss=float("inf")), rlk.RLK_ERR_INVALID_ARG),
    (dict(softcap=-1.0), rlk.RLK_ERR_INVALID_ARG), (dict(softcap=float("nan")), rlk.RLK_ERR_INVALID_ARG),
])
def test_ce_contract(built, kw, status):
    assert ctypes.sizeof(rlk.LinearCeContract) == 104
    c = contract(**kw)
    assert rlk.rlk_linear_ce_check(c) == status
    sizes = [rlk.rlk_linear_ce_workspace_size(c, g) for g in (0, 1)]
    assert (min(sizes) > 0) == (status == rlk.RLK_OK)
    if status != rlk.RLK_OK:
        assert rlk.rlk_last_error_message()


def test_ce_workspace_does_not_grow_with_the_logits(built):
    a = rlk.rlk_linear_ce_workspace_size(contract(T=65536, V=150000, H=4096), 1)
    assert a < 65536 * 150000 // 4  # the logits alone, in BF16, are 2 bytes each
    # dx of a piece, the FP32 sums and the active rows' hidden
    T, H, piece = 4096, 4096, 2048
    b = rlk.rlk_linear_ce_workspace_size(contract(T=T, V=150000, H=H, piece=piece), 1)
    assert b < 2 * T * piece + 6 * T * H + (1 << 20)


def test_ce_calls_refuse_before_any_device_work(built):
    c, ig = contract(), contract(mask_mode=rlk.MASK_IGNORE_INDEX)
    bad, mis = rlk.RLK_ERR_INVALID_ARG, rlk.RLK_ERR_MISALIGNED
    ok = [0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000, 0x70000]
    fwd = rlk.rlk_linear_ce_fwd
    assert rlk.library().rlk_linear_ce_check(None) == bad
    assert fwd(contract(T=-1), *ok, None) == bad
    for i in range(7):
        args = list(ok)
        args[i] = None
        assert fwd(c, *args, None) == bad, i
    for i in (0, 1, 6):
        args = list(ok)
        args[i] += 8
        assert fwd(c, *args, None) == mis
    assert fwd(ig, *ok, None) == bad  # ignore_index mode takes no mask
    # hidden, weight, targets, mask, lse, grad, dhidden, dweight, workspace
    bwd = rlk.rlk_linear_ce_bwd
    ok = [0x100000, 0x200000, 0x300000, 0x400000, 0x500000, 0x600000, 0x700000, 0x800000, 0x900000]
    for i in (0, 1, 2, 3, 4, 5, 8):
        args = list(ok)
        args[i] = None
        assert bwd(c, *args, None) == bad, i
    assert bwd(c, *ok[:6], None, None, ok[8], None) == bad  # no output at all
    for i in (6, 7):
        args = list(ok)
        args[i] += 2
        assert bwd(c, *args, None) == mis
    for i, j in ((6, 0), (6, 1), (7, 0), (7, 1), (7, 6)):
        args = list(ok)
        args[i] = args[j] + 512  # inside the other
        assert bwd(c, *args, None) == bad and "overlap" in rlk.rlk_last_error_message()
    assert fwd(contract(T=0), *[None] * 7, None) == rlk.RLK_OK
    assert bwd(contract(T=0), *[None] * 6, 0x700000, None, None, None) == rlk.RLK_OK


def test_fp8_calls_refuse_before_any_device_work(built):
    bad, mis, no = rlk.RLK_ERR_INVALID_ARG, rlk.RLK_ERR_MISALIGNED, rlk.RLK_ERR_UNSUPPORTED

    def quant(rows=4, cols=100, x=0x10000, kind=rlk.RLK_BF16, ldx=100, block=1, q=0x20000, ldq=112, s=0x30000,
              qt=0x40000, ldt=16, st=0x50000):
        return rlk.rlk_fp8_quantize(rows, cols, x, kind, ldx, block, q, ldq, s, qt, ldt, st, None)
    for kw, status in ((dict(rows=-1), bad), (dict(cols=-1), bad), (dict(kind=2), bad), (dict(block=64), bad),
                       (dict(x=None), bad), (dict(q=None), bad), (dict(s=None), bad), (dict(st=None), bad),
                       (dict(q=None, s=None, qt=None, st=None), bad), (dict(ldx=99), bad), (dict(ldq=96), bad),
                       (dict(ldq=104), mis), (dict(ldt=8), mis), (dict(q=0x20008), mis), (dict(x=0x10001), mis),
                       (dict(s=0x30002), mis), (dict(rows=1 << 31), no), (dict(q=0x10010), bad),
                       (dict(qt=0x20010), bad), (dict(s=0x20100), bad), (dict(st=0x30008), bad)):
        assert quant(**kw) == status, kw
        assert rlk.rlk_last_error_message()
    assert quant(rows=0) == rlk.RLK_OK and quant(cols=0, ldx=0) == rlk.RLK_OK

    def mm(M=4, N=100, K=200, a=0x10000, lda=208, sa=0x20000, b=0x30000, ldb=208, sb=0x40000, block=128, c=0x50000,
           kind=rlk.RLK_BF16, ldc=100, acc=0, ws=0x60000):
        return rlk.rlk_fp8_matmul(M, N, K, a, lda, sa, b, ldb, sb, block, c, kind, ldc, acc, ws, None)
    for kw, status in ((dict(M=-1), bad), (dict(N=-1), bad), (dict(K=0), bad), (dict(block=2), bad),
                       (dict(kind=5), bad), (dict(acc=2), bad), (dict(acc=1), bad), (dict(a=None), bad),
                       (dict(sa=None), bad), (dict(b=None), bad), (dict(sb=None), bad), (dict(c=None), bad),
                       (dict(ws=None), bad), (dict(lda=199), bad), (dict(lda=200), mis), (dict(a=0x10004), mis),
                       (dict(b=0x30008), mis), (dict(ws=0x60004), mis), (dict(c=0x50001), mis), (dict(ldc=99), bad),
                       (dict(sa=0x20001), mis), (dict(K=1 << 31), no), (dict(M=1 << 30, N=1 << 30), no),
                       (dict(c=0x10010), bad), (dict(c=0x30010), bad), (dict(c=0x60000 - 200), bad)):
        assert mm(**kw) == status, kw
        assert rlk.rlk_last_error_message()
    assert mm(M=0) == rlk.RLK_OK and mm(N=0) == rlk.RLK_OK
