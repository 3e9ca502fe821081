"""The FP8 product with a layer's epilogue, its backward, and layers of rows that belong to groups, against plain 64-bit
forms, on the GPU.

Bounds count the product's FP32 roundings (fp8_reference.bound), the activations' (fp8_layer_reference.act_error) and
one rounding of the result, half a step of its type; quantisation without arithmetic in front of it is held to equality.
"""
import numpy as np
import pytest
import torch

import fp8_layer_reference as layer
import fp8_reference as ref
import vocab_selected_token_tile_gb300 as rlk
from vocab_selected_token_tile_gb300 import autograd

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(shape, seed, sigma=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape).astype(np.float32) * np.float32(sigma)
    x *= np.where(rng.random(shape[-1]) < 0.05, np.float32(10), np.float32(1))  # a few large channels
    return x


def tensor(x, dtype="bf16"):
    return torch.from_numpy(x).cuda().to(DT[dtype])


def f64(t):
    return t.detach().double().cpu().numpy()


def values(q):
    return q.float().cpu().numpy().astype(np.float64)


def half_step(t, y):
    """Half a step of the tensor's type at y."""
    return torch.finfo(t.dtype).eps / 2 * np.abs(y) + 1e-37


def within(got, want, err):
    d = np.abs(f64(got) - want)
    lim = err + half_step(got, np.abs(want) + err)
    assert d.shape == lim.shape and np.all(d <= lim), f"worst {np.nanmax(d / lim):.3g} of the bound"


def operands(M, rows, K, seed, lead=()):
    a, b = tensor(rand((M, K), seed)), tensor(rand((*lead, rows, K), seed + 1, 0.05))
    return (*rlk.fp8_quantize(a), *rlk.fp8_quantize(b, block_rows=128))


def check_layer(M, N, K, act="none", gated=False, bias=None, residual=None, out="bf16", keep=False, seed=0):
    rows = 2 * N if gated else N
    qa, sa, qb, sb = operands(M, rows, K, seed + M + N + K)
    tb = None if bias is None else tensor(rand((1, rows), seed + 5, 0.5)[0], bias)
    tr = None if residual is None else tensor(rand((M, N), seed + 6), residual)
    got = rlk.fp8_matmul_act(qa, sa, qb, sb, bias=tb, activation=act, gated=gated, residual=tr, keep=keep,
                             out_dtype=DT[out], validate=True)
    z, y, dz, err = layer.layer(values(qa), sa.cpu().numpy(), values(qb), sb.cpu().numpy(),
                                None if tb is None else f64(tb), act, gated, None if tr is None else f64(tr))
    if keep:
        got, gz = got
        within(gz, z, dz)
    assert got.dtype == DT[out] and got.shape == (M, N)
    within(got, y, err)
    return got


# each kernel and each of its joins: 16, 32 and 64 rows with K split or not, tiles of pairs, few of them, a last round
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 4096, 4096), (3, 130, 200), (16, 257, 1000), (17, 40, 129),
                                   (33, 255, 640), (64, 1024, 128), (64, 129, 2100), (65, 128, 1024), (100, 515, 500),
                                   (129, 1, 128), (256, 256, 2048), (300, 1000, 1000), (520, 900, 2300), (7, 40001, 200)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_layer_sizes(built, M, N, K, out):
    check_layer(M, N, K, "silu", bias="f32", residual="bf16", out=out, keep=True)


@pytest.mark.parametrize("M,N,K", [(1, 64, 1), (1, 1024, 2048), (5, 192, 384), (16, 128, 1000), (31, 320, 520),
                                   (64, 64, 4096), (64, 4096, 256), (65, 64, 640), (200, 192, 300), (513, 1024, 1000),
                                   (300, 128, 4096), (2, 20032, 300)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_gated_sizes(built, M, N, K, out):
    check_layer(M, N, K, "gelu_tanh", True, bias="bf16", residual="f32", out=out, keep=True)


@pytest.mark.parametrize("act", layer.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [4, 150, 700])
def test_activations(built, M, gated, act):
    check_layer(M, 320, 512, act, gated, bias="bf16", out="f32", keep=True)


@pytest.mark.parametrize("bias", [None, "bf16", "f32"])
@pytest.mark.parametrize("residual", [None, "bf16", "f32"])
@pytest.mark.parametrize("M", [6, 140])
def test_what_is_left_out(built, M, residual, bias):
    for out in ("bf16", "f32"):
        check_layer(M, 333, 260, "relu", False, bias, residual, out)


def test_without_an_epilogue(built):
    for M, N, K in ((5, 300, 700), (64, 4096, 1024), (400, 1300, 2000), (2100, 2500, 300)):
        for out in ("bf16", "f32"):
            check_layer(M, N, K, out=out)


def test_special_arguments_of_the_activations(built):
    # zeros in B leave the bias: a NaN or an infinity beside numbers reaches its own column only
    z = np.array([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 60.0, -60.0, 1e4, np.nan, -1e4, 3e38, -3e38, np.inf, np.nan, -np.inf],
                 np.float32)
    n, big = len(z), (0.0, -1e4, -3e38, -np.inf)
    for M in (2, 130):
        qa, sa, qb, sb = operands(M, n, 128, 1)
        qb = torch.zeros_like(qb.view(torch.uint8)).view(torch.float8_e4m3fn)
        for act in layer.ACTS:
            got = f64(rlk.fp8_matmul_act(qa, sa, qb, sb, bias=torch.from_numpy(z).cuda(), activation=act,
                                         out_dtype=torch.float32))
            with np.errstate(all="ignore"):
                want = layer.act(z.astype(np.float64), act)
            if act != "none":
                want[np.isin(z, big)] = 0.0  # the limits
            assert (np.isnan(got) == np.isnan(z)).all()
            for j in range(n):
                if np.isinf(want[j]):
                    assert (got[:, j] == want[j]).all(), (act, z[j])
                elif not np.isnan(want[j]):
                    err = layer.act_error(np.float64(z[j:j + 1]) if abs(z[j]) < 1e5 else np.zeros(1), act)[0]
                    assert np.all(np.abs(got[:, j] - want[j]) <= err + 2.0 ** -20 * abs(want[j])), (act, z[j])


def test_gradients_of_special_arguments(built):
    z = np.tile(np.array([0.0, -0.0, 3.0, -3.0, 30.0, -30.0, np.inf, -np.inf, 3e38, -3e38, np.nan], np.float32), 2)
    dy = np.ones((130, len(z)), np.float32)
    t = torch.from_numpy(np.tile(z, (130, 1))).cuda().to(torch.bfloat16)
    for act in layer.ACTS[1:]:
        q, s, _, _, db = rlk.fp8_act_grad(torch.from_numpy(dy).cuda(), t, act, bias_dtype=torch.float32)
        got = f64(db) / 130
        want = np.where(z > 0, 1.0, 0.0)
        few = np.abs(z) < 10
        want[few] = layer.slope(z[few].astype(np.float64), act)
        assert (np.isnan(got) == np.isnan(z)).all()
        ok = ~np.isnan(z)
        assert np.all(np.abs(got - want)[ok] <= 2.0 ** -17)
    # relu passes an infinite gradient on where z > 0 and nowhere else
    dy[:, 3] = np.inf
    db = f64(rlk.fp8_act_grad(torch.from_numpy(dy).cuda(), t, "relu", bias_dtype=torch.float32)[4])
    assert db[3] == 0 and np.isfinite(db[~np.isnan(z)]).all()


@pytest.mark.parametrize("M", [9, 300])
def test_strided_and_unaligned_operands(built, M):
    N, K = 190, 260
    qa, sa, qb, sb = operands(M, N, K, 11)
    want = f64(rlk.fp8_matmul_act(qa, sa, qb, sb, activation="gelu", out_dtype=torch.float32))
    for dtype in (torch.bfloat16, torch.float32):
        for offset, stride in ((0, 192), (1, 191), (3, 200), (8, 208)):
            buf = torch.full((M * stride + 16,), 7.0, device="cuda", dtype=dtype)
            out = buf.as_strided((M, N), (stride, 1), offset)
            resb = tensor(rand((1, M * stride + 16), 12)[0], "f32").to(dtype)
            res = resb.as_strided((M, N), (stride, 1), offset)
            biasb = tensor(rand((1, N + 5), 13)[0], "bf16")[offset % 5:][:N]
            z, y, dz, err = layer.layer(values(qa), sa.cpu().numpy(), values(qb), sb.cpu().numpy(), f64(biasb), "gelu",
                                        False, f64(res))
            got = rlk.fp8_matmul_act(qa, sa, qb, sb, bias=biasb, activation="gelu", residual=res, out=out)
            assert got is out
            within(out, y, err)
            rest = buf.clone()
            rest.as_strided((M, N), (stride, 1), offset).fill_(7.0)
            assert (rest == 7.0).all()  # nothing beside the result is touched
    assert np.isfinite(want).all()


@pytest.mark.parametrize("M,N,K", [(4, 500, 4000), (200, 500, 4000), (3000, 1500, 300)])
def test_residual_in_place(built, M, N, K):
    qa, sa, qb, sb = operands(M, N, K, 21)
    for dtype in ("bf16", "f32"):
        res = tensor(rand((M, N), 22), dtype)
        want = rlk.fp8_matmul_act(qa, sa, qb, sb, activation="relu", residual=res, out_dtype=DT[dtype])
        rlk.fp8_matmul_act(qa, sa, qb, sb, activation="relu", residual=res, out=res)
        assert torch.equal(res, want)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,rows,K", [(2304, 2304, 5632), (2500, 2176, 6000)])
def test_last_tiles_in_a_launch_of_their_own(built, M, rows, K, gated):
    # a round of the pairs and a few tiles more, which are split along K
    N = rows // 2 if gated else rows
    qa, sa, qb, sb = operands(M, rows, K, 14)
    bias, res = tensor(rand((1, rows), 15, 0.5)[0], "f32"), tensor(rand((M, N), 16), "f32")
    y, z = rlk.fp8_matmul_act(qa, sa, qb, sb, bias=bias, activation="gelu_tanh", gated=gated, residual=res, keep=True,
                              out_dtype=torch.float32, validate=True)

    def stands_for(q, s, r):
        s = s.double().t().repeat_interleave(r, dim=0)[:q.shape[0]]
        return q.double() * s.repeat_interleave(128, dim=1)[:, :K]

    a, b = stands_for(qa, sa, 1), stands_for(qb, sb, 128)
    want = a @ b.t() + bias.double()
    err = ref.bound(K, (a.abs() @ b.abs().t()).cpu().numpy())
    within(z, f64(want), err + 2.0 ** -24 * np.abs(f64(want)))
    n = want.shape[1] // 2 if gated else want.shape[1]
    act = torch.nn.functional.gelu(want[:, :n], approximate="tanh")
    out = f64(act * want[:, n:] if gated else act) + f64(res)
    lim = 1.13 * err[:, :n] + layer.act_error(f64(want[:, :n]), "gelu_tanh")
    if gated:
        lim = lim * (np.abs(f64(want[:, n:])) + err[:, n:]) + np.abs(f64(act)) * err[:, n:]
    within(y, out, lim + 3 * 2.0 ** -24 * (np.abs(out) + np.abs(f64(res))))


# ------------------------------------------------------------------ the epilogue's backward

# The derivatives are sums of a few products, each with 2^-21 for e^x and 1 / x and an exponent rounded to 2^-23 of
# itself (a derivative falls off faster than the exponent grows): within 2^-17 of the largest value that they can take.
SLOPE = 2.0 ** -17


def check_codes(q, s, dz, terms):
    """q * s against dz [R, C] (float64), groups of 128 along the rows: half a step of E4M3 of the value, half the
    smallest step, dz's own error (SLOPE of its terms) and the roundings of the scale, its reciprocal and the product."""
    scale = f64(s)
    for g in range(-(-dz.shape[1] // 128)):
        piece, own = dz[:, g * 128:(g + 1) * 128], SLOPE * terms[:, g * 128:(g + 1) * 128]
        top = np.maximum(np.abs(piece).max(axis=1), 2.0 ** -100) / 448.0
        assert np.all(np.abs(scale[g] - top) <= 2.0 ** -22 * top + own.max(axis=1) / 448.0)
        got = values(q[:, g * 128:(g + 1) * 128]) * scale[g][:, None]
        lim = (2.0 ** -4 + 2.0 ** -21) * np.abs(piece) + scale[g][:, None] * 2.0 ** -10 + 1.1 * own
        assert np.all(np.abs(got - piece) <= lim)


@pytest.mark.parametrize("R,N", [(1, 1), (3, 129), (128, 128), (130, 200), (300, 1000), (1000, 72)])
@pytest.mark.parametrize("dy_type", ["bf16", "f32"])
@pytest.mark.parametrize("act", layer.ACTS)
def test_act_grad(built, R, N, dy_type, act):
    dy, z = tensor(rand((R, N), 31, 1e-3), dy_type), tensor(rand((R, N), 32))
    q, s, qt, st, db = rlk.fp8_act_grad(dy, z, act, bias_dtype=torch.float32)
    dz = layer.backward(f64(z), f64(dy), act, False)
    if act in ("none", "relu"):
        exact = rlk.fp8_quantize_both(torch.from_numpy(dz.astype(np.float32)).cuda())
        for a, b in zip((q, s, qt, st), exact):
            assert torch.equal(a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a,
                               b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b)
    terms = np.abs(f64(dy)) * 1.13
    check_codes(q, s, dz, terms)
    check_codes(qt, st, dz.T, terms.T)
    assert np.all(np.abs(f64(db) - dz.sum(axis=0)) <= ((R + 4) * 2.0 ** -24 + SLOPE) * terms.sum(axis=0) + 1e-37)
    only = rlk.fp8_act_grad(dy, z, act, rowwise=False)
    assert only[0] is None and only[4] is None and torch.equal(only[2].view(torch.uint8), qt.view(torch.uint8))
    assert torch.equal(rlk.fp8_act_grad(dy, z, act, transpose=False)[0].view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("R,N", [(1, 64), (130, 128), (257, 320)])
@pytest.mark.parametrize("act", layer.ACTS)
def test_act_grad_gated(built, R, N, act):
    dy, z = tensor(rand((R, N), 33, 1e-3)), tensor(rand((R, 2 * N), 34))
    q, s, qt, st, db = rlk.fp8_act_grad(dy, z, act, gated=True, bias_dtype=torch.float32)
    assert q.shape == (R, 2 * N) and qt.shape == (2 * N, R) and db.shape == (2 * N,)
    dz = layer.backward(f64(z), f64(dy), act, True)
    terms = np.abs(f64(dy)) * 1.13
    terms = np.concatenate((terms * np.abs(f64(z)[:, N:]), np.abs(f64(dy)) * (np.abs(f64(z)[:, :N]) + 1)), axis=1)
    assert np.all(np.abs(f64(db) - dz.sum(axis=0)) <= ((R + 5) * 2.0 ** -24 + SLOPE) * terms.sum(axis=0) + 1e-37)
    check_codes(q, s, dz, terms)
    check_codes(qt, st, dz.T, terms.T)


# ------------------------------------------------------------------ rows of groups

SPLITS = {
    "one": ([37], 0), "all in the last": ([0, 0, 0, 90], 0), "all in the first": ([200, 0, 0], 3),
    "even": ([64, 64, 64, 64], 0), "ragged": ([1, 0, 130, 7, 0, 256, 33, 129], 21), "none at all": ([0, 0, 0], 50),
    "single rows": ([1] * 40, 0), "few of many": ([0] * 60 + [2, 0, 1] + [0] * 65, 5), "large": ([700, 3, 515, 0, 300], 0),
    "1024 groups": ([1, 0, 2, 0] * 256, 1), "some tens": ([20, 35, 0, 12, 66, 1, 40], 9), "hundreds": ([300, 129, 513], 70),
    "a hundred each": ([128, 100, 129, 64, 65, 1], 130),
}


def split_of(name):
    counts, pad = SPLITS[name]
    ends = np.cumsum(counts).astype(np.int32)
    return counts, int(ends[-1]) + pad, torch.from_numpy(ends).cuda(), [0, *ends.tolist()]


@pytest.mark.parametrize("name", SPLITS)
@pytest.mark.parametrize("gated,N,K", [(False, 200, 300), (True, 192, 520)])
def test_grouped_layer(built, name, gated, N, K):
    counts, M, ends, at = split_of(name)
    G, rows = len(counts), 2 * N if gated else N
    qa, sa, qb, sb = operands(M, rows, K, 41, (G,))
    bias = tensor(rand((G, rows), 42, 0.5), "f32")
    for out in ("bf16", "f32"):
        y, z = rlk.fp8_grouped_matmul(qa, sa, qb, sb, ends, bias=bias, activation="silu", gated=gated, keep=True,
                                      out_dtype=DT[out], validate=True)
        held = torch.full((M, N), 3.0, device="cuda", dtype=DT[out])
        rlk.fp8_grouped_matmul(qa, sa, qb, sb, ends, bias=bias, activation="silu", gated=gated, out=held)
        assert torch.equal(held[:at[-1]], y[:at[-1]])
        assert (y[at[-1]:] == 0).all() and (held[at[-1]:] == 3.0).all()
        for e in range(G):
            lo, hi = at[e], at[e + 1]
            if hi > lo:
                wz, wy, dz, err = layer.layer(values(qa[lo:hi]), sa[:, lo:hi].cpu().numpy(), values(qb[e]),
                                              sb[e].cpu().numpy(), f64(bias[e]), "silu", gated, None)
                within(z[lo:hi], wz, dz)
                within(y[lo:hi], wy, err)


def test_what_the_rows_behind_the_groups_hold_reaches_nothing(built):
    counts, M, ends, at = split_of("ragged")
    qa, sa, qb, sb = operands(M, 128, 256, 43, (len(counts),))
    want = rlk.fp8_grouped_matmul(qa, sa, qb, sb, ends)
    qa.view(torch.uint8)[at[-1]:] = 0x7F  # NaN
    sa[:, at[-1]:] = float("nan")
    assert torch.equal(rlk.fp8_grouped_matmul(qa, sa, qb, sb, ends), want)
    # and one group's NaN stays with it
    qa.view(torch.uint8)[at[2]:at[3]] = 0x7F
    got = rlk.fp8_grouped_matmul(qa, sa, qb, sb, ends)
    assert torch.equal(got[:at[2]], want[:at[2]]) and torch.equal(got[at[3]:], want[at[3]:])
    assert got[at[2]:at[3]].isnan().all()


@pytest.mark.parametrize("bad", [[50, 20, 70, 10, 90], [-5, 30, -1, 60, 2 ** 31 - 1], [0, 0, 500, 100, 90], [-1, -2, -3, -4, -5]])
def test_ends_out_of_order_are_held_to_their_running_maximum(built, bad):
    M, N, K, G = 100, 130, 200, 5
    qa, sa, qb, sb = operands(M, N, K, 44, (G,))
    ends = torch.tensor(bad, dtype=torch.int32, device="cuda")
    tidy = torch.tensor(np.maximum.accumulate(np.clip(bad, 0, M)), dtype=torch.int32, device="cuda")
    assert torch.equal(rlk.fp8_grouped_matmul(qa, sa, qb, sb, ends), rlk.fp8_grouped_matmul(qa, sa, qb, sb, tidy))
    x = tensor(rand((M, N), 45))
    a, b = rlk.fp8_quantize_grouped(x, ends), rlk.fp8_quantize_grouped(x, tidy)
    used = int(tidy[-1])
    assert torch.equal(a[0][:used].view(torch.uint8), b[0][:used].view(torch.uint8))
    dw = [rlk.fp8_grouped_dweight(v[2], v[3], v[2], v[3], e, M) for v, e in ((a, ends), (b, tidy))]
    assert torch.equal(dw[0], dw[1])


@pytest.mark.parametrize("name", SPLITS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [1, 130, 264])
def test_quantize_grouped(built, name, C, dtype):
    counts, M, ends, at = split_of(name)
    x = tensor(rand((M, C), 51), dtype)
    q, s, qt, st = rlk.fp8_quantize_grouped(x, ends)
    assert qt.shape == (C, 128 * rlk.group_tiles(len(counts), M))
    p = 0
    for e, n in enumerate(counts):
        if n == 0:
            continue
        lo, hi, tiles = at[e], at[e + 1], -(-n // 128)
        wq, ws, wqt, wst = rlk.fp8_quantize_both(x[lo:hi])
        assert torch.equal(q[lo:hi].view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s[:, lo:hi], ws)
        got = qt[:, 128 * p:128 * (p + tiles)].view(torch.uint8)
        assert torch.equal(got[:, :n], wqt.view(torch.uint8)) and (got[:, n:] == 0).all()
        assert torch.equal(st[p:p + tiles], wst)
        p += tiles
    alone = rlk.fp8_quantize_grouped(x, ends, rowwise=False)
    assert alone[0] is None and torch.equal(alone[2][:, :128 * p].view(torch.uint8), qt[:, :128 * p].view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,R,C", [(1, 1, 1), (3, 130, 200), (5, 128, 384), (4, 300, 129)])
def test_quantize_of_several_matrices(built, G, R, C, dtype):
    x = tensor(rand((G, R, C), 52), dtype)
    for t in (x, tensor(rand((G, R + 3, C + 8), 53), dtype)[:, :R, :C]):
        q, s, qt, st = rlk.fp8_quantize_both(t, block_rows=128)
        for e in range(G):
            for got, want in zip((q[e], s[e], qt[e], st[e]), rlk.fp8_quantize_both(t[e], block_rows=128)):
                assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(rlk.fp8_quantize(x, 128)[0].view(torch.uint8), rlk.fp8_quantize_both(x, 128)[0].view(torch.uint8))
    assert torch.equal(rlk.fp8_quantize(x, 128, True)[0].view(torch.uint8),
                       rlk.fp8_quantize_both(x, 128)[2].view(torch.uint8))


@pytest.mark.parametrize("name", SPLITS)
def test_grouped_dweight(built, name):
    counts, rows, ends, at = split_of(name)
    G = len(counts)
    M, N = (20, 33) if G > 100 else (300, 140)
    dy, x = tensor(rand((rows, M), 61)), tensor(rand((rows, N), 62))
    _, _, at_q, at_s = rlk.fp8_quantize_grouped(dy, ends, rowwise=False)
    _, _, bt_q, bt_s = rlk.fp8_quantize_grouped(x, ends, rowwise=False)
    old = tensor(rand((G, M, N), 63), "f32")
    f32 = rlk.fp8_grouped_dweight(at_q, at_s, bt_q, bt_s, ends, rows, out_dtype=torch.float32, validate=True)
    bf16 = rlk.fp8_grouped_dweight(at_q, at_s, bt_q, bt_s, ends, rows)
    assert torch.equal(bf16, f32.to(torch.bfloat16))
    added = rlk.fp8_grouped_dweight(at_q, at_s, bt_q, bt_s, ends, rows, out=old.clone(), accumulate=True)
    assert torch.equal(added, old + f32)
    p = 0
    for e, n in enumerate(counts):
        tiles = -(-n // 128)
        if n == 0:
            assert (f32[e] == 0).all()
            continue
        cols = slice(128 * p, 128 * (p + tiles))
        want, terms = ref.matmul(values(at_q[:, cols]), at_s[p:p + tiles].cpu().numpy(), values(bt_q[:, cols]),
                                 bt_s[p:p + tiles].cpu().numpy(), 1)
        assert np.all(np.abs(f64(f32[e]) - want) <= ref.bound(128 * tiles, terms))
        p += tiles


def test_grouped_offsets_past_32_bits(built):
    # a weight of 2.3e9 codes: the last groups lie past 2^31 bytes
    G, N, K, M = 36, 8000, 8192, 40
    free, _ = torch.cuda.mem_get_info()
    if free < 8 << 30:  # pragma: no cover
        pytest.skip("needs 8 GB")
    ends = torch.zeros(G, dtype=torch.int32, device="cuda")
    ends[-1] = M
    q1, s1 = rlk.fp8_quantize(tensor(rand((N, K), 71, 0.05)), block_rows=128)
    qb = torch.zeros((G, N, K), dtype=torch.uint8, device="cuda")
    qb[-1] = q1.view(torch.uint8)
    sb = torch.zeros((G, *s1.shape), device="cuda")
    sb[-1] = s1
    qa, sa = rlk.fp8_quantize(tensor(rand((M, K), 72)))
    got = rlk.fp8_grouped_matmul(qa, sa, qb.view(torch.float8_e4m3fn), sb, ends, out_dtype=torch.float32)
    want = rlk.fp8_matmul(qa, sa, q1, s1, out_dtype=torch.float32)
    assert float((got - want).abs().max()) <= 1e-4 * float(want.abs().max())


# ------------------------------------------------------------------ training

def relative(got, want):
    return float(np.linalg.norm(f64(got) - want) / np.linalg.norm(want))


# Each operand of a product is within half a step of E4M3, 2^-4 of its value: over a binade that is 2^-4 / sqrt 3 on
# average at most, and two independent operands give sqrt 2 of it, 5.1%; the kept z and a BF16 result add 2^-8 each,
# and the backward starts from a forward that is that far off.
FP8_TOLERANCE = 0.051 * 1.5


@pytest.mark.parametrize("act,gated,bias,residual", [("gelu", False, True, True), ("silu", True, False, False),
                                                     ("gelu_tanh", True, True, True), ("none", False, True, False),
                                                     ("none", False, False, True), ("relu", False, True, False)])
@pytest.mark.parametrize("lead", [(5,), (3, 67), (300,)])
def test_linear_gradients_against_the_formula(built, lead, act, gated, bias, residual):
    K, N = 200, 192
    rows = 2 * N if gated else N
    x = tensor(rand((*lead, K), 81)).requires_grad_()
    w = tensor(rand((rows, K), 82, 0.07), "f32").requires_grad_()
    b = tensor(rand((1, rows), 83, 0.3)[0], "f32").requires_grad_() if bias else None
    r = tensor(rand((*lead, N), 84)).requires_grad_() if residual else None
    y = autograd.fp8_linear(x, w, bias=b, activation=act, gated=gated, residual=r)
    assert y.shape == (*lead, N) and y.dtype == torch.bfloat16
    dy = tensor(rand((*lead, N), 85))
    leaves = [t for t in (x, w, b, r) if t is not None]
    grads = dict(zip([n for n, t in zip("xwbr", (x, w, b, r)) if t is not None],
                     torch.autograd.grad(y, leaves, dy)))
    X, W = f64(x).reshape(-1, K), f64(w)
    Z = X @ W.T + (0 if b is None else f64(b))
    D = f64(dy).reshape(-1, N)
    want_y = layer.forward(Z, act, gated) + (0 if r is None else f64(r).reshape(-1, N))
    dz = layer.backward(Z, D, act, gated)
    # the backward at z as the forward had it: of the quantised operands, in BF16
    assert relative(y.reshape(-1, N), want_y) <= FP8_TOLERANCE
    slack = 1.0 if act != "relu" else 3.0  # a step's derivative jumps where z's sign changes
    assert relative(grads["x"].reshape(-1, K), dz @ W) <= FP8_TOLERANCE * 1.5 * slack
    assert relative(grads["w"], dz.T @ X) <= FP8_TOLERANCE * 1.5 * slack
    assert grads["x"].dtype == torch.bfloat16 and grads["w"].dtype == torch.float32
    if bias:
        assert relative(grads["b"], dz.sum(axis=0)) <= FP8_TOLERANCE * 1.5 * slack
    if residual:
        assert torch.equal(grads["r"], dy)


def test_linear_inference_is_the_training_forward(built):
    x, w, b = tensor(rand((70, 128), 86)), tensor(rand((256, 128), 87, 0.1)), tensor(rand((1, 256), 88)[0])
    y = autograd.fp8_linear(x, w, bias=b, activation="silu", gated=True)
    wg = w.clone().requires_grad_()
    assert torch.equal(autograd.fp8_linear(x, wg, bias=b, activation="silu", gated=True).detach(), y)


@pytest.mark.parametrize("frozen", ["x", "w", "b", "xw", "xb", "wb"])
def test_frozen_inputs(built, frozen):
    x, w, b = tensor(rand((90, 160), 89)), tensor(rand((128, 160), 90, 0.1)), tensor(rand((1, 128), 91)[0])
    ends = torch.tensor([40, 40, 85], dtype=torch.int32, device="cuda")
    w3, b3 = torch.stack([w, w * 2, w * 0.5]), torch.stack([b, b, -b])
    for call, ts in ((lambda x, w, b: autograd.fp8_linear(x, w, b, "gelu"), (x, w, b)),
                     (lambda x, w, b: autograd.fp8_grouped_linear(x, w, ends, b, "gelu"), (x, w3, b3))):
        full = [t.clone().requires_grad_() for t in ts]
        dy = torch.ones((90, 128), device="cuda", dtype=torch.bfloat16)
        want = torch.autograd.grad(call(*full), full, dy)
        part = [t.clone().requires_grad_(n not in frozen) for n, t in zip("xwb", ts)]
        got = torch.autograd.grad(call(*part), [t for t in part if t.requires_grad], dy)
        for g, t in zip(got, [t for n, t in zip("xwb", want) if n not in frozen]):
            assert torch.equal(g, t)


@pytest.mark.parametrize("name", ["one", "all in the last", "ragged", "none at all", "few of many", "large"])
@pytest.mark.parametrize("act,gated,bias", [("silu", True, False), ("gelu", False, True), ("none", False, False),
                                            ("none", False, True)])
def test_grouped_gradients_against_the_formula(built, name, act, gated, bias):
    counts, M, ends, at = split_of(name)
    G, N, K = len(counts), 128, 136
    rows = 2 * N if gated else N
    xs = rand((M, K), 92)
    xs[at[-1]:] = np.nan  # padding holds anything
    x = tensor(xs).requires_grad_()
    w = tensor(rand((G, rows, K), 93, 0.08)).requires_grad_()
    b = tensor(rand((G, rows), 94, 0.3)).requires_grad_() if bias else None
    dys = rand((M, N), 95)
    dys[at[-1]:] = np.inf
    y = autograd.fp8_grouped_linear(x, w, ends, bias=b, activation=act, gated=gated)
    grads = torch.autograd.grad(y, [x, w] + ([b] if bias else []), tensor(dys))
    assert (y[at[-1]:] == 0).all() and (grads[0][at[-1]:] == 0).all()
    want = [np.zeros((M, N)), np.zeros((M, K)), np.zeros((G, rows, K)), np.zeros((G, rows))]
    X, W, D = f64(x), f64(w), f64(tensor(dys))
    for e in range(G):
        lo, hi = at[e], at[e + 1]
        if hi > lo:
            Z = X[lo:hi] @ W[e].T + (f64(b)[e] if bias else 0)
            want[0][lo:hi] = layer.forward(Z, act, gated)
            dz = layer.backward(Z, D[lo:hi], act, gated)
            want[1][lo:hi], want[2][e], want[3][e] = dz @ W[e], dz.T @ X[lo:hi], dz.sum(axis=0)
        else:
            assert (grads[1][e] == 0).all() and (not bias or (grads[2][e] == 0).all())
    if at[-1]:
        assert relative(y, want[0]) <= FP8_TOLERANCE
        for g, t in zip(grads, want[1:]):
            assert relative(g, t) <= FP8_TOLERANCE * 1.5


def test_no_rows(built):
    w = tensor(rand((2, 128, 64), 96)).requires_grad_()
    b = torch.zeros((2, 128), device="cuda", requires_grad=True)
    x = torch.zeros((0, 64), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    ends = torch.zeros(2, dtype=torch.int32, device="cuda")
    y = autograd.fp8_grouped_linear(x, w, ends, bias=b, activation="relu")
    assert y.shape == (0, 128)
    for g, t in zip(torch.autograd.grad(y.sum(), (x, w, b)), (x, w, b)):
        assert g.shape == t.shape and (g == 0).all()
    w2, b2 = w[0].detach().requires_grad_(), b[0].detach().requires_grad_()
    y = autograd.fp8_linear(x, w2, bias=b2, activation="silu", gated=True)
    assert y.shape == (0, 64)
    for g, t in zip(torch.autograd.grad(y.sum(), (x, w2, b2)), (x, w2, b2)):
        assert g.shape == t.shape and (g == 0).all()


# ------------------------------------------------------------------ together, and on streams

def test_a_block_of_experts_together(built):
    """Routing, the experts' gated layer and their second one, the shared dense block with its residual, the head's
    cross entropy: one training step, its gradients against the same in FP32."""
    torch.manual_seed(0)
    T, D, F, G, top, V = 200, 128, 192, 6, 2, 500
    p = [torch.randn(s, device="cuda") * sc for s, sc in (((T, D), 1.0), ((G, D), 0.3), ((G, 2 * F, D), 0.09), ((G, D, F), 0.07),
                                                          ((2 * F, D), 0.09), ((D, F), 0.07), ((D,), 0.1), ((V, D), 0.05))]
    p = [t.to(torch.bfloat16) for t in p]
    target = torch.randint(0, V, (T,), device="cuda")
    choice = (p[0].float() @ p[1].float().t()).topk(top).indices  # the same routing for both

    def step(x, router, up, down, sup, sdown, bias, head, own):
        gate = torch.softmax(x.float() @ router.float().t(), dim=1).gather(1, choice)
        expert = choice.reshape(-1)
        order = expert.argsort(stable=True)
        ends = torch.bincount(expert, minlength=G).cumsum(0).to(torch.int32)
        rows = x[order // top]
        if own:
            h = autograd.fp8_grouped_linear(rows, up, ends, activation="silu", gated=True)
            out = autograd.fp8_grouped_linear(h, down, ends)
            mixed = torch.zeros((T, D), device="cuda").index_add(0, order // top, out.float() * gate.reshape(-1)[order][:, None])
            h = autograd.fp8_linear(x, sup, activation="silu", gated=True)
            y = autograd.fp8_linear(h, sdown, bias=bias, residual=(x.float() + mixed).to(torch.bfloat16))
            return autograd.linear_cross_entropy(y, head, target)
        f = lambda v, w: torch.nn.functional.silu(v @ w[:F].float().t()) * (v @ w[F:].float().t())  # noqa: E731
        e = expert[order]
        v = rows.float()
        h = torch.stack([f(v[i:i + 1], up[k])[0] for i, k in enumerate(e.tolist())])
        out = torch.einsum("rf,rdf->rd", h, down.float()[e])
        mixed = torch.zeros((T, D), device="cuda").index_add(0, order // top, out * gate.reshape(-1)[order][:, None])
        y = f(x.float(), sup) @ sdown.float().t() + bias.float() + x.float() + mixed
        return torch.nn.functional.cross_entropy(y @ head.float().t(), target)

    results = []
    for own in (True, False):
        leaves = [t.clone().requires_grad_() for t in p]
        loss = step(*leaves, own)
        results.append((loss, torch.autograd.grad(loss, leaves)))
    # the logits are within the products' error of theirs, and the loss moves by no more than the logits do
    assert abs(float(results[0][0]) - float(results[1][0])) <= FP8_TOLERANCE
    for a, b in zip(results[0][1], results[1][1]):
        # three layers deep: each adds its own error
        assert relative(a, f64(b)) <= 3 * FP8_TOLERANCE


def test_given_streams_and_two_calls_at_once(built):
    qa, sa, qb, sb = operands(300, 640, 512, 101)
    counts, M, ends, _ = split_of("ragged")
    ga, gsa, gb, gsb = operands(M, 256, 384, 102, (len(counts),))
    want = rlk.fp8_matmul_act(qa, sa, qb, sb, activation="gelu"), rlk.fp8_grouped_matmul(ga, gsa, gb, gsb, ends)
    x = tensor(rand((M, 130), 103))
    want_q = rlk.fp8_quantize_grouped(x, ends)[0].clone()
    used = int(ends[-1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        got.append(rlk.fp8_matmul_act(qa, sa, qb, sb, activation="gelu", stream=streams[0]))
        got.append(rlk.fp8_grouped_matmul(ga, gsa, gb, gsb, ends, stream=streams[1]))
        q = rlk.fp8_quantize_grouped(x, ends, stream=streams[0])[0]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i & 1])
    assert torch.equal(q[:used].view(torch.uint8), want_q[:used].view(torch.uint8))


def test_captured_steps(built):
    """A step captured once and replayed on other inputs, other group sizes among them."""
    G, M, N, K = 5, 260, 128, 192
    x, w = tensor(rand((M, K), 104)).requires_grad_(), tensor(rand((G, 2 * N, K), 105, 0.08)).requires_grad_()
    dy = tensor(rand((M, N), 106))
    ends = torch.tensor([50, 50, 120, 121, 250], dtype=torch.int32, device="cuda")

    def step():
        y = autograd.fp8_grouped_linear(x, w, ends, activation="silu", gated=True)
        return (y, *torch.autograd.grad(y, (x, w), dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k, new in enumerate(([50, 50, 120, 121, 250], [0, 200, 200, 200, 260], [260] * 5, [0] * 5)):
        ends.copy_(torch.tensor(new, dtype=torch.int32))
        with torch.no_grad():
            x.copy_(tensor(rand((M, K), 107 + k)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_two_captured_graphs_at_once(built):
    """Graphs that share the stream's status word, replayed on two streams."""
    counts, M, ends, _ = split_of("large")
    ga, gsa, gb, gsb = operands(M, 256, 384, 112, (len(counts),))
    qa, sa, qb, sb = operands(300, 640, 512, 113)
    want = rlk.fp8_grouped_matmul(ga, gsa, gb, gsb, ends), rlk.fp8_matmul_act(qa, sa, qb, sb, activation="silu", gated=True)
    calls = (lambda: rlk.fp8_grouped_matmul(ga, gsa, gb, gsb, ends),
             lambda: rlk.fp8_matmul_act(qa, sa, qb, sb, activation="silu", gated=True))
    graphs, held = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g, call in zip(graphs, calls):
        with torch.cuda.graph(g):
            held.append(call())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1])


def test_same_bits_again(built):
    counts, M, ends, _ = split_of("large")
    x, w = tensor(rand((M, 300), 108)).requires_grad_(), tensor(rand((len(counts), 384, 300), 109, 0.06)).requires_grad_()
    b = tensor(rand((len(counts), 384), 110)).requires_grad_()
    dy = tensor(rand((M, 192), 111))
    runs = [torch.autograd.grad(autograd.fp8_grouped_linear(x, w, ends, b, "gelu", True), (x, w, b), dy) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, c) for a, c in zip(r, runs[0]))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
def test_a_rows_result_is_its_own(built, act, gated):
    """Other rows of the call, of the next group and behind the groups leave a row's bits as they are."""
    N, K = 192, 130
    for M in (3, 8, 23, 50, 64, 100, 300):
        qb, sb = operands(1, 2 * N if gated else N, K, 130)[2:]
        x = tensor(rand((M, K), 131 + M))
        other = tensor(rand((M, K), 132 + M, 3.0))
        mine = torch.arange(M, device="cuda") % 3 == 0  # no row beside it, nor two away, is
        other[mine] = x[mine]
        a, b = (rlk.fp8_matmul_act(*rlk.fp8_quantize(v), qb, sb, activation=act, gated=gated, out_dtype=torch.float32)
                for v in (x, other))
        assert torch.equal(a[mine], b[mine]), M
        assert not torch.equal(a, b)
    G = 6
    qb, sb = operands(1, 2 * N if gated else N, K, 133, (G,))[2:]
    for counts in ([1, 0, 2, 1, 3, 1], [5, 1, 1, 20, 7, 1], [30, 1, 0, 33, 20, 3], [50, 1, 70, 40, 1, 60], [200, 1, 300, 0, 129, 1]):
        used = sum(counts)
        M = used + 7
        ends = torch.tensor(counts, device="cuda").cumsum(0).to(torch.int32)
        x = tensor(rand((M, K), 134 + M))
        other = tensor(rand((M, K), 135 + M, 3.0))
        mine = torch.arange(M, device="cuda") % 3 == 0
        mine[used - 1], mine[used:] = True, False
        other[mine] = x[mine]
        a, b = (rlk.fp8_grouped_matmul(*rlk.fp8_quantize(v), qb, sb, ends, activation=act, gated=gated,
                                       out_dtype=torch.float32) for v in (x, other))
        assert torch.equal(a[mine], b[mine]), counts
        assert not torch.equal(a, b)
