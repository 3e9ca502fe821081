"""FP8 quantisation and the FP8 product against plain 64-bit forms, on the GPU.

Quantisation is held to equality: its definition fixes every rounding.  The
product's bound (fp8_reference.bound) counts its FP32 roundings against the
sum of the terms' magnitudes; a BF16 result is the FP32 one rounded once.
"""
import numpy as np
import pytest
import torch

import fp8_reference as ref
import vocab_selected_token_tile_gb300 as rlk

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def rand(shape, seed, sigma=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape).astype(np.float32) * np.float32(sigma)
    x *= np.where(rng.random(shape[1]) < 0.05, np.float32(20), np.float32(1))  # a few large channels
    return x


def as_input(x, dtype):
    t = torch.from_numpy(x)
    return t.to(torch.bfloat16).cuda() if dtype == "bf16" else t.cuda()


def values(q):
    return q.float().cpu().numpy().astype(np.float64)


def same(got, want):
    return np.array_equal(np.nan_to_num(got, nan=1e9), np.nan_to_num(want, nan=1e9)) and \
        np.array_equal(np.isnan(got), np.isnan(want))


def check_quantized(x, block, result, transposed=False):
    q, s = result
    want_q, want_s = ref.quantize(x.T if transposed else x, block)
    assert same(values(q), want_q)
    assert same(s.cpu().numpy(), want_s)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 128), (1, 4096), (2, 7), (3, 129), (8, 136), (127, 128), (128, 127),
                                 (129, 1000), (200, 385), (257, 264)])
def test_quantize_matches_the_definition(built, R, C, dtype, block):
    t = as_input(rand((R, C), R * 1000 + C), dtype)
    x = t.float().cpu().numpy()
    check_quantized(x, block, rlk.fp8_quantize(t, block_rows=block))
    check_quantized(x, block, rlk.fp8_quantize(t, block_rows=block, transpose=True), transposed=True)
    q, s, qt, st = rlk.fp8_quantize_both(t, block_rows=block)
    check_quantized(x, block, (q, s))
    check_quantized(x, block, (qt, st), transposed=True)
    assert q.stride(0) % 16 == 0 and q.data_ptr() % 16 == 0 and (C == 1 or qt.stride(0) % 16 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset,stride", [(0, 300), (1, 301), (8, 304), (3, 512)])
def test_quantize_strided_and_unaligned_rows(built, offset, stride, dtype):
    R, C = 140, 290
    buf = as_input(rand((1, R * stride + 16), 5), dtype)[0]
    t = buf[offset:offset + R * stride].as_strided((R, C), (stride, 1), storage_offset=offset)
    x = t.float().cpu().numpy()
    q, s, qt, st = rlk.fp8_quantize_both(t)
    check_quantized(x, 1, (q, s))
    check_quantized(x, 1, (qt, st), transposed=True)


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_special_values(built, block):
    R, C = 260, 400
    x = rand((R, C), 9)
    x[0, :] = 0.0                      # a whole row of zeros
    x[3, 128:256] = -0.0
    x[5, 10] = np.nan                  # one NaN, one infinity: their groups stand for NaN
    x[7, 300] = np.inf
    x[9, 0] = -np.inf
    x[11, :128] = np.float32(1e-38)    # below the floor: zeros
    x[12, :128] = np.float32(2.0 ** -99)
    x[13, :128] = np.float32(3.0e38)
    x[14, :] = 448.0                   # the largest value, at scale 1
    x[15, :128] = np.linspace(0, 448, 128, dtype=np.float32)
    t = torch.from_numpy(x).cuda()
    q, s, qt, st = rlk.fp8_quantize_both(t, block_rows=block)
    check_quantized(x, block, (q, s))
    check_quantized(x, block, (qt, st), transposed=True)
    if block == 1:
        assert np.all(values(q)[0] == 0) and np.isfinite(s[:, 0].cpu().numpy()).all()
        assert np.isnan(values(q)[5, :128] * s[0, 5].item()).all()


def test_quantize_writes_nothing_past_its_columns(built):
    R, C = 130, 130
    t = as_input(rand((R, C), 2), "bf16")
    q = torch.full((R, 160), 0xAB, dtype=torch.uint8, device="cuda")
    qt = torch.full((C, 176), 0xCD, dtype=torch.uint8, device="cuda")
    s = torch.empty((2, R), device="cuda")
    st = torch.empty((2, C), device="cuda")
    rlk.check(rlk.rlk_fp8_quantize(R, C, t.data_ptr(), rlk.RLK_BF16, C, 1, q.data_ptr(), 160, s.data_ptr(),
                                   qt.data_ptr(), 176, st.data_ptr(), torch.cuda.current_stream().cuda_stream))
    check_quantized(t.float().cpu().numpy(), 1, (q[:, :C].view(torch.float8_e4m3fn), s))
    check_quantized(t.float().cpu().numpy(), 1, (qt[:, :R].view(torch.float8_e4m3fn), st), transposed=True)
    assert (q[:, C:] == 0xAB).all() and (qt[:, R:] == 0xCD).all()


def operands(M, N, K, block, seed=1):
    a, b = as_input(rand((M, K), seed), "bf16"), as_input(rand((N, K), seed + 1, 0.05), "bf16")
    qa, sa = rlk.fp8_quantize(a)
    qb, sb = rlk.fp8_quantize(b, block_rows=block)
    return qa, sa, qb, sb


def expect(qa, sa, qb, sb, block):
    return ref.matmul(values(qa), sa.cpu().numpy(), values(qb), sb.cpu().numpy(), block)


def check_product(got, want, terms, K):
    err, lim = np.abs(got.cpu().numpy().astype(np.float64) - want), ref.bound(K, terms)
    assert (err <= lim).all(), f"worst {np.max(err / lim):.3g} of the bound"


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 128, 128), (1, 1000, 100), (1, 4096, 4096), (5, 129, 384), (16, 257, 1000), (17, 100, 129),
    (32, 300, 2048), (33, 255, 640), (64, 1024, 128), (65, 128, 1024), (100, 515, 500), (128, 260, 5000),
    (129, 1, 128), (129, 256, 128), (200, 257, 129), (300, 1000, 1000), (1000, 384, 16), (520, 900, 2300)])
def test_product_matches_64_bits(built, M, N, K, block):
    qa, sa, qb, sb = operands(M, N, K, block, seed=M + N + K)
    want, terms = expect(qa, sa, qb, sb, block)
    f32 = rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=block, out_dtype=torch.float32, validate=True)
    check_product(f32, want, terms, K)
    bf16 = rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=block)
    assert torch.equal(bf16, f32.to(torch.bfloat16))  # the same sums, rounded once
    again = rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=block, out_dtype=torch.float32)
    assert torch.equal(again, f32)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M,N,K", [
    (2100, 2501, 130),    # more tiles than pairs of CTAs, odd rows of C
    (700, 20002, 300), (256, 20480, 128),
    (65, 300, 9000), (257, 511, 4001),  # K split over a cluster, many granules of scales
    (3, 40000, 700), (40, 40001, 260)])  # more tiles than the persistent CTAs of few rows
def test_product_of_many_tiles(built, M, N, K, block):
    qa, sa, qb, sb = operands(M, N, K, block, seed=N)
    a = qa.double() * sa.double().t().repeat_interleave(128, dim=1)[:, :K]
    b = qb.double() * sb.double().t().repeat_interleave(128, dim=1)[:, :K].repeat_interleave(block, dim=0)[:N]
    want, terms = a @ b.t(), a.abs() @ b.abs().t()
    f32 = rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=block, out_dtype=torch.float32, validate=True)
    assert ((f32.double() - want).abs() <= ref.bound(K, terms)).all()
    assert torch.equal(rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=block), f32.to(torch.bfloat16))
    base = torch.randn((M, N), device="cuda")
    out = base.clone()
    rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=block, out=out, accumulate=True)
    assert torch.equal(out, base + f32)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M,N,K", [(2309, 2100, 4100), (2560, 4090, 2816), (2100, 2820, 9000)])
def test_product_whose_last_tiles_are_split(built, M, N, K, block):
    # 90, 160 and 108 tiles of 256 x 256, K long enough for a second launch that overlaps the first's end: what
    # follows in the stream, on the same C, must follow both
    qa, sa, qb, sb = operands(M, N, K, block, seed=K)
    a = qa.double() * sa.double().t().repeat_interleave(128, dim=1)[:, :K]
    b = qb.double() * sb.double().t().repeat_interleave(128, dim=1)[:, :K].repeat_interleave(block, dim=0)[:N]
    f32 = rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=block, out_dtype=torch.float32, validate=True)
    assert ((f32.double() - a @ b.t()).abs() <= ref.bound(K, a.abs() @ b.abs().t())).all()
    ws = torch.zeros(rlk.RLK_FP8_WORKSPACE, dtype=torch.uint8, device="cuda")
    out, want = torch.zeros((M, N), device="cuda"), torch.zeros((M, N), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=block, out=out, accumulate=True, workspace=ws)
            out.mul_(0.5)
    graph.replay()
    for _ in range(4):
        want.add_(f32).mul_(0.5)
    assert torch.equal(out, want)
    for _ in range(4):
        rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=block, out=out, accumulate=True, workspace=ws)
        want.add_(f32)
    assert torch.equal(out, want)


@pytest.mark.parametrize("M,K", [(3, 300), (200, 300), (130, 3000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,stride", [(0, 264), (1, 263), (4, 300)])
def test_product_into_strided_rows(built, M, K, dtype, offset, stride):
    N = 259
    qa, sa, qb, sb = operands(M, N, K, 128)
    plain = rlk.fp8_matmul(qa, sa, qb, sb, out_dtype=dtype)
    buf = torch.full((M * stride + 16,), 7.0, dtype=dtype, device="cuda")
    out = buf.as_strided((M, N), (stride, 1), storage_offset=offset)
    assert rlk.fp8_matmul(qa, sa, qb, sb, out=out) is out
    assert torch.equal(out, plain)
    untouched = torch.ones_like(buf, dtype=torch.bool)
    untouched.as_strided((M, N), (stride, 1), storage_offset=offset).zero_()
    assert (buf[untouched] == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(2, 300, 700), (150, 300, 700)])
def test_product_accumulates(built, M, N, K):
    qa, sa, qb, sb = operands(M, N, K, 1)
    plain = rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=1, out_dtype=torch.float32)
    base = torch.randn((M, N), device="cuda")
    out = base.clone()
    rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=1, out=out, accumulate=True)
    assert torch.equal(out, base + plain)


def test_product_of_nan_and_infinite_groups(built):
    M, N, K = 40, 200, 256
    a = as_input(rand((M, K), 3), "bf16")
    a[7, 130] = float("nan")
    a[9, 5] = float("inf")
    qa, sa = rlk.fp8_quantize(a)
    qb, sb = rlk.fp8_quantize(as_input(rand((N, K), 4), "bf16"), block_rows=128)
    out = rlk.fp8_matmul(qa, sa, qb, sb)
    bad = torch.isnan(out).all(dim=1).cpu()
    assert bad[7] and bad[9] and int(bad.sum()) == 2
    assert torch.isfinite(out[[r for r in range(M) if r not in (7, 9)]]).all()


def test_product_takes_rows_of_other_strides(built):
    M, N, K = 20, 300, 200
    qa, sa, qb, sb = operands(M, N, K, 128)
    want = rlk.fp8_matmul(qa, sa, qb, sb)
    wide = torch.full((M, 512), 0x7F, dtype=torch.uint8, device="cuda")  # NaN codes around the operand
    wide[:, 64:64 + K] = qa.view(torch.uint8)
    assert torch.equal(rlk.fp8_matmul(wide[:, 64:64 + K], sa, qb, sb), want)


def test_product_past_2_to_31_elements(built):
    M, N, K = 8300, 260000, 128  # 2.16e9 elements of C
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    qa, sa, qb, sb = operands(M, N, K, 1, seed=11)
    out = rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=1, validate=True)
    rows = [0, 4129, 8299]
    part = rlk.fp8_matmul(qa[rows], sa[:, rows].contiguous(), qb, sb, b_block_rows=1)
    assert torch.equal(out[rows], part)


def test_product_on_another_stream_and_in_a_graph(built):
    qa, sa, qb, sb = operands(3, 1000, 1024, 128)
    want = rlk.fp8_matmul(qa, sa, qb, sb)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = rlk.fp8_matmul(qa, sa, qb, sb)
    side.synchronize()
    assert torch.equal(got, want)
    x = as_input(rand((3, 1024), 77), "bf16")
    out = torch.empty_like(want)
    ws = torch.zeros(rlk.RLK_FP8_WORKSPACE, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, s = rlk.fp8_quantize(x)
        rlk.fp8_matmul(q, s, qb, sb, out=out, workspace=ws)
    x.copy_(as_input(rand((3, 1024), 78), "bf16"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, rlk.fp8_matmul(*rlk.fp8_quantize(x), qb, sb))


def test_stream_argument(built):
    # the calls enqueue on the given stream, whatever the current one is, and their results may be freed at once
    x, w = as_input(rand((5, 512), 1), "bf16"), as_input(rand((300, 512), 2), "bf16")
    want = rlk.fp8_matmul(*rlk.fp8_quantize(x), *rlk.fp8_quantize(w, block_rows=128))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rlk.fp8_matmul(*rlk.fp8_quantize(x, stream=side), *rlk.fp8_quantize(w, block_rows=128, stream=side),
                         stream=side)
    junk = [torch.full((300, 512), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(4)]  # noqa: F841
    side.synchronize()
    assert torch.equal(got, want)


def test_binding_refuses_what_the_call_cannot_read(built):
    qa, sa, qb, sb = operands(4, 130, 200, 128)
    with pytest.raises(ValueError):
        rlk.fp8_matmul(qa, sa, qb[:, :100], sb)
    with pytest.raises(ValueError):
        rlk.fp8_matmul(qa, sa[:1], qb, sb)
    with pytest.raises(ValueError):
        rlk.fp8_matmul(qa, sa, qb, sb, b_block_rows=1)
    with pytest.raises(TypeError):
        rlk.fp8_matmul(qa.float(), sa, qb, sb)
    with pytest.raises(ValueError):
        rlk.fp8_matmul(qa.t(), sa, qb, sb)
    with pytest.raises(ValueError):
        rlk.fp8_matmul(qa, sa, qb, sb, accumulate=True)
    with pytest.raises(rlk.RlkError):  # accumulation is in FP32
        rlk.fp8_matmul(qa, sa, qb, sb, out=torch.zeros((4, 130), dtype=torch.bfloat16, device="cuda"), accumulate=True)
    with pytest.raises(TypeError):
        rlk.fp8_matmul(qa, sa, qb, sb, out_dtype=torch.float16)
    with pytest.raises(rlk.RlkError) as e:  # rows off the 16-byte grid
        rlk.fp8_matmul(torch.zeros((4, 201), dtype=torch.uint8, device="cuda")[:, :200], sa, qb, sb)
    assert e.value.status == rlk.RLK_ERR_MISALIGNED
    with pytest.raises(ValueError):
        rlk.fp8_quantize(torch.zeros(8, device="cuda"))
    with pytest.raises(TypeError):
        rlk.fp8_quantize(torch.zeros((8, 8), device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        rlk.fp8_quantize(torch.zeros((8, 8)))


def test_empty_products_and_matrices(built):
    q, s = rlk.fp8_quantize(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (1, 0)
    qb, sb = rlk.fp8_quantize(torch.ones((5, 64), dtype=torch.bfloat16, device="cuda"), block_rows=128)
    assert rlk.fp8_matmul(q, s, qb, sb).shape == (0, 5)
