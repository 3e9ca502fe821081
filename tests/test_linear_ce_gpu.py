"""The cross entropy of hidden @ weight^T and its gradients against the 64-bit reference, on the GPU.

The tolerances are ce_reference's bounds: counts of the FP32 roundings on the
way, each against the magnitude it applies to, and the BF16 rounding of the
logits' gradient and of the results.
"""
import numpy as np
import pytest
import torch

import ce_reference as ref
import vocab_selected_token_tile_gb300 as rlk
from vocab_selected_token_tile_gb300.autograd import fp8_linear, linear_cross_entropy

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

REDUCTIONS = {"none": rlk.REDUCE_NONE, "sum": rlk.REDUCE_SUM, "mean": rlk.REDUCE_MEAN}


def bf16_matrix(rows, cols, seed, sigma, pad=0):
    """A [rows, cols] BF16 CUDA matrix whose rows are 16-byte aligned, NaN in the padding."""
    rng = np.random.default_rng(seed)
    t = torch.from_numpy((rng.standard_normal((rows, cols)) * sigma).astype(np.float32)).to(torch.bfloat16).cuda()
    stride = -(-cols // 8) * 8 + pad
    if stride == cols:
        return t
    buf = torch.full((rows, stride), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:, :cols] = t
    return buf[:, :cols]


def case(T, V, H, seed=0, pad=0, inactive=0.25):
    h, w = bf16_matrix(T, H, seed, 1.0, pad), bf16_matrix(V, H, seed + 1, 2.0 / np.sqrt(H), pad)
    rng = np.random.default_rng(seed + 2)
    t = rng.integers(0, V, T)
    on = rng.random(T) >= inactive
    t[~on] = rng.choice([-100, -1, V, V + 7, 1 << 40], int((~on).sum()))  # never used as an index
    return h, w, t, on


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def check_forward(h, w, t, on, loss, lse, reduction, eps, z, cap):
    want, want_lse, y = ref.forward(host(h), host(w), t, on, eps, z, cap)
    b = ref.loss_bound(host(h), host(w), y, want_lse, eps, z, cap)
    assert (np.abs(host(lse) - want_lse) <= ref.lse_bound(host(h), host(w), y, cap)).all()
    if reduction == "none":
        assert (np.abs(host(loss) - want) <= np.where(on, b, 0)).all()
    else:
        total = ref.reduce(want, on, reduction)
        lim = ref.reduce(np.where(on, b, 0), on, reduction) + 2.0 ** -22 * abs(total)
        assert abs(float(loss) - total) <= lim
    return want_lse, y


def check_backward(h, w, t, on, dh, dw, rows, lse, y, eps, z, cap):
    want_h, want_w = ref.backward(host(h), host(w), t, on, rows, eps, z, cap)
    bh, bw = ref.gradient_bounds(host(h), host(w), y, lse, t, on, rows, eps, z, cap, float(np.abs(rows).max(initial=0)))
    for got, want, b in ((dh, want_h, bh), (dw, want_w, bw)):
        if got is not None:
            err = np.abs(host(got) - want)
            assert (err <= b).all(), f"worst {np.nanmax(err / b):.3g} of the bound"
    if dh is not None:
        assert (host(dh)[~on] == 0).all()


def run(T, V, H, reduction="mean", eps=0.0, z=0.0, cap=0.0, piece=0, pad=0, inactive=0.25, ignore=False, seed=0):
    h, w, t, on = case(T, V, H, seed, pad, inactive)
    if ignore:
        t = np.where(on, t, -100)
    mask = None if ignore else torch.from_numpy(on.astype(np.uint8)).cuda()
    targets = torch.from_numpy(t).cuda()
    c = rlk.linear_ce_contract(h, w, mask, reduction=REDUCTIONS[reduction], label_smoothing=eps, z_loss=z,
                               softcap=cap, piece=piece, validate=1)
    loss, lse = rlk.linear_ce_fwd(c, h, w, targets, mask)
    want_lse, y = check_forward(h, w, t, on, loss, lse, reduction, eps, z, cap)
    g = np.linspace(-1.5, 1.0, T).astype(np.float32) if reduction == "none" else np.float32(0.75)
    grad = torch.tensor(g, device="cuda")
    dh, dw = rlk.linear_ce_bwd(c, h, w, targets, mask, lse, grad)
    check_backward(h, w, t, on, dh, dw, ref.row_gradients(g.astype(np.float64), on, reduction), want_lse, y, eps, z, cap)
    again = rlk.linear_ce_bwd(c, h, w, targets, mask, lse, grad)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)
    return c, h, w, targets, mask, loss, lse, grad, dh, dw


@pytest.mark.parametrize("T,V,H", [
    (1, 1, 1), (1, 2, 8), (1, 300, 64), (3, 255, 100), (17, 256, 63), (64, 257, 65), (127, 1000, 128), (128, 512, 256),
    (129, 1023, 200), (200, 2049, 320), (300, 5000, 130), (513, 700, 1000), (40, 33000, 72)])
@pytest.mark.parametrize("reduction", ["none", "mean"])
def test_matches_64_bits(built, T, V, H, reduction):
    run(T, V, H, reduction, seed=T + V + H)


@pytest.mark.parametrize("eps,z,cap", [(0.1, 0, 0), (1.0, 0, 0), (0, 1e-2, 0), (0, 0, 5.0), (0, 0, 0.5),
                                       (0.05, 1e-3, 30.0)])
@pytest.mark.parametrize("T,V,H", [(5, 130, 40), (150, 1100, 136)])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_options_match_64_bits(built, T, V, H, reduction, eps, z, cap):
    run(T, V, H, reduction, eps, z, cap)


@pytest.mark.parametrize("piece", [1, 256, 300, 1024, 100000])
@pytest.mark.parametrize("T", [9, 260])
def test_pieces_of_the_vocabulary(built, T, piece):
    # the last piece a few rows, K slices without a block in it among the others
    run(T, 2310, 192, "mean", piece=piece)
    run(T, 2049, 100, "none", 0.1, 1e-3, 10.0, piece=piece)


def test_strided_rows_and_ignore_index(built):
    run(70, 900, 96, "mean", pad=40)
    run(70, 900, 99, "none", pad=8, ignore=True)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_no_active_row(built, reduction):
    h, w, t, _ = case(40, 300, 64)
    mask = torch.zeros(40, dtype=torch.uint8, device="cuda")
    targets = torch.from_numpy(t).cuda()
    h, w = h.requires_grad_(), w.requires_grad_()
    loss = linear_cross_entropy(h, w, targets, mask, reduction=reduction, label_smoothing=0.1, z_loss=1e-3)
    assert (loss == 0).all()
    loss.sum().backward()
    assert (h.grad == 0).all() and (w.grad == 0).all()


def test_no_row(built):
    h, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), bf16_matrix(300, 64, 1, 1.0)
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    h, w = h.requires_grad_(), w.requires_grad_()
    loss = linear_cross_entropy(h, w, t, None)
    assert loss.item() == 0
    loss.backward()
    assert h.grad.shape == (0, 64) and (w.grad == 0).all()
    assert linear_cross_entropy(h, w, t, None, reduction="none").shape == (0,)


def test_inactive_rows_do_not_touch_the_others(built):
    c, h, w, targets, mask, loss, lse, grad, dh, dw = run(100, 500, 64, "none")
    keep = mask.bool()
    sub = rlk.linear_ce_contract(h[keep].contiguous(), w, mask[keep], validate=1)
    part, part_lse = rlk.linear_ce_fwd(sub, h[keep].contiguous(), w, targets[keep], mask[keep])
    assert torch.equal(part, loss[keep]) and torch.equal(part_lse, lse[keep])


@pytest.mark.parametrize("T", [30, 300, 900])
def test_masked_rows_may_hold_anything(built, T):
    # NaN and infinities in an inactive row's hidden reach nothing but that row's lse
    h, w, t, on = case(T, 700, 100, seed=T, inactive=0.6)
    targets, mask = torch.from_numpy(t).cuda(), torch.from_numpy(on.astype(np.uint8)).cuda()
    c = rlk.linear_ce_contract(h, w, mask, reduction=rlk.REDUCE_MEAN, validate=1)
    loss, lse = rlk.linear_ce_fwd(c, h, w, targets, mask)
    one = torch.ones((), device="cuda")
    want = rlk.linear_ce_bwd(c, h, w, targets, mask, lse, one)
    dirty = torch.empty_strided(h.shape, h.stride(), dtype=h.dtype, device=h.device).copy_(h)
    off = torch.from_numpy(np.flatnonzero(~on)).cuda()
    dirty[off[::2]] = float("nan")
    dirty[off[1::2]] = float("inf")
    c = rlk.linear_ce_contract(dirty, w, mask, reduction=rlk.REDUCE_MEAN, validate=1)
    loss2, lse2 = rlk.linear_ce_fwd(c, dirty, w, targets, mask)
    got = rlk.linear_ce_bwd(c, dirty, w, targets, mask, lse2, one)
    assert torch.equal(loss2, loss) and torch.equal(lse2[mask.bool()], lse[mask.bool()])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.isfinite(got[1]).all()


def test_rows_between_lines_give_the_same(built):
    # large enough for the forward to copy hidden onto 128-byte lines: the bits of rows that lie there already
    T, V, H = 701, 40003, 1000
    gen = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn((T, 1024), generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn((V, H), generator=gen, device="cuda") * 0.03).to(torch.bfloat16)
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda")
    targets[::9] = -100
    out = []
    for h in (wide[:, :H], wide[:, :H].contiguous()):
        c = rlk.linear_ce_contract(h, w, reduction=rlk.REDUCE_NONE, label_smoothing=0.1, softcap=20.0, validate=1)
        out.append(rlk.linear_ce_fwd(c, h, w, targets))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    # FP32 sums of H exact products: H 2^-24 of their magnitudes' sum at the worst, the cap's slope is at most 1
    a = wide[:, :H].double()
    x = a @ w.double().t()
    lse = torch.logsumexp(20.0 * torch.tanh(x / 20.0), dim=1)
    lim = H * 2.0 ** -24 * (a.abs() @ w.double().abs().t()).amax(dim=1) + 2.0 ** -18 * (lse.abs() + 20.0)
    assert ((out[1][1].double() - lse).abs() <= lim).all()


def test_weight_past_2_to_31_elements(built):
    T, V, H = 40, 560000, 4000  # 2.24e9 elements
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    gen = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.empty((V, H), dtype=torch.bfloat16, device="cuda").normal_(0.0, 0.02, generator=gen)
    rows = torch.tensor([0, 3, 280000, 536871, V - 1], device="cuda")
    some = torch.arange(T, device="cuda") % len(rows)
    c = rlk.linear_ce_contract(h, w, reduction=rlk.REDUCE_SUM, validate=1)
    loss, lse = rlk.linear_ce_fwd(c, h, w, rows[some])
    parts = [torch.logsumexp(h.double() @ w[v:v + 40000].double().t(), dim=1) for v in range(0, V, 40000)]
    want = torch.logsumexp(torch.stack(parts), dim=0)
    # FP32 sums of H products: H 2^-24 of their magnitudes' sum at the worst, and that is under 5 H 0.02
    lim = H * 2.0 ** -24 * 5 * H * 0.02 + 2.0 ** -18 * (want.abs() + 20.0)
    assert ((lse.double() - want).abs() <= lim).all()
    one = torch.ones((), device="cuda")
    dh, dw = rlk.linear_ce_bwd(c, h, w, rows[some], None, lse, one)
    # a row of dweight depends on its own row of weight and on lse: the same bits from those rows alone
    few = w[rows].contiguous()
    c2 = rlk.linear_ce_contract(h, few, reduction=rlk.REDUCE_SUM, validate=1)
    _, dw2 = rlk.linear_ce_bwd(c2, h, few, some, None, lse, one)
    assert torch.equal(dw[rows], dw2)
    assert torch.isfinite(dh).all()


def test_only_the_gradient_that_is_asked_for(built):
    c, h, w, targets, mask, loss, lse, grad, dh, dw = run(100, 700, 128, "mean")
    a, b = rlk.linear_ce_bwd(c, h, w, targets, mask, lse, grad, need_dweight=False)
    assert b is None and torch.equal(a, dh)
    a, b = rlk.linear_ce_bwd(c, h, w, targets, mask, lse, grad, need_dhidden=False)
    assert a is None and torch.equal(b, dw)


def test_gradients_match_differences(built):
    # hidden and weight on a grid of 1/16, a step of 1/64: all exact in BF16
    rng = np.random.default_rng(3)
    T, V, H = 40, 300, 48
    grid = lambda r, c, top: torch.from_numpy(rng.integers(-top, top, (r, c)) / 16.0).to(torch.bfloat16).cuda()  # noqa: E731
    h, w = grid(T, H, 28), grid(V, H, 5)
    t = torch.from_numpy(rng.integers(0, V, T)).cuda()
    kw = dict(reduction="none", label_smoothing=0.1, z_loss=1e-2, softcap=20.0)
    hr, wr = h.clone().requires_grad_(), w.clone().requires_grad_()
    linear_cross_entropy(hr, wr, t, None, **kw).sum().backward()
    for which, grad in ((h, hr.grad), (w, wr.grad)):
        for k in range(4):
            # one element of each row (a direction across rows of hidden; of weight, rows far apart)
            d = torch.zeros_like(which)
            rows = torch.arange(0, which.shape[0], 1 if which is h else 97, device="cuda")
            d[rows, (rows * 7 + k * 5) % H] = 1 / 64
            plus = (h + d, w) if which is h else (h, w + d)
            minus = (h - d, w) if which is h else (h, w - d)
            up = linear_cross_entropy(*plus, t, None, **kw).double().sum()
            down = linear_cross_entropy(*minus, t, None, **kw).double().sum()
            got = float((grad.double() * d.double()).sum())
            # BF16 gradients: 2^-8 of each term twice over; FP32 losses: 1e-6 of about 10 a row; the third
            # derivative's share of a step this small is below 1e-4 of the terms
            terms = float((grad.double() * d.double()).abs().sum())
            assert abs(float(up - down) / 2 - got) <= 2.0 ** -7 * terms + T * 1e-5


def test_errors_are_reported(built):
    h, w, t, on = case(20, 300, 64, inactive=0.0)
    t[3] = 300
    targets, mask = torch.from_numpy(t).cuda(), torch.ones(20, dtype=torch.uint8, device="cuda")
    c = rlk.linear_ce_contract(h, w, mask, validate=1)
    with pytest.raises(rlk.RlkError) as e:
        rlk.linear_ce_fwd(c, h, w, targets, mask)
    assert e.value.status == rlk.RLK_ERR_TARGET_RANGE
    loss, lse = rlk.linear_ce_fwd(c.replace(validate=0), h, w, targets, mask)
    assert torch.isnan(loss[3]) and torch.isfinite(loss[[0, 1, 2, 4, 19]]).all()
    with pytest.raises(rlk.RlkError) as e:
        rlk.linear_ce_bwd(c, h, w, targets, mask, lse, loss)
    assert e.value.status == rlk.RLK_ERR_TARGET_RANGE
    h2 = h.clone()
    h2[5, 3] = float("nan")
    targets[3] = 0
    with pytest.raises(rlk.RlkError) as e:
        rlk.linear_ce_fwd(c, h2, w, targets, mask)
    assert e.value.status == rlk.RLK_ERR_NONFINITE_LSE
    loss, lse = rlk.linear_ce_fwd(c.replace(validate=0), h2, w, targets, mask)
    assert torch.isnan(lse[5]) and int(torch.isnan(loss).sum()) == 1


def test_non_finite_upstream_gradients_stay_in_their_rows(built):
    h, w, t, on = case(30, 400, 64, inactive=0.0)
    targets, mask = torch.from_numpy(t).cuda(), torch.ones(30, dtype=torch.uint8, device="cuda")
    c = rlk.linear_ce_contract(h, w, mask)
    loss, lse = rlk.linear_ce_fwd(c, h, w, targets, mask)
    g = torch.linspace(-2, 2, 30, device="cuda")
    want, _ = rlk.linear_ce_bwd(c, h, w, targets, mask, lse, g)
    bad = g.clone()
    bad[4] = float("nan")
    got, _ = rlk.linear_ce_bwd(c, h, w, targets, mask, lse, bad)
    rows = [r for r in range(30) if r != 4]
    assert torch.isnan(got[4]).all() and torch.equal(got[rows], want[rows])


def test_binding_refuses_what_the_call_cannot_read(built):
    h, w, t, on = case(10, 100, 64)
    targets, mask = torch.from_numpy(t).cuda(), torch.from_numpy(on.astype(np.uint8)).cuda()
    c = rlk.linear_ce_contract(h, w, mask)
    with pytest.raises(ValueError):
        rlk.linear_ce_contract(h, w[:, :32], mask)
    with pytest.raises(TypeError):
        rlk.linear_ce_contract(h.float(), w, mask)
    with pytest.raises(rlk.RlkError):
        rlk.linear_ce_contract(torch.zeros((10, 63), dtype=torch.bfloat16, device="cuda"), w[:, :63], mask)
    with pytest.raises(ValueError):
        rlk.linear_ce_fwd(c, h[:5], w, targets, mask)
    with pytest.raises(ValueError):
        rlk.linear_ce_fwd(c, h, w, targets[:5], mask)
    with pytest.raises(TypeError):
        rlk.linear_ce_fwd(c, h, w, targets.int(), mask)
    with pytest.raises(ValueError):
        rlk.linear_ce_fwd(c, h, w, targets, mask, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        linear_cross_entropy(h, w, targets, mask, reduction="batchmean")


def test_on_another_stream_and_in_a_graph(built):
    c, h, w, targets, mask, loss, lse, grad, dh, dw = run(50, 600, 64, "mean")
    c = c.replace(validate=0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss2, lse2 = rlk.linear_ce_fwd(c, h, w, targets, mask)
        dh2, dw2 = rlk.linear_ce_bwd(c, h, w, targets, mask, lse2, grad)
    side.synchronize()
    assert torch.equal(loss2, loss) and torch.equal(dh2, dh) and torch.equal(dw2, dw)
    ws = torch.empty(rlk.rlk_linear_ce_workspace_size(c, 1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss3, lse3 = rlk.linear_ce_fwd(c, h, w, targets, mask, workspace=ws)
        dh3, dw3 = rlk.linear_ce_bwd(c, h, w, targets, mask, lse3, grad, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss3, loss) and torch.equal(dh3, dh) and torch.equal(dw3, dw)


def test_large_vocabulary_against_a_blocked_64_bit_form(built):
    # a vocabulary of the size the framework scores, two pieces, sampled rows and columns
    T, V, H = 256, 151936, 128
    h, w, t, on = case(T, V, H, seed=8)
    targets, mask = torch.from_numpy(t).cuda(), torch.from_numpy(on.astype(np.uint8)).cuda()
    c = rlk.linear_ce_contract(h, w, mask, reduction=rlk.REDUCE_SUM, piece=76032, validate=1)
    loss, lse = rlk.linear_ce_fwd(c, h, w, targets, mask)
    one = torch.ones((), device="cuda")
    dh, dw = rlk.linear_ce_bwd(c, h, w, targets, mask, lse, one)
    h64, w64 = h.double(), w.double()
    y = h64 @ w64.t()
    want_lse = torch.logsumexp(y, dim=1)
    assert (lse.double() - want_lse).abs().max() <= float(ref.lse_bound(host(h), host(w), np.array([[20.0] * 8] * T)).max()) + 1200 * 2.0 ** -23
    d = torch.exp(y - want_lse[:, None])
    m = torch.from_numpy(on).cuda()
    d[torch.arange(T, device="cuda")[m], targets[m]] -= 1
    d[~m] = 0
    for got, want, terms in ((dh, d @ w64, d.abs() @ w64.abs()), (dw, d.t() @ h64, d.abs().t() @ h64.abs())):
        assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2e-4) * terms + 1e-30).all()
        assert float((got.double() - want).norm() / want.norm()) < 4e-3


@pytest.mark.parametrize("T,V,H,piece", [
    (300, 700, 2500, 0),      # bands of H blocks, the last one narrow
    (7100, 600, 2500, 0),     # two bands of token blocks
    (520, 3000, 136, 512),    # more tiles of dweight than of dhidden, then the reverse
    (5000, 300, 72, 256)])
def test_tile_orders_against_64_bits_on_the_gpu(built, T, V, H, piece):
    h, w, t, on = case(T, V, H, seed=T + V)
    targets, mask = torch.from_numpy(t).cuda(), torch.from_numpy(on.astype(np.uint8)).cuda()
    c = rlk.linear_ce_contract(h, w, mask, reduction=rlk.REDUCE_SUM, piece=piece, validate=1)
    loss, lse = rlk.linear_ce_fwd(c, h, w, targets, mask)
    dh, dw = rlk.linear_ce_bwd(c, h, w, targets, mask, lse, torch.ones((), device="cuda"))
    h64, w64, m = h.double(), w.double(), torch.from_numpy(on).cuda()
    y = h64 @ w64.t()
    want = torch.logsumexp(y, dim=1)
    b = torch.from_numpy(ref.lse_bound(host(h), host(w), y.cpu().numpy())).cuda()
    assert ((lse.double() - want).abs() <= b).all()
    d = torch.exp(y - want[:, None])
    d[torch.arange(T, device="cuda")[m], targets[m]] -= 1
    d[~m] = 0
    p = torch.exp(y - want[:, None]) * m[:, None]
    # dx: rounded to BF16, the probabilities off by the logits' and lse's errors; sums of V or T terms in FP32
    err = 2.0 ** -8 * d.abs() + p * (2 * b[:, None] + 2.0 ** -19 * (1 + want.abs()[:, None])) + 2.0 ** -21 * d.abs()
    for got, exact, e, terms, n in ((dh, d @ w64, err @ w64.abs(), d.abs() @ w64.abs(), V + 600),
                                    (dw, d.t() @ h64, err.t() @ h64.abs(), d.abs().t() @ h64.abs(), T + 16)):
        assert ((got.double() - exact).abs() <= e + n * 2.0 ** -23 * terms + 2.0 ** -8 * exact.abs() + 1e-30).all()


def test_fp8_linear_gradients(built):
    # the product's own error is tested elsewhere: here the formulas, through exactly quantised operands
    rng = np.random.default_rng(1)
    T, K, N = 70, 200, 130
    ints = lambda r, c: torch.from_numpy(rng.integers(-8, 9, (r, c)).astype(np.float32))  # noqa: E731
    x, w, dy = ints(T, K), ints(N, K), ints(T, N)
    for a in (x, w, dy):
        # every group's largest magnitude 448 / 32 = 14 (by rows, columns and blocks): the scales are powers of two
        a[:, ::64] = 14.0
        a[::64, :] = 14.0
    xg, wg = x.to(torch.bfloat16).cuda().requires_grad_(), w.cuda().requires_grad_()
    y = fp8_linear(xg.view(7, 10, K), wg)
    assert y.shape == (7, 10, N) and y.dtype == torch.bfloat16
    y.backward(dy.to(torch.bfloat16).cuda().view(7, 10, N))
    want = x.double() @ w.double().t()
    assert torch.equal(y.view(T, N).cpu(), want.to(torch.bfloat16))
    assert xg.grad.dtype == torch.bfloat16 and torch.equal(xg.grad.cpu(), (dy.double() @ w.double()).to(torch.bfloat16))
    assert wg.grad.dtype == torch.float32 and torch.equal(wg.grad.cpu().double(), dy.double().t() @ x.double())
    xo = x.to(torch.bfloat16).cuda().requires_grad_()
    fp8_linear(xo, w.cuda()).backward(dy.to(torch.bfloat16).cuda())
    assert torch.equal(xo.grad, xg.grad)
    wo = w.cuda().requires_grad_()
    fp8_linear(x.to(torch.bfloat16).cuda(), wo).backward(dy.to(torch.bfloat16).cuda())
    assert torch.equal(wo.grad, wg.grad)
