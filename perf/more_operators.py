"""The operators of feed-forward blocks in 8 bits, dense and by experts, as cases to measure.

``run`` makes one pass: with ``own`` the calls that a user makes of this package, without it the same
mathematics in elementary torch operations in 32 bits.

linear        y = act(A B^T + bias) + residual of E4M3 operands (A with a scale for each 1 x 128 group of a row,
              B for each 128 x 128 block), all sums in FP32, y rounded once.  gated: B holds the gate's n rows, then
              n more, and y = act(gate) * up + residual.
linear step   that layer on BF16 inputs and weights, and its gradients: x and w are quantised, z = A B^T + bias is
              kept in BF16, dz = dy act'(z) in FP32; dx is the product of dz's rows with w, dw that of the columns of
              dz and x in groups of 128 tokens, dbias the sum of dz over the tokens.
experts       the rows of A belong to experts, group e ending at row ends[e], each with a B and a bias of its own;
              rows behind the last group are zero.
experts step  that layer with its gradients; the groups of 128 tokens start anew with each expert.
"""
import math

import numpy as np
import torch

own = False

_GROUP = 128
_E4M3_MAX = 448.0
_FLOOR = 2.0 ** -100  # an all-zero group's amax counts as this: its scale stays normal and its values are 0
_GELU = math.sqrt(2.0 / math.pi)


def _linear(name, m, n, k, act, gated, bias, residual, out):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "act": act, "gated": gated, "bias": bias,
            "residual": residual, "out": out}


def _experts(name, op, tokens, top, experts, pad, n, k, act, gated, bias, out):
    return {"name": name, "op": op, "tokens": tokens, "top": top, "experts": experts, "pad": pad, "n": n, "k": k,
            "act": act, "gated": gated, "bias": bias, "out": out}


def listed():
    return [
        # one decoded token through a block's last projection, added to the residual stream: the weight's bytes
        _linear("linear 1 token", 1, 4096, 4096, "none", False, "bf16", "bf16", "bf16"),
        # a ragged decode batch through a gated block's first projection: the bytes of two weights
        _linear("linear 37 tokens gated", 37, 12288, 4096, "silu", True, "none", "none", "bf16"),
        # a prompt of odd sizes into an FP32 residual stream
        _linear("linear prompt odd", 1000, 5003, 2000, "relu", False, "f32", "f32", "f32"),
        # a training batch through a wide projection
        _linear("linear batch gelu", 8192, 12288, 4096, "gelu", False, "bf16", "none", "bf16"),
        # a small model's training step: odd sizes, every part of the epilogue
        {"name": "linear step small odd", "op": "linear step", "m": 600, "n": 2000, "k": 1000, "act": "gelu_tanh", "gated": False,
         "bias": True, "residual": True},
        # a gated block's first projection in a training step
        {"name": "linear step gated", "op": "linear step", "m": 4096, "n": 6144, "k": 4096, "act": "silu", "gated": True,
         "bias": False, "residual": False},
        # one decoded token's experts
        _experts("experts 1 token", "experts", 1, 8, 128, 0, 768, 2048, "silu", True, "none", "bf16"),
        # a decode batch: few rows for each of many experts, and the rows of absent sequences behind them
        _experts("experts 64 tokens", "experts", 64, 8, 128, 24, 2048, 4096, "none", False, "bf16", "bf16"),
        # a prompt
        _experts("experts prompt", "experts", 2048, 8, 64, 0, 4096, 2048, "none", False, "none", "f32"),
        # a small model's training step: odd sizes, padded rows
        _experts("experts step small odd", "experts step", 499, 2, 5, 30, 641, 520, "relu", False, "bf16", "bf16"),
        # a training step
        _experts("experts step", "experts step", 4096, 4, 32, 256, 1408, 2048, "silu", True, "none", "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear step", "experts", "experts step"))
    act = rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh"))
    gated = act != "none" and rng.random() < 0.4
    two = 2 if gated else 1

    def columns(lo, hi):
        n = _log(rng, lo, hi)
        return -(-n // 64) * 64 if gated else n

    if op == "linear":
        k = _log(rng, 256, 8192)
        n = columns(256, 12288 // two)
        m = _log(rng, 1, max(1, min(8192, 4 * 10 ** 11 // (two * n * k))))
        return {"op": op, "m": m, "n": n, "k": k, "act": act, "gated": gated, "bias": rng.choice(("none", "bf16", "f32")),
                "residual": rng.choice(("none", "bf16", "f32")), "out": rng.choice(("bf16", "bf16", "f32"))}
    if op == "linear step":
        k = _log(rng, 256, 4096)
        n = columns(256, 8192 // two)
        m = _log(rng, 1, max(1, min(4096, 10 ** 11 // (two * n * k))))
        return {"op": op, "m": m, "n": n, "k": k, "act": act, "gated": gated, "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.5}
    step = op == "experts step"
    experts = _log(rng, 2, 128)
    top = rng.randint(1, min(8, experts))
    k = _log(rng, 256, 4096)
    n = columns(256, max(256, min(4096, 5 * 10 ** 8 // (experts * k)) // two))
    tokens = _log(rng, 1, max(1, min(16384, 5 * 10 ** 10 // (two * n * k)) // top))
    return {"op": op, "tokens": tokens, "top": top, "experts": experts, "pad": rng.choice((0, 0, rng.randint(1, 300))), "n": n, "k": k,
            "act": act, "gated": gated, "bias": rng.choice(("none", "bf16") if step else ("none", "bf16", "f32")),
            "out": "bf16" if step else rng.choice(("bf16", "bf16", "f32"))}


# ------------------------------------------------------------------ the plain forms

def _quantized(x, r, c):
    """(values, scales) of x [..., R, C] in 32 bits, a scale for each r x c group: values as x, scales [..., R / r, C / c]."""
    R, C = x.shape[-2:]
    g = torch.nn.functional.pad(x.float(), (0, -C % c, 0, -R % r))
    g = g.view(*x.shape[:-2], -(-R // r), r, -(-C // c), c)
    top = torch.clamp_min(g.abs().amax(dim=(-3, -1), keepdim=True), _FLOOR)
    s = top / torch.full_like(top, _E4M3_MAX)  # by a number it would be a product: many BF16 values lie on a tie of the codes
    q = (g * (1.0 / s)).to(torch.float8_e4m3fn).view(*x.shape[:-2], g.shape[-4] * r, -1)[..., :R, :C]
    return q, s[..., :, 0, :, 0]


def _values(q, s, r, c):
    """What codes [..., R, C] with scales [..., R / r, C / c] stand for, in 32 bits."""
    s = s.repeat_interleave(r, dim=-2) if r > 1 else s
    return q.float() * s.repeat_interleave(c, dim=-1)[..., :q.shape[-2], :q.shape[-1]]


def _rounded(x, r, c):
    return _values(*_quantized(x, r, c), r, c)


def _act(z, kind):
    if kind == "relu":
        return z.clamp_min(0)
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_GELU * (z + 0.044715 * z * z * z)))
    return z


def _slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        t = torch.tanh(_GELU * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _GELU * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _forward(z, c):
    n = c["n"]
    return _act(z[..., :n], c["act"]) * z[..., n:] if c["gated"] else _act(z, c["act"])


def _backward(z, dy, c):
    """dz from dy and the pre-activation, both of one width of type."""
    n = c["n"]
    if c["gated"]:
        return torch.cat((dy * z[..., n:] * _slope(z[..., :n], c["act"]), dy * _act(z[..., :n], c["act"])), dim=-1)
    return dy * _slope(z, c["act"]) if c["act"] != "none" else dy


def _plain_linear(s, c):
    z = _values(s["a"], s["a_scale"].t(), 1, _GROUP) @ _values(s["b"], s["b_scale"].t(), _GROUP, _GROUP).t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _forward(z, c)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(_TYPES[c["out"]])


def _plain_linear_step(s, c):
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
    wq = _rounded(w, _GROUP, _GROUP)
    z = _rounded(x, 1, _GROUP) @ wq.t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _forward(z, c)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    dz = _backward(z.to(torch.bfloat16).float(), dy, c)
    bf16 = torch.bfloat16
    out = {"y": y.to(bf16), "dx": (_rounded(dz, 1, _GROUP) @ wq).to(bf16),
           "dw": (_rounded(dz, _GROUP, 1).t() @ _rounded(x, _GROUP, 1)).to(bf16)}
    if s["bias"] is not None:
        out["dbias"] = dz.sum(dim=0).to(bf16)
    return out


def _places(s, c):
    """Each row's expert and place among its rows (the last place of the last expert for rows behind the groups), whether it
    has an expert, and the number of places: the largest group's in whole groups of 128, and one more."""
    ends = s["ends"].long()
    rows = torch.arange(s["rows"], device=ends.device)
    e = torch.searchsorted(ends, rows, right=True)
    used = e < c["experts"]
    e = e.clamp_max(c["experts"] - 1)
    places = -(-s["largest"] // _GROUP) * _GROUP
    begin = torch.cat((torch.zeros_like(ends[:1]), ends[:-1]))
    return e, torch.where(used, rows - begin[e], places), used[:, None], places


def _spread(x, experts, e, i, places):
    """Rows [R, C] in 32 bits as [experts, places, C], zero where an expert has no row."""
    out = torch.zeros((experts, places + 1, x.shape[1]), device=x.device)
    out[e, i] = x.float()
    return out[:, :places]


def _plain_experts(s, c):
    e, i, used, places = _places(s, c)
    a = _spread(_values(s["a"], s["a_scale"].t(), 1, _GROUP), c["experts"], e, i, places)
    z = torch.bmm(a, _values(s["b"], s["b_scale"].transpose(1, 2), _GROUP, _GROUP).transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"].float()[:, None]
    y = _forward(z, c)[e, i.clamp_max(places - 1)]
    return torch.where(used, y, 0.0).to(_TYPES[c["out"]])


def _plain_experts_step(s, c):
    e, i, used, places = _places(s, c)
    at = i.clamp_max(places - 1)
    x = s["x"].float()
    wq = _rounded(s["w"].float(), _GROUP, _GROUP)
    z = torch.bmm(_spread(_rounded(x, 1, _GROUP), c["experts"], e, i, places), wq.transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"].float()[:, None]
    y = torch.where(used, _forward(z, c)[e, at], 0.0)
    dy = _spread(s["dy"], c["experts"], e, i, places)
    dz = _backward(z.to(torch.bfloat16).float(), dy, c)
    dx = torch.where(used, torch.bmm(_rounded(dz, 1, _GROUP), wq)[e, at], 0.0)
    xs = _spread(x, c["experts"], e, i, places)
    dw = torch.bmm(_rounded(dz, _GROUP, 1).transpose(1, 2), _rounded(xs, _GROUP, 1))
    bf16 = torch.bfloat16
    out = {"y": y.to(bf16), "dx": dx.to(bf16), "dw": dw.to(bf16)}
    if s["bias"] is not None:
        out["dbias"] = dz.sum(dim=1).to(bf16)
    return out


# ------------------------------------------------------------------ the interface

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _counts(case, seed):
    """The rows of each expert: every token picks `top` of them, from a router that favours some a little."""
    rng = np.random.default_rng(seed)
    lean = rng.normal(0.0, 0.4, case["experts"])
    picked = np.argsort(-(lean + rng.gumbel(size=(case["tokens"], case["experts"]))), axis=1)[:, :case["top"]]
    return np.bincount(picked.ravel(), minlength=case["experts"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(sigma)

    def activations(r, k):
        # a few channels of a transformer's activations are much larger than the rest
        x = normal(r, k)
        big = torch.rand((k,), generator=gen, device="cuda") < 0.01
        return x.mul_(torch.where(big, 20.0, 1.0))

    def codes(x, r):
        """(E4M3 with rows on 16-byte boundaries, scales laid out [..., group along the row, row or block of rows])."""
        q, s = _quantized(x, r, _GROUP)
        pad = -q.shape[-1] % 16
        if pad:
            q = torch.nn.functional.pad(q.contiguous().view(torch.uint8), (0, pad)).view(torch.float8_e4m3fn)[..., :x.shape[-1]]
        else:
            q = q.contiguous()
        return q, s.transpose(-1, -2).contiguous()

    c = dict(case)
    state = {"case": c, "bias": None, "residual": None}
    n, k, wide = c["n"], c["k"], c["n"] * (2 if c["gated"] else 1)
    by_expert = c["op"].startswith("experts")
    lead = (c["experts"],) if by_expert else ()
    if by_expert:
        counts = _counts(c, seed)
        rows = int(counts.sum()) + c["pad"]
        state["ends"] = torch.from_numpy(np.cumsum(counts)).to(device="cuda", dtype=torch.int32)
        state["rows"], state["largest"] = rows, int(counts.max())
    else:
        rows = c["m"]
    x, w = activations(rows, k), normal(*lead, wide, k, sigma=0.02)
    if c["op"].endswith("step"):
        state["x"], state["w"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
        state["dy"] = normal(rows, n, sigma=1e-3).to(torch.bfloat16)
        bias = "bf16" if c["bias"] in (True, "bf16") else "none"
        residual = "bf16" if c.get("residual") else "none"
    else:
        state["a"], state["a_scale"] = codes(x, 1)
        state["b"], state["b_scale"] = codes(w, _GROUP)
        bias, residual = c["bias"], c.get("residual", "none")
    if bias != "none":
        state["bias"] = normal(*lead, wide, sigma=0.5).to(_TYPES[bias])
    if residual != "none":
        state["residual"] = normal(rows, n).to(_TYPES[residual])
    return state


def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    if c["op"] == "linear":
        return _plain_linear(state, c)
    if c["op"] == "linear step":
        return _plain_linear_step(state, c)
    if c["op"] == "experts":
        return _plain_experts(state, c)
    return _plain_experts_step(state, c)


def _run_own(c, s):
    import vocab_selected_token_tile_gb300 as rlk
    from vocab_selected_token_tile_gb300 import autograd
    if c["op"] == "linear":
        return rlk.fp8_matmul_act(s["a"], s["a_scale"], s["b"], s["b_scale"], bias=s["bias"], activation=c["act"],
                                  gated=c["gated"], residual=s["residual"], out_dtype=_TYPES[c["out"]])
    if c["op"] == "experts":
        return rlk.fp8_grouped_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], s["ends"], bias=s["bias"],
                                      activation=c["act"], gated=c["gated"], out_dtype=_TYPES[c["out"]])
    leaves = [s["x"].requires_grad_(), s["w"].requires_grad_()]
    if s["bias"] is not None:
        leaves.append(s["bias"].requires_grad_())
    if c["op"] == "linear step":
        y = autograd.fp8_linear(s["x"], s["w"], bias=s["bias"], activation=c["act"], gated=c["gated"], residual=s["residual"])
    else:
        y = autograd.fp8_grouped_linear(s["x"], s["w"], s["ends"], bias=s["bias"], activation=c["act"], gated=c["gated"])
    grads = torch.autograd.grad(y, leaves, s["dy"])
    return {"y": y.detach(), **dict(zip(("dx", "dw", "dbias"), grads))}


def work(case):
    n, k, wide, step = case["n"], case["k"], case["n"] * (2 if case["gated"] else 1), case["op"].endswith("step")
    size = {"none": 0, "bf16": 2, "f32": 4, True: 2, False: 0}
    bias, res = size[case["bias"]], size[case.get("residual", "none")]
    if case["op"].startswith("experts"):
        rows, experts = case["tokens"] * case["top"], case["experts"]
        # the experts that a step of evenly spread tokens reaches: only their weights are read
        live = experts * (1 - (1 - case["top"] / experts) ** case["tokens"])
        out_rows, weights = rows + case["pad"], live
    else:
        rows = out_rows = case["m"]
        experts = weights = 1
    flops = 2 * rows * wide * k
    if not step:
        kb = -(-k // _GROUP)
        scales = 4 * kb * (rows + weights * -(-wide // _GROUP))
        return {"bytes": rows * k + weights * wide * k + scales + out_rows * n * size[case["out"]] + weights * wide * bias
                + rows * n * res, "flops": flops}
    # x, w, dy and what is added once; y and the gradients once
    once = 2 * (rows * k + weights * wide * k + rows * n) + weights * wide * bias + rows * n * res
    return {"bytes": once + 2 * (out_rows * (n + k) + experts * wide * k) + experts * wide * bias, "flops": 3 * flops}


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3(v):
    """The nearest of 8 steps a binade, subnormals below 2^-6, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-_E4M3_MAX, _E4M3_MAX)


def _exact_rows(x, block):
    """x [R, C] in 64 bits after quantisation in groups of 128 columns of `block` rows; the definition rounds the scale, its
    reciprocal and the product to 32 bits."""
    out = torch.empty_like(x)
    R = x.shape[0]
    for c0 in range(0, x.shape[1], _GROUP):
        g = x[:, c0:c0 + _GROUP]
        top = torch.nn.functional.pad(g.abs().amax(dim=1), (0, -R % block)).view(-1, block).amax(dim=1)
        sc = (top.clamp_min(_FLOOR) / _E4M3_MAX).float().double()
        rec = (1.0 / sc).float().double().repeat_interleave(block)[:R, None]
        out[:, c0:c0 + _GROUP] = _e4m3((g * rec).float().double()) * sc.repeat_interleave(block)[:R, None]
    return out


def _exact_step(x, w, bias, dy, c):
    """(z, dx, dw, dbias) of one weight's rows in 64 bits; dz is rounded to 32 before its quantisation."""
    wq = _exact_rows(w.double(), _GROUP)
    z = _exact_rows(x.double(), 1) @ wq.t()
    if bias is not None:
        z = z + bias.double()
    dz = _backward(z.float().to(torch.bfloat16).double(), dy.double(), c)
    d32 = dz.float().double()
    dx = _exact_rows(d32, 1) @ wq
    dw = _exact_rows(d32.t().contiguous(), 1) @ _exact_rows(x.double().t().contiguous(), 1).t()
    return z, dx, dw, dz.sum(dim=0)


def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    if work(case)["flops"] > 1.6e13:
        return None  # over about 20 seconds at the rate of 64-bit products
    s, c = prepare(case, seed), case

    def stands_for(q, scale, block):
        t = scale.double().t().repeat_interleave(block, dim=0)[:q.shape[0]]
        return q.double() * t.repeat_interleave(_GROUP, dim=1)[:, :q.shape[1]]

    if case["op"] == "linear":
        z = stands_for(s["a"], s["a_scale"], 1) @ stands_for(s["b"], s["b_scale"], _GROUP).t()
        y = _forward(z + (0 if s["bias"] is None else s["bias"].double()), c)
        return y if s["residual"] is None else y + s["residual"].double()
    if case["op"] == "linear step":
        z, dx, dw, db = _exact_step(s["x"], s["w"], s["bias"], s["dy"], c)
        y = _forward(z, c)
        out = {"y": y if s["residual"] is None else y + s["residual"].double(), "dx": dx, "dw": dw}
        return out if s["bias"] is None else {**out, "dbias": db}
    ends = [0] + s["ends"].tolist()
    rows, n, k, wide = s["rows"], c["n"], c["k"], c["n"] * (2 if c["gated"] else 1)
    new = dict(dtype=torch.float64, device="cuda")
    y = torch.zeros((rows, n), **new)
    if case["op"] == "experts":
        a = stands_for(s["a"], s["a_scale"], 1)
        for e in range(c["experts"]):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                z = a[lo:hi] @ stands_for(s["b"][e], s["b_scale"][e], _GROUP).t()
                y[lo:hi] = _forward(z + (0 if s["bias"] is None else s["bias"][e].double()), c)
        return y
    dx, dw = torch.zeros((rows, k), **new), torch.zeros((c["experts"], wide, k), **new)
    db = torch.zeros((c["experts"], wide), **new)
    for e in range(c["experts"]):
        lo, hi = ends[e], ends[e + 1]
        if hi > lo:
            z, dx[lo:hi], dw[e], db[e] = _exact_step(s["x"][lo:hi], s["w"][e], None if s["bias"] is None else s["bias"][e],
                                                     s["dy"][lo:hi], c)
            y[lo:hi] = _forward(z, c)
    out = {"y": y, "dx": dx, "dw": dw}
    return out if s["bias"] is None else {**out, "dbias": db}
