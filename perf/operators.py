"""The operators of the 8-bit projections and of the cross entropy over a large vocabulary, as cases to measure.

``run`` makes one pass: with ``own`` the calls that a user makes of this package, without it the same
mathematics in elementary torch operations in 32 bits.

quantize   E4M3 values with one FP32 scale for each 1 x 128 group of a row (or each 128 x 128 block): for a
           group with largest magnitude amax, s = max(amax, 2^-100) / 448 and q = e4m3(x * (1 / s)), each step
           one FP32 rounding.  Scales are laid out [group along the row, row (or block of rows)].
matmul     C = A B^T of such operands, summed in FP32; A has 1 x 128 groups, B either kind.
ce         the cross entropy of logits = hidden weight^T with label smoothing, z-loss and a soft cap of the
           logits; per token, or its mean with the gradients of hidden and weight.
"""
import math

import torch

own = False

_GROUP = 128
_E4M3_MAX = 448.0
_FLOOR = 2.0 ** -100  # an all-zero group's amax counts as this: its scale stays normal and its values are 0


def listed():
    return [
        # one decoded token's activation before an FP8 projection: latency
        {"name": "quantize 1 token", "op": "quantize", "rows": 1, "cols": 4096, "block": 1, "both": False, "dtype": "bf16"},
        # a training batch's activation: rows for the forward, the transpose for the weight gradient
        {"name": "quantize batch both", "op": "quantize", "rows": 8192, "cols": 4096, "block": 1, "both": True, "dtype": "bf16"},
        # an FP32 master copy of a vocabulary's head, once per optimiser step, in 128 x 128 blocks
        {"name": "quantize head blocks", "op": "quantize", "rows": 151936, "cols": 4096, "block": 128, "both": False, "dtype": "f32"},
        # one token through a projection: the weight's bytes
        {"name": "matmul 1 token", "op": "matmul", "m": 1, "n": 4096, "k": 4096, "block": 128, "out": "bf16"},
        # a ragged decode batch through the head: the logits of 37 sequences
        {"name": "matmul 37 tokens head", "op": "matmul", "m": 37, "n": 151936, "k": 4096, "block": 128, "out": "bf16"},
        # a training batch through a wide projection, forward
        {"name": "matmul batch", "op": "matmul", "m": 8192, "n": 12288, "k": 4096, "block": 128, "out": "bf16"},
        # the weight gradient: both sides grouped along an odd number of tokens, FP32 out
        {"name": "matmul weight gradient", "op": "matmul", "m": 4096, "n": 4096, "k": 8191, "block": 1, "out": "f32"},
        # scoring one short continuation: the weight's bytes
        {"name": "ce 16 tokens", "op": "ce", "t": 16, "v": 151936, "h": 1024, "grad": False, "eps": 0.0, "z": 0.0, "cap": 0.0},
        # scoring a batch of sequences
        {"name": "ce score 2048", "op": "ce", "t": 2048, "v": 151936, "h": 4096, "grad": False, "eps": 0.0, "z": 0.0, "cap": 0.0},
        # a fine-tuning step of a small model: odd sizes, smoothing and a capped head
        {"name": "ce step small odd", "op": "ce", "t": 1000, "v": 50257, "h": 1000, "grad": True, "eps": 0.1, "z": 0.0, "cap": 30.0},
        # a fine-tuning step of a large vocabulary with z-loss
        {"name": "ce step large", "op": "ce", "t": 4096, "v": 151936, "h": 4096, "grad": True, "eps": 0.0, "z": 1e-4, "cap": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "matmul", "ce"))
    if op == "quantize":
        cols = _log(rng, 256, 16384)
        rows = _log(rng, 1, min(151936, 151936 * 4096 // cols))
        block = rng.choice((1, 1, 128))
        return {"op": op, "rows": rows, "cols": cols, "block": block, "both": rng.random() < 0.5, "dtype": rng.choice(("bf16", "f32"))}
    if op == "matmul":
        out = rng.choice(("bf16", "bf16", "f32"))
        k = _log(rng, 512, 16384)
        n = _log(rng, 512, 151936 if k <= 4096 else 16384)
        m = _log(rng, 1, max(1, min(8192, 5 * 10 ** 11 // (n * k))))
        return {"op": op, "m": m, "n": n, "k": k, "block": rng.choice((1, 128, 128)), "out": out}
    h = _log(rng, 256, 4096)
    v = _log(rng, 2000, 151936)
    grad = rng.random() < 0.6
    t = _log(rng, 1, 4096)
    return {"op": op, "t": t, "v": v, "h": h, "grad": grad, "eps": rng.choice((0.0, 0.05, 0.1)), "z": rng.choice((0.0, 1e-4)),
            "cap": rng.choice((0.0, 0.0, 30.0))}


# ------------------------------------------------------------------ the plain forms

def _grouped(x, block):
    """x [R, C] in 32 bits, padded with zeros to whole groups, as [R / block, block, C / 128, 128]."""
    R, C = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -C % _GROUP, 0, -R % block))
    return x.view(-1, block, x.shape[1] // _GROUP, _GROUP)


def _plain_quantize(x, block):
    R, C = x.shape
    g = _grouped(x, block)
    s = torch.clamp_min(g.abs().amax(dim=(1, 3), keepdim=True), _FLOOR) / _E4M3_MAX
    q = (g * (1.0 / s)).to(torch.float8_e4m3fn).view(g.shape[0] * block, -1)[:R, :C].contiguous()
    return q, s[:, 0, :, 0].t().contiguous()


def _dequantized(q, scale, block):
    R, C = q.shape
    s = scale.t().repeat_interleave(_GROUP, dim=1)[:, :C]
    return q.float() * (s if block == 1 else s.repeat_interleave(block, dim=0)[:R])


def _plain_ce(state):
    c, h, w, t, m = state["case"], state["hidden"].float(), state["weight"].float(), state["targets"], state["mask"]
    V, eps, z, cap = c["v"], c["eps"], c["z"], c["cap"]
    y = h @ w.t()
    if cap:
        y = cap * torch.tanh(y / cap)
    top = y.amax(dim=1, keepdim=True)
    lse = (top + torch.log(torch.exp(y - top).sum(dim=1, keepdim=True)))[:, 0]
    active = m != 0
    loss = lse - (1 - eps) * y.gather(1, t[:, None])[:, 0] + z * lse * lse
    if eps:
        loss = loss - eps / V * y.sum(dim=1)
    loss = torch.where(active, loss, torch.zeros_like(loss))
    if not c["grad"]:
        return {"loss": loss, "lse": lse}
    n = active.sum().clamp_min(1)
    g = active.float() / n
    d = torch.exp(y - lse[:, None]) * (1 + 2 * z * lse)[:, None]
    d.scatter_add_(1, t[:, None], torch.full_like(lse, eps - 1)[:, None])
    if eps:
        d -= eps / V
    if cap:
        d *= 1 - (y / cap) ** 2
    d *= g[:, None]
    return {"loss": loss.sum() / n, "dhidden": (d @ w).to(torch.bfloat16), "dweight": (d.t() @ h).to(torch.bfloat16)}


# ------------------------------------------------------------------ the interface

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(r, c, sigma):
        return torch.randn((r, c), generator=gen, device="cuda", dtype=torch.float32).mul_(sigma)

    def activations(r, c):
        # a few channels of a transformer's activations are much larger than the rest
        x = normal(r, c, 1.0)
        big = torch.rand((c,), generator=gen, device="cuda") < 0.01
        return x.mul_(torch.where(big, 20.0, 1.0))

    state = {"case": dict(case)}
    if case["op"] == "quantize":
        x = activations(case["rows"], case["cols"]) if case["block"] == 1 else normal(case["rows"], case["cols"], 0.02)
        state["x"] = x if case["dtype"] == "f32" else x.to(torch.bfloat16)
    elif case["op"] == "matmul":
        a = activations(case["m"], case["k"])
        b = normal(case["n"], case["k"], 0.02) if case["block"] == 128 else activations(case["n"], case["k"])
        for name, x, block in (("a", a, 1), ("b", b, case["block"])):
            q, s = _plain_quantize(x, block)
            pad = -case["k"] % 16  # rows on 16-byte boundaries
            if pad:
                q = torch.nn.functional.pad(q.view(torch.uint8), (0, pad)).view(torch.float8_e4m3fn)[:, :case["k"]]
            state[name], state[name + "_scale"] = q, s
    else:
        pad = -case["h"] % 8  # rows on 16-byte boundaries
        hidden, weight = normal(case["t"], case["h"] + pad, 1.0), normal(case["v"], case["h"] + pad, 0.02)
        state["hidden"] = hidden.to(torch.bfloat16)[:, :case["h"]]
        state["weight"] = weight.to(torch.bfloat16)[:, :case["h"]]
        state["targets"] = torch.randint(0, case["v"], (case["t"],), generator=gen, device="cuda")
        state["mask"] = (torch.rand((case["t"],), generator=gen, device="cuda") < 0.9).to(torch.uint8)
        state["mask"][0] = 1  # prompts and padding aside, a batch has at least one scored token
    return state


def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    if c["op"] == "quantize":
        q, s = _plain_quantize(state["x"], c["block"])
        out = {"q": q, "scale": s}
        if c["both"]:
            out["qt"], out["scale_t"] = _plain_quantize(state["x"].t(), c["block"])
        return out
    if c["op"] == "matmul":
        y = _dequantized(state["a"], state["a_scale"], 1) @ _dequantized(state["b"], state["b_scale"], c["block"]).t()
        return y.to(torch.bfloat16) if c["out"] == "bf16" else y
    return _plain_ce(state)


def _run_own(c, state):
    import vocab_selected_token_tile_gb300 as rlk
    from vocab_selected_token_tile_gb300 import autograd
    if c["op"] == "quantize":
        if c["both"]:
            q, s, qt, st = rlk.fp8_quantize_both(state["x"], block_rows=c["block"])
            return {"q": q, "scale": s, "qt": qt, "scale_t": st}
        q, s = rlk.fp8_quantize(state["x"], block_rows=c["block"])
        return {"q": q, "scale": s}
    if c["op"] == "matmul":
        return rlk.fp8_matmul(state["a"], state["a_scale"], state["b"], state["b_scale"], b_block_rows=c["block"],
                              out_dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    options = {"label_smoothing": c["eps"], "z_loss": c["z"], "softcap": c["cap"]}
    if not c["grad"]:
        loss, lse = autograd.linear_cross_entropy(state["hidden"], state["weight"], state["targets"], state["mask"],
                                                  reduction="none", return_lse=True, **options)
        return {"loss": loss, "lse": lse}
    hidden, weight = state["hidden"].requires_grad_(), state["weight"].requires_grad_()
    loss = autograd.linear_cross_entropy(hidden, weight, state["targets"], state["mask"], reduction="mean", **options)
    dh, dw = torch.autograd.grad(loss, (hidden, weight))
    return {"loss": loss.detach(), "dhidden": dh, "dweight": dw}


def work(case):
    if case["op"] == "quantize":
        n, size = case["rows"] * case["cols"], 4 if case["dtype"] == "f32" else 2
        groups = -(-case["cols"] // _GROUP) * -(-case["rows"] // case["block"])
        groups_t = -(-case["rows"] // _GROUP) * -(-case["cols"] // case["block"])
        return {"bytes": n * size + (2 * n + 4 * (groups + groups_t) if case["both"] else n + 4 * groups), "flops": 3 * n}
    if case["op"] == "matmul":
        m, n, k, kb = case["m"], case["n"], case["k"], -(-case["k"] // _GROUP)
        scales = 4 * kb * (m + -(-n // case["block"]))
        return {"bytes": (m + n) * k + scales + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    t, v, h = case["t"], case["v"], case["h"]
    one = 2 * (t + v) * h + 9 * t  # hidden, weight, targets and mask once
    return {"bytes": one + (2 * (t + v) * h + 4 if case["grad"] else 8 * t), "flops": (6 if case["grad"] else 2) * t * v * h}


def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    if work(case)["flops"] > 1.6e13:
        return None  # over about 20 seconds at the rate of 64-bit products
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "quantize":
        def one(x, block):
            R, C = x.shape
            q = torch.empty((R, C), dtype=f64, device=x.device)
            scale = torch.empty((-(-C // _GROUP), -(-R // block)), dtype=f64, device=x.device)
            for c0 in range(0, C, _GROUP):
                g = x[:, c0:c0 + _GROUP].double()
                top = torch.nn.functional.pad(g.abs().amax(dim=1), (0, -R % block)).view(-1, block).amax(dim=1)
                sc = top.clamp_min(_FLOOR) / _E4M3_MAX
                scale[c0 // _GROUP] = sc
                # the definition rounds the scale, its reciprocal and the product to 32 bits
                v = g * (1.0 / sc.float().double()).float().double().repeat_interleave(block)[:R, None]
                v = v.float().double()
                # the nearest of 8 steps a binade, subnormals below 2^-6, ties to even
                step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
                q[:, c0:c0 + _GROUP] = (torch.round(v / step) * step).clamp(-_E4M3_MAX, _E4M3_MAX)
            return q, scale
        out = dict(zip(("q", "scale"), one(s["x"], case["block"])))
        if case["both"]:
            out.update(zip(("qt", "scale_t"), one(s["x"].t(), case["block"])))
        return out
    if case["op"] == "matmul":
        acc = torch.zeros((case["m"], case["n"]), dtype=f64, device="cuda")
        rows = torch.arange(case["n"], device="cuda") // case["block"]
        for kb in range(s["a_scale"].shape[0]):
            k0, k1 = kb * _GROUP, min((kb + 1) * _GROUP, case["k"])
            a = s["a"][:, k0:k1].double() * s["a_scale"][kb].double()[:, None]
            b = s["b"][:, k0:k1].double() * s["b_scale"][kb].double()[rows][:, None]
            acc.addmm_(a, b.t())
        return acc
    V, eps, z, cap = case["v"], case["eps"], case["z"], case["cap"]
    w = s["weight"].double()
    active = (s["mask"] != 0).double()
    n = max(1.0, float(active.sum()))
    losses, lses, dhs = [], [], []
    dw = torch.zeros_like(w) if case["grad"] else None
    for r0 in range(0, case["t"], 512):
        h, t, on = s["hidden"][r0:r0 + 512].double(), s["targets"][r0:r0 + 512], active[r0:r0 + 512]
        x = h @ w.t()
        y = torch.tanh(x / cap) * cap if cap else x
        lse = torch.logsumexp(y, dim=1)
        pick = torch.nn.functional.one_hot(t, V).double()
        want = (1 - eps) * pick + eps / V
        losses.append(on * (lse - (want * y).sum(dim=1) + z * lse ** 2))
        lses.append(lse)
        if case["grad"]:
            d = (torch.softmax(y, dim=1) * (1 + 2 * z * lse)[:, None] - want) * (on / n)[:, None]
            if cap:
                d = d * (1 - (y / cap) ** 2)
            dhs.append(d @ w)
            dw.addmm_(d.t(), h)
    loss, lse = torch.cat(losses), torch.cat(lses)
    if not case["grad"]:
        return {"loss": loss, "lse": lse}
    return {"loss": loss.sum() / n, "dhidden": torch.cat(dhs), "dweight": dw}
