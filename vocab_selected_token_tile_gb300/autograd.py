"""torch.autograd entry points of the selected-token log-probability.

Argument marshalling only: ``SelectedTokenLogprob``'s forward calls
``rlk_logp_fwd`` and its backward ``rlk_logp_bwd`` with the saved LSE;
``FusedLmHeadLogprob``'s forward calls ``rlk_logp_fused_lmhead`` (logits =
hidden @ weight^T, never materialised) and its backward
``rlk_logp_fused_lmhead_bwd`` with the saved LSE -- or, with keep_logits,
``rlk_logp_fused_lmhead_keep`` and ``rlk_logp_fused_lmhead_bwd_kept`` with the
saved FP32 logits.  Every step of the
arithmetic runs in the CUDA library.  The outputs follow the typed contract of PR #289
("[WS2][PR4][Logp] feat: add distributed TP/CP logprob drift report",
"typed contract" commit: FP32 logprob and FP32 LSE outputs); the LSE is not
differentiable.

``LinearCrossEntropy`` (``linear_cross_entropy``) runs ``rlk_linear_ce_fwd``
and ``rlk_linear_ce_bwd``; ``Fp8Linear`` (``fp8_linear``) quantises with
``rlk_fp8_quantize`` and forms its output and both gradients with
``rlk_fp8_matmul``; ``Fp8Layer`` (``fp8_linear`` with a bias, an activation, a
gate or a residual, and ``fp8_grouped_linear``) runs ``rlk_fp8_matmul_act`` or
``rlk_fp8_grouped_matmul``, ``rlk_fp8_act_grad`` and the products of the
gradients.
"""
import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import (MASK_EXPLICIT, MASK_IGNORE_INDEX, REDUCE_MEAN, REDUCE_NONE, REDUCE_SUM, Contract, Fp8LayerStep,
               fp8_grouped_matmul, fp8_matmul, fp8_matmul_act, fp8_quantize, fp8_quantize_both, linear_ce_bwd,
               linear_ce_contract, linear_ce_fwd, logp_bwd, logp_fused_lmhead, logp_fused_lmhead_bwd,
               logp_fused_lmhead_bwd_kept, logp_fused_lmhead_keep, logp_fwd)

_LOGIT_DTYPES = (torch.bfloat16, torch.int16)  # int16: BF16 bits viewed as integers


class SelectedTokenLogprob(torch.autograd.Function):
    """(logp, lse) of BF16 logits [T, row_stride]; d logits = g (onehot - softmax) in BF16."""

    @staticmethod
    def forward(ctx, logits, targets, mask, contract):
        if logits.dtype not in _LOGIT_DTYPES or not logits.is_cuda:
            raise TypeError("logits must be a CUDA tensor of BF16 (or its int16 bits)")
        logp, lse = logp_fwd(contract, logits, targets, mask)
        ctx.save_for_backward(logits, targets, mask, lse)
        ctx.contract = contract
        ctx.mark_non_differentiable(lse)
        return logp, lse

    @staticmethod
    def backward(ctx, grad_logp, grad_lse):
        logits, targets, mask, lse = ctx.saved_tensors
        if grad_logp is None:
            return None, None, None, None
        g = grad_logp if (grad_logp.dtype == torch.float32 and grad_logp.is_contiguous()) else \
            grad_logp.to(torch.float32).contiguous()
        c = ctx.contract
        # columns [V_padded, row_stride) are not the kernel's: their gradient is zero
        out = torch.zeros_like(logits) if c.row_stride > c.V_padded else None
        dlogits = logp_bwd(c, logits, targets, mask, lse, g, dlogits=out)
        return dlogits, None, None, None


def selected_logprob(logits, targets, mask=None, v_real=None, v_padded=None, num_tiles=64, virtual_tp=1,
                     ignore_index=-100):
    """(logp, lse) with autograd; ``mask`` None selects ignore_index mode.

    ``logits`` is [T, row_stride] BF16 on the GPU; columns [v_real, v_padded)
    are padding (v_padded defaults to row_stride, v_real to v_padded).
    """
    T, stride = logits.shape
    vp = stride if v_padded is None else v_padded
    vr = vp if v_real is None else v_real
    c = Contract(T=T, V_real=vr, V_padded=vp, num_tiles=num_tiles, virtual_tp=virtual_tp,
                 mask_mode=MASK_EXPLICIT if mask is not None else MASK_IGNORE_INDEX, ignore_index=ignore_index,
                 row_stride=stride)
    return SelectedTokenLogprob.apply(logits, targets, mask, c)


class FusedLmHeadLogprob(torch.autograd.Function):
    """(logp, lse) of logits = hidden @ weight^T over a tiled vocabulary; d hidden and d weight in BF16
    (the dtype of the inputs).  hidden [T, H], weight [V_padded, H].  With keep_logits False the logits
    are never materialised and the backward re-runs the GEMM; with True the forward keeps its FP32
    logits (T * V_padded * 4 bytes, held until the backward) and the backward forms dlogits from them
    instead.  The gradients are bitwise the same either way."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, mask, contract, keep_logits=False):
        for name, t in (("hidden", hidden), ("weight", weight)):
            if t.dtype not in _LOGIT_DTYPES or not t.is_cuda or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous CUDA tensor of BF16 (or its int16 bits)")
        logits = None
        if keep_logits and (ctx.needs_input_grad[0] or ctx.needs_input_grad[1]):
            logp, lse, logits = logp_fused_lmhead_keep(contract, hidden, weight, targets, mask)
        else:
            logp, lse = logp_fused_lmhead(contract, hidden, weight, targets, mask)
        ctx.save_for_backward(hidden, weight, targets, mask, lse, logits)
        ctx.contract = contract
        ctx.mark_non_differentiable(lse)
        return logp, lse

    @staticmethod
    def backward(ctx, grad_logp, grad_lse):
        hidden, weight, targets, mask, lse, logits = ctx.saved_tensors
        if grad_logp is None:
            return None, None, None, None, None, None
        g = grad_logp if (grad_logp.dtype == torch.float32 and grad_logp.is_contiguous()) else \
            grad_logp.to(torch.float32).contiguous()
        if logits is not None:
            dh, dw = logp_fused_lmhead_bwd_kept(ctx.contract, hidden, weight, targets, mask, lse, logits, g)
        else:
            dh, dw = logp_fused_lmhead_bwd(ctx.contract, hidden, weight, targets, mask, lse, g)
        return dh, dw, None, None, None, None


def lmhead_logprob(hidden, weight, targets, mask=None, v_real=None, num_tiles=64, virtual_tp=1, ignore_index=-100,
                   keep_logits=False):
    """(logp, lse) of hidden @ weight^T with autograd; ``mask`` None selects ignore_index mode.

    ``weight`` is [V_padded, H]; rows [v_real, V_padded) are padding (v_real defaults to V_padded).
    ``keep_logits`` trades T * V_padded * 4 bytes, held from the forward to the backward, for the
    backward's recompute GEMM (a third of the forward+backward's tensor work).
    """
    T = hidden.shape[0]
    vp = weight.shape[0]
    vr = vp if v_real is None else v_real
    c = Contract(T=T, V_real=vr, V_padded=vp, num_tiles=num_tiles, virtual_tp=virtual_tp,
                 mask_mode=MASK_EXPLICIT if mask is not None else MASK_IGNORE_INDEX, ignore_index=ignore_index)
    return FusedLmHeadLogprob.apply(hidden, weight, targets, mask, c, keep_logits)


def _differentiated(*tensors):
    """Whether a derivative may be asked for through these tensors: a gradient, or the tangent of a dual tensor, which
    the functions here refuse, as they have no forward-mode rule."""
    return torch.is_grad_enabled() and any(t.requires_grad for t in tensors) or \
        any(forward_ad.unpack_dual(t).tangent is not None for t in tensors)


class LinearCrossEntropy(torch.autograd.Function):
    """(loss, lse) of the cross entropy of hidden @ weight^T; the backward forms the logits again, a piece of the
    vocabulary at a time."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, mask, contract):
        loss, lse = linear_ce_fwd(contract, hidden, weight, targets, mask)
        ctx.save_for_backward(hidden, weight, targets, mask, lse)
        ctx.contract = contract
        ctx.mark_non_differentiable(lse)
        return loss, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss, grad_lse):
        if grad_loss is None:
            return None, None, None, None, None
        hidden, weight, targets, mask, lse = ctx.saved_tensors
        g = grad_loss if grad_loss.dtype is torch.float32 and grad_loss.is_contiguous() else \
            grad_loss.to(torch.float32).contiguous()
        dh, dw = linear_ce_bwd(ctx.contract, hidden, weight, targets, mask, lse, g, ctx.needs_input_grad[0],
                               ctx.needs_input_grad[1])
        return dh, dw, None, None, None


def linear_cross_entropy(hidden, weight, targets, mask=None, ignore_index=-100, reduction="mean", label_smoothing=0.0,
                         z_loss=0.0, softcap=0.0, piece=0, return_lse=False):
    """The cross entropy of hidden @ weight^T against ``targets``, with autograd, without keeping the logits.

    ``hidden`` [T, H] and ``weight`` [V, H] are BF16 with rows on 16-byte boundaries; ``mask`` None selects
    ignore_index mode.  ``reduction`` is "mean" (over the active rows; 0 without any), "sum" or "none" (FP32 [T], 0 on
    inactive rows).  ``softcap`` caps the logits at +-softcap by tanh, ``label_smoothing`` mixes the target with the
    uniform distribution and ``z_loss`` adds z_loss * lse^2.  ``piece`` bounds the vocabulary rows whose logits'
    gradient is held at a time (0: 512 MB of it).  With ``return_lse`` the result is (loss, lse).
    """
    kinds = {"none": REDUCE_NONE, "sum": REDUCE_SUM, "mean": REDUCE_MEAN}
    if reduction not in kinds:
        raise ValueError("reduction must be none, sum or mean")
    c = linear_ce_contract(hidden, weight, mask, ignore_index, kinds[reduction], label_smoothing, z_loss, softcap,
                           piece)
    if _differentiated(hidden, weight):
        loss, lse = LinearCrossEntropy.apply(hidden, weight, targets, mask, c)
    else:
        loss, lse = linear_ce_fwd(c, hidden, weight, targets, mask)
    return (loss, lse) if return_lse else loss


class Fp8Linear(torch.autograd.Function):
    """y = x @ weight^T in FP8: x in 1 x 128 groups of its rows, weight in 128 x 128 blocks.  The backward quantises dy
    along its rows for dx = dy @ weight, and dy and x along the tokens for dweight = dy^T @ x."""

    @staticmethod
    def forward(ctx, x, weight, to):
        need_x, need_w = ctx.needs_input_grad[:2]
        xq, xs, xtq, xts = fp8_quantize_both(x) if need_w else (*fp8_quantize(x), None, None)
        wq, ws, wtq, wts = fp8_quantize_both(weight, block_rows=128) if need_x else \
            (*fp8_quantize(weight, block_rows=128), None, None)
        y = fp8_matmul(xq, xs, wq, ws, **to)
        ctx.save_for_backward(xtq, xts, wtq, wts)
        ctx.types = x.dtype, weight.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        xtq, xts, wtq, wts = ctx.saved_tensors
        need_x, need_w = ctx.needs_input_grad[:2]
        dy = dy if dy.dtype in (torch.bfloat16, torch.float32) else dy.to(torch.bfloat16)
        dy = dy if dy.stride(-1) == 1 and (dy.shape[0] <= 1 or dy.stride(0) >= dy.shape[1]) else dy.contiguous()
        q = s = qt = st = None
        if need_x and need_w:
            q, s, qt, st = fp8_quantize_both(dy)
        elif need_x:
            q, s = fp8_quantize(dy)
        elif need_w:
            qt, st = fp8_quantize(dy, transpose=True)
        dx = fp8_matmul(q, s, wtq, wts, out_dtype=ctx.types[0]) if need_x else None
        dw = fp8_matmul(qt, st, xtq, xts, b_block_rows=1, out_dtype=ctx.types[1]) if need_w else None
        return dx, dw, None


def _dense_rows(t):
    """t with contiguous rows that do not overlap: a copy of what is transposed, or expanded from fewer rows."""
    return t if t.stride(-1) == 1 and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1]) else t.contiguous()


def _rows_of(dy):
    """dy as the quantisations take it: BF16 or FP32, contiguous rows that do not overlap."""
    return _dense_rows(dy if dy.dtype in (torch.bfloat16, torch.float32) else dy.to(torch.bfloat16))


class Fp8Layer(torch.autograd.Function):
    """y = act(x @ weight^T + bias) + residual in FP8, dense or (with ends) of rows that belong to groups, each with a
    weight and a bias of its own.  z, the argument of the activation, is kept in BF16; the backward forms dz, the sum of
    its rows for the bias, and its codes along the rows and along the tokens in one pass, then the two products of
    Fp8Linear's (Fp8LayerStep makes the calls)."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, ends, activation, gated, out_dtype):
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        step = Fp8LayerStep(x, weight, bias, residual, ends, activation, gated, need_x, need_w, need_b, out_dtype)
        y, z, saved = step.forward(x, weight)
        ctx.save_for_backward(z, saved, ends)
        ctx.step = step
        ctx.residual = None if residual is None else residual.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        dres = dy.to(ctx.residual) if ctx.needs_input_grad[3] else None
        if not any(ctx.needs_input_grad[:3]):
            return None, None, None, dres, None, None, None, None
        z, saved, ends = ctx.saved_tensors
        return *ctx.step.backward(_rows_of(dy), z, saved, ends), dres, None, None, None, None


def fp8_linear(x, weight, bias=None, activation=None, gated=False, residual=None, out_dtype=None):
    """act(x [..., K] @ weight [N, K]^T + bias) + residual in FP8 with autograd: BF16 out, or FP32 with ``out_dtype``
    torch.float32, rounded once; gradients in the inputs' types (BF16 or FP32).

    Forward and backward quantise with one FP32 scale per 128 elements (or 128 x 128 weights) and sum in FP32; what is
    saved for the backward are the E4M3 transposes, one byte an element, and with an activation or a gate its argument
    in BF16.  ``activation`` is None, "relu", "silu", "gelu" or "gelu_tanh"; with ``gated`` the weight holds the gate's
    rows, then as many more (a multiple of 64 each), and the result is act(gate) * other.  ``bias`` has a value for each
    row of the weight; ``residual`` has the result's shape (an FP32 stream keeps its digits in an FP32 result only).

    The weight is quantised at every call: a server, whose weights stay, does that once (fp8_quantize with block_rows
    128) and calls fp8_matmul_act.
    """
    if bias is None and residual is None and not gated and activation in (None, "none"):
        return _linear(x, weight, out_dtype)
    lead = x.shape[:-1]
    rows = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    n = weight.shape[0] // 2 if gated else weight.shape[0]
    if residual is not None:
        if residual.shape != (*lead, n):
            raise ValueError(f"residual is {list(residual.shape)}; the result is {[*lead, n]}")
        residual = _dense_rows(residual if x.dim() == 2 else residual.reshape(rows.shape[0], n))
    if _differentiated(*(t for t in (x, weight, bias, residual) if t is not None)):
        y = Fp8Layer.apply(rows, weight, bias, residual, None, activation, gated, out_dtype)
    else:
        y = fp8_matmul_act(*fp8_quantize(rows), *fp8_quantize(weight, block_rows=128), bias, activation, gated, residual,
                           False, out_dtype)
    return y if x.dim() == 2 else y.reshape(*lead, n)


def fp8_grouped_linear(x, weight, ends, bias=None, activation=None, gated=False, out_dtype=None):
    """fp8_linear for rows that belong to groups (a mixture's experts), with autograd: group e is rows
    [ends[e - 1], ends[e]) of x [M, K], with weight[e] of weight [G, N, K] and bias[e] of bias [G, N].

    ``ends`` is int32 [G] on the GPU, the running sum of the groups' counts of rows; nothing is read back.  Rows behind
    the last group (padding) have a zero result and a zero gradient, and reach nothing whatever they hold; a group
    without rows has zero gradients.  All weights are quantised at every call; fp8_grouped_matmul takes kept codes.
    """
    if _differentiated(*(t for t in (x, weight, bias) if t is not None)):
        return Fp8Layer.apply(x, weight, bias, None, ends, activation, gated, out_dtype)
    return fp8_grouped_matmul(*fp8_quantize(x), *fp8_quantize(weight, block_rows=128), ends, bias, activation, gated,
                              False, out_dtype)


def _linear(x, weight, out_dtype):
    """fp8_linear without an epilogue."""
    lead = x.shape[:-1]
    rows = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    to = {} if out_dtype is None else {"out_dtype": out_dtype}
    if _differentiated(x, weight):
        y = Fp8Linear.apply(rows, weight, to)
    else:
        y = fp8_matmul(*fp8_quantize(rows), *fp8_quantize(weight, block_rows=128), **to)
    return y if x.dim() == 2 else y.reshape(*lead, weight.shape[0])
