"""Deterministic selected-token log-probability over a tiled vocabulary (GB300, sm_103a).

A thin ctypes binding of ``librlk_logp.so`` (declared in ``include/rlk_logp.h``).
The functions named ``rlk_*`` mirror the C entry points one to one and take
raw device pointers; ``logp_fwd``, ``logp_bwd`` and ``logp_fwd_bwd`` only
marshal torch tensors (allocate outputs, pass ``data_ptr()`` and the current
stream).  Every step of the computation runs in the CUDA library: if it is
missing or fails to load, these functions raise -- there is no fallback.
"""
import contextlib
import ctypes
import os

from . import _build

RLK_OK = 0
RLK_ERR_INVALID_ARG = 1
RLK_ERR_UNSUPPORTED = 2
RLK_ERR_NON_TILEABLE = 3
RLK_ERR_MISALIGNED = 4
RLK_ERR_TARGET_RANGE = 5
RLK_ERR_NONFINITE_LSE = 6
RLK_ERR_TIMEOUT = 7
RLK_ERR_CUDA = 8

RLK_BF16 = 0
RLK_F32 = 1

RLK_FP8_WORKSPACE = 256

ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

REDUCE_NONE = 0
REDUCE_SUM = 1
REDUCE_MEAN = 2

MASK_EXPLICIT = 0
MASK_IGNORE_INDEX = 1

EXPORTED = (
    "rlk_logp_check_contract",
    "rlk_logp_workspace_size",
    "rlk_logp_fwd",
    "rlk_logp_bwd",
    "rlk_logp_fwd_noalloc",
    "rlk_logp_fwd_entropy",
    "rlk_logp_fwd_bwd_entropy",
    "rlk_grpo_loss",
    "rlk_grpo_fused_workspace_size",
    "rlk_grpo_fused_step",
    "rlk_logp_lmhead_workspace_size",
    "rlk_logp_fused_lmhead",
    "rlk_logp_fused_lmhead_bwd",
    "rlk_logp_fused_lmhead_keep",
    "rlk_logp_fused_lmhead_bwd_kept",
    "rlk_logp_check_shard_contract",
    "rlk_logp_shard_workspace_size",
    "rlk_logp_shard_fwd",
    "rlk_logp_fold",
    "rlk_logp_shard_bwd",
    "rlk_linear_ce_check",
    "rlk_linear_ce_workspace_size",
    "rlk_linear_ce_fwd",
    "rlk_linear_ce_bwd",
    "rlk_fp8_quantize",
    "rlk_fp8_matmul",
    "rlk_fp8_matmul_act",
    "rlk_fp8_grouped_matmul",
    "rlk_fp8_quantize_grouped",
    "rlk_fp8_quantize_batch",
    "rlk_fp8_grouped_dweight",
    "rlk_fp8_act_grad_workspace_size",
    "rlk_fp8_act_grad",
    "rlk_logp_workspace_status",
    "rlk_selftest_bounded_wait",
    "rlk_status_string",
    "rlk_last_error_message",
)


class Contract(ctypes.Structure):
    """Mirror of ``rlk_logp_contract`` (64 bytes)."""
    _fields_ = [
        ("T", ctypes.c_int64),
        ("V_real", ctypes.c_int64),
        ("V_padded", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
        ("num_tiles", ctypes.c_int32),
        ("virtual_tp", ctypes.c_int32),
        ("mask_mode", ctypes.c_int32),
        ("validate", ctypes.c_int32),
        ("ignore_index", ctypes.c_int64),
        ("wait_timeout_ns", ctypes.c_int64),
    ]

    def __init__(self, T, V_real, V_padded, num_tiles=64, virtual_tp=1, mask_mode=MASK_EXPLICIT,
                 ignore_index=-100, validate=0, row_stride=0, wait_timeout_ns=0):
        super().__init__(T, V_real, V_padded, row_stride, num_tiles, virtual_tp, mask_mode, validate,
                         ignore_index, wait_timeout_ns)

    def replace(self, **kw):
        d = {name: getattr(self, name) for name, _ in self._fields_}
        d.update(kw)
        return Contract(**d)


class LinearCeContract(ctypes.Structure):
    """Mirror of ``rlk_linear_ce_contract`` (104 bytes); strides and piece 0 take the header's defaults."""
    _fields_ = [(n, ctypes.c_int64) for n in ("T", "V", "H", "hidden_stride", "weight_stride", "dhidden_stride",
                                              "dweight_stride", "ignore_index", "wait_timeout_ns", "piece")] + \
               [(n, ctypes.c_int32) for n in ("mask_mode", "reduction", "validate")] + \
               [(n, ctypes.c_float) for n in ("label_smoothing", "z_loss", "softcap")]

    def __init__(self, T, V, H, hidden_stride=0, weight_stride=0, dhidden_stride=0, dweight_stride=0,
                 ignore_index=-100, wait_timeout_ns=0, piece=0, mask_mode=MASK_EXPLICIT, reduction=REDUCE_NONE,
                 validate=0, label_smoothing=0.0, z_loss=0.0, softcap=0.0):
        super().__init__(T, V, H, hidden_stride, weight_stride, dhidden_stride, dweight_stride, ignore_index,
                         wait_timeout_ns, piece, mask_mode, reduction, validate, label_smoothing, z_loss, softcap)

    def replace(self, **kw):
        d = {name: getattr(self, name) for name, _ in self._fields_}
        d.update(kw)
        return LinearCeContract(**d)


class Fp8Epilogue(ctypes.Structure):
    """Mirror of ``rlk_fp8_epilogue`` (56 bytes)."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("z", ctypes.c_void_p),
                ("residual_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64), ("bias_type", ctypes.c_int32),
                ("residual_type", ctypes.c_int32), ("activation", ctypes.c_int32), ("gated", ctypes.c_int32)]


class RlkError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{rlk_status_string(status)}: {message}")
        self.status = status


_lib = None


def library():
    """Load librlk_logp.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"CUDA library not built: {_build.LIB} (run __graft_entry__.build())")
        lib = ctypes.CDLL(_build.LIB)
        P = ctypes.POINTER(Contract)
        vp, i = ctypes.c_void_p, ctypes.c_int
        lib.rlk_logp_check_contract.argtypes = [P]
        lib.rlk_logp_check_contract.restype = i
        lib.rlk_logp_workspace_size.argtypes = [P]
        lib.rlk_logp_workspace_size.restype = ctypes.c_size_t
        lib.rlk_logp_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logp_fwd.restype = i
        lib.rlk_logp_bwd.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logp_bwd.restype = i
        lib.rlk_logp_lmhead_workspace_size.argtypes = [P, ctypes.c_int64]
        lib.rlk_logp_lmhead_workspace_size.restype = ctypes.c_size_t
        lib.rlk_logp_fused_lmhead.argtypes = [P, vp, ctypes.c_int64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logp_fused_lmhead.restype = i
        lib.rlk_logp_fused_lmhead_bwd.argtypes = [P, vp, ctypes.c_int64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logp_fused_lmhead_bwd.restype = i
        lib.rlk_logp_fused_lmhead_keep.argtypes = [P, vp, ctypes.c_int64, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logp_fused_lmhead_keep.restype = i
        lib.rlk_logp_fused_lmhead_bwd_kept.argtypes = [P, vp, ctypes.c_int64, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                       vp, vp]
        lib.rlk_logp_fused_lmhead_bwd_kept.restype = i
        lib.rlk_logp_fwd_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logp_fwd_noalloc.restype = i
        lib.rlk_logp_fwd_entropy.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logp_fwd_entropy.restype = i
        lib.rlk_logp_fwd_bwd_entropy.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logp_fwd_bwd_entropy.restype = i
        lib.rlk_grpo_loss.argtypes = [ctypes.c_int64, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp]
        lib.rlk_grpo_loss.restype = i
        lib.rlk_grpo_fused_workspace_size.argtypes = [P]
        lib.rlk_grpo_fused_workspace_size.restype = ctypes.c_size_t
        lib.rlk_grpo_fused_step.argtypes = [P, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_grpo_fused_step.restype = i
        lib.rlk_logp_check_shard_contract.argtypes = [P, ctypes.c_int32]
        lib.rlk_logp_check_shard_contract.restype = i
        lib.rlk_logp_shard_workspace_size.argtypes = [P]
        lib.rlk_logp_shard_workspace_size.restype = ctypes.c_size_t
        lib.rlk_logp_shard_fwd.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logp_shard_fwd.restype = i
        lib.rlk_logp_fold.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logp_fold.restype = i
        lib.rlk_logp_shard_bwd.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_logp_shard_bwd.restype = i
        C = ctypes.POINTER(LinearCeContract)
        lib.rlk_linear_ce_check.argtypes = [C]
        lib.rlk_linear_ce_check.restype = i
        lib.rlk_linear_ce_workspace_size.argtypes = [C, ctypes.c_int32]
        lib.rlk_linear_ce_workspace_size.restype = ctypes.c_size_t
        lib.rlk_linear_ce_fwd.argtypes = [C, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_linear_ce_fwd.restype = i
        lib.rlk_linear_ce_bwd.argtypes = [C, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.rlk_linear_ce_bwd.restype = i
        i64, i32 = ctypes.c_int64, ctypes.c_int32
        lib.rlk_fp8_quantize.argtypes = [i64, i64, vp, ctypes.c_int32, i64, ctypes.c_int32, vp, i64, vp, vp, i64, vp,
                                         vp]
        lib.rlk_fp8_quantize.restype = i
        lib.rlk_fp8_matmul.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, vp, ctypes.c_int32, vp, ctypes.c_int32,
                                       i64, ctypes.c_int32, vp, vp]
        lib.rlk_fp8_matmul.restype = i
        E = ctypes.POINTER(Fp8Epilogue)
        lib.rlk_fp8_matmul_act.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, vp, E, vp, i32, i64, vp, vp]
        lib.rlk_fp8_grouped_matmul.argtypes = [i64, i64, i64, i64, vp, vp, i64, vp, vp, i64, i64, vp, E, vp, i32, i64,
                                               i32, vp, vp]
        lib.rlk_fp8_quantize_grouped.argtypes = [i64, i64, i64, vp, vp, i32, i64, vp, i64, vp, vp, i64, vp, vp]
        lib.rlk_fp8_quantize_batch.argtypes = [i64, i64, i64, vp, i32, i64, i64, vp, i64, i64, vp, vp, i64, i64, vp, vp]
        lib.rlk_fp8_grouped_dweight.argtypes = [i64, i64, i64, i64, vp, vp, i64, vp, vp, i64, vp, vp, i32, i64, i64,
                                                i32, vp, vp]
        lib.rlk_fp8_act_grad_workspace_size.argtypes = [i64, i64, i64, i32]
        lib.rlk_fp8_act_grad_workspace_size.restype = ctypes.c_size_t
        lib.rlk_fp8_act_grad.argtypes = [i64, i64, i64, vp, vp, i32, i64, vp, i64, i32, i32, vp, i64, vp, vp, i64, vp,
                                         vp, i32, vp, vp]
        for name in ("matmul_act", "grouped_matmul", "quantize_grouped", "quantize_batch", "grouped_dweight",
                     "act_grad"):
            getattr(lib, "rlk_fp8_" + name).restype = i
        lib.rlk_logp_workspace_status.argtypes = [vp, vp]
        lib.rlk_logp_workspace_status.restype = i
        lib.rlk_selftest_bounded_wait.argtypes = [ctypes.c_int64, vp, vp]
        lib.rlk_selftest_bounded_wait.restype = i
        lib.rlk_status_string.argtypes = [i]
        lib.rlk_status_string.restype = ctypes.c_char_p
        lib.rlk_last_error_message.argtypes = []
        lib.rlk_last_error_message.restype = ctypes.c_char_p
        _lib = lib
    return _lib


# ------------------------------------------------------------------ C names

def rlk_logp_check_contract(contract):
    return library().rlk_logp_check_contract(ctypes.byref(contract))


def rlk_logp_workspace_size(contract):
    return library().rlk_logp_workspace_size(ctypes.byref(contract))


def rlk_logp_fwd(contract, logits, targets, active_mask, logp, lse, partials, workspace, stream):
    return library().rlk_logp_fwd(ctypes.byref(contract), logits, targets, active_mask, logp, lse, partials,
                                  workspace, stream)


def rlk_logp_bwd(contract, logits, targets, active_mask, lse_in, grad_logp, dlogits, logp_out, lse_out,
                 workspace, stream):
    return library().rlk_logp_bwd(ctypes.byref(contract), logits, targets, active_mask, lse_in, grad_logp,
                                  dlogits, logp_out, lse_out, workspace, stream)


def rlk_logp_lmhead_workspace_size(contract, H):
    return library().rlk_logp_lmhead_workspace_size(ctypes.byref(contract), H)


def rlk_logp_fused_lmhead(contract, hidden, H, weight, targets, active_mask, grad_logp, logp, lse, dhidden,
                          dweight_f32, dweight_bf16, workspace, stream):
    return library().rlk_logp_fused_lmhead(ctypes.byref(contract), hidden, H, weight, targets, active_mask,
                                           grad_logp, logp, lse, dhidden, dweight_f32, dweight_bf16, workspace,
                                           stream)


def rlk_logp_fused_lmhead_bwd(contract, hidden, H, weight, targets, active_mask, lse_in, grad_logp, dhidden,
                              dweight_f32, dweight_bf16, workspace, stream):
    return library().rlk_logp_fused_lmhead_bwd(ctypes.byref(contract), hidden, H, weight, targets, active_mask,
                                               lse_in, grad_logp, dhidden, dweight_f32, dweight_bf16, workspace,
                                               stream)


def rlk_logp_fused_lmhead_keep(contract, hidden, H, weight, targets, active_mask, logp, lse, logits_f32, workspace,
                               stream):
    return library().rlk_logp_fused_lmhead_keep(ctypes.byref(contract), hidden, H, weight, targets, active_mask,
                                                logp, lse, logits_f32, workspace, stream)


def rlk_logp_fused_lmhead_bwd_kept(contract, hidden, H, weight, targets, active_mask, lse_in, logits_f32, grad_logp,
                                   dhidden, dweight_f32, dweight_bf16, workspace, stream):
    return library().rlk_logp_fused_lmhead_bwd_kept(ctypes.byref(contract), hidden, H, weight, targets, active_mask,
                                                    lse_in, logits_f32, grad_logp, dhidden, dweight_f32,
                                                    dweight_bf16, workspace, stream)


def rlk_logp_fwd_entropy(contract, logits, targets, active_mask, logp, lse, entropy, workspace, stream):
    return library().rlk_logp_fwd_entropy(ctypes.byref(contract), logits, targets, active_mask, logp, lse, entropy,
                                          workspace, stream)


def rlk_logp_fwd_bwd_entropy(contract, logits, targets, active_mask, grad_logp, dlogits, logp_out, lse_out,
                             entropy_out, workspace, stream):
    return library().rlk_logp_fwd_bwd_entropy(ctypes.byref(contract), logits, targets, active_mask, grad_logp,
                                              dlogits, logp_out, lse_out, entropy_out, workspace, stream)


def rlk_grpo_loss(T, logp, advantage, active_mask, ref_logp, beta, loss, grad_logp, active_count, stream):
    return library().rlk_grpo_loss(T, logp, advantage, active_mask, ref_logp, beta, loss, grad_logp, active_count,
                                   stream)


def rlk_grpo_fused_workspace_size(contract):
    return library().rlk_grpo_fused_workspace_size(ctypes.byref(contract))


def rlk_grpo_fused_step(contract, logits, targets, active_mask, advantage, ref_logp, beta, dlogits, logp_out, lse_out,
                        grad_out, entropy_out, loss, active_count, workspace, stream):
    return library().rlk_grpo_fused_step(ctypes.byref(contract), logits, targets, active_mask, advantage, ref_logp,
                                         beta, dlogits, logp_out, lse_out, grad_out, entropy_out, loss, active_count,
                                         workspace, stream)


def rlk_logp_fwd_noalloc(contract, logits, targets, active_mask, logp, lse, partials, stream):
    return library().rlk_logp_fwd_noalloc(ctypes.byref(contract), logits, targets, active_mask, logp, lse,
                                          partials, stream)


def rlk_logp_check_shard_contract(contract, shard):
    return library().rlk_logp_check_shard_contract(ctypes.byref(contract), shard)


def rlk_logp_shard_workspace_size(contract):
    return library().rlk_logp_shard_workspace_size(ctypes.byref(contract))


def rlk_logp_shard_fwd(contract, shard, logits_shard, targets, active_mask, partials_shard, target_logit, workspace,
                       stream):
    return library().rlk_logp_shard_fwd(ctypes.byref(contract), shard, logits_shard, targets, active_mask,
                                        partials_shard, target_logit, workspace, stream)


def rlk_logp_fold(contract, gathered_partials, gathered_target_logit, targets, active_mask, logp, lse, workspace,
                  stream):
    return library().rlk_logp_fold(ctypes.byref(contract), gathered_partials, gathered_target_logit, targets,
                                   active_mask, logp, lse, workspace, stream)


def rlk_logp_shard_bwd(contract, shard, logits_shard, targets, active_mask, lse_in, grad_logp, dlogits_shard,
                       workspace, stream):
    return library().rlk_logp_shard_bwd(ctypes.byref(contract), shard, logits_shard, targets, active_mask, lse_in,
                                        grad_logp, dlogits_shard, workspace, stream)


def rlk_linear_ce_check(contract):
    return library().rlk_linear_ce_check(ctypes.byref(contract))


def rlk_linear_ce_workspace_size(contract, with_grad):
    return library().rlk_linear_ce_workspace_size(ctypes.byref(contract), with_grad)


def rlk_linear_ce_fwd(contract, hidden, weight, targets, active_mask, loss, lse, workspace, stream):
    return library().rlk_linear_ce_fwd(ctypes.byref(contract), hidden, weight, targets, active_mask, loss, lse,
                                       workspace, stream)


def rlk_linear_ce_bwd(contract, hidden, weight, targets, active_mask, lse, grad_loss, dhidden, dweight, workspace,
                      stream):
    return library().rlk_linear_ce_bwd(ctypes.byref(contract), hidden, weight, targets, active_mask, lse, grad_loss,
                                       dhidden, dweight, workspace, stream)


def rlk_fp8_quantize(rows, cols, x, x_type, x_stride, block_rows, q, q_stride, scale, qt, qt_stride, scale_t, stream):
    return library().rlk_fp8_quantize(rows, cols, x, x_type, x_stride, block_rows, q, q_stride, scale, qt, qt_stride,
                                      scale_t, stream)


def rlk_fp8_matmul(M, N, K, a, a_stride, a_scale, b, b_stride, b_scale, b_block_rows, c, c_type, c_stride, accumulate,
                   workspace, stream):
    return library().rlk_fp8_matmul(M, N, K, a, a_stride, a_scale, b, b_stride, b_scale, b_block_rows, c, c_type,
                                    c_stride, accumulate, workspace, stream)


def rlk_fp8_matmul_act(M, N, K, a, a_stride, a_scale, b, b_stride, b_scale, epilogue, c, c_type, c_stride, workspace,
                       stream):
    return library().rlk_fp8_matmul_act(M, N, K, a, a_stride, a_scale, b, b_stride, b_scale,
                                        None if epilogue is None else ctypes.byref(epilogue), c, c_type, c_stride,
                                        workspace, stream)


def rlk_fp8_grouped_matmul(groups, M, N, K, ends, a, a_stride, a_scale, b, b_stride, b_group_stride, b_scale, epilogue,
                           c, c_type, c_stride, zero_rest, workspace, stream):
    return library().rlk_fp8_grouped_matmul(groups, M, N, K, ends, a, a_stride, a_scale, b, b_stride, b_group_stride,
                                            b_scale, None if epilogue is None else ctypes.byref(epilogue), c, c_type,
                                            c_stride, zero_rest, workspace, stream)


def rlk_fp8_quantize_grouped(groups, rows, cols, ends, x, x_type, x_stride, q, q_stride, scale, qt, qt_stride, scale_t,
                             stream):
    return library().rlk_fp8_quantize_grouped(groups, rows, cols, ends, x, x_type, x_stride, q, q_stride, scale, qt,
                                              qt_stride, scale_t, stream)


def rlk_fp8_quantize_batch(count, rows, cols, x, x_type, x_stride, x_batch_stride, q, q_stride, q_batch_stride, scale,
                           qt, qt_stride, qt_batch_stride, scale_t, stream):
    return library().rlk_fp8_quantize_batch(count, rows, cols, x, x_type, x_stride, x_batch_stride, q, q_stride,
                                            q_batch_stride, scale, qt, qt_stride, qt_batch_stride, scale_t, stream)


def rlk_fp8_grouped_dweight(groups, rows, M, N, ends, a, a_stride, a_scale, b, b_stride, b_scale, c, c_type, c_stride,
                            c_group_stride, accumulate, workspace, stream):
    return library().rlk_fp8_grouped_dweight(groups, rows, M, N, ends, a, a_stride, a_scale, b, b_stride, b_scale, c,
                                             c_type, c_stride, c_group_stride, accumulate, workspace, stream)


def rlk_fp8_act_grad_workspace_size(groups, rows, cols, gated):
    return library().rlk_fp8_act_grad_workspace_size(groups, rows, cols, gated)


def rlk_fp8_act_grad(groups, rows, cols, ends, dy, dy_type, dy_stride, z, z_stride, activation, gated, q, q_stride,
                     scale, qt, qt_stride, scale_t, dbias, dbias_type, workspace, stream):
    return library().rlk_fp8_act_grad(groups, rows, cols, ends, dy, dy_type, dy_stride, z, z_stride, activation, gated,
                                      q, q_stride, scale, qt, qt_stride, scale_t, dbias, dbias_type, workspace, stream)


def rlk_logp_workspace_status(workspace, stream):
    return library().rlk_logp_workspace_status(workspace, stream)


def rlk_selftest_bounded_wait(timeout_ns, workspace, stream):
    return library().rlk_selftest_bounded_wait(timeout_ns, workspace, stream)


def rlk_status_string(status):
    return library().rlk_status_string(status).decode()


def rlk_last_error_message():
    return library().rlk_last_error_message().decode()


def check(status):
    if status != RLK_OK:
        raise RlkError(status, rlk_last_error_message())


# ------------------------------------------------------------------ torch marshalling

def _ptr(t):
    return None if t is None else t.data_ptr()


_BF16 = ("bfloat16", "int16", "uint16")  # BF16 logits, or their bits as 16-bit integers
_I64 = ("int64",)
_U8 = ("uint8", "bool")
_F32 = ("float32",)


def _need(t, name, nbytes, kinds, optional=False):
    """Fails before any launch when ``t`` cannot be what the call reads or writes through its pointer:
    a CUDA tensor of one of ``kinds`` whose storage holds ``nbytes`` from its first element on (so no
    access leaves it) and, when it is contiguous, whose own elements cover them (a short view of a
    larger buffer is a mistake too).  The C entry points check pointers, alignment and the device;
    only the caller knows the sizes."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    kind = str(t.dtype).replace("torch.", "")
    if kind not in kinds:
        raise TypeError(f"{name} must be {' or '.join(kinds)}, not {kind}")
    have = t.untyped_storage().nbytes() - t.storage_offset() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name} holds {have} bytes from its first element; the call touches {nbytes}")
    if t.is_contiguous() and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} has {t.numel()} elements; the call touches {nbytes} bytes")


def _need_rows(t, name, T, stride, width, kinds):
    """A [T, stride] row buffer of 16-bit elements of which the call touches ``width`` a row; a 2-D
    view must also have those rows and that row stride (a shard read in place from the whole row
    buffer is such a view)."""
    _need(t, name, _rows(T, stride, width, 2), kinds)
    if t.dim() == 2 and T > 0 and (t.shape[0] < T or t.shape[1] < width or t.stride(1) != 1 or
                                   (T > 1 and t.stride(0) != stride)):
        raise ValueError(f"{name} is a {list(t.shape)} view with strides {list(t.stride())}; the call reads {T} "
                         f"rows of {width} elements, {stride} apart")


def _rows(T, stride, width, esize):
    """Bytes from the first element of a [T, stride] row-major buffer to the end of row T-1's width."""
    return 0 if T <= 0 else ((T - 1) * stride + width) * esize


def _dlogits_out(contract, logits, dlogits, stride=None, width=None):
    """The dlogits buffer: the given one, checked, or a new [T, row stride] one like the logits."""
    import torch
    stride = stride or contract.row_stride or contract.V_padded
    width = width or contract.V_padded
    if dlogits is None:
        return torch.empty((contract.T, stride), dtype=logits.dtype, device=logits.device)
    _need_rows(dlogits, "dlogits", contract.T, stride, width, _BF16)
    return dlogits


def _lmhead_operands(contract, hidden, weight):
    """hidden [T, H] and weight [V_padded, H], BF16, contiguous; returns H."""
    if hidden.dim() != 2 or hidden.shape[0] != contract.T:
        raise ValueError(f"hidden must be [T = {contract.T}, H], not {list(hidden.shape)}")
    H = hidden.shape[1]
    if weight.dim() != 2 or weight.shape[0] != contract.V_padded or weight.shape[1] != H:
        raise ValueError(f"weight must be [V_padded = {contract.V_padded}, H = {H}], not {list(weight.shape)}")
    for name, t in (("hidden", hidden), ("weight", weight)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        _need(t, name, 2 * t.numel(), _BF16)
    return H


def _lmhead_workspace(contract, H, dev, workspace):
    import torch
    n = rlk_logp_lmhead_workspace_size(contract, H)
    if n == 0:
        check(rlk_logp_check_contract(contract) or RLK_ERR_UNSUPPORTED)
    if workspace is None:
        return torch.empty(n, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", n, ("uint8",))
    return workspace


def _rowwise(contract, targets, mask, **f32):
    """targets int64 [T], mask uint8/bool [T] (None in ignore_index mode) and FP32 [T] vectors."""
    T = contract.T
    _need(targets, "targets", 8 * T, _I64)
    _need(mask, "mask", T, _U8, optional=True)
    for name, t in f32.items():
        _need(t, name, 4 * T, _F32)


def _stream(stream):
    import torch
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


_workspaces = {}


def workspace_for(contract, device, stream=None):
    """A per-(device, stream) status workspace; calls on one stream never overlap."""
    import torch
    key = (str(device), _stream(stream))
    n = max(rlk_logp_workspace_size(contract), 256)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < n:
        ws = torch.zeros(n, dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def logp_fwd(contract, logits, targets, mask=None, partials=False, stream=None, out=None):
    """(logp, lse[, partials]) for BF16 ``logits`` [T, row_stride] (bf16/int16 storage) on the GPU."""
    import torch
    dev = logits.device
    T = contract.T
    _need_rows(logits, "logits", contract.T, contract.row_stride or contract.V_padded, contract.V_padded, _BF16)
    logp, lse = out if out is not None else (torch.empty(T, dtype=torch.float32, device=dev),
                                             torch.empty(T, dtype=torch.float32, device=dev))
    _rowwise(contract, targets, mask, logp=logp, lse=lse)
    part = torch.empty((T, contract.num_tiles, 2), dtype=torch.float32, device=dev) if partials else None
    ws = workspace_for(contract, dev, stream)
    check(rlk_logp_fwd(contract, _ptr(logits), _ptr(targets), _ptr(mask), _ptr(logp), _ptr(lse), _ptr(part),
                       _ptr(ws), _stream(stream)))
    return (logp, lse, part) if partials else (logp, lse)


def logp_bwd(contract, logits, targets, mask, lse, grad, dlogits=None, stream=None):
    """BF16 dlogits [T, row_stride] from the forward's LSE (the logits are re-read)."""
    dev = logits.device
    _need_rows(logits, "logits", contract.T, contract.row_stride or contract.V_padded, contract.V_padded, _BF16)
    _rowwise(contract, targets, mask, lse=lse, grad=grad)
    dlogits = _dlogits_out(contract, logits, dlogits)
    ws = workspace_for(contract, dev, stream)
    check(rlk_logp_bwd(contract, _ptr(logits), _ptr(targets), _ptr(mask), _ptr(lse), _ptr(grad),
                       _ptr(dlogits), None, None, _ptr(ws), _stream(stream)))
    return dlogits


def logp_fwd_entropy(contract, logits, targets, mask=None, stream=None):
    """(logp, lse, entropy) for BF16 ``logits`` on the GPU, in one pass; entropy of each row's softmax."""
    import torch
    dev = logits.device
    T = contract.T
    _need_rows(logits, "logits", contract.T, contract.row_stride or contract.V_padded, contract.V_padded, _BF16)
    _rowwise(contract, targets, mask)
    logp, lse, ent = (torch.empty(T, dtype=torch.float32, device=dev) for _ in range(3))
    ws = workspace_for(contract, dev, stream)
    check(rlk_logp_fwd_entropy(contract, _ptr(logits), _ptr(targets), _ptr(mask), _ptr(logp), _ptr(lse), _ptr(ent),
                               _ptr(ws), _stream(stream)))
    return logp, lse, ent


def grpo_loss(logp, advantage, mask, ref_logp=None, beta=0.0, stream=None):
    """(loss, grad_logp, active_count) of the token-mean GRPO loss (GPU tensors; loss and count are 1-element)."""
    import torch
    dev = logp.device
    T = logp.numel()
    _need(logp, "logp", 4 * T, _F32)
    _need(advantage, "advantage", 4 * T, _F32)
    _need(mask, "mask", T, _U8, optional=True)
    _need(ref_logp, "ref_logp", 4 * T, _F32, optional=True)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    count = torch.empty(1, dtype=torch.float32, device=dev)
    g = torch.empty(T, dtype=torch.float32, device=dev)
    check(rlk_grpo_loss(T, _ptr(logp), _ptr(advantage), _ptr(mask), _ptr(ref_logp), float(beta), _ptr(loss),
                        _ptr(g), _ptr(count), _stream(stream)))
    return loss, g, count


def grpo_fused_step(contract, logits, targets, mask, advantage, ref_logp=None, beta=0.0, dlogits=None,
                    entropy=False, stream=None, workspace=None):
    """The GRPO step in one pass over the logits: a dict of dlogits, logp, lse, grad (g), loss and active_count
    (1-element), and entropy if asked; bitwise logp_fwd -> grpo_loss -> logp_bwd(lse, g)."""
    import torch
    dev = logits.device
    T = contract.T
    _need_rows(logits, "logits", contract.T, contract.row_stride or contract.V_padded, contract.V_padded, _BF16)
    _rowwise(contract, targets, mask, advantage=advantage)
    _need(ref_logp, "ref_logp", 4 * T, _F32, optional=True)
    dlogits = _dlogits_out(contract, logits, dlogits)
    out = {"dlogits": dlogits}
    for k in ("logp", "lse", "grad"):
        out[k] = torch.empty(T, dtype=torch.float32, device=dev)
    out["entropy"] = torch.empty(T, dtype=torch.float32, device=dev) if entropy else None
    out["loss"] = torch.empty(1, dtype=torch.float32, device=dev)
    out["active_count"] = torch.empty(1, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(rlk_grpo_fused_workspace_size(contract), 256), dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", rlk_grpo_fused_workspace_size(contract), ("uint8",))
    check(rlk_grpo_fused_step(contract, _ptr(logits), _ptr(targets), _ptr(mask), _ptr(advantage), _ptr(ref_logp),
                              float(beta), _ptr(dlogits), _ptr(out["logp"]), _ptr(out["lse"]), _ptr(out["grad"]),
                              _ptr(out["entropy"]), _ptr(out["loss"]), _ptr(out["active_count"]), _ptr(workspace),
                              _stream(stream)))
    return out


def logp_fwd_bwd(contract, logits, targets, mask, grad, dlogits=None, stream=None, out=None):
    """Fused single pass: (dlogits, logp, lse); each logits row is read from HBM once."""
    import torch
    dev = logits.device
    T = contract.T
    _need_rows(logits, "logits", contract.T, contract.row_stride or contract.V_padded, contract.V_padded, _BF16)
    dlogits = _dlogits_out(contract, logits, dlogits)
    logp, lse = out if out is not None else (torch.empty(T, dtype=torch.float32, device=dev),
                                             torch.empty(T, dtype=torch.float32, device=dev))
    _rowwise(contract, targets, mask, grad=grad, logp=logp, lse=lse)
    ws = workspace_for(contract, dev, stream)
    check(rlk_logp_bwd(contract, _ptr(logits), _ptr(targets), _ptr(mask), None, _ptr(grad), _ptr(dlogits),
                       _ptr(logp), _ptr(lse), _ptr(ws), _stream(stream)))
    return dlogits, logp, lse


def logp_fwd_bwd_entropy(contract, logits, targets, mask, grad, dlogits=None, stream=None):
    """Fused single pass plus each row's entropy: (dlogits, logp, lse, entropy)."""
    import torch
    dev = logits.device
    T = contract.T
    _need_rows(logits, "logits", contract.T, contract.row_stride or contract.V_padded, contract.V_padded, _BF16)
    _rowwise(contract, targets, mask, grad=grad)
    dlogits = _dlogits_out(contract, logits, dlogits)
    logp, lse, ent = (torch.empty(T, dtype=torch.float32, device=dev) for _ in range(3))
    ws = workspace_for(contract, dev, stream)
    check(rlk_logp_fwd_bwd_entropy(contract, _ptr(logits), _ptr(targets), _ptr(mask), _ptr(grad), _ptr(dlogits),
                                   _ptr(logp), _ptr(lse), _ptr(ent), _ptr(ws), _stream(stream)))
    return dlogits, logp, lse, ent


def logp_fwd_bwd_host(contract, logits, targets, mask, grad, device, chunk_rows=8192, dlogits=None,
                      staging=None):
    """Fused forward+backward of inputs in (pinned) host memory.

    Row chunks of ``logits`` (host, [T, row_stride] bf16/int16) are copied to
    the device on a copy stream while the previous chunk computes on the
    current stream; rows are independent, so the results are bitwise those of
    one call on the whole batch.  ``targets`` int64 [T], ``mask`` uint8 [T]
    (None in ignore_index mode) and ``grad`` float32 [T] are host tensors too.
    ``staging`` (device, like ``logits``) and ``dlogits`` (device) may be
    passed to reuse allocations.  Returns (dlogits on the device, logp and LSE
    in pinned host memory); the copies back are enqueued on the current
    stream, so synchronise it before reading them.  With contract.validate the
    call synchronises and checks every chunk's status.
    """
    import torch
    T = contract.T
    stride = contract.row_stride or contract.V_padded
    if logits.dim() != 2 or logits.shape[0] < T or logits.shape[1] < stride:
        raise ValueError(f"logits must be [T >= {T}, row_stride >= {stride}], not {list(logits.shape)}")
    for name, t in (("targets", targets), ("mask", mask), ("grad", grad)):
        if t is not None and t.numel() < T:
            raise ValueError(f"{name} must hold T = {T} values")
    comp = torch.cuda.current_stream(device)
    copy = torch.cuda.Stream(device)
    d_logits = staging if staging is not None else torch.empty(logits.shape, dtype=logits.dtype, device=device)
    d_dl = dlogits if dlogits is not None else torch.empty(logits.shape, dtype=logits.dtype, device=device)
    d_tgt = torch.empty(T, dtype=torch.int64, device=device)
    d_mask = torch.empty(T, dtype=torch.uint8, device=device) if mask is not None else None
    d_g = torch.empty(T, dtype=torch.float32, device=device)
    d_logp = torch.empty(T, dtype=torch.float32, device=device)
    d_lse = torch.empty(T, dtype=torch.float32, device=device)
    h_logp = torch.empty(T, dtype=torch.float32, pin_memory=True)
    h_lse = torch.empty(T, dtype=torch.float32, pin_memory=True)
    starts = list(range(0, T, chunk_rows))
    ws = torch.zeros(max(len(starts), 1) * 256, dtype=torch.uint8, device=device)  # a status word per chunk
    copy.wait_stream(comp)  # the buffers above exist before the copy stream writes them
    with torch.cuda.stream(copy):
        d_tgt.copy_(targets, non_blocking=True)
        if mask is not None:
            d_mask.copy_(mask, non_blocking=True)
        d_g.copy_(grad, non_blocking=True)
    for i, r0 in enumerate(starts):
        r1 = min(T, r0 + chunk_rows)
        with torch.cuda.stream(copy):
            d_logits[r0:r1].copy_(logits[r0:r1], non_blocking=True)
            landed = torch.cuda.Event()
            landed.record(copy)
        comp.wait_event(landed)
        c = contract.replace(T=r1 - r0, validate=0)
        check(rlk_logp_bwd(c, d_logits[r0].data_ptr(), d_tgt[r0:].data_ptr(),
                           None if d_mask is None else d_mask[r0:].data_ptr(), None, d_g[r0:].data_ptr(),
                           d_dl[r0].data_ptr(), d_logp[r0:].data_ptr(), d_lse[r0:].data_ptr(),
                           ws[i * 256:].data_ptr(), comp.cuda_stream))
    comp.wait_stream(copy)
    h_logp.copy_(d_logp, non_blocking=True)
    h_lse.copy_(d_lse, non_blocking=True)
    if contract.validate:
        for i in range(len(starts)):
            check(rlk_logp_workspace_status(ws[i * 256:].data_ptr(), comp.cuda_stream))
    return d_dl, h_logp, h_lse


def logp_fused_lmhead(contract, hidden, weight, targets, mask=None, grad=None, stream=None, workspace=None,
                      dweight_dtype="bf16"):
    """Fused lm_head on BF16 hidden [T, H] and weight [V_padded, H] (GPU tensors).

    Forward only: returns (logp, lse).  With ``grad`` (FP32 [T]): returns
    (logp, lse, dhidden [T, H] BF16, dweight [V_padded, H]); ``dweight_dtype``
    "bf16" (default), "f32", or "both" (then dweight is a (f32, bf16) pair).
    """
    import torch
    dev = hidden.device
    H = _lmhead_operands(contract, hidden, weight)
    T = contract.T
    _rowwise(contract, targets, mask)
    _need(grad, "grad", 4 * T, _F32, optional=True)
    logp = torch.empty(T, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    dh = dwf = dwb = None
    if grad is not None:
        if dweight_dtype not in ("bf16", "f32", "both"):
            raise ValueError("dweight_dtype must be bf16, f32 or both")
        dh = torch.empty_like(hidden)
        if dweight_dtype in ("f32", "both"):
            dwf = torch.empty(weight.shape, dtype=torch.float32, device=dev)
        if dweight_dtype in ("bf16", "both"):
            dwb = torch.empty_like(weight)
    ws = _lmhead_workspace(contract, H, dev, workspace)
    check(rlk_logp_fused_lmhead(contract, _ptr(hidden), H, _ptr(weight), _ptr(targets), _ptr(mask), _ptr(grad),
                                _ptr(logp), _ptr(lse), _ptr(dh), _ptr(dwf), _ptr(dwb), _ptr(ws), _stream(stream)))
    if grad is None:
        return logp, lse
    dw = {"bf16": dwb, "f32": dwf, "both": (dwf, dwb)}[dweight_dtype]
    return logp, lse, dh, dw


def logp_fused_lmhead_bwd(contract, hidden, weight, targets, mask, lse, grad, stream=None, workspace=None,
                          dweight_dtype="bf16"):
    """(dhidden [T, H] BF16, dweight [V_padded, H]) from the forward's LSE; ``dweight_dtype`` as for
    logp_fused_lmhead."""
    import torch
    dev = hidden.device
    H = _lmhead_operands(contract, hidden, weight)
    _rowwise(contract, targets, mask, lse=lse, grad=grad)
    if dweight_dtype not in ("bf16", "f32", "both"):
        raise ValueError("dweight_dtype must be bf16, f32 or both")
    dh = torch.empty_like(hidden)
    dwf = torch.empty(weight.shape, dtype=torch.float32, device=dev) if dweight_dtype in ("f32", "both") else None
    dwb = torch.empty_like(weight) if dweight_dtype in ("bf16", "both") else None
    ws = _lmhead_workspace(contract, H, dev, workspace)
    check(rlk_logp_fused_lmhead_bwd(contract, _ptr(hidden), H, _ptr(weight), _ptr(targets), _ptr(mask), _ptr(lse),
                                    _ptr(grad), _ptr(dh), _ptr(dwf), _ptr(dwb), _ptr(ws), _stream(stream)))
    return dh, {"bf16": dwb, "f32": dwf, "both": (dwf, dwb)}[dweight_dtype]


def logp_fused_lmhead_keep(contract, hidden, weight, targets, mask=None, stream=None, workspace=None):
    """(logp, lse, logits): the fused lm_head forward that also keeps its FP32 logits [T, V_padded] for
    logp_fused_lmhead_bwd_kept (T * V_padded * 4 bytes)."""
    import torch
    dev = hidden.device
    H = _lmhead_operands(contract, hidden, weight)
    T = contract.T
    _rowwise(contract, targets, mask)
    logp = torch.empty(T, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    logits = torch.empty((T, weight.shape[0]), dtype=torch.float32, device=dev)
    ws = _lmhead_workspace(contract, H, dev, workspace)
    check(rlk_logp_fused_lmhead_keep(contract, _ptr(hidden), H, _ptr(weight), _ptr(targets), _ptr(mask), _ptr(logp),
                                     _ptr(lse), _ptr(logits), _ptr(ws), _stream(stream)))
    return logp, lse, logits


def logp_fused_lmhead_bwd_kept(contract, hidden, weight, targets, mask, lse, logits, grad, stream=None, workspace=None,
                               dweight_dtype="bf16"):
    """(dhidden, dweight) from the logits and LSE of logp_fused_lmhead_keep; bitwise logp_fused_lmhead_bwd's."""
    import torch
    dev = hidden.device
    H = _lmhead_operands(contract, hidden, weight)
    _rowwise(contract, targets, mask, lse=lse, grad=grad)
    _need(logits, "logits", 4 * contract.T * contract.V_padded, _F32)
    if dweight_dtype not in ("bf16", "f32", "both"):
        raise ValueError("dweight_dtype must be bf16, f32 or both")
    dh = torch.empty_like(hidden)
    dwf = torch.empty(weight.shape, dtype=torch.float32, device=dev) if dweight_dtype in ("f32", "both") else None
    dwb = torch.empty_like(weight) if dweight_dtype in ("bf16", "both") else None
    ws = _lmhead_workspace(contract, H, dev, workspace)
    check(rlk_logp_fused_lmhead_bwd_kept(contract, _ptr(hidden), H, _ptr(weight), _ptr(targets), _ptr(mask),
                                         _ptr(lse), _ptr(logits), _ptr(grad), _ptr(dh), _ptr(dwf), _ptr(dwb), _ptr(ws),
                                         _stream(stream)))
    return dh, {"bf16": dwb, "f32": dwf, "both": (dwf, dwb)}[dweight_dtype]


# ------------------------------------------------------------------ vocabulary shards (one rank's calls)

def shard_workspace(contract, device):
    import torch
    n = rlk_logp_shard_workspace_size(contract)
    if n == 0:
        check(rlk_logp_check_shard_contract(contract, 0) or RLK_ERR_INVALID_ARG)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def shard_fwd(contract, shard, logits_shard, targets, mask=None, stream=None, workspace=None):
    """(partials [T, num_tiles/tp, 2], target_logit [T]) of one vocabulary shard (GPU tensors)."""
    import torch
    dev = logits_shard.device
    T = contract.T
    vs = contract.V_padded // contract.virtual_tp
    _need_rows(logits_shard, "logits_shard", T, contract.row_stride or vs, vs, _BF16)
    _rowwise(contract, targets, mask)
    part = torch.empty((T, contract.num_tiles // contract.virtual_tp, 2), dtype=torch.float32, device=dev)
    xt = torch.empty(T, dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else shard_workspace(contract, dev)
    check(rlk_logp_shard_fwd(contract, shard, _ptr(logits_shard), _ptr(targets), _ptr(mask), _ptr(part), _ptr(xt),
                             _ptr(ws), _stream(stream)))
    return part, xt


def fold_gathered(contract, gathered_partials, gathered_target_logit, targets, mask=None, stream=None,
                  workspace=None):
    """(logp, lse) from every shard's partials [tp, T, num_tiles/tp, 2] and target logits [tp, T]."""
    import torch
    dev = gathered_partials.device
    T = contract.T
    _need(gathered_partials, "gathered_partials", 8 * T * contract.num_tiles, _F32)
    _need(gathered_target_logit, "gathered_target_logit", 4 * T * contract.virtual_tp, _F32)
    _rowwise(contract, targets, mask)
    logp = torch.empty(T, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else shard_workspace(contract, dev)
    check(rlk_logp_fold(contract, _ptr(gathered_partials), _ptr(gathered_target_logit), _ptr(targets), _ptr(mask),
                        _ptr(logp), _ptr(lse), _ptr(ws), _stream(stream)))
    return logp, lse


def shard_bwd(contract, shard, logits_shard, targets, mask, lse, grad, dlogits=None, stream=None, workspace=None):
    """BF16 dlogits of one vocabulary shard [T, row_stride] (columns [0, V_padded/tp) written)."""
    dev = logits_shard.device
    vs = contract.V_padded // contract.virtual_tp
    stride = contract.row_stride or vs
    _need_rows(logits_shard, "logits_shard", contract.T, stride, vs, _BF16)
    _rowwise(contract, targets, mask, lse=lse, grad=grad)
    dlogits = _dlogits_out(contract, logits_shard, dlogits, stride=stride, width=vs)
    ws = workspace if workspace is not None else shard_workspace(contract, dev)
    check(rlk_logp_shard_bwd(contract, shard, _ptr(logits_shard), _ptr(targets), _ptr(mask), _ptr(lse), _ptr(grad),
                             _ptr(dlogits), _ptr(ws), _stream(stream)))
    return dlogits


# ------------------------------------------------------------------ FP8 projections

_torch = None
_HERE = contextlib.nullcontext()


def _t():
    """torch, imported at the first call that marshals tensors."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _raw_stream(t, stream):
    """The stream's handle: the given one's, or the current one's of the tensor's device."""
    return stream.cuda_stream if stream is not None else _t()._C._cuda_getCurrentRawStream(t.device.index)


def _allocating(stream):
    """Within it, new tensors come from the memory of the given stream (None: the current one): the current stream's
    may still be in use by work that is queued there."""
    return _HERE if stream is None else _t().cuda.stream(stream)


def _used_here(stream, *tensors):
    """Tells the allocator that the current stream, too, uses these tensors of the given stream's memory, so that it is
    not handed out again before the work queued here by then is done."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(_t().cuda.current_stream(t.device))


def _matrix(t, name, dtypes):
    """A 2-D CUDA tensor of one of ``dtypes`` with contiguous rows: (rows, columns, row stride in elements)."""
    shape = t.shape
    if len(shape) != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor, not {list(shape)} on {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d)[6:] for d in dtypes)}, not {str(t.dtype)[6:]}")
    rows, cols = shape
    stride, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name}'s rows must be contiguous: its strides are {list(t.stride())}")
    if rows <= 1:
        return rows, cols, max(cols, stride)
    if stride < cols:
        raise ValueError(f"{name}'s rows overlap: its strides are {list(t.stride())}")
    return rows, cols, stride


def _padded(stride, rows, cols, piece):
    """A row stride; that of a single row, which may come with any, in whole 16-byte pieces."""
    return -(-cols // piece) * piece if rows <= 1 else stride


def _code_stride(cols):
    """Bytes from one row of codes to the next: whole 16-byte pieces.

    Long rows that need padding at all start on 128-byte lines, which each of their 128-byte groups then fills
    (8000 x 3517: written in 22.6 us against 23.4; as a weight of 37 tokens read in 40.5 us against 41.8).
    """
    return -(-cols // 128) * 128 if cols % 16 and cols >= 2048 else -(-cols // 16) * 16


def _codes(x, rows, cols):
    """An E4M3 [rows, cols] tensor whose rows start on 16-byte boundaries, and its row stride."""
    stride = _code_stride(cols)
    return _new(x, rows, cols, _t().float8_e4m3fn, stride), stride


def _new(x, rows, cols, dtype, stride=None):
    """A [rows, cols] tensor on x's device, contiguous or with rows `stride` apart (empty_strided takes half the host
    time of new_empty, and a slice of a wider tensor several times that)."""
    return _t().empty_strided((rows, cols), (cols if stride is None else stride, 1), dtype=dtype, device=x.device)


def _quantize(x, block_rows, rowwise, transposed, stream):
    torch = _t()
    R, C, stride = _matrix(x, "x", (torch.bfloat16, torch.float32))
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    q = scale = qt = scale_t = None
    ldq = ldt = 0
    gr, gc = -(-R // 128), -(-C // 128)
    with _allocating(stream):
        if rowwise:
            q, ldq = _codes(x, R, C)
            scale = _new(x, gc, R if block_rows == 1 else gr, torch.float32)
        if transposed:
            qt, ldt = _codes(x, C, R)
            scale_t = _new(x, gr, C if block_rows == 1 else gc, torch.float32)
    st = rlk_fp8_quantize(R, C, x.data_ptr(), RLK_F32 if x.dtype is torch.float32 else RLK_BF16, stride, block_rows,
                          _ptr(q), ldq, _ptr(scale), _ptr(qt), ldt, _ptr(scale_t), _raw_stream(x, stream))
    if st:
        check(st)
    _used_here(stream, q, scale, qt, scale_t)
    return q, scale, qt, scale_t


def _type(t):
    return RLK_F32 if t.dtype is _t().float32 else RLK_BF16


def _matrices(t, name, dtypes):
    """A 3-D CUDA tensor of matrices with contiguous rows: (count, rows, columns, row stride, matrix stride)."""
    shape = t.shape
    if len(shape) != 3 or not t.is_cuda:
        raise ValueError(f"{name} must be a 3-D CUDA tensor, not {list(shape)} on {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d)[6:] for d in dtypes)}, not {str(t.dtype)[6:]}")
    count, rows, cols = shape
    between, stride, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name}'s rows must be contiguous: its strides are {list(t.stride())}")
    if rows <= 1:
        stride = max(cols, stride)
    elif stride < cols:
        raise ValueError(f"{name}'s rows overlap: its strides are {list(t.stride())}")
    if count > 1 and between < (rows - 1) * stride + cols:
        raise ValueError(f"{name}'s matrices overlap: its strides are {list(t.stride())}")
    return count, rows, cols, stride, between


def _batch_codes(x, count, rows, cols):
    """E4M3 matrices whose rows start on 16-byte boundaries, and their row stride."""
    stride = -(-cols // 16) * 16
    return _t().empty_strided((count, rows, cols), (rows * stride, stride, 1), dtype=_t().float8_e4m3fn,
                              device=x.device), stride


def _quantize_batch(x, block_rows, rowwise, transposed, stream):
    torch = _t()
    G, R, C, stride, between = _matrices(x, "x", (torch.bfloat16, torch.float32))
    if block_rows != 128:
        raise ValueError("several matrices are quantised with block_rows 128")
    q = scale = qt = scale_t = None
    ldq = ldt = 0
    gr, gc = -(-R // 128), -(-C // 128)
    with _allocating(stream):
        if rowwise:
            q, ldq = _batch_codes(x, G, R, C)
            scale = torch.empty((G, gc, gr), dtype=torch.float32, device=x.device)
        if transposed:
            qt, ldt = _batch_codes(x, G, C, R)
            scale_t = torch.empty((G, gr, gc), dtype=torch.float32, device=x.device)
    st = rlk_fp8_quantize_batch(G, R, C, x.data_ptr(), _type(x), stride, between, _ptr(q), ldq, R * ldq, _ptr(scale),
                                _ptr(qt), ldt, C * ldt, _ptr(scale_t), _raw_stream(x, stream))
    if st:
        check(st)
    _used_here(stream, q, scale, qt, scale_t)
    return q, scale, qt, scale_t


def fp8_quantize(x, block_rows=1, transpose=False, stream=None):
    """(q, scale) of a BF16 or FP32 matrix [R, C]: E4M3 values and one FP32 scale for each 1 x 128 group of a row
    (block_rows 1) or each 128 x 128 block (128), so that x ~ q * scale.

    ``scale`` is group-major: [ceil(C / 128), R] or [ceil(C / 128), ceil(R / 128)].  With ``transpose`` the result
    is that of x's transpose [C, R].  q's rows start on 16-byte boundaries (a view where C is not a multiple of 16).
    Several matrices [G, R, C] (experts' weights, block_rows 128) give q [G, R, C] and scale [G, ...], each its own.
    """
    q, scale, qt, scale_t = (_quantize if x.dim() != 3 else _quantize_batch)(x, block_rows, not transpose, transpose, stream)
    return (qt, scale_t) if transpose else (q, scale)


def fp8_quantize_both(x, block_rows=1, stream=None):
    """(q, scale, qt, scale_t): fp8_quantize of x and of its transpose from one read of x."""
    return (_quantize if x.dim() != 3 else _quantize_batch)(x, block_rows, True, True, stream)


def _ends(ends, like):
    """The groups that int32 ends [G] describe: (G, pointer)."""
    if ends.dtype is not _t().int32 or ends.dim() != 1 or not ends.is_contiguous() or not ends.is_cuda:
        raise TypeError(f"ends must be a contiguous int32 CUDA tensor [G], not {str(ends.dtype)[6:]} "
                        f"{list(ends.shape)} on {ends.device}")
    if not 1 <= ends.shape[0] <= 1024:
        raise ValueError(f"ends has {ends.shape[0]} groups; 1 to 1024 are taken")
    return ends.shape[0], ends.data_ptr()


def group_tiles(groups, rows):
    """Groups of 128 rows that fp8_quantize_grouped leaves room for: what any division of `rows` can ask for."""
    return rows // 128 + min(groups, rows)


def fp8_quantize_grouped(x, ends, rowwise=True, transpose=True, stream=None):
    """(q, scale, qt, scale_t): fp8_quantize_both of rows that belong to groups, group e ending at row ends[e].

    The transpose's groups of 128 start anew with each group of rows, padded with zeros to whole 128s: qt is
    [C, 128 * group_tiles(G, R)] and scale_t [group_tiles(G, R), C], of which the first ceil(rows / 128) of each group,
    one group after the other, are written.  Rows of q and scale behind the last group are not written.  ``rowwise`` or
    ``transpose`` False leaves the one pair out (None).
    """
    torch = _t()
    R, C, stride = _matrix(x, "x", (torch.bfloat16, torch.float32))
    G, pe = _ends(ends, x)
    q = scale = qt = scale_t = None
    ldq = ldt = 0
    tiles = group_tiles(G, R)
    with _allocating(stream):
        if rowwise:
            q, ldq = _codes(x, R, C)
            scale = _new(x, -(-C // 128), R, torch.float32)
        if transpose:
            qt, ldt = _codes(x, C, 128 * tiles)
            scale_t = _new(x, tiles, C, torch.float32)
    st = rlk_fp8_quantize_grouped(G, R, C, pe, x.data_ptr(), _type(x), stride, _ptr(q), ldq, _ptr(scale), _ptr(qt),
                                  ldt, _ptr(scale_t), _raw_stream(x, stream))
    if st:
        check(st)
    _used_here(stream, q, scale, qt, scale_t)
    return q, scale, qt, scale_t


_fp8_workspaces = {}


def _fp8_workspace(t, raw, stream):
    """The status word of a device and stream (``raw``: its handle): zeroed there once, only ever set by a call, and
    cleared where fp8_matmul has reported it."""
    key = (t.device.index, raw)
    ws = _fp8_workspaces.get(key)
    if ws is None:
        torch = _t()
        with _allocating(stream):
            ws = torch.zeros(RLK_FP8_WORKSPACE, dtype=torch.uint8, device=t.device)
            if torch.cuda.is_current_stream_capturing():
                return ws  # the graph's memory, not to be kept beyond it
        _fp8_workspaces[key] = ws
    return ws


def _scale_operand(s, name, groups, n):
    if s.dtype is not _t().float32 or s.shape != (groups, n) or not s.is_contiguous() or not s.is_cuda:
        raise ValueError(f"{name} must be a contiguous FP32 CUDA tensor [{groups}, {n}], not "
                         f"{str(s.dtype)[6:]} {list(s.shape)}")
    return s.data_ptr()


def fp8_matmul(a, a_scale, b, b_scale, b_block_rows=128, out_dtype=None, out=None, accumulate=False, workspace=None,
               validate=False, stream=None):
    """a @ b^T [M, N] of E4M3 operands a [M, K] and b [N, K] with the scales fp8_quantize gives them.

    ``a_scale`` is [ceil(K / 128), M]; ``b_scale`` [ceil(K / 128), N] (b_block_rows 1) or [ceil(K / 128),
    ceil(N / 128)] (128).  The result is BF16 (or FP32 with ``out_dtype`` torch.float32), in ``out`` if given (its rows
    may be strided); ``accumulate`` adds the product to an FP32 ``out``.  K = 0 is an empty sum: zeros, or ``out`` as it
    was.  ``validate`` synchronises and raises if a device-side wait expired, in this call or in one before it
    on this stream that was not validated, and clears the record (in a ``workspace`` of the caller's it stays).
    """
    torch = _t()
    codes = (torch.float8_e4m3fn, torch.uint8)  # E4M3 values, or their codes as bytes
    M, K, lda = _matrix(a, "a", codes)
    N, Kb, ldb = _matrix(b, "b", codes)
    if Kb != K:
        raise ValueError(f"a is [{M}, {K}] and b [{N}, {Kb}]: their rows must have one length")
    if b_block_rows not in (1, 128):
        raise ValueError("b_block_rows must be 1 or 128")
    groups = -(-K // 128)
    pa = _scale_operand(a_scale, "a_scale", groups, M)
    pb = _scale_operand(b_scale, "b_scale", groups, N if b_block_rows == 1 else -(-N // 128))
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out_dtype = out_dtype or torch.bfloat16
        if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
            raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
        with _allocating(stream):
            out = _new(a, M, N, out_dtype)
        _used_here(stream, out)
        ldc = N
    else:
        rows, cols, ldc = _matrix(out, "out", (torch.bfloat16, torch.float32))
        if (rows, cols) != (M, N) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out is {str(out.dtype)[6:]} {list(out.shape)}; the product is [{M}, {N}]")
    if K == 0:
        if accumulate and out.dtype is not torch.float32:
            raise TypeError("accumulate needs an FP32 out")
        if not accumulate:
            with _allocating(stream):
                out.zero_()
        return out
    st = _raw_stream(a, stream)
    given = workspace is not None
    if given:
        _need(workspace, "workspace", RLK_FP8_WORKSPACE, ("uint8",))
    else:
        workspace = _fp8_workspace(a, st, stream)
    status = rlk_fp8_matmul(M, N, K, a.data_ptr(), _padded(lda, M, K, 16), pa, b.data_ptr(), _padded(ldb, N, K, 16),
                            pb, b_block_rows, out.data_ptr(), RLK_F32 if out.dtype is torch.float32 else RLK_BF16, ldc,
                            int(accumulate), workspace.data_ptr(), st)
    if status:
        check(status)
    if validate:
        status = rlk_logp_workspace_status(workspace.data_ptr(), st)
        if status and not given:
            with _allocating(stream):
                workspace.zero_()  # reported once, not with every later call
        check(status)
    return out


def _validated(validate, workspace, given, st, stream):
    """Reports an expired wait of this call or of ones before it on its stream, once where the record is ours."""
    if not validate:
        return
    status = rlk_logp_workspace_status(workspace.data_ptr(), st)
    if status and not given:
        with _allocating(stream):
            workspace.zero_()
    check(status)


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(str(a) for a in ACTIVATIONS)}, not {name!r}")
    return ACTIVATIONS[name]


def _layer(a, a_scale, b, b_scale, ends, bias, activation, gated, residual, keep, out_dtype, out, workspace, validate,
           stream):
    torch = _t()
    codes = (torch.float8_e4m3fn, torch.uint8)
    both = (torch.bfloat16, torch.float32)
    M, K, lda = _matrix(a, "a", codes)
    if ends is None:
        rows, Kb, ldb = _matrix(b, "b", codes)
        lead, group = (), 0
    else:
        G, pe = _ends(ends, a)
        Gb, rows, Kb, ldb, group = _matrices(b, "b", codes)
        if Gb != G:
            raise ValueError(f"ends has {G} groups and b {Gb}")
        lead = (G,)
    if Kb != K or K < 1:
        raise ValueError(f"a is [{M}, {K}] and b {list(b.shape)}: their rows must have one length, at least 1")
    act = _activation(activation)
    if gated and rows % 128:
        raise ValueError(f"a gated layer's b holds two halves of a multiple of 64 rows, not {rows} rows")
    N = rows // 2 if gated else rows
    groups = -(-K // 128)
    pa = _scale_operand(a_scale, "a_scale", groups, M)
    want = lead + (groups, -(-rows // 128))
    if b_scale.dtype is not torch.float32 or b_scale.shape != want or not b_scale.is_contiguous() or \
            not b_scale.is_cuda:
        raise ValueError(f"b_scale must be a contiguous FP32 CUDA tensor {list(want)}, not "
                         f"{str(b_scale.dtype)[6:]} {list(b_scale.shape)}")
    e = Fp8Epilogue(activation=act, gated=int(bool(gated)))
    if bias is not None:
        if bias.shape != lead + (rows,):
            raise ValueError(f"bias is {list(bias.shape)}; the layer's is {list(lead + (rows,))}")
        e.bias, e.bias_type = _vector(bias, "bias", bias.numel(), both), _type(bias)
    if residual is not None:
        r, c, e.residual_stride = _matrix(residual, "residual", both)
        if (r, c) != (M, N):
            raise ValueError(f"residual is {list(residual.shape)}; the result is [{M}, {N}]")
        e.residual, e.residual_type = residual.data_ptr(), _type(residual)
    z = None
    fresh = out is None
    if fresh:
        out_dtype = out_dtype or torch.bfloat16
        if out_dtype not in both:
            raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    else:
        r, c, ldc = _matrix(out, "out", both)
        if (r, c) != (M, N) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out is {str(out.dtype)[6:]} {list(out.shape)}; the result is [{M}, {N}]")
    with _allocating(stream):
        if fresh:
            out, ldc = _new(a, M, N, out_dtype), N
        if keep:  # rows on 16-byte boundaries, for the backward's loads
            e.z_stride = -(-rows // 8) * 8
            z = _new(a, M, rows, torch.bfloat16, e.z_stride)
            e.z = z.data_ptr()
    _used_here(stream, out if fresh else None, z)
    st = _raw_stream(a, stream)
    given = workspace is not None
    if given:
        _need(workspace, "workspace", RLK_FP8_WORKSPACE, ("uint8",))
    else:
        workspace = _fp8_workspace(a, st, stream)
    lda, ldb = _padded(lda, M, K, 16), _padded(ldb, rows, K, 16)
    if ends is None:
        status = rlk_fp8_matmul_act(M, N, K, a.data_ptr(), lda, pa, b.data_ptr(), ldb, b_scale.data_ptr(), e,
                                    out.data_ptr(), _type(out), ldc, workspace.data_ptr(), st)
    else:
        status = rlk_fp8_grouped_matmul(G, M, N, K, pe, a.data_ptr(), lda, pa, b.data_ptr(), ldb, group,
                                        b_scale.data_ptr(), e, out.data_ptr(), _type(out), ldc, int(fresh),
                                        workspace.data_ptr(), st)
    if status:
        check(status)
    _validated(validate, workspace, given, st, stream)
    return (out, z) if keep else out


def fp8_matmul_act(a, a_scale, b, b_scale, bias=None, activation=None, gated=False, residual=None, keep=False,
                   out_dtype=None, out=None, workspace=None, validate=False, stream=None):
    """act(a @ b^T + bias) + residual [M, N] of E4M3 operands: fp8_matmul (b in 128 x 128 blocks, K at least 1) with a
    layer's epilogue, all in FP32 and rounded once.

    ``activation`` is None, "relu", "silu", "gelu" or "gelu_tanh".  With ``gated`` b holds N rows of the gate, then N
    more (N a multiple of 64), and the result is act(gate) * other + residual.  ``bias`` [rows of b] and ``residual``
    [M, N] (rows may be strided; ``out`` itself is allowed) are BF16 or FP32.  With ``keep`` the result is (out, z), z
    the pre-activation in BF16 as fp8_act_grad needs it.  ``out_dtype``, ``out``, ``workspace``, ``validate``: as
    fp8_matmul's.
    """
    return _layer(a, a_scale, b, b_scale, None, bias, activation, gated, residual, keep, out_dtype, out, workspace,
                  validate, stream)


def fp8_grouped_matmul(a, a_scale, b, b_scale, ends, bias=None, activation=None, gated=False, keep=False,
                       out_dtype=None, out=None, workspace=None, validate=False, stream=None):
    """fp8_matmul_act for rows that belong to groups (a mixture's experts): group e is rows [ends[e - 1], ends[e]) of a.

    ``ends`` is int32 [G] on the GPU (nothing is read back), b [G, rows, K], b_scale [G, ceil(K / 128), ceil(rows / 128)]
    and ``bias`` [G, rows], as fp8_quantize gives them for [G, rows, K] weights.  Rows behind the last group are zero, or
    in an ``out`` of the caller's as they were (those of z are undefined).  A group without rows is allowed and costs
    nothing.
    """
    return _layer(a, a_scale, b, b_scale, ends, bias, activation, gated, None, keep, out_dtype, out, workspace,
                  validate, stream)


def fp8_grouped_dweight(at, at_scale, bt, bt_scale, ends, rows, out_dtype=None, out=None, accumulate=False,
                        workspace=None, validate=False, stream=None):
    """[G, M, N]: for each group, its columns of ``at`` [M, ...] times those of ``bt`` [N, ...] transposed: the weight
    gradients dy_e^T x_e, with (at, at_scale) and (bt, bt_scale) the qt and scale_t that fp8_quantize_grouped (or
    fp8_act_grad) gives for dy and x of ``rows`` rows.

    BF16 or FP32 (``out_dtype``), in ``out`` if given; ``accumulate`` adds to an FP32 ``out``.  Zero (or unchanged) for a
    group without rows.
    """
    torch = _t()
    codes = (torch.float8_e4m3fn, torch.uint8)
    both = (torch.bfloat16, torch.float32)
    G, pe = _ends(ends, at)
    tiles = group_tiles(G, rows)
    M, deep, lda = _matrix(at, "at", codes)
    N, deep_b, ldb = _matrix(bt, "bt", codes)
    if deep != 128 * tiles or deep_b != deep:
        raise ValueError(f"at and bt are {list(at.shape)} and {list(bt.shape)}; {G} groups of {rows} rows have "
                         f"{128 * tiles} columns")
    pa = _scale_operand(at_scale, "at_scale", tiles, M)
    pb = _scale_operand(bt_scale, "bt_scale", tiles, N)
    fresh = out is None
    if fresh:
        if accumulate:
            raise ValueError("accumulate needs out")
        out_dtype = out_dtype or torch.bfloat16
        if out_dtype not in both:
            raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
        with _allocating(stream):
            out = torch.empty((G, M, N), dtype=out_dtype, device=at.device)
        _used_here(stream, out)
        ldc, between = N, M * N
    else:
        Go, Mo, No, ldc, between = _matrices(out, "out", both)
        if (Go, Mo, No) != (G, M, N) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out is {str(out.dtype)[6:]} {list(out.shape)}; the result is [{G}, {M}, {N}]")
    if rows == 0:
        if not accumulate:
            with _allocating(stream):
                out.zero_()
        return out
    st = _raw_stream(at, stream)
    given = workspace is not None
    if given:
        _need(workspace, "workspace", RLK_FP8_WORKSPACE, ("uint8",))
    else:
        workspace = _fp8_workspace(at, st, stream)
    status = rlk_fp8_grouped_dweight(G, rows, M, N, pe, at.data_ptr(), _padded(lda, M, deep, 16), pa, bt.data_ptr(),
                                     _padded(ldb, N, deep, 16), pb, out.data_ptr(), _type(out), ldc, between,
                                     int(accumulate), workspace.data_ptr(), st)
    if status:
        check(status)
    _validated(validate, workspace, given, st, stream)
    return out


def fp8_act_grad(dy, z=None, activation=None, gated=False, ends=None, rowwise=True, transpose=True, bias_dtype=None,
                 stream=None):
    """(q, scale, qt, scale_t, dbias): the backward of fp8_matmul_act's epilogue, quantised as the products that follow
    need it, in one pass.

    From dy [R, N] (BF16 or FP32) and the kept z, in FP32: dz = dy * act'(z), or (gated) the gate's half
    dy * z_other * act'(z_gate), then the other half dy * act(z_gate).  q, scale, qt, scale_t are fp8_quantize_both of dz,
    with ``ends`` fp8_quantize_grouped's.  ``bias_dtype`` asks for dbias, the sum of dz over the rows ([G, ...] with
    ``ends``).  What is not asked for is None.  z may be None without an activation and a gate.  No rows (R = 0) give
    empty codes and a zero dbias.
    """
    torch = _t()
    both = (torch.bfloat16, torch.float32)
    R, N, stride = _matrix(dy, "dy", both)
    act = _activation(activation)
    wide = 2 * N if gated else N
    pz = ldz = 0
    if act or gated:
        if z is None:
            raise ValueError("an activation or a gate needs z")
        rz, cz, ldz = _matrix(z, "z", (torch.bfloat16,))
        if (rz, cz) != (R, wide):
            raise ValueError(f"z is {list(z.shape)} and dy {list(dy.shape)}: z must be [{R}, {wide}]")
        pz = z.data_ptr()
    G, pe = (0, None) if ends is None else _ends(ends, dy)
    q = scale = qt = scale_t = dbias = ws = None
    ldq = ldt = 0
    tiles = group_tiles(G, R) if G else -(-R // 128)
    with _allocating(stream):
        if rowwise:
            q, ldq = _codes(dy, R, wide)
            scale = _new(dy, -(-wide // 128), R, torch.float32)
        if transpose:
            qt, ldt = _codes(dy, wide, 128 * tiles if G else R)
            scale_t = _new(dy, tiles, wide, torch.float32)
        if bias_dtype is not None:
            if bias_dtype not in both:
                raise TypeError("bias_dtype must be torch.bfloat16 or torch.float32")
            dbias = torch.empty((G, wide) if ends is not None else (wide,), dtype=bias_dtype, device=dy.device)
            ws = torch.empty(max(1, rlk_fp8_act_grad_workspace_size(G, R, N, int(bool(gated)))), dtype=torch.uint8,
                             device=dy.device)
            if R == 0:
                dbias.zero_()
    if R == 0:  # a batch without rows, which the C call refuses
        _used_here(stream, q, scale, qt, scale_t, dbias)
        return q, scale, qt, scale_t, dbias
    st = rlk_fp8_act_grad(G, R, N, pe, dy.data_ptr(), _type(dy), stride, pz or None, ldz, act, int(bool(gated)),
                          _ptr(q), ldq, _ptr(scale), _ptr(qt), ldt, _ptr(scale_t), _ptr(dbias),
                          RLK_F32 if bias_dtype is torch.float32 else RLK_BF16, _ptr(ws), _raw_stream(dy, stream))
    if st:
        check(st)
    _used_here(stream, q, scale, qt, scale_t, dbias)
    return q, scale, qt, scale_t, dbias


class _Places:
    """Pieces of one buffer: codes, scales and partial sums that live and die together (an allocation each costs 3 us of
    host time, ten of them a training step)."""

    def __init__(self):
        self.size = 0

    def take(self, nbytes):
        at = self.size
        self.size = (at + nbytes + 255) & ~255
        return at


class Fp8LayerStep:
    """The forward and the backward of a layer act(x @ weight^T + bias) + residual, dense or (with ``ends``) of rows that
    belong to groups, as autograd's functions call them: the operands' quantisation and the products as
    fp8_quantize_both, fp8_quantize_grouped, fp8_matmul_act, fp8_grouped_matmul, fp8_act_grad, fp8_matmul and
    fp8_grouped_dweight make them, with what a pass quantises in one buffer.

    forward gives (y, z, saved): z the pre-activation (None where no derivative needs it) and saved the transposes' codes
    and scales; backward takes them back.
    """

    def __init__(self, x, weight, bias, residual, ends, activation, gated, need_x, need_w, need_b, out_dtype=None):
        torch = _t()
        both = (torch.bfloat16, torch.float32)
        self.out = out_dtype or torch.bfloat16
        if self.out not in both:
            raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
        self.M, self.K, self.sx = _matrix(x, "x", both)
        self.G, self.pe = (0, None) if ends is None else _ends(ends, x)
        if ends is None:
            self.rows, Kw, self.sw = _matrix(weight, "weight", both)
            self.between, lead = 0, ()
        else:
            Gw, self.rows, Kw, self.sw, self.between = _matrices(weight, "weight", both)
            lead = (self.G,)
            if Gw != self.G:
                raise ValueError(f"ends has {self.G} groups and weight {Gw}")
        if Kw != self.K or Kw < 1:
            raise ValueError(f"x is {list(x.shape)} and weight {list(weight.shape)}: their rows must have one length, "
                             "at least 1")
        if gated and self.rows % 128:
            raise ValueError(f"a gated layer's weight holds two halves of a multiple of 64 rows, not {self.rows} rows")
        self.N = self.rows // 2 if gated else self.rows
        self.act, self.gated = _activation(activation), int(bool(gated))
        self.e = Fp8Epilogue(activation=self.act, gated=self.gated)
        self.tb = None if bias is None else bias.dtype
        if bias is not None:
            if bias.shape != lead + (self.rows,):
                raise ValueError(f"bias is {list(bias.shape)}; the layer's is {list(lead + (self.rows,))}")
            self.e.bias, self.e.bias_type = _vector(bias, "bias", bias.numel(), both), _type(bias)
        if residual is not None:
            r, c, self.e.residual_stride = _matrix(residual, "residual", both)
            if (r, c) != (self.M, self.N):
                raise ValueError(f"residual is {list(residual.shape)}; the result is [{self.M}, {self.N}]")
            self.e.residual, self.e.residual_type = residual.data_ptr(), _type(residual)
        self.types = x.dtype, weight.dtype
        self.weight_shape, self.device = weight.shape, x.device
        self.need_x, self.need_w, self.need_b = need_x, need_w, need_b
        count = max(1, self.G)
        self.kg, self.rg = -(-self.K // 128), -(-self.rows // 128)
        self.tiles = group_tiles(self.G, self.M) if self.G else -(-self.M // 128)
        self.ldm = 128 * self.tiles if self.G else _code_stride(self.M)  # of codes along the rows of x
        self.ldk, self.ldr = _code_stride(self.K), _code_stride(self.rows)
        keep = _Places()
        self.xt, self.xts = (keep.take(self.K * self.ldm), keep.take(4 * self.tiles * self.K)) if need_w else (0, 0)
        self.wt, self.wts = (keep.take(count * self.K * self.ldr), keep.take(4 * count * self.rg * self.kg)) if need_x \
            else (0, 0)
        self.kept = keep.size

    def _buffer(self, size):
        return _t().empty((size,), dtype=_t().uint8, device=self.device)

    def forward(self, x, weight):
        torch = _t()
        M, K, rows, G, kg, rg, ldk = self.M, self.K, self.rows, self.G, self.kg, self.rg, self.ldk
        count = max(1, G)
        own = _Places()
        xq, xs = own.take(M * ldk), own.take(4 * kg * M)
        wq, ws = own.take(count * rows * ldk), own.take(4 * count * kg * rg)
        scratch = self._buffer(own.size)
        saved = self._buffer(self.kept) if self.kept else None
        b, k = scratch.data_ptr(), 0 if saved is None else saved.data_ptr()
        st = _raw_stream(x, None)
        xt, xts = (k + self.xt, k + self.xts) if self.need_w else (None, None)
        wt, wts = (k + self.wt, k + self.wts) if self.need_x else (None, None)
        tx, tw = _type(x), _type(weight)
        if G and self.need_w:
            status = rlk_fp8_quantize_grouped(G, M, K, self.pe, x.data_ptr(), tx, self.sx, b + xq, ldk, b + xs, xt,
                                              self.ldm, xts, st)
        else:
            status = rlk_fp8_quantize(M, K, x.data_ptr(), tx, self.sx, 1, b + xq, ldk, b + xs, xt, self.ldm, xts, st)
        if G:
            status = status or rlk_fp8_quantize_batch(G, rows, K, weight.data_ptr(), tw, self.sw, self.between, b + wq,
                                                      ldk, rows * ldk, b + ws, wt, self.ldr, K * self.ldr, wts, st)
        else:
            status = status or rlk_fp8_quantize(rows, K, weight.data_ptr(), tw, self.sw, 128, b + wq, ldk, b + ws, wt,
                                                self.ldr, wts, st)
        if status:
            check(status)
        y, z, e = _new(x, M, self.N, self.out), None, self.e
        if (self.act or self.gated) and (self.need_x or self.need_w or self.need_b):
            e.z_stride = -(-rows // 8) * 8
            z = _new(x, M, rows, torch.bfloat16, e.z_stride)
            e.z = z.data_ptr()
        w = _fp8_workspace(x, st, None).data_ptr()
        if G:
            status = rlk_fp8_grouped_matmul(G, M, self.N, K, self.pe, b + xq, ldk, b + xs, b + wq, ldk, rows * ldk, b + ws,
                                            e, y.data_ptr(), _type(y), self.N, 1, w, st)
        else:
            status = rlk_fp8_matmul_act(M, self.N, K, b + xq, ldk, b + xs, b + wq, ldk, b + ws, e, y.data_ptr(),
                                        _type(y), self.N, w, st)
        if status:
            check(status)
        return y, z, saved

    def backward(self, dy, z, saved, ends):
        """(dx, dweight, dbias), None where none is needed."""
        torch = _t()
        M, K, rows, G, rg, tiles = self.M, self.K, self.rows, self.G, self.rg, self.tiles
        need_x, need_w, need_b = self.need_x, self.need_w, self.need_b
        tx, tw = self.types
        dx = _new(dy, M, K, tx) if need_x else None
        dw = torch.empty(self.weight_shape, dtype=tw, device=dy.device) if need_w else None
        db = torch.empty(self.weight_shape[:-1], dtype=self.tb, device=dy.device) if need_b else None
        if M == 0 or rows == 0:
            for t in (dx, dw, db):
                if t is not None:
                    t.zero_()
            return dx, dw, db
        R, N, sy = _matrix(dy, "dy", (torch.bfloat16, torch.float32))
        if (R, N) != (M, self.N):
            raise ValueError(f"dy is {list(dy.shape)}; the result is [{M}, {self.N}]")
        pe = None if ends is None else ends.data_ptr()
        own = _Places()
        q, s = (own.take(M * self.ldr), own.take(4 * rg * M)) if need_x else (0, 0)
        qt, sq = (own.take(rows * self.ldm), own.take(4 * tiles * rows)) if need_w else (0, 0)
        part = own.take(4 * tiles * rows) if need_b else 0
        scratch = self._buffer(own.size)
        b = scratch.data_ptr()
        q, s = (b + q, b + s) if need_x else (None, None)
        qt, sq = (b + qt, b + sq) if need_w else (None, None)
        st = _raw_stream(dy, None)
        if z is None and not need_b and G:
            status = rlk_fp8_quantize_grouped(G, M, rows, pe, dy.data_ptr(), _type(dy), sy, q, self.ldr, s, qt, self.ldm,
                                              sq, st)
        elif z is None and not need_b:
            status = rlk_fp8_quantize(M, rows, dy.data_ptr(), _type(dy), sy, 1, q, self.ldr, s, qt, self.ldm, sq, st)
        else:
            status = rlk_fp8_act_grad(G, M, N, pe, dy.data_ptr(), _type(dy), sy, _ptr(z), 0 if z is None else z.stride(0),
                                      self.act, self.gated, q, self.ldr, s, qt, self.ldm, sq, _ptr(db),
                                      RLK_F32 if self.tb is torch.float32 else RLK_BF16, b + part if need_b else None, st)
        if status:
            check(status)
        k = 0 if saved is None else saved.data_ptr()
        w = _fp8_workspace(dy, st, None).data_ptr()
        if need_x:
            out, kind = dx.data_ptr(), _type(dx)
            if G:
                status = rlk_fp8_grouped_matmul(G, M, K, rows, pe, q, self.ldr, s, k + self.wt, self.ldr, K * self.ldr,
                                                k + self.wts, None, out, kind, K, 1, w, st)
            else:
                status = rlk_fp8_matmul(M, K, rows, q, self.ldr, s, k + self.wt, self.ldr, k + self.wts, 128, out, kind, K,
                                        0, w, st)
        if need_w and not status:
            out, kind = dw.data_ptr(), _type(dw)
            if G:
                status = rlk_fp8_grouped_dweight(G, M, rows, K, pe, qt, self.ldm, sq, k + self.xt, self.ldm, k + self.xts,
                                                 out, kind, K, rows * K, 0, w, st)
            else:
                status = rlk_fp8_matmul(rows, K, M, qt, self.ldm, sq, k + self.xt, self.ldm, k + self.xts, 1, out, kind, K,
                                        0, w, st)
        if status:
            check(status)
        return dx, dw, db


# ------------------------------------------------------------------ cross entropy over a large vocabulary

def _head_operand(t, name):
    """A BF16 (or its int16 bits) matrix's (rows, columns, row stride)."""
    torch = _t()
    rows, cols, stride = _matrix(t, name, (torch.bfloat16, torch.int16, torch.uint16))
    return rows, cols, _padded(stride, rows, cols, 8)


def linear_ce_contract(hidden, weight, mask=None, ignore_index=-100, reduction=REDUCE_NONE, label_smoothing=0.0,
                       z_loss=0.0, softcap=0.0, piece=0, validate=0, wait_timeout_ns=0):
    """The contract of linear_ce_fwd and linear_ce_bwd for these operands: hidden [T, H] and weight [V, H], BF16,
    rows on 16-byte boundaries.  The gradients have rows of whole 16-byte pieces."""
    T, H, hs = _head_operand(hidden, "hidden")
    V, Hw, wstr = _head_operand(weight, "weight")
    if Hw != H:
        raise ValueError(f"hidden is [{T}, {H}] and weight [{V}, {Hw}]: their rows must have one length")
    out = -(-H // 8) * 8
    c = LinearCeContract(T, V, H, hs, wstr, out, out, ignore_index, wait_timeout_ns, piece,
                         MASK_EXPLICIT if mask is not None else MASK_IGNORE_INDEX, reduction, validate,
                         label_smoothing, z_loss, softcap)
    status = rlk_linear_ce_check(c)
    if status:
        check(status)
    return c


def _ce_workspace(contract, with_grad, like, workspace):
    n = rlk_linear_ce_workspace_size(contract, with_grad)
    if n == 0:
        check(rlk_linear_ce_check(contract) or RLK_ERR_UNSUPPORTED)
    if workspace is None:
        return _t().empty_strided((n,), (1,), dtype=_t().uint8, device=like.device)
    _need(workspace, "workspace", n, ("uint8",))
    return workspace


def _vector(t, name, n, dtypes):
    """A contiguous CUDA tensor of n elements (or more) of one of ``dtypes``; its pointer."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d)[6:] for d in dtypes)}, not {str(t.dtype)[6:]}")
    if not t.is_cuda or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {n} elements, not {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _ce_operands(c, hidden, weight, targets, mask):
    for name, t, rows, stride in (("hidden", hidden, c.T, c.hidden_stride or c.H),
                                  ("weight", weight, c.V, c.weight_stride or c.H)):
        r, cols, s = _head_operand(t, name)
        if r != rows or cols != c.H or (s != stride and rows > 1):
            raise ValueError(f"{name} is {list(t.shape)} with strides {list(t.stride())}; the contract's is "
                             f"[{rows}, {c.H}] with rows {stride} apart")
    torch = _t()
    return (hidden.data_ptr(), weight.data_ptr(), _vector(targets, "targets", c.T, (torch.int64,)),
            None if mask is None else _vector(mask, "mask", c.T, (torch.uint8, torch.bool)))


def linear_ce_fwd(contract, hidden, weight, targets, mask=None, stream=None, workspace=None):
    """(loss, lse) of the cross entropy of hidden @ weight^T: loss [T], or one value with a reduction; lse [T]."""
    operands = _ce_operands(contract, hidden, weight, targets, mask)
    f32 = _t().float32
    new = _t().empty_strided
    with _allocating(stream):
        loss = new((contract.T,), (1,), dtype=f32, device=hidden.device) if contract.reduction == REDUCE_NONE else \
            new((), (), dtype=f32, device=hidden.device)
        lse = new((contract.T,), (1,), dtype=f32, device=hidden.device)
        ws = _ce_workspace(contract, 0, hidden, workspace)
    _used_here(stream, loss, lse)
    status = rlk_linear_ce_fwd(contract, *operands, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                               _raw_stream(hidden, stream))
    if status:
        check(status)
    return loss, lse


def linear_ce_bwd(contract, hidden, weight, targets, mask, lse, grad_loss, need_dhidden=True, need_dweight=True,
                  stream=None, workspace=None):
    """(dhidden [T, H], dweight [V, H]) in BF16 from the forward's lse and the loss's FP32 gradient ([T], or one value
    with a reduction); a gradient that is not needed is None and costs nothing."""
    operands = _ce_operands(contract, hidden, weight, targets, mask)
    T, V, H, f32 = contract.T, contract.V, contract.H, (_t().float32,)
    pl = _vector(lse, "lse", T, f32)
    pg = _vector(grad_loss, "grad_loss", T if contract.reduction == REDUCE_NONE else 1, f32)

    with _allocating(stream):
        dh = _new(hidden, T, H, hidden.dtype, contract.dhidden_stride or H) if need_dhidden else None
        dw = _new(hidden, V, H, hidden.dtype, contract.dweight_stride or H) if need_dweight else None
        ws = _ce_workspace(contract, 1, hidden, workspace)
    _used_here(stream, dh, dw)
    status = rlk_linear_ce_bwd(contract, *operands, pl, pg, _ptr(dh), _ptr(dw), ws.data_ptr(),
                               _raw_stream(hidden, stream))
    if status:
        check(status)
    return dh, dw
