"""ctypes view of the C ABI in include/psk.h (argument marshalling only).

Loads ``_build/libpsk.so`` from this package's directory.  There is no
fallback: if the library is missing, importing the binding raises.
"""

from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libpsk.so")

PSK_F32, PSK_BF16, PSK_I32, PSK_I64 = 0, 1, 2, 3
PSK_ORDER_SEQUENTIAL, PSK_ORDER_BLOCKED, PSK_ORDER_INTERLEAVED = 0, 1, 2
PSK_EXP_EXACT, PSK_EXP_FAST = 0, 1
PSK_NORM_RMS, PSK_NORM_LAYER = 0, 1
PSK_LR_CONSTANT, PSK_LR_LINEAR, PSK_LR_COSINE = 0, 1, 2
PSK_MAX_RANK = 4
PSK_ADAMW_MAX_LEAVES = 512
PSK_W_IN_OUT, PSK_W_OUT_IN = 0, 1
PSK_ACT_NONE, PSK_ACT_RELU, PSK_ACT_GELU, PSK_ACT_SILU = 0, 1, 2, 3
PSK_ORTHO_MAX_LEAVES = 512
PSK_HEAD_NORM_NONE, PSK_HEAD_NORM_RMS = 0, 1
PSK_PAIRS_HALVES, PSK_PAIRS_NEIGHBOURS = 0, 1

ERRORS = {
    -1: "PSK_E_PROGRAM", -2: "PSK_E_TOO_MANY_NODES", -3: "PSK_E_SHAPE", -4: "PSK_E_DTYPE",
    -5: "PSK_E_NULL", -6: "PSK_E_ORDER", -7: "PSK_E_CUDA", -8: "PSK_E_ALIAS", -9: "PSK_E_ARG",
}

EXPORTS = ("psk_group_run", "psk_group_run_ex", "psk_group_run_interp", "psk_group_check", "psk_group_prepare", "psk_group_prepare_ex", "psk_softmax_region", "psk_softmax_masked",
           "psk_softmax_backward", "psk_norm_region",
           "psk_adamw_tree", "psk_adamw_tree_ex", "psk_adamw_tree_static", "psk_adamw_lr", "psk_adamw_workspace",
           "psk_adamw_scalars", "psk_adamw_group_sqsums", "psk_adamw_clip_scale", "psk_adamw_tree_scaled",
           "psk_embed", "psk_embed_workspace", "psk_embed_backward", "psk_dropout",
           "psk_norm_backward_workspace", "psk_norm_backward",
           "psk_token_logp", "psk_policy_loss_workspace", "psk_policy_loss",
           "psk_linear_workspace", "psk_linear", "psk_linear_backward_workspace", "psk_linear_backward",
           "psk_orthogonalize_workspace", "psk_orthogonalize",
           "psk_qk_norm_rotary", "psk_qk_norm_rotary_backward_workspace", "psk_qk_norm_rotary_backward",
           "psk_device_status", "psk_test_drop_row", "psk_test_fast_exp", "psk_last_error")


class psk_program(ctypes.Structure):
    _fields_ = [("tokens", ctypes.POINTER(ctypes.c_uint32)), ("n_tokens", ctypes.c_int32),
                ("imm", ctypes.POINTER(ctypes.c_float)), ("n_imm", ctypes.c_int32)]


class psk_input(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("stride", ctypes.c_int64 * PSK_MAX_RANK)]


class psk_output(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("shape", ctypes.c_int64 * PSK_MAX_RANK)]


class psk_order(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("param", ctypes.c_int32)]


class psk_leaf(ctypes.Structure):
    _fields_ = [("theta", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("grad_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32),
                ("numel", ctypes.c_int64)]


class psk_adamw_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("t", ctypes.c_int64)]


class psk_adamw_schedule(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("warmup", ctypes.c_int64), ("total", ctypes.c_int64),
                ("grad_clip", ctypes.c_double)]


class psk_ortho_leaf(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64)]


class PskError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code
        self.name = ERRORS.get(code, str(code))


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        L.psk_group_run.argtypes = [P(psk_program), P(psk_input), ctypes.c_int32, P(psk_output), ctypes.c_void_p]
        L.psk_group_check.argtypes = [P(psk_program), ctypes.c_int32, P(ctypes.c_int32), P(ctypes.c_int32)]
        L.psk_group_prepare.argtypes = [P(psk_program), P(psk_input), ctypes.c_int32, P(psk_output)]
        L.psk_group_run_ex.argtypes = [P(psk_program), P(psk_input), ctypes.c_int32, P(psk_output), ctypes.c_int32,
                                       ctypes.c_void_p]
        L.psk_group_prepare_ex.argtypes = [P(psk_program), P(psk_input), ctypes.c_int32, P(psk_output), ctypes.c_int32]
        L.psk_group_run_interp.argtypes = [P(psk_program), P(psk_input), ctypes.c_int32, P(psk_output),
                                           ctypes.c_int32, ctypes.c_void_p]
        L.psk_softmax_region.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                                         ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                         psk_order, ctypes.c_int32, ctypes.c_void_p]
        L.psk_softmax_masked.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                                         ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_int64, psk_order, ctypes.c_int32, ctypes.c_void_p]
        L.psk_softmax_backward.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                                           ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, psk_order, ctypes.c_void_p]
        L.psk_norm_region.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_int32, ctypes.c_double, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_int32, psk_order, ctypes.c_void_p]
        L.psk_adamw_tree.argtypes = [P(psk_leaf), ctypes.c_int32, P(psk_adamw_hparams), ctypes.c_void_p]
        L.psk_adamw_scalars.argtypes = [P(psk_adamw_hparams), P(ctypes.c_float)]
        L.psk_adamw_lr.argtypes = [P(psk_adamw_hparams), P(psk_adamw_schedule), P(ctypes.c_float)]
        L.psk_adamw_workspace.argtypes = [P(psk_leaf), ctypes.c_int32, P(psk_adamw_schedule), P(ctypes.c_uint64)]
        L.psk_adamw_tree_ex.argtypes = [P(psk_leaf), ctypes.c_int32, P(psk_adamw_hparams), P(psk_adamw_schedule),
                                        ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]
        L.psk_adamw_tree_static.argtypes = [P(psk_leaf), ctypes.c_int32, P(psk_adamw_hparams),
                                            P(psk_adamw_schedule), ctypes.c_void_p]
        L.psk_device_status.argtypes = [P(ctypes.c_uint32), ctypes.c_int32]
        L.psk_test_drop_row.argtypes = [ctypes.c_int64]
        L.psk_test_fast_exp.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]
        L.psk_adamw_group_sqsums.argtypes = [P(psk_leaf), ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_uint64, ctypes.c_void_p]
        L.psk_adamw_clip_scale.argtypes = [ctypes.c_void_p, P(ctypes.c_int64), ctypes.c_int32, ctypes.c_double,
                                           ctypes.c_void_p, ctypes.c_void_p]
        L.psk_adamw_tree_scaled.argtypes = [P(psk_leaf), ctypes.c_int32, P(psk_adamw_hparams),
                                            P(psk_adamw_schedule), ctypes.c_void_p, ctypes.c_void_p]
        V, I32, I64, U64, F64 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_double)
        L.psk_embed.argtypes = [V, I32, I64, V, I32, I64, I64, I64, F64, V, I32, I64, V]
        L.psk_embed_workspace.argtypes = [I64, I64, I64, P(U64)]
        L.psk_embed_backward.argtypes = [V, I32, I64, V, I32, I64, F64, V, I32, I64, I64, I64, I32, V, U64, V]
        L.psk_dropout.argtypes = [V, I32, V, I32, V, I32, I64, I64, I64, I64, I64, F64, U64, U64, V, V]
        L.psk_norm_backward_workspace.argtypes = [I64, I64, P(U64)]
        L.psk_norm_backward.argtypes = [V, I32, V, I32, V, I32, I64, I64, I64, I64, I64, I32, F64, V, I32, V, V, I32,
                                        V, U64, V]
        L.psk_token_logp.argtypes = [V, I32, I64, I64, I64, F64, V, I32, V, V]
        L.psk_policy_loss_workspace.argtypes = [I64, I64, P(U64)]
        L.psk_policy_loss.argtypes = [V, I32, I64, I64, I64, F64, V, I32, V, V, V, V, F64, F64, F64, V, V, V, I32, I64,
                                      V, U64, V]
        mat, head = [V, I32, I64], [I64, I64]
        L.psk_linear_workspace.argtypes = mat + mat + [I32, I64, I64, I64, P(U64)]
        L.psk_linear.argtypes = mat + mat + [I32, I64, I64, I64, V, I32, I32] + mat + mat + mat + [V, U64, V]
        L.psk_linear_backward_workspace.argtypes = (mat + mat + mat + [I32, I64, I64, I64, I32, V, I32, V, I32, V, I32,
                                                                       P(U64)])
        L.psk_linear_backward.argtypes = (mat + mat + mat + [I32, I64, I64, I64, I32] + mat + mat + mat
                                          + [V, I32, I32, V, U64, V])
        L.psk_orthogonalize_workspace.argtypes = [I32, I64, I64, I32, P(U64)]
        L.psk_orthogonalize.argtypes = [P(psk_ortho_leaf), I32, I64, I64, I32, I32, P(F64), I32, F64, F64, V, U64, V]
        rot = [I64, I64, I64, I64, I64, V, I32, V, I32, I32, F64, V, V, I32]
        L.psk_qk_norm_rotary.argtypes = [V, V, I32] + head * 2 + [V, V, I32] + head * 2 + rot + [V]
        L.psk_qk_norm_rotary_backward_workspace.argtypes = [I64, I64, I64, I64, P(U64)]
        L.psk_qk_norm_rotary_backward.argtypes = (([V, V, I32] + head * 2) * 3 + rot + [V, V, I32, V, U64, V])
        L.psk_last_error.restype = ctypes.c_char_p
        for f in ("psk_group_run", "psk_group_run_ex", "psk_group_run_interp", "psk_group_check", "psk_group_prepare", "psk_group_prepare_ex",
                  "psk_softmax_region", "psk_norm_region",
                  "psk_softmax_masked", "psk_softmax_backward",
                  "psk_adamw_tree",
                  "psk_adamw_scalars", "psk_adamw_lr", "psk_adamw_workspace", "psk_adamw_tree_ex",
                  "psk_adamw_tree_static",
                  "psk_adamw_group_sqsums", "psk_adamw_clip_scale", "psk_adamw_tree_scaled",
                  "psk_embed", "psk_embed_workspace", "psk_embed_backward", "psk_dropout",
                  "psk_norm_backward_workspace", "psk_norm_backward",
                  "psk_token_logp", "psk_policy_loss_workspace", "psk_policy_loss",
                  "psk_linear_workspace", "psk_linear", "psk_linear_backward_workspace", "psk_linear_backward",
                  "psk_orthogonalize_workspace", "psk_orthogonalize",
                  "psk_qk_norm_rotary", "psk_qk_norm_rotary_backward_workspace", "psk_qk_norm_rotary_backward",
                  "psk_device_status", "psk_test_drop_row", "psk_test_fast_exp"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def check(rc: int) -> None:
    if rc != 0:
        raise PskError(rc, lib().psk_last_error().decode())
