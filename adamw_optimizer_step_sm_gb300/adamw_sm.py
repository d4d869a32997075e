"""Python binding of the adamw_sm C ABI (include/adamw_sm.h,
include/adamw_losses.h and include/adamw_matrix.h).

Argument marshalling only: every step of the optimizer runs in the library's
CUDA kernels.  The functions keep the C names; a non-zero status raises
``AdamWError``.  ``Plan`` is a small convenience wrapper that builds the
tensor table from torch tensors (torch supplies device memory and streams).

The library is built in-tree (``build.build``) on first use when its sources
are newer than the shared object (or taken from the path in the environment
variable ADAMW_SM_LIBRARY, for a build made with other tuning constants); if
it cannot be built or loaded, every call raises -- there is no fallback
implementation.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

from . import build as _build

MODE_BF16_KAHAN = 0
MODE_MIXED_FP32_MASTER = 1
MODE_MIXED_BF16_REMAINDER = 2
MODE_BF16_PLAIN = 3
MODE_BF16_KAHAN_FP32_VAR = 4
# AnyPrecisionAdamW storage: MODE_ANYPREC | ANYPREC_* flags (bf16 param and
# grad; each flag makes one optimizer buffer fp32, or drops the compensation).
MODE_ANYPREC = 16
ANYPREC_M_FP32 = 1
ANYPREC_V_FP32 = 2
ANYPREC_C_FP32 = 4
ANYPREC_NO_KAHAN = 8
ANYPREC_MODES = tuple(MODE_ANYPREC | f for f in range(16) if (f & 12) != 12)
PLAN_NORM = 1
BUILD_CHECK_BOUNDS = 1
BUILD_BULK_STAGING = 2
STATUS_WAIT_RAN_OUT = 1
STATUS_BOUNDS = 2
PLAN_NO_FUSE = 2
STEP_CLIP = 1
STEP_NORM = 2

ADAMW_OK = 0
ADAMW_ERR_INVALID_ARG = -1
ADAMW_ERR_MISALIGNED = -2
ADAMW_ERR_CUDA = -3
ADAMW_ERR_NO_NORM = -4
ADAMW_ERR_TOO_LARGE = -5
ADAMW_ERR_NOT_ACCESSIBLE = -6

# the fine-tuning operators (include/adamw_losses.h)
DTYPE_BF16 = 0
DTYPE_FP16 = 1
DTYPE_FP32 = 2
KL = {"k1": 1, "k2": 2, "k3": 3}
REDUCE = {"token": 0, "sequence": 1, "fixed": 2}
PREFERENCE = {"sigmoid": 0, "hinge": 1, "ipo": 2}
REF_NONE = 0
REF_TOKEN = 1
REF_SEQUENCE = 2
NORM = {"l2": 0, "max": 1}

# the matrix operators (include/adamw_matrix.h)
MUON_SCALE = {"spectral": 0, "rms": 1}
EXPERT_STREAM_ROWS = 16


class AdamWError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status}: {adamw_status_string(status)}")


class adamw_tensor_t(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("aux", ctypes.c_void_p), ("numel", ctypes.c_int64)]


class adamw_hparams_t(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float),
                ("beta2", ctypes.c_float), ("eps", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("max_grad_norm", ctypes.c_float)]


class adamw_plan_info_t(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("n_tensors", ctypes.c_int32),
                ("total_elems", ctypes.c_int64), ("grid", ctypes.c_int32),
                ("block", ctypes.c_int32), ("n_chunks", ctypes.c_int64),
                ("scalar_elems", ctypes.c_int64), ("device", ctypes.c_int32),
                ("has_norm", ctypes.c_int32), ("norm_grid", ctypes.c_int32),
                ("fused", ctypes.c_int32)]


class adamw_chunk_t(ctypes.Structure):
    _fields_ = [("tensor", ctypes.c_int32), ("vec", ctypes.c_int32),
                ("offset", ctypes.c_int64), ("len", ctypes.c_int64),
                ("cta", ctypes.c_int32), ("pad_", ctypes.c_int32)]


class adamw_rows_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("inner", ctypes.c_int64),
                ("outer_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("cols", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class adamw_tokens_t(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("sequences", ctypes.c_int64),
                ("offsets", ctypes.c_void_p), ("mask", ctypes.c_void_p)]


class adamw_policy_t(ctypes.Structure):
    _fields_ = [("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float),
                ("dual_clip", ctypes.c_float), ("kl_coef", ctypes.c_float),
                ("entropy_coef", ctypes.c_float), ("divisor", ctypes.c_float),
                ("grad_scale", ctypes.c_float), ("kl", ctypes.c_int32),
                ("reduce", ctypes.c_int32), ("advantage_per_token", ctypes.c_int32)]


class adamw_preference_t(ctypes.Structure):
    _fields_ = [("beta", ctypes.c_float), ("margin", ctypes.c_float),
                ("label_smoothing", ctypes.c_float), ("grad_scale", ctypes.c_float),
                ("kind", ctypes.c_int32), ("length_average", ctypes.c_int32),
                ("ref", ctypes.c_int32)]


class adamw_grad_t(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("src_dtype", ctypes.c_int32), ("dst_dtype", ctypes.c_int32)]


class adamw_matrices_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("batch_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("pad_", ctypes.c_int32)]


class adamw_ortho_t(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("n_coefficients", ctypes.c_int32),
                ("coefficients", ctypes.POINTER(ctypes.c_float)), ("eps", ctypes.c_float)]


class adamw_muon_tensor_t(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("momentum", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("batch", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class adamw_muon_options_t(ctypes.Structure):
    _fields_ = [("ortho", adamw_ortho_t), ("nesterov", ctypes.c_int32), ("scale", ctypes.c_int32),
                ("momentum_dtype", ctypes.c_int32)]


class adamw_muon_hparams_t(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("pad_", ctypes.c_float)]


_lock = threading.Lock()
_lib: ctypes.CDLL | None = None


def load() -> ctypes.CDLL:
    """Build if needed and load the shared library (raises on failure)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = os.environ.get("ADAMW_SM_LIBRARY") or _build.build()
            L = ctypes.CDLL(path)
            vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
            L.adamw_plan_create.argtypes = [ctypes.POINTER(adamw_tensor_t), i32, i32, i32,
                                            ctypes.POINTER(vp)]
            L.adamw_step.argtypes = [vp, ctypes.POINTER(adamw_hparams_t), i64, vp, vp, vp]
            L.adamw_grad_norm.argtypes = [vp, vp, vp, vp]
            L.adamw_step_device.argtypes = [vp, vp, vp, i32, vp, vp, vp]
            L.adamw_plan_destroy.argtypes = [vp]
            L.adamw_plan_device_status.argtypes = [vp, ctypes.POINTER(i32)]
            L.adamw_plan_test_skew_barrier.argtypes = [vp, i64]
            L.adamw_plan_test_corrupt_chunk.argtypes = [vp, i64, i64]
            L.adamw_build_flags.argtypes = []
            L.adamw_build_flags.restype = i32
            L.adamw_lr_linear_warmup.argtypes = [ctypes.c_float, i64, i64, i64]
            L.adamw_lr_linear_warmup.restype = ctypes.c_float
            L.adamw_lr_linear_warmup_device.argtypes = [vp, vp, ctypes.c_float, i64, i64, vp]
            L.adamw_plan_get_info.argtypes = [vp, ctypes.POINTER(adamw_plan_info_t)]
            L.adamw_plan_chunks.argtypes = [ctypes.POINTER(adamw_tensor_t), i32, i32, i32,
                                            ctypes.POINTER(adamw_chunk_t), i64,
                                            ctypes.POINTER(i64)]
            L.adamw_step_scalars.argtypes = [ctypes.POINTER(adamw_hparams_t), i64,
                                             ctypes.POINTER(ctypes.c_float)]
            L.adamw_copy_probe.argtypes = [vp, vp, i64, vp]
            L.adamw_grad_norm_noalloc.argtypes = [ctypes.POINTER(adamw_tensor_t), i32, vp, vp, vp]
            L.adamw_step_table.argtypes = [vp, i32, i32, ctypes.POINTER(adamw_hparams_t), i64,
                                           vp, vp, vp]
            L.adamw_step_table_cache_clear.argtypes = []
            f32, P = ctypes.c_float, ctypes.POINTER
            rows, tokens, policy = P(adamw_rows_t), P(adamw_tokens_t), P(adamw_policy_t)
            L.adamw_token_logprob.argtypes = [rows, vp, i64, f32, vp, vp, vp, vp]
            L.adamw_token_logprob_backward.argtypes = [rows, vp, i64, f32, vp, vp, vp, vp, rows, vp]
            L.adamw_policy_loss.argtypes = [tokens, policy, *([vp] * 11)]
            L.adamw_policy_loss_logits.argtypes = [rows, vp, i64, f32, tokens, policy,
                                                   *([vp] * 7), rows, vp, vp]
            L.adamw_preference_loss.argtypes = [tokens, P(adamw_preference_t), *([vp] * 7)]
            L.adamw_clip_plan_create.argtypes = [P(adamw_grad_t), i32, P(vp)]
            L.adamw_clip_grads.argtypes = [vp, f32, i32, vp, vp]
            L.adamw_clip_plan_destroy.argtypes = [vp]
            for name in ("adamw_policy_workspace", "adamw_policy_logits_workspace"):
                getattr(L, name).argtypes = [i64, i64]
                getattr(L, name).restype = i64
            mats = P(adamw_matrices_t)
            L.adamw_orthogonalize.argtypes = [mats, mats, P(adamw_ortho_t), vp, vp]
            L.adamw_orthogonalize_workspace.argtypes = [i64, i64, i64]
            L.adamw_orthogonalize_workspace.restype = i64
            L.adamw_muon_plan_create.argtypes = [P(adamw_muon_tensor_t), i32, P(adamw_muon_options_t), P(vp)]
            L.adamw_muon_step.argtypes = [vp, vp, vp, vp]
            L.adamw_muon_plan_destroy.argtypes = [vp]
            L.adamw_expert_rows.argtypes = [mats, mats, i32, vp, mats, vp, vp]
            L.adamw_expert_outer.argtypes = [mats, mats, vp, mats, i32, vp, vp]
            L.adamw_expert_workspace.argtypes = [mats, mats]
            L.adamw_expert_workspace.restype = i64
            L.adamw_expert_backward.argtypes = [mats, mats, mats, i32, vp, mats, mats, i32, i32, vp, vp]
            L.adamw_expert_backward_workspace.argtypes = [mats, mats, mats]
            L.adamw_expert_backward_workspace.restype = i64
            L.adamw_matrix_status.argtypes = [P(i32)]
            L.adamw_matrix_test_expire.argtypes = [i32]
            L.adamw_matrix_test_expire.restype = None
            L.adamw_status_string.argtypes = [ctypes.c_int]
            L.adamw_status_string.restype = ctypes.c_char_p
            for name in ("adamw_plan_create", "adamw_step", "adamw_grad_norm", "adamw_step_device",
                         "adamw_plan_destroy", "adamw_plan_get_info", "adamw_plan_chunks",
                         "adamw_step_scalars", "adamw_copy_probe", "adamw_grad_norm_noalloc",
                         "adamw_step_table", "adamw_step_table_cache_clear",
                         "adamw_plan_device_status", "adamw_lr_linear_warmup_device",
                         "adamw_plan_test_skew_barrier", "adamw_plan_test_corrupt_chunk",
                         "adamw_token_logprob", "adamw_token_logprob_backward",
                         "adamw_policy_loss", "adamw_policy_loss_logits", "adamw_preference_loss",
                         "adamw_clip_plan_create", "adamw_clip_grads", "adamw_clip_plan_destroy",
                         "adamw_orthogonalize", "adamw_muon_plan_create", "adamw_muon_step",
                         "adamw_muon_plan_destroy", "adamw_expert_rows", "adamw_expert_outer",
                         "adamw_expert_backward", "adamw_matrix_status"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
        return _lib


def _check(rc: int, where: str):
    if rc != ADAMW_OK:
        raise AdamWError(rc, where)


def _table(entries) -> tuple[ctypes.Array, int]:
    entries = list(entries)
    arr = (adamw_tensor_t * max(1, len(entries)))()
    for i, e in enumerate(entries):
        arr[i] = e if isinstance(e, adamw_tensor_t) else adamw_tensor_t(*e)
    return arr, len(entries)


# ------------------------------------------------------------ C functions --

def adamw_status_string(status: int) -> str:
    return load().adamw_status_string(status).decode()


def adamw_plan_create(entries, mode: int, flags: int = 0) -> int:
    """entries: adamw_tensor_t or (param, grad, exp_avg, exp_avg_sq, aux, numel)
    tuples of device addresses.  Returns the plan handle."""
    arr, n = _table(entries)
    out = ctypes.c_void_p()
    _check(load().adamw_plan_create(arr, n, mode, flags, ctypes.byref(out)), "adamw_plan_create")
    return out.value


def adamw_step(plan: int, hp: adamw_hparams_t, step: int, d_grad_norm: int = 0,
               d_nonfinite: int = 0, stream: int = 0) -> None:
    _check(load().adamw_step(plan, ctypes.byref(hp), step, d_grad_norm or None,
                             d_nonfinite or None, stream or None), "adamw_step")


def adamw_step_device(plan: int, d_hp: int, d_step: int, flags: int = 0, d_grad_norm: int = 0,
                      d_nonfinite: int = 0, stream: int = 0) -> None:
    """A step whose hyperparameters (device adamw_hparams_t at d_hp) and
    applied-step counter (device int64 at d_step) live on the device."""
    _check(load().adamw_step_device(plan, d_hp, d_step, flags, d_grad_norm or None,
                                    d_nonfinite or None, stream or None), "adamw_step_device")


def adamw_grad_norm(plan: int, d_grad_norm: int = 0, d_nonfinite: int = 0,
                    stream: int = 0) -> None:
    _check(load().adamw_grad_norm(plan, d_grad_norm or None, d_nonfinite or None,
                                  stream or None), "adamw_grad_norm")


NOALLOC_MAX_TENSORS = 4096


def adamw_grad_norm_noalloc(entries, d_grad_norm: int = 0, d_nonfinite: int = 0,
                            stream: int = 0) -> None:
    """Global gradient norm of a tensor list without any device allocation
    (no plan; only .grad and .numel of each entry are read).  For callers
    that cannot call cudaMalloc; see include/adamw_sm.h."""
    arr, n = _table(entries)
    _check(load().adamw_grad_norm_noalloc(arr, n, d_grad_norm or None, d_nonfinite or None,
                                          stream or None), "adamw_grad_norm_noalloc")


def adamw_step_table(d_table: int, n_tensors: int, mode: int, hp: adamw_hparams_t, step: int,
                     d_grad_norm: int = 0, d_nonfinite: int = 0, stream: int = 0) -> None:
    """One step over a tensor table held in device memory at address d_table
    (n_tensors adamw_tensor_t entries); plans are cached by table contents."""
    _check(load().adamw_step_table(d_table, n_tensors, mode, ctypes.byref(hp), step,
                                   d_grad_norm or None, d_nonfinite or None, stream or None),
           "adamw_step_table")


def adamw_step_table_cache_clear() -> int:
    return load().adamw_step_table_cache_clear()


def adamw_plan_destroy(plan: int) -> None:
    _check(load().adamw_plan_destroy(plan), "adamw_plan_destroy")


def adamw_lr_linear_warmup(base_lr: float, step: int, warmup: int, total: int) -> float:
    return float(load().adamw_lr_linear_warmup(base_lr, step, warmup, total))


def adamw_lr_linear_warmup_device(d_hp: int, d_step: int, base_lr: float, warmup: int,
                                  total: int, stream: int = 0) -> None:
    _check(load().adamw_lr_linear_warmup_device(d_hp, d_step, base_lr, warmup, total,
                                                stream or None), "adamw_lr_linear_warmup_device")


def adamw_plan_device_status(plan: int) -> int:
    """Reads and clears the plan's device status word (1: a bounded wait in
    one of its kernels ran out)."""
    out = ctypes.c_int32(0)
    _check(load().adamw_plan_device_status(plan, ctypes.byref(out)), "adamw_plan_device_status")
    return out.value


def adamw_build_flags() -> int:
    """BUILD_CHECK_BOUNDS / BUILD_BULK_STAGING bits of the loaded library."""
    return int(load().adamw_build_flags())


def adamw_plan_test_corrupt_chunk(plan: int, chunk: int, delta: int) -> None:
    """Bounds-checked builds only: lengthen update chunk ``chunk`` by ``delta``."""
    _check(load().adamw_plan_test_corrupt_chunk(plan, chunk, delta), "adamw_plan_test_corrupt_chunk")


def adamw_plan_test_skew_barrier(plan: int, delta: int) -> None:
    """Failure-path tests only: misalign the fused step's barrier counter."""
    _check(load().adamw_plan_test_skew_barrier(plan, delta), "adamw_plan_test_skew_barrier")


def adamw_plan_get_info(plan: int) -> adamw_plan_info_t:
    info = adamw_plan_info_t()
    _check(load().adamw_plan_get_info(plan, ctypes.byref(info)), "adamw_plan_get_info")
    return info


def adamw_plan_chunks(entries, mode: int, grid: int) -> list[adamw_chunk_t]:
    arr, n = _table(entries)
    count = ctypes.c_int64(0)
    rc = load().adamw_plan_chunks(arr, n, mode, grid, None, 0, ctypes.byref(count))
    if rc not in (ADAMW_OK, ADAMW_ERR_TOO_LARGE):
        _check(rc, "adamw_plan_chunks")
    out = (adamw_chunk_t * max(1, count.value))()
    _check(load().adamw_plan_chunks(arr, n, mode, grid, out, count.value, ctypes.byref(count)),
           "adamw_plan_chunks")
    return list(out[:count.value])


def adamw_step_scalars(hp: adamw_hparams_t, step: int) -> list[float]:
    out = (ctypes.c_float * 5)()
    _check(load().adamw_step_scalars(ctypes.byref(hp), step, out), "adamw_step_scalars")
    return list(out)


def adamw_copy_probe(dst: int, src: int, nbytes: int, stream: int = 0) -> None:
    _check(load().adamw_copy_probe(dst, src, nbytes, stream or None), "adamw_copy_probe")


# The C functions of adamw_losses.h.  rows, tokens, policy and pref are the
# structures above; every other argument is a device address (0: NULL), a
# number or a stream.  losses.py has them over torch tensors.

def adamw_token_logprob(logits: adamw_rows_t, targets: int, ignore_index: int, scale: float, logp: int,
                        entropy: int = 0, stats: int = 0, stream: int = 0) -> None:
    rc = load().adamw_token_logprob(ctypes.byref(logits), targets, ignore_index, scale, logp,
                                    entropy or None, stats or None, stream or None)
    _check(rc, "adamw_token_logprob")


def adamw_token_logprob_backward(logits: adamw_rows_t, targets: int, ignore_index: int, scale: float,
                                 stats: int, entropy: int, d_logp: int, d_entropy: int,
                                 d_logits: adamw_rows_t, stream: int = 0) -> None:
    rc = load().adamw_token_logprob_backward(ctypes.byref(logits), targets, ignore_index, scale, stats,
                                             entropy or None, d_logp, d_entropy or None,
                                             ctypes.byref(d_logits), stream or None)
    _check(rc, "adamw_token_logprob_backward")


def adamw_policy_workspace(n: int, sequences: int) -> int:
    return load().adamw_policy_workspace(n, sequences)


def adamw_policy_logits_workspace(n: int, sequences: int) -> int:
    return load().adamw_policy_logits_workspace(n, sequences)


def adamw_policy_loss(tokens: adamw_tokens_t, policy: adamw_policy_t, logp: int, old_logp: int,
                      ref_logp: int, advantages: int, entropy: int, stats: int, counts: int, d_logp: int,
                      d_entropy: int, workspace: int, stream: int = 0) -> None:
    rc = load().adamw_policy_loss(ctypes.byref(tokens), ctypes.byref(policy), logp, old_logp,
                                  ref_logp or None, advantages, entropy or None, stats, counts, d_logp,
                                  d_entropy or None, workspace, stream or None)
    _check(rc, "adamw_policy_loss")


def adamw_policy_loss_logits(logits: adamw_rows_t, targets: int, ignore_index: int, scale: float,
                             tokens: adamw_tokens_t, policy: adamw_policy_t, old_logp: int, ref_logp: int,
                             advantages: int, stats: int, counts: int, logp: int, entropy: int,
                             d_logits: adamw_rows_t, workspace: int, stream: int = 0) -> None:
    rc = load().adamw_policy_loss_logits(ctypes.byref(logits), targets, ignore_index, scale,
                                         ctypes.byref(tokens), ctypes.byref(policy), old_logp,
                                         ref_logp or None, advantages, stats, counts, logp, entropy or None,
                                         ctypes.byref(d_logits), workspace, stream or None)
    _check(rc, "adamw_policy_loss_logits")


def adamw_preference_loss(tokens: adamw_tokens_t, pref: adamw_preference_t, logp: int, ref_logp: int,
                          stats: int, losses: int, rewards: int, d_logp: int, stream: int = 0) -> None:
    rc = load().adamw_preference_loss(ctypes.byref(tokens), ctypes.byref(pref), logp, ref_logp or None,
                                      stats, losses, rewards, d_logp, stream or None)
    _check(rc, "adamw_preference_loss")


def adamw_clip_plan_create(entries) -> int:
    """entries: adamw_grad_t or (src, dst, numel, src_dtype, dst_dtype)
    tuples.  Returns the plan handle."""
    entries = list(entries)
    arr = (adamw_grad_t * max(1, len(entries)))()
    for i, e in enumerate(entries):
        arr[i] = e if isinstance(e, adamw_grad_t) else adamw_grad_t(*e)
    out = ctypes.c_void_p()
    _check(load().adamw_clip_plan_create(arr, len(entries), ctypes.byref(out)), "adamw_clip_plan_create")
    return out.value


def adamw_clip_grads(plan: int, max_norm: float, norm: int, result: int, stream: int = 0) -> None:
    rc = load().adamw_clip_grads(plan, max_norm, norm, result, stream or None)
    _check(rc, "adamw_clip_grads")


def adamw_clip_plan_destroy(plan: int) -> None:
    _check(load().adamw_clip_plan_destroy(plan), "adamw_clip_plan_destroy")


# The C functions of adamw_matrix.h; matrix.py has them over torch tensors.

def ortho_options(steps: int, coefficients, eps: float) -> adamw_ortho_t:
    """coefficients: (a, b, c), or a sequence of them, one for each step (the
    last one for the steps beyond)."""
    rows = [coefficients] if not hasattr(coefficients[0], "__len__") else list(coefficients)
    if any(len(r) != 3 for r in rows):
        raise ValueError("want three coefficients a step")
    flat = (ctypes.c_float * (3 * len(rows)))(*[float(x) for r in rows for x in r])
    return adamw_ortho_t(steps, len(rows), flat, eps)


def adamw_orthogonalize(src: adamw_matrices_t, dst: adamw_matrices_t, ortho: adamw_ortho_t, workspace: int,
                        stream: int = 0) -> None:
    rc = load().adamw_orthogonalize(ctypes.byref(src), ctypes.byref(dst), ctypes.byref(ortho), workspace or None,
                                    stream or None)
    _check(rc, "adamw_orthogonalize")


def adamw_orthogonalize_workspace(batch: int, rows: int, cols: int) -> int:
    return load().adamw_orthogonalize_workspace(batch, rows, cols)


def adamw_muon_plan_create(entries, options: adamw_muon_options_t) -> int:
    """entries: adamw_muon_tensor_t or (param, grad, momentum, master, batch,
    rows, cols) tuples.  Returns the plan handle."""
    entries = list(entries)
    arr = (adamw_muon_tensor_t * max(1, len(entries)))()
    for i, e in enumerate(entries):
        arr[i] = e if isinstance(e, adamw_muon_tensor_t) else adamw_muon_tensor_t(*e)
    out = ctypes.c_void_p()
    rc = load().adamw_muon_plan_create(arr, len(entries), ctypes.byref(options), ctypes.byref(out))
    _check(rc, "adamw_muon_plan_create")
    return out.value


def adamw_muon_step(plan: int, d_hparams: int, d_nonfinite: int, stream: int = 0) -> None:
    _check(load().adamw_muon_step(plan, d_hparams, d_nonfinite, stream or None), "adamw_muon_step")


def adamw_muon_plan_destroy(plan: int) -> None:
    _check(load().adamw_muon_plan_destroy(plan), "adamw_muon_plan_destroy")


def adamw_expert_rows(x: adamw_matrices_t, w: adamw_matrices_t, transposed: int, offsets: int, y: adamw_matrices_t,
                      workspace: int = 0, stream: int = 0) -> None:
    rc = load().adamw_expert_rows(ctypes.byref(x), ctypes.byref(w), transposed, offsets, ctypes.byref(y),
                                  workspace or None, stream or None)
    _check(rc, "adamw_expert_rows")


def adamw_expert_outer(dy: adamw_matrices_t, x: adamw_matrices_t, offsets: int, dw: adamw_matrices_t,
                       accumulate: int = 0, workspace: int = 0, stream: int = 0) -> None:
    rc = load().adamw_expert_outer(ctypes.byref(dy), ctypes.byref(x), offsets, ctypes.byref(dw), accumulate,
                                   workspace or None, stream or None)
    _check(rc, "adamw_expert_outer")


def adamw_expert_workspace(a: adamw_matrices_t, b: adamw_matrices_t) -> int:
    return load().adamw_expert_workspace(ctypes.byref(a), ctypes.byref(b))


def adamw_expert_backward(dy: adamw_matrices_t, x: adamw_matrices_t, w: adamw_matrices_t, transposed: int, offsets: int,
                          dx: adamw_matrices_t | None, dw: adamw_matrices_t | None, dw_transposed: int = 0,
                          accumulate: int = 0, workspace: int = 0, stream: int = 0) -> None:
    ref = lambda m: None if m is None else ctypes.byref(m)
    rc = load().adamw_expert_backward(ref(dy), ref(x), ref(w), transposed, offsets, ref(dx), ref(dw), dw_transposed,
                                      accumulate, workspace or None, stream or None)
    _check(rc, "adamw_expert_backward")


def adamw_expert_backward_workspace(dy: adamw_matrices_t, x: adamw_matrices_t, w: adamw_matrices_t) -> int:
    return load().adamw_expert_backward_workspace(ctypes.byref(dy), ctypes.byref(x), ctypes.byref(w))


def adamw_matrix_status() -> int:
    """Reads and clears the current device's status word of the matrix
    operators (1: a bounded wait ran out)."""
    out = ctypes.c_int32(0)
    _check(load().adamw_matrix_status(ctypes.byref(out)), "adamw_matrix_status")
    return out.value


def adamw_matrix_test_expire(on: bool) -> None:
    load().adamw_matrix_test_expire(int(on))


def hparams(lr=2e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1,
            max_grad_norm=0.0) -> adamw_hparams_t:
    return adamw_hparams_t(lr, beta1, beta2, eps, weight_decay, max_grad_norm)


# --------------------------------------------------------- torch wrapper --

def buffer_dtypes(mode: int):
    """torch dtypes of param, grad, exp_avg, exp_avg_sq and aux in a storage
    mode (None: the mode does not use that buffer)."""
    import torch
    bf, f32 = torch.bfloat16, torch.float32
    named = {MODE_BF16_KAHAN: (bf,) * 5,
             MODE_MIXED_FP32_MASTER: (f32, bf, f32, f32, bf),
             MODE_MIXED_BF16_REMAINDER: (bf, bf, f32, f32, torch.int16),
             MODE_BF16_PLAIN: (bf,) * 4 + (None,),
             MODE_BF16_KAHAN_FP32_VAR: (bf, bf, bf, f32, bf)}
    if mode in named:
        return named[mode]
    if mode not in ANYPREC_MODES:
        raise ValueError(f"unknown storage mode {mode}")
    f = mode & 15
    return (bf, bf, f32 if f & ANYPREC_M_FP32 else bf, f32 if f & ANYPREC_V_FP32 else bf,
            None if f & ANYPREC_NO_KAHAN else (f32 if f & ANYPREC_C_FP32 else bf))


class Plan:
    """A plan over lists of torch CUDA tensors (one list per buffer kind).

    bf16 Kahan mode: params, exp_avg, exp_avg_sq, aux (= compensation) bf16.
    Mixed mode: params (= fp32 master), exp_avg, exp_avg_sq fp32; aux = bf16
    param out.  Remainder mode: params bf16, exp_avg, exp_avg_sq fp32, aux =
    int16 remainder of the fp32 master.  Any-precision modes: as
    ``buffer_dtypes(mode)``.  grads are bf16 in all modes.  The tensors must stay alive and in
    place for the plan's lifetime (the plan holds references to them).
    """

    def __init__(self, params, grads, exp_avgs, exp_avg_sqs, auxs, mode: int,
                 norm: bool = False, fuse: bool = True):
        import torch
        if auxs is None:
            auxs = [None] * len(list(params))
        lists = [list(x) for x in (params, grads, exp_avgs, exp_avg_sqs, auxs)]
        n = len(lists[0])
        if any(len(x) != n for x in lists):
            raise ValueError("tensor lists differ in length")
        want = buffer_dtypes(mode)
        entries = []
        for k in range(n):
            ts = [x[k] for x in lists]
            numel = ts[0].numel()
            for j, (t, dt) in enumerate(zip(ts, want)):
                if dt is None:       # a buffer the mode does not use
                    continue
                # gradients may live in pinned host memory (read over the
                # CPU-GPU link); everything else on the device
                where_ok = t.is_cuda or (j == 1 and t.is_pinned())
                if not where_ok or t.dtype != dt or not t.is_contiguous() or t.numel() != numel:
                    raise TypeError(f"tensor {k}: want contiguous CUDA {dt} of {numel} elements"
                                    + (" (or pinned host memory)" if j == 1 else ""))
            entries.append(adamw_tensor_t(*(t.data_ptr() if t is not None else None for t in ts),
                                          numel))
        self._keep = lists
        self.mode = mode
        dev = lists[0][0].device if n else torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.device(dev):
            self.handle = adamw_plan_create(entries, mode, (PLAN_NORM if norm else 0)
                                            | (0 if fuse else PLAN_NO_FUSE))
        self.device = dev
        self.info = adamw_plan_get_info(self.handle)
        self.last_nonfinite = None

    def step(self, hp: adamw_hparams_t, step: int, grad_norm=None, nonfinite=None,
             stream=None) -> None:
        """One step at t = ``step``.  A clipped step (hp.max_grad_norm > 0)
        needs a non-finite flag; without ``nonfinite`` it goes to the plan's
        own int32 device tensor ``last_nonfinite`` (1: the step was skipped,
        so the caller must pass the same ``step`` again)."""
        import torch
        st = stream if stream is not None else torch.cuda.current_stream(self.device)
        if nonfinite is None and hp.max_grad_norm > 0:
            if self.last_nonfinite is None:
                self.last_nonfinite = torch.zeros(1, dtype=torch.int32, device=self.device)
            nonfinite = self.last_nonfinite
        adamw_step(self.handle, hp, step,
                   grad_norm.data_ptr() if grad_norm is not None else 0,
                   nonfinite.data_ptr() if nonfinite is not None else 0,
                   st.cuda_stream)

    def step_device(self, d_hp, d_step, flags: int = 0, grad_norm=None, nonfinite=None,
                    stream=None) -> None:
        """d_hp: CUDA uint8 tensor holding one adamw_hparams_t (see
        ``device_hparams``); d_step: CUDA int64 tensor, the applied-step count."""
        import torch
        st = stream if stream is not None else torch.cuda.current_stream(self.device)
        adamw_step_device(self.handle, d_hp.data_ptr(), d_step.data_ptr(), flags,
                          grad_norm.data_ptr() if grad_norm is not None else 0,
                          nonfinite.data_ptr() if nonfinite is not None else 0, st.cuda_stream)

    def grad_norm(self, grad_norm=None, nonfinite=None, stream=None) -> None:
        import torch
        st = stream if stream is not None else torch.cuda.current_stream(self.device)
        adamw_grad_norm(self.handle, grad_norm.data_ptr() if grad_norm is not None else 0,
                        nonfinite.data_ptr() if nonfinite is not None else 0, st.cuda_stream)

    def close(self) -> None:
        if getattr(self, "handle", None):
            adamw_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def device_hparams(hp: adamw_hparams_t, device="cuda"):
    """An adamw_hparams_t as a CUDA uint8 tensor, for adamw_step_device."""
    import torch
    raw = bytes(hp)
    return torch.frombuffer(bytearray(raw), dtype=torch.uint8).to(device)


def dtype_code(dtype) -> int:
    """The library's code of a torch dtype of logits or gradients."""
    import torch
    codes = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32}
    if dtype not in codes:
        raise TypeError(f"want bfloat16, float16 or float32, not {dtype}")
    return codes[dtype]


class ClipResult(NamedTuple):
    """The plan's own device tensors, overwritten by its next ``clip``."""
    norm: object       # fp32, the global norm
    coef: object       # fp32, what the gradients were multiplied by
    nonfinite: object  # int32, 1: a gradient was inf or NaN (then coef is 1)


class ClipPlan:
    """Clips a list of gradients by their global norm, over every parameter
    group and optimizer and over bf16, fp16 and fp32 tensors alike.

    ``grads``: contiguous CUDA tensors of one device.  ``outs``: where the
    clipped gradients go, tensors of the same sizes and any of the three
    types (for example the bf16 gradients that an optimizer reads, from fp32
    accumulators); None clips in place.  No tensor twice, and none that reaches
    into another.  ``norm_only``: nothing is written but the result.  The tensors must stay alive and in place for the plan's
    lifetime (the plan holds references to them); calls on one plan must not
    overlap on the GPU."""

    def __init__(self, grads, outs=None, norm_only: bool = False):
        import torch
        grads = list(grads)
        if norm_only and outs is not None:
            raise ValueError("norm_only writes no outs")
        outs = list(outs) if outs is not None else grads
        if len(outs) != len(grads):
            raise ValueError("tensor lists differ in length")
        if not grads:
            raise ValueError("empty gradient list")
        dev = grads[0].device
        entries = []
        for k, (g, o) in enumerate(zip(grads, outs)):
            for t in (g, o):
                if not t.is_cuda or t.device != dev or not t.is_contiguous() or t.numel() != g.numel():
                    raise TypeError(f"tensor {k}: want contiguous CUDA tensors of one device and of equal sizes")
            entries.append(adamw_grad_t(g.data_ptr() or None, None if norm_only else o.data_ptr() or None,
                                        g.numel(), dtype_code(g.dtype), dtype_code(o.dtype)))
        self._keep = (grads, outs)
        self.device = dev
        with torch.cuda.device(dev):
            self.handle = adamw_clip_plan_create(entries)
        self._result = torch.zeros(4, dtype=torch.float32, device=dev)
        # the memory may still be in use on the stream current here, by its zeroing
        # if nothing else, and the first clip may be on another
        torch.cuda.current_stream(dev).synchronize()
        self._at = self._result.data_ptr()
        self.result = ClipResult(self._result[0], self._result[1], self._result.view(torch.int32)[2])
        # what a clip writes, for autograd: a buffer once for all views of it
        bases = [] if norm_only else [o if o._base is None else o._base for o in outs]
        self._written = list({id(b): b for b in [self._result, *bases]}.values())

    def clip(self, max_norm: float, norm: str = "l2", stream=None) -> ClipResult:
        """One clip to ``max_norm`` (infinity: only copies or converts) by the
        l2 norm of all elements or their largest magnitude ("max"); returns
        ``self.result`` without waiting for the GPU.  To autograd it is an
        in-place write of the outs.  With a non-finite gradient nothing is
        scaled: the values reach the optimizer, which skips or reports the
        step."""
        import torch
        if norm not in NORM:
            raise ValueError('norm must be "l2" or "max"')
        if not max_norm > 0:
            raise ValueError("want max_norm > 0")
        st = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(self.device.index)
        adamw_clip_grads(self.handle, max_norm, NORM[norm], self._at, st)
        torch.autograd.graph.increment_version(self._written)
        return self.result

    def close(self) -> None:
        if getattr(self, "handle", None):
            adamw_clip_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MuonPlan:
    """The Muon step over lists of torch CUDA tensors of one device: params and
    grads bf16, momenta fp32 or bf16 (all of one type), masters fp32, each
    contiguous [..., rows, cols] (leading dimensions are a batch of matrices).
    No buffer may reach into another.  The tensors must stay alive and in place
    for the plan's lifetime (the plan holds references to them); steps of one
    plan must not overlap on the GPU."""

    def __init__(self, params, grads, momenta, masters, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315),
                 eps: float = 1e-7, nesterov: bool = True, scale: str = "rms"):
        import torch
        lists = [list(x) for x in (params, grads, momenta, masters)]
        if any(len(x) != len(lists[0]) for x in lists):
            raise ValueError("tensor lists differ in length")
        if not lists[0]:
            raise ValueError("empty parameter list")
        if scale not in MUON_SCALE:
            raise ValueError('want scale "rms" or "spectral"')
        dev, mdt = lists[0][0].device, lists[2][0].dtype
        if mdt not in (torch.float32, torch.bfloat16):
            raise TypeError(f"want fp32 or bf16 momenta, not {mdt}")
        want = (torch.bfloat16, torch.bfloat16, mdt, torch.float32)
        entries = []
        for k, ts in enumerate(zip(*lists)):
            shape = ts[0].shape
            if len(shape) < 2:
                raise ValueError(f"tensor {k}: want [..., rows, cols]")
            for t, dt in zip(ts, want):
                if not t.is_cuda or t.device != dev or t.dtype != dt or not t.is_contiguous() or t.shape != shape:
                    raise TypeError(f"tensor {k}: want contiguous CUDA {dt} {tuple(shape)} of one device")
            entries.append(adamw_muon_tensor_t(*(t.data_ptr() or None for t in ts), shape[:-2].numel(), *shape[-2:]))
        self._keep = lists
        self.device = dev
        self._options = adamw_muon_options_t(ortho_options(steps, coefficients, eps), int(nesterov), MUON_SCALE[scale],
                                             DTYPE_FP32 if mdt == torch.float32 else DTYPE_BF16)
        with torch.cuda.device(dev):
            self.handle = adamw_muon_plan_create(entries, self._options)

    def step(self, d_hparams, nonfinite, stream=None) -> None:
        """d_hparams: CUDA fp32 [4]: lr, momentum, weight decay, unused;
        nonfinite: CUDA int32 [1], 1 after a step that wrote nothing, 2 after one
        whose results are undefined as a kernel's bounded wait ran out."""
        import torch
        for name, t, dt, n in (("d_hparams", d_hparams, torch.float32, 4), ("nonfinite", nonfinite, torch.int32, 1)):
            if t.dtype != dt or t.device != self.device or t.numel() < n or not t.is_contiguous():
                raise TypeError(f"want {name} contiguous {dt} [{n}] on {self.device}")
        st = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(self.device.index)
        adamw_muon_step(self.handle, d_hparams.data_ptr(), nonfinite.data_ptr(), st)

    def close(self) -> None:
        if getattr(self, "handle", None):
            adamw_muon_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
