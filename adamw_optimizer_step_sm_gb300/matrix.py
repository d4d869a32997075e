"""Matrix operators of a training step, over torch tensors.

    orthogonalize           Newton-Schulz orthogonalisation of matrices
    expert_linear           products grouped by expert, of ragged sizes
    expert_linear_backward  the gradients of both factors

Every function is one or a few calls into the library (include/adamw_matrix.h
has the formulas) on the current stream of the tensors' device, and waits for
nothing.  ``optim.Muon`` is the optimizer whose step orthogonalises.  Every wait
in a kernel is bounded; one that ran out (results are then undefined) shows in
``adamw_sm.adamw_matrix_status()``, which synchronises.

Experts: rows offsets[e] to offsets[e + 1] - 1 of [tokens, features] belong to
expert e; ``offsets`` is int64 [experts + 1] on the device, as for packed
sequences, so that no call waits for the router's counts.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import adamw_sm as A
from .losses import _call, _tangent, _written

_byref = ctypes.byref
_empty = torch.empty
_matrices_t = A.adamw_matrices_t
_CODES = {torch.bfloat16: A.DTYPE_BF16, torch.float16: A.DTYPE_FP16, torch.float32: A.DTYPE_FP32}
_HALVES = (torch.bfloat16, torch.float16)
_BYTES = torch.uint8

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _matrices(x: torch.Tensor) -> A.adamw_matrices_t:
    """x, [rows, cols] or [batch, rows, cols] with consecutive elements in a row."""
    s, d = x.stride(), x.shape
    if len(d) == 2:
        return _matrices_t(x.data_ptr(), 1, d[0], d[1], 0, s[0], _CODES[x.dtype])
    return _matrices_t(x.data_ptr(), d[0], d[1], d[2], s[0], s[1], _CODES[x.dtype])


# ------------------------------------------------------- orthogonalisation --

_options: dict = {}


def _ortho(steps, coefficients, eps):
    key = (steps, coefficients, eps) if type(coefficients) is tuple and type(coefficients[0]) is float else None
    o = _options.get(key) if key else None
    if o is None:
        if not 1 <= steps <= 32:
            raise ValueError("want 1 to 32 steps")
        if not eps > 0:
            raise ValueError("want eps > 0")
        o = A.ortho_options(steps, coefficients, eps)
        if not 1 <= o.n_coefficients <= 32:
            raise ValueError("want coefficients (a, b, c), or up to 32 of them")
        if key and len(_options) < 64:
            _options[key] = o
    return o


def orthogonalize(x: torch.Tensor, *, steps: int = 5, coefficients=COEFFICIENTS, eps: float = 1e-7,
                  dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The Newton-Schulz iteration of each matrix of x ([..., rows, cols], bf16,
    fp16 or fp32): X / max(norm, eps), then ``steps`` times a X + (b G + c G G) X
    with G = X X^T.  ``coefficients``: (a, b, c), or one such triple a step (the
    last for the steps beyond).  The result is of ``dtype``, or written to
    ``out`` (which may be x).  A matrix holding inf or NaN gives NaN, a zero
    matrix zeros.  Not differentiable: it is what optimizers do to gradients."""
    code, shape = _CODES.get(x.dtype), x.shape
    nd = len(shape)
    if code is None or nd < 2 or not x.is_cuda:
        if not x.is_cuda:
            raise TypeError("want CUDA tensors")
        if code is None:
            raise TypeError(f"want bfloat16, float16 or float32 matrices, not {x.dtype}")
        raise ValueError("want matrices [..., rows, cols]")
    if x.requires_grad and torch.is_grad_enabled() or _tangent(x).tangent is not None:
        raise RuntimeError("orthogonalize has no gradient: detach its input")
    dev = x.device
    if out is not None:
        dtype = out.dtype
        if out.shape != shape or out.device != dev or dtype not in _CODES or not out.is_contiguous():
            raise ValueError("out must be contiguous, of x's shape and device, in bfloat16, float16 or float32")
        if out.requires_grad and torch.is_grad_enabled():
            raise RuntimeError("out requires a gradient")
    elif dtype not in _CODES:
        raise TypeError(f"want a result in bfloat16, float16 or float32, not {dtype}")
    ortho = _ortho(steps, coefficients, eps)
    if x.numel() == 0:
        return out if out is not None else _empty(shape, dtype=dtype, device=dev)
    if nd > 3:   # one batch dimension, a copy where the others do not make one
        x = x.detach().reshape(-1, *shape[-2:])
    stride = x.stride()
    rows, cols = shape[-2], shape[-1]
    turned = False
    if stride[-1] != 1 and cols > 1:
        if stride[-2] == 1 and out is None and nd <= 3:
            turned = True   # a transposed view: the transpose's result, transposed
        else:
            x = x.detach().contiguous()
            stride = x.stride()
    batch, between = (1, 0) if nd == 2 else (x.shape[0], stride[0])
    y = out
    if turned:
        rows, cols = cols, rows
        y = _empty((*shape[:-2], rows, cols), dtype=dtype, device=dev)
    elif y is None:
        y = _empty(shape, dtype=dtype, device=dev)
    lib = A.load()
    nbytes = lib.adamw_orthogonalize_workspace(batch, rows, cols)
    # torch's allocations start at multiples of 512 bytes
    work = _empty(nbytes, dtype=_BYTES, device=dev) if nbytes else None
    _call(lib.adamw_orthogonalize, "adamw_orthogonalize", dev,
          _byref(_matrices_t(x.data_ptr(), batch, rows, cols, between, stride[-1] if turned else stride[-2], code)),
          _byref(_matrices_t(y.data_ptr(), batch, rows, cols, rows * cols, cols, _CODES[dtype])),
          _byref(ortho), work.data_ptr() if nbytes else None)
    if out is not None:
        _written(out)
    return y.mT if turned else y


# ----------------------------------------------------------------- experts --

def _tokens_of(name: str, x: torch.Tensor) -> torch.Tensor:
    if x.is_cuda and x.dtype in _HALVES and x.dim() == 2 and x.stride(1) == 1:
        return x
    if not x.is_cuda:
        raise TypeError("want CUDA tensors")
    if x.dtype not in _HALVES:
        raise TypeError(f"want bfloat16 or float16 {name}, not {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"want {name} [tokens, features]")
    return x if x.shape[1] <= 1 else x.detach().contiguous()


def _weight_of(w: torch.Tensor, x: torch.Tensor):
    """(the experts' matrices, whether they are the transposes of w's)"""
    if w.dtype != x.dtype or w.device != x.device:
        raise TypeError("want weights of the tokens' type and device")
    shape, stride = w.shape, w.stride()
    if len(shape) != 3 or shape[0] < 1:
        raise ValueError("want weights [experts, out features, in features]")
    if stride[2] != 1 and shape[2] > 1:
        if stride[1] == 1:
            return _matrices_t(w.data_ptr(), shape[0], shape[2], shape[1], stride[0], stride[2], _CODES[w.dtype]), 1, w
        w = w.detach().contiguous()
        stride = w.stride()
    return _matrices_t(w.data_ptr(), *shape, stride[0], stride[1], _CODES[w.dtype]), 0, w


def _offsets_of(offsets: torch.Tensor, experts: int, device) -> torch.Tensor:
    if offsets.dtype is torch.int64 and offsets.device == device and offsets.shape == (experts + 1,) and offsets.is_contiguous():
        return offsets
    if offsets.dtype != torch.int64 or offsets.device != device:
        raise TypeError("want int64 offsets on the tokens' device")
    if offsets.shape != (experts + 1,):
        raise ValueError(f"want {experts + 1} offsets for {experts} experts, not {tuple(offsets.shape)}")
    return offsets.contiguous()


def _rows_product(x, w, transposed, offsets, y):
    lib = A.load()
    a = _byref(_matrices(x))
    b = _byref(w)
    # few tokens are multiplied by the weights as they lie
    nbytes = 0 if x.shape[0] <= A.EXPERT_STREAM_ROWS and not transposed and y.shape[1] < 1 << 24 \
        else lib.adamw_expert_workspace(a, b)
    work = _empty(nbytes, dtype=_BYTES, device=x.device) if nbytes else None
    _call(lib.adamw_expert_rows, "adamw_expert_rows", x.device, a, b, transposed, offsets.data_ptr(),
          _byref(_matrices(y)), work.data_ptr() if nbytes else None)
    return y


def _expert_linear(x, weight, offsets, out):
    x = _tokens_of("tokens", x)
    w, transposed, _keep = _weight_of(weight, x)
    experts, n, k = weight.shape
    if k != x.shape[1]:
        raise ValueError(f"weights {tuple(weight.shape)} do not match tokens {tuple(x.shape)}")
    offsets = _offsets_of(offsets, experts, x.device)
    if out is None:
        out = _empty((x.shape[0], n), dtype=x.dtype, device=x.device)
    elif out.shape != (x.shape[0], n) or out.device != x.device or out.dtype not in _CODES or (n > 1 and out.stride(1) != 1):
        raise ValueError("out must be [tokens, out features] on the tokens' device, rows of consecutive elements")
    return _rows_product(x, w, transposed, offsets, out)


class _ExpertLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, offsets):
        y = _expert_linear(x, weight, offsets, None)
        ctx.save_for_backward(x, weight, offsets)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, offsets = ctx.saved_tensors   # checked by the forward pass
        return (*_gradients(dy, x, weight, offsets, ctx.needs_input_grad, None, False), None)


def expert_linear(x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor, *,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[t] = weight[e] x[t] for every token t of expert e: x [tokens, in],
    weight [experts, out, in] (or a transposed view of [experts, in, out]),
    bf16 or fp16; sums in fp32, rounded once.  Tokens of no expert give zeros.
    Differentiable in x and weight; forward mode has no rule and is refused.
    ``out`` (bf16, fp16 or fp32) takes the result where no gradient is wanted."""
    wanted = torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad)
    if wanted or _tangent(x).tangent is not None or _tangent(weight).tangent is not None:
        if out is not None:
            raise RuntimeError("out= takes no part in autograd")
        return _ExpertLinear.apply(x, weight, offsets)
    if out is not None and out.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("out requires a gradient")
    y = _expert_linear(x, weight, offsets, out)
    if out is not None:
        _written(out)
    return y


def expert_linear_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor, *,
                           need=(True, True), d_weight: Optional[torch.Tensor] = None, accumulate: bool = False):
    """(gradient of x, gradient of weight) of ``expert_linear``; ``need`` says
    which are wanted (None for the other).  ``d_weight``: where the weights'
    gradient goes, [experts, out, in] in bf16, fp16 or fp32 (for example an
    optimizer's own gradient buffer); with ``accumulate`` it is added there, in
    fp32 before the rounding."""
    x = _tokens_of("tokens", x)
    w, _, _ = _weight_of(weight, x)
    if dy.dtype != x.dtype or dy.device != x.device:
        raise TypeError("want gradients of the tokens' type and device")
    if dy.shape != (x.shape[0], weight.shape[1]) or weight.shape[2] != x.shape[1]:
        raise ValueError(f"gradients {tuple(dy.shape)}, tokens {tuple(x.shape)} and weights {tuple(weight.shape)} do not match")
    offsets = _offsets_of(offsets, weight.shape[0], x.device)
    if accumulate and d_weight is None:
        raise ValueError("accumulate needs d_weight")
    if d_weight is not None:
        if d_weight.requires_grad and torch.is_grad_enabled():
            raise RuntimeError("d_weight requires a gradient")
        if d_weight.shape != weight.shape or d_weight.device != x.device or d_weight.dtype not in _CODES:
            raise ValueError("d_weight must have the weights' shape and device, in bfloat16, float16 or float32")
        s = d_weight.stride()
        if not (s[2] == 1 or d_weight.shape[2] <= 1 or s[1] == 1):
            raise ValueError("d_weight needs consecutive elements along one of its last two dimensions")
    return _gradients(dy, x, weight, offsets, need, d_weight, accumulate)


def _gradients(dy, x, weight, offsets, need, dw, accumulate):
    """Of arguments that fit each other."""
    dy, x = _tokens_of("gradients", dy), _tokens_of("tokens", x)
    w, transposed, _keep = _weight_of(weight, x)
    if not offsets.is_contiguous():
        offsets = offsets.contiguous()
    dev, dtype = x.device, x.dtype
    dx = _empty(x.shape, dtype=dtype, device=dev) if need[0] else None
    given = dw is not None and need[1]
    turned, d = 0, None
    if need[1]:
        e, n, k = weight.shape
        if dw is None:   # laid out as the weights are
            dw = _empty((e, k, n), dtype=dtype, device=dev).mT if transposed else _empty((e, n, k), dtype=dtype, device=dev)
        s = dw.stride()
        turned = 0 if s[2] == 1 or k <= 1 else 1
        d = _matrices_t(dw.data_ptr(), e, k, n, s[0], s[2], _CODES[dw.dtype]) if turned else \
            _matrices_t(dw.data_ptr(), e, n, k, s[0], s[1], _CODES[dw.dtype])
    else:
        dw = None
    lib = A.load()
    a, b, c = _byref(_matrices(dy)), _byref(_matrices(x)), _byref(w)
    nbytes = lib.adamw_expert_backward_workspace(a, b, c)
    work = _empty(nbytes, dtype=_BYTES, device=dev) if nbytes else None
    _call(lib.adamw_expert_backward, "adamw_expert_backward", dev, a, b, c, transposed, offsets.data_ptr(),
          _byref(_matrices(dx)) if need[0] else None, _byref(d) if need[1] else None, turned, int(accumulate),
          work.data_ptr() if nbytes else None)
    if given:
        _written(dw)
    return dx, dw
