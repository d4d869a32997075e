"""Token losses for fine-tuning, over torch tensors: what happens between a
model's logits and the optimizer step.

    token_logprob            log-probability (and entropy) of each token
    token_logprob_backward   its gradient with respect to the logits
    policy_loss              clipped policy loss with a KL term, and gradients
    policy_loss_logits       the same from logits, in one pass over them
    preference_loss          loss over pairs of sequences, and gradients

Every function is one call into the library (include/adamw_losses.h has the
formulas) on the current stream of the tensors' device, and waits for
nothing.  The losses return their gradients beside their values, for

    r = policy_loss_logits(logits, targets, old_logp, advantages)
    logits.backward(r.d_logits)

or ``logp.backward(r.d_logp)``: ``token_logprob`` is differentiable when its
logits require a gradient.

Layouts: logits are [vocabulary], [tokens, vocabulary] or [batch, tokens,
vocabulary] in bf16, fp16 or fp32, any strides as long as a row's elements
are consecutive (``logits[:, :-1]`` needs no copy); targets int64 of the
logits' leading shape.  Token arrays (log-probabilities, masks, advantages)
are fp32 [sequences, tokens], or [tokens] packed with ``offsets``, int64
[sequences + 1]: sequence i is tokens offsets[i] to offsets[i + 1] - 1.
Without offsets a flat array is one sequence.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import adamw_sm as A

# names looked up once: small calls are mostly host time
_byref = ctypes.byref
_empty = torch.empty
_rows_t, _tokens_t = A.adamw_rows_t, A.adamw_tokens_t
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
# what autograd has to be told of a tensor of the caller's that was written, so
# that a graph which saved its earlier values refuses to go on with the new ones
_written = torch.autograd.graph.increment_version
_tangent = torch.autograd.forward_ad.unpack_dual
_F32 = torch.float32
_CODES = {torch.bfloat16: A.DTYPE_BF16, torch.float16: A.DTYPE_FP16, torch.float32: A.DTYPE_FP32}


class TokenLogprob(NamedTuple):
    logp: torch.Tensor                # fp32, the targets' shape
    entropy: Optional[torch.Tensor]   # the same, when asked
    stats: torch.Tensor               # fp32 [..., 2], for the backward pass


class PolicyLoss(NamedTuple):
    stats: torch.Tensor               # fp32 [6]: loss, policy term, KL, entropy, clipped share, KL from old
    counts: torch.Tensor              # int64 [2]: tokens, sequences that count
    d_logp: torch.Tensor
    d_entropy: Optional[torch.Tensor]


class PolicyLogits(NamedTuple):
    stats: torch.Tensor
    counts: torch.Tensor
    logp: torch.Tensor
    entropy: Optional[torch.Tensor]
    d_logits: torch.Tensor


class PreferenceLoss(NamedTuple):
    stats: torch.Tensor               # fp32 [3]: loss, share of pairs in the right order, mean margin
    losses: torch.Tensor              # fp32 [pairs]
    rewards: torch.Tensor             # fp32 [2 * pairs]: beta times each sequence's log ratio
    d_logp: torch.Tensor


# ---------------------------------------------------------------- checking --

# The checks take the usual case first, in one condition.

def _call(f, name: str, device: torch.device, *args) -> None:
    """One library call on the device's current stream."""
    index = device.index
    if index == _current_device():
        rc = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = f(*args, _raw_stream(index))
    if rc:
        raise A.AdamWError(rc, name)


def _geometry(x: torch.Tensor):
    """(rows, inner, outer_stride, row_stride) of a tensor whose last dimension
    is a row."""
    shape, stride = x.shape, x.stride()
    nd = len(shape)
    if nd == 2:
        return shape[0], shape[0] or 1, 0, stride[0]
    if nd == 3:
        return shape[0] * shape[1], shape[1] or 1, stride[0], stride[1]
    if nd == 1:
        return 1, 1, 0, 0
    levels = []
    for n, s in zip(shape[:-1], stride[:-1]):
        if n == 1:
            continue
        if levels and levels[-1][1] == n * s:
            levels[-1] = (levels[-1][0] * n, s)
        else:
            levels.append((n, s))
    if len(levels) > 2:
        raise ValueError("the leading dimensions of the logits need more than two levels of strides")
    levels = [(1, 0)] * (2 - len(levels)) + levels
    return levels[0][0] * levels[1][0], max(1, levels[1][0]), levels[0][1], levels[1][1]


def _rows(x: torch.Tensor) -> A.adamw_rows_t:
    code, shape, stride = _CODES.get(x.dtype), x.shape, x.stride()
    nd = len(shape)
    if code is None or not x.is_cuda or nd == 0 or shape[-1] < 1 or (stride[-1] != 1 and shape[-1] > 1):
        if not x.is_cuda:
            raise TypeError("want CUDA tensors")
        if code is None:
            raise TypeError(f"want bfloat16, float16 or float32 logits, not {x.dtype}")
        if nd == 0 or shape[-1] < 1:
            raise ValueError("want logits of [..., vocabulary]")
        raise ValueError("the elements of a row of logits must be consecutive")
    if nd == 2:
        return _rows_t(x.data_ptr(), shape[0], shape[0] or 1, 0, stride[0], shape[1], code)
    if nd == 3:
        return _rows_t(x.data_ptr(), shape[0] * shape[1], shape[1] or 1, stride[0], stride[1], shape[2], code)
    return _rows_t(x.data_ptr(), *_geometry(x), shape[-1], code)


def _targets(t: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
    if t.dtype is torch.int64 and t.device == logits.device and t.shape == logits.shape[:-1] and t.is_contiguous():
        return t
    if t.dtype != torch.int64 or t.device != logits.device:
        raise TypeError("want int64 targets on the logits' device")
    if t.shape != logits.shape[:-1]:
        raise ValueError(f"targets {tuple(t.shape)} do not match logits {tuple(logits.shape)}")
    return t if t.is_contiguous() else t.contiguous()


def _floats(name: str, t: torch.Tensor, shape, device) -> torch.Tensor:
    if t.dtype is _F32 and t.shape == shape and t.device == device and t.is_contiguous():
        return t
    if t.dtype != torch.float32 or t.device != device:
        raise TypeError(f"want fp32 {name} on the same device")
    if t.shape != shape:
        raise ValueError(f"{name} {tuple(t.shape)} does not match {tuple(shape)}")
    return t if t.is_contiguous() else t.contiguous()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _like_rows(x: torch.Tensor) -> torch.Tensor:
    """A new tensor for the gradient of x, its rows at the same strides and the
    same distance from a 16-byte boundary (both sides then take 16-byte
    accesses whatever the vocabulary's size), unless x is spread too thin: more
    than a quarter beyond its own size, and 64 rows that a short batch may skip
    (``logits[:, :-1]`` of a few tokens), would be memory for nothing."""
    shape, stride, n = x.shape, x.stride(), x.numel()
    if len(shape) == 3 and n and stride[0] < stride[1]:   # [batch, tokens] stored as [tokens, batch]
        return _like_rows(x.transpose(0, 1)).transpose(0, 1)
    span = 1   # elements from the first to the last, so far
    for s, k in zip(reversed(stride), reversed(shape)):
        if k > 1:
            if s < span:   # overlapping rows (an expanded tensor), or dimensions in another order
                return _empty(shape, dtype=x.dtype, device=x.device)
            span += s * (k - 1)
    if n == 0 or span > n + n // 4 + 64 * shape[-1]:
        return _empty(shape, dtype=x.dtype, device=x.device)
    phase = x.data_ptr() % 16 // x.element_size()
    if phase == 0:
        return torch.empty_strided(shape, stride, dtype=x.dtype, device=x.device)
    return _empty(span + phase, dtype=x.dtype, device=x.device).as_strided(shape, stride, phase)


def _out_rows(out: Optional[torch.Tensor], x: torch.Tensor, rows: A.adamw_rows_t):
    """The tensor for the gradient of x, and its adamw_rows_t."""
    if out is None:
        size = 4 if rows.dtype == A.DTYPE_FP32 else 2
        if ((rows.data or 0) | (rows.row_stride | rows.outer_stride | rows.cols) * size) % 16 == 0:
            # every row starts at a 16-byte boundary: so do a contiguous tensor's
            out = _empty(x.shape, dtype=x.dtype, device=x.device)
            d = _rows_t.from_buffer_copy(rows)
            d.data, d.row_stride, d.outer_stride = out.data_ptr(), rows.cols, rows.inner * rows.cols
            return out, d
        out = _like_rows(x)
    elif out.shape != x.shape or out.dtype != x.dtype or out.device != x.device:
        raise ValueError("out must have the logits' shape, type and device")
    if out.stride() == x.stride():
        d = _rows_t.from_buffer_copy(rows)
        d.data = out.data_ptr()
        return out, d
    return out, _rows(out)


def _scale(temperature: float) -> float:
    if not temperature > 0:
        raise ValueError("want temperature > 0")
    return 1.0 / temperature


# ------------------------------------------------------ log-probabilities --

def _token_logprob(logits, targets, ignore_index, temperature, entropy) -> TokenLogprob:
    rows, t = _rows(logits), _targets(targets, logits)
    dev, shape = logits.device, targets.shape
    logp = _empty(shape, dtype=_F32, device=dev)
    ent = _empty(shape, dtype=_F32, device=dev) if entropy else None
    stats = _empty((*shape, 2), dtype=_F32, device=dev)
    _call(A.load().adamw_token_logprob, "adamw_token_logprob", dev, _byref(rows), t.data_ptr(), ignore_index, _scale(temperature),
          logp.data_ptr(), _ptr(ent), stats.data_ptr())
    return TokenLogprob(logp, ent, stats)


class _TokenLogprob(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, ignore_index, temperature, entropy):
        r = _token_logprob(logits, targets, ignore_index, temperature, entropy)
        ctx.save_for_backward(logits, targets, *r)
        ctx.options = (ignore_index, temperature)
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(r.stats)
        return tuple(r)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_logp, d_entropy, _):
        logits, targets, logp, ent, stats = ctx.saved_tensors
        if d_logp is None and d_entropy is None:
            return None, None, None, None, None
        if d_logp is None:
            d_logp = torch.zeros_like(logp)
        d = token_logprob_backward(logits, targets, TokenLogprob(logp, ent, stats), d_logp, d_entropy,
                                   ignore_index=ctx.options[0], temperature=ctx.options[1])
        return d, None, None, None, None


def token_logprob(logits: torch.Tensor, targets: torch.Tensor, *, ignore_index: int = -100,
                  temperature: float = 1.0, entropy: bool = False) -> TokenLogprob:
    """log softmax(logits / temperature) at the targets, and with ``entropy``
    the softmax's entropy; fp32.  Tokens whose target is ``ignore_index`` are
    not read and give 0.  Differentiable (logp and entropy) when the logits
    require a gradient; forward mode has no rule and is refused."""
    if logits.requires_grad and torch.is_grad_enabled() or _tangent(logits).tangent is not None:
        return TokenLogprob(*_TokenLogprob.apply(logits, targets, ignore_index, temperature, entropy))
    return _token_logprob(logits, targets, ignore_index, temperature, entropy)


def token_logprob_backward(logits: torch.Tensor, targets: torch.Tensor, result: TokenLogprob,
                           d_logp: torch.Tensor, d_entropy: Optional[torch.Tensor] = None, *,
                           ignore_index: int = -100, temperature: float = 1.0,
                           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient with respect to the logits, from ``token_logprob``'s result
    for the same arguments.  ``out=logits`` writes it over the logits."""
    rows, t = _rows(logits), _targets(targets, logits)
    dev, shape = logits.device, targets.shape
    stats = _floats("stats", result.stats, (*shape, 2), dev)
    dl = _floats("d_logp", d_logp, shape, dev)
    dh = ent = None
    if d_entropy is not None:
        if result.entropy is None:
            raise ValueError("a gradient of the entropy needs the forward pass's entropy")
        dh = _floats("d_entropy", d_entropy, shape, dev)
        ent = _floats("entropy", result.entropy, shape, dev)
    d, d_rows = _out_rows(out, logits, rows)
    _call(A.load().adamw_token_logprob_backward, "adamw_token_logprob_backward", dev, _byref(rows), t.data_ptr(), ignore_index, _scale(temperature),
          stats.data_ptr(), _ptr(ent), dl.data_ptr(), _ptr(dh), _byref(d_rows))
    if out is not None:
        _written(out)
    return d


# ------------------------------------------------------------ token losses --

def _tokens(shape, offsets, mask, device):
    """(adamw_tokens_t, sequences, what must stay alive) of token arrays."""
    n = shape.numel()
    if offsets is None and mask is not None and mask.dtype is torch.bool and mask.shape == shape \
            and mask.device == device and mask.is_contiguous():
        sequences = shape[0] if len(shape) > 1 else 1
        return _tokens_t(n, sequences, None, mask.data_ptr()), sequences, mask
    keep = []
    if offsets is not None:
        if offsets.dtype != torch.int64 or offsets.device != device or offsets.dim() != 1 or offsets.numel() < 1:
            raise TypeError("want int64 offsets [sequences + 1] on the same device")
        offsets = offsets if offsets.is_contiguous() else offsets.contiguous()
        keep.append(offsets)
        sequences = offsets.numel() - 1
    else:
        sequences = shape[0] if len(shape) > 1 else 1
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8) or mask.device != device:
            raise TypeError("want a bool or uint8 mask on the same device")
        if mask.shape != shape:
            raise ValueError(f"mask {tuple(mask.shape)} does not match {tuple(shape)}")
        mask = mask if mask.is_contiguous() else mask.contiguous()
        keep.append(mask)
    return _tokens_t(n, sequences, _ptr(offsets), _ptr(mask)), sequences, keep


def _detached(t):
    return t.detach() if t.requires_grad else t


def _per_token(name, v, shape, sequences, offsets, per_token):
    """Whether v is per token, as said or by its shape; as many packed tokens as
    sequences fit both, and then have to be told."""
    if per_token is not None:
        return bool(per_token)
    if v.shape != shape:
        return False
    if offsets is not None and sequences > 1 and shape == (sequences,):
        raise ValueError(f"as many sequences as tokens: say {name}_per_token=True or False")
    return True


def _advantages(a, shape, sequences, offsets, per_token, device):
    """(tensor, per token) of advantages."""
    if _per_token("advantage", a, shape, sequences, offsets, per_token):
        return _floats("advantages", a, shape, device), 1
    return _floats("advantages", a, (sequences,), device), 0


def _policy(clip_low, clip_high, dual_clip, kl, kl_coef, entropy_coef, reduce, divisor, grad_scale, per_token):
    if kl not in A.KL or reduce not in A.REDUCE:
        raise ValueError('want kl "k1", "k2" or "k3" and reduce "token", "sequence" or "fixed"')
    return A.adamw_policy_t(clip_low, clip_high, dual_clip, kl_coef, entropy_coef, divisor, grad_scale,
                            A.KL[kl], A.REDUCE[reduce], per_token)


def policy_loss(logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, *,
                ref_logp: Optional[torch.Tensor] = None, entropy: Optional[torch.Tensor] = None,
                mask: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                clip_low: float = 0.2, clip_high: float = 0.2, dual_clip: float = 0.0, kl: str = "k3",
                kl_coef: float = 0.0, entropy_coef: float = 0.0, reduce: str = "token",
                divisor: float = 1.0, grad_scale: float = 1.0,
                advantage_per_token: Optional[bool] = None) -> PolicyLoss:
    """The clipped policy loss of tokens, with a KL term to a reference and an
    entropy bonus, and its gradients with respect to ``logp`` and ``entropy``.

    ``advantages``: per token, or one per sequence, as their shape says; where
    it fits both (packed, as many sequences as tokens) ``advantage_per_token``
    has to say which.  ``mask``: tokens that count.  ``reduce``: mean over the
    tokens ("token"), mean over the sequences of their means ("sequence"), or a
    sum divided by ``divisor`` ("fixed").  ``grad_scale`` multiplies the
    gradients."""
    dev, shape = logp.device, logp.shape
    if not logp.is_cuda:
        raise TypeError("want CUDA tensors")
    logp = _floats("logp", _detached(logp), shape, dev)
    old = _floats("old_logp", old_logp, shape, dev)
    ref = None if ref_logp is None else _floats("ref_logp", ref_logp, shape, dev)
    ent = None if entropy is None else _floats("entropy", _detached(entropy), shape, dev)
    if kl_coef != 0.0 and ref is None:
        raise ValueError("a KL term needs ref_logp")
    if entropy_coef != 0.0 and ent is None:
        raise ValueError("an entropy term needs the entropy")
    tokens, sequences, _keep = _tokens(shape, offsets, mask, dev)
    adv, per_token = _advantages(advantages, shape, sequences, offsets, advantage_per_token, dev)
    policy = _policy(clip_low, clip_high, dual_clip, kl, kl_coef, entropy_coef, reduce, divisor, grad_scale,
                     per_token)
    stats = _empty(6, dtype=_F32, device=dev)
    counts = _empty(2, dtype=torch.int64, device=dev)
    d_logp = _empty(shape, dtype=_F32, device=dev)
    d_entropy = _empty(shape, dtype=_F32, device=dev) if ent is not None else None
    lib = A.load()
    work = _empty(lib.adamw_policy_workspace(tokens.n, sequences), dtype=torch.uint8, device=dev)
    _call(lib.adamw_policy_loss, "adamw_policy_loss", dev, _byref(tokens), _byref(policy), logp.data_ptr(), old.data_ptr(), _ptr(ref),
          adv.data_ptr(), _ptr(ent), stats.data_ptr(), counts.data_ptr(), d_logp.data_ptr(), _ptr(d_entropy),
          work.data_ptr())
    return PolicyLoss(stats, counts, d_logp, d_entropy)


def policy_loss_logits(logits: torch.Tensor, targets: torch.Tensor, old_logp: torch.Tensor,
                       advantages: torch.Tensor, *, ref_logp: Optional[torch.Tensor] = None,
                       entropy: bool = False, offsets: Optional[torch.Tensor] = None,
                       ignore_index: int = -100, temperature: float = 1.0, clip_low: float = 0.2,
                       clip_high: float = 0.2, dual_clip: float = 0.0, kl: str = "k3", kl_coef: float = 0.0,
                       entropy_coef: float = 0.0, reduce: str = "token", divisor: float = 1.0,
                       grad_scale: float = 1.0, out: Optional[torch.Tensor] = None,
                       advantage_per_token: Optional[bool] = None) -> PolicyLogits:
    """``token_logprob``, ``policy_loss`` and ``token_logprob_backward`` in one
    pass over the logits: each row is read once, and its gradient written once
    (to ``out``, which may be the logits themselves).  Tokens whose target is
    ``ignore_index`` do not count.  ``entropy`` asks for the entropy (implied
    by ``entropy_coef``)."""
    logits = _detached(logits)
    rows, t = _rows(logits), _targets(targets, logits)
    dev, shape = logits.device, targets.shape
    old = _floats("old_logp", old_logp, shape, dev)
    ref = None if ref_logp is None else _floats("ref_logp", ref_logp, shape, dev)
    if kl_coef != 0.0 and ref is None:
        raise ValueError("a KL term needs ref_logp")
    tokens, sequences, _keep = _tokens(shape, offsets, None, dev)
    adv, per_token = _advantages(advantages, shape, sequences, offsets, advantage_per_token, dev)
    policy = _policy(clip_low, clip_high, dual_clip, kl, kl_coef, entropy_coef, reduce, divisor, grad_scale,
                     per_token)
    d, d_rows = _out_rows(None if out is None else _detached(out), logits, rows)
    stats = _empty(6, dtype=_F32, device=dev)
    counts = _empty(2, dtype=torch.int64, device=dev)
    logp = _empty(shape, dtype=_F32, device=dev)
    ent = _empty(shape, dtype=_F32, device=dev) if entropy or entropy_coef != 0.0 else None
    lib = A.load()
    work = _empty(lib.adamw_policy_logits_workspace(tokens.n, sequences), dtype=torch.uint8, device=dev)
    _call(lib.adamw_policy_loss_logits, "adamw_policy_loss_logits", dev, _byref(rows), t.data_ptr(), ignore_index, _scale(temperature),
          _byref(tokens), _byref(policy), old.data_ptr(), _ptr(ref), adv.data_ptr(), stats.data_ptr(),
          counts.data_ptr(), logp.data_ptr(), _ptr(ent), _byref(d_rows), work.data_ptr())
    if out is not None:
        _written(out)
    return PolicyLogits(stats, counts, logp, ent, d)


def preference_loss(logp: torch.Tensor, ref_logp: Optional[torch.Tensor] = None, *,
                    mask: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                    beta: float = 0.1, margin: float = 0.0, kind: str = "sigmoid",
                    label_smoothing: float = 0.0, length_average: bool = False,
                    grad_scale: float = 1.0, ref_per_token: Optional[bool] = None) -> PreferenceLoss:
    """The preference loss of pairs and its gradient with respect to ``logp``:
    of 2 B sequences, i is preferred over B + i.  ``ref_logp``: the frozen
    reference's log-probabilities per token, its sums per sequence, or None;
    where its shape fits both (packed, as many sequences as tokens)
    ``ref_per_token`` has to say which.
    ``kind``: "sigmoid", "hinge" or "ipo".  ``length_average`` takes means
    over a sequence's tokens instead of sums."""
    dev, shape = logp.device, logp.shape
    if not logp.is_cuda:
        raise TypeError("want CUDA tensors")
    if kind not in A.PREFERENCE:
        raise ValueError('want kind "sigmoid", "hinge" or "ipo"')
    logp = _floats("logp", _detached(logp), shape, dev)
    tokens, sequences, _keep = _tokens(shape, offsets, mask, dev)
    if sequences < 2 or sequences % 2:
        raise ValueError("want an even number of sequences, the preferred ones first")
    pairs = sequences // 2
    ref, how = None, A.REF_NONE
    if ref_logp is not None:
        how = A.REF_TOKEN if _per_token("ref", ref_logp, shape, sequences, offsets, ref_per_token) else A.REF_SEQUENCE
        ref = _floats("ref_logp", ref_logp, shape if how == A.REF_TOKEN else (sequences,), dev)
    pref = A.adamw_preference_t(beta, margin, label_smoothing, grad_scale, A.PREFERENCE[kind],
                                1 if length_average else 0, how)
    stats = _empty(3, dtype=_F32, device=dev)
    losses = _empty(pairs, dtype=_F32, device=dev)
    rewards = _empty(sequences, dtype=_F32, device=dev)
    d_logp = _empty(shape, dtype=_F32, device=dev)
    _call(A.load().adamw_preference_loss, "adamw_preference_loss", dev, _byref(tokens), _byref(pref), logp.data_ptr(), _ptr(ref),
          stats.data_ptr(), losses.data_ptr(), rewards.data_ptr(), d_logp.data_ptr())
    return PreferenceLoss(stats, losses, rewards, d_logp)
