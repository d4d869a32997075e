"""Host-side checks of the fine-tuning operators' C ABI: workspace sizes and
refusals.  No GPU: every call here is refused before anything is launched
(addresses are never dereferenced)."""
import ctypes
import math

import pytest
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A
from adamw_optimizer_step_sm_gb300 import losses as L

BAD, MIS, BIG = A.ADAMW_ERR_INVALID_ARG, A.ADAMW_ERR_MISALIGNED, A.ADAMW_ERR_TOO_LARGE
P = 1 << 40   # an address that is never read


def _rows(**k):
    d = dict(data=P, rows=8, inner=8, outer_stride=0, row_stride=100, cols=100, dtype=A.DTYPE_BF16)
    d.update(k)
    return A.adamw_rows_t(*(d[n] for n, _ in A.adamw_rows_t._fields_))


def _status(f, *args):
    with pytest.raises(A.AdamWError) as e:
        f(*args)
    return e.value.status


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), BAD), (dict(cols=-1), BAD), (dict(cols=0), BAD), (dict(inner=0), BAD), (dict(inner=3), BAD),
    (dict(row_stride=-100), BAD), (dict(outer_stride=-1), BAD), (dict(dtype=3), BAD), (dict(data=None), BAD),
    (dict(data=P + 1), MIS), (dict(rows=1 << 31, inner=1 << 31), BIG), (dict(row_stride=1 << 41), BIG),
])
def test_logits_are_checked(change, status):
    bad, good = _rows(**change), _rows()
    assert _status(A.adamw_token_logprob, bad, P, -100, 1.0, P) == status
    big = 2 << 40
    assert _status(A.adamw_token_logprob_backward, bad, P, -100, 1.0, P, 0, P, 0, _rows(data=P + big)) == status
    rc = _status(A.adamw_token_logprob_backward, good, P, -100, 1.0, P, 0, P, 0,
                 _rows(**dict(dict(data=P + big), **change)))
    assert rc == status


@pytest.mark.parametrize("scale", [0.0, -1.0, math.inf, math.nan, 3e38])
def test_scale_is_checked(scale):
    assert _status(A.adamw_token_logprob, _rows(), P, -100, scale, P) == BAD


def test_token_logprob_pointers():
    x = _rows()
    assert _status(A.adamw_token_logprob, x, 0, -100, 1.0, P) == BAD
    assert _status(A.adamw_token_logprob, x, P, -100, 1.0, 0) == BAD
    assert _status(A.adamw_token_logprob, x, P + 4, -100, 1.0, P) == MIS
    assert _status(A.adamw_token_logprob, x, P, -100, 1.0, P + 2) == MIS
    assert _status(A.adamw_token_logprob, x, P, -100, 1.0, P, 0, P + 4) == MIS
    # no rows: nothing to do, nothing looked at
    A.adamw_token_logprob(_rows(rows=0, data=None), 0, -100, 1.0, 0)


def test_gradient_rows_may_not_overlap():
    back = lambda x, d, **k: _status(A.adamw_token_logprob_backward, x, P, -100, 1.0, P, k.get("ent", 0), P,
                                     k.get("dh", 0), d)
    far = P + (1 << 30)
    x = _rows()
    assert back(x, _rows(data=far, row_stride=99)) == BAD              # rows into one another
    assert back(x, _rows(data=far, row_stride=0)) == BAD
    assert back(x, _rows(data=far, rows=8, inner=4, outer_stride=399, row_stride=100)) == BAD
    assert back(x, _rows(data=far, rows=8, inner=4, outer_stride=100, row_stride=199)) == BAD
    assert back(x, _rows(data=P + 16)) == BAD                          # into the logits
    assert back(x, _rows(row_stride=104)) == BAD                       # the same start, other rows
    assert back(x, _rows(data=far, cols=96)) == BAD                    # another shape
    assert back(x, _rows(data=far, dtype=A.DTYPE_FP16)) == BAD
    assert back(x, _rows(data=far), dh=P) == BAD                       # entropy's gradient without the entropy


def _policy(**k):
    d = dict(clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0, divisor=1.0, grad_scale=1.0,
             kl=3, reduce=0, advantage_per_token=0)
    d.update(k)
    return A.adamw_policy_t(*(d[n] for n, _ in A.adamw_policy_t._fields_))


def _call_policy(t=None, p=None, **k):
    a = dict(logp=P, old=P, ref=0, adv=P, ent=0, stats=P, counts=P, d_logp=P, d_ent=0, work=P)
    a.update(k)
    return _status(A.adamw_policy_loss, t or A.adamw_tokens_t(100, 10, None, None), p or _policy(), *a.values())


@pytest.mark.parametrize("change", [
    dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_high=-0.1), dict(clip_high=math.inf), dict(dual_clip=1.0),
    dict(dual_clip=-1.0), dict(dual_clip=math.inf), dict(kl_coef=math.nan), dict(entropy_coef=math.inf),
    dict(grad_scale=math.nan), dict(kl=0), dict(kl=4), dict(reduce=3), dict(reduce=2, divisor=0.0),
    dict(reduce=2, divisor=math.inf), dict(advantage_per_token=2), dict(kl_coef=0.1), dict(entropy_coef=0.1),
])
def test_policy_options_are_checked(change):
    assert _call_policy(p=_policy(**change)) == BAD


def test_policy_tokens_and_pointers_are_checked():
    T = A.adamw_tokens_t
    assert _call_policy(t=T(101, 10, None, None)) == BAD
    assert _call_policy(t=T(-1, 10, None, None)) == BAD
    assert _call_policy(t=T(5, 0, None, None)) == BAD
    assert _call_policy(t=T(1 << 31, 1, None, None)) == BIG
    assert _call_policy(t=T(100, 10, P + 4, None)) == MIS
    for k in ("logp", "old", "adv", "stats", "counts", "d_logp", "work"):
        assert _call_policy(**{k: 0}) == BAD
    for k in ("logp", "old", "ref", "adv", "ent", "stats", "d_logp", "d_ent"):
        assert _call_policy(**{k: P + 2}) == MIS
    assert _call_policy(counts=P + 4) == MIS and _call_policy(work=P + 8) == MIS
    assert _call_policy(p=_policy(entropy_coef=0.1), ent=P) == BAD    # no place for its gradient
    logits = lambda t, x: _status(A.adamw_policy_loss_logits, x, P, -100, 1.0, t, _policy(), P, 0, P, P, P, P, 0,
                                  _rows(data=P + (1 << 30)), P)
    assert logits(T(8, 2, None, P), _rows()) == BAD                   # a mask beside targets
    assert logits(T(9, 3, None, None), _rows()) == BAD                # other rows than tokens


def test_workspaces():
    assert A.adamw_policy_workspace(-1, 1) == 0 and A.adamw_policy_workspace(1, 1 << 31) == 0
    sizes = [A.adamw_policy_workspace(n, s) for n, s in ((0, 0), (1, 1), (1000, 8), (40000, 8), (40000, 9000),
                                                         (2_000_000, 2048))]
    assert sizes == sorted(sizes) and all(s > 0 and s % 16 == 0 for s in sizes)
    for n, s in ((1000, 8), (2_000_000, 2048)):
        more = A.adamw_policy_logits_workspace(n, s) - A.adamw_policy_workspace(n, s)
        assert more >= 16 * n   # row statistics and two gradients


def test_preference_is_checked():
    def call(t=None, n=4, **k):
        d = dict(beta=0.1, margin=0.0, label_smoothing=0.0, grad_scale=1.0, kind=0, length_average=0, ref=0)
        a = dict(logp=P, ref_logp=0, stats=P, losses=P, rewards=P, d_logp=P)
        for key, v in k.items():
            (a if key in a else d)[key] = v
        pref = A.adamw_preference_t(*(d[n] for n, _ in A.adamw_preference_t._fields_))
        return _status(A.adamw_preference_loss, t or A.adamw_tokens_t(40, n, None, None), pref, *a.values())
    for change in (dict(beta=0.0), dict(beta=-1.0), dict(beta=math.inf), dict(beta=1e-45), dict(margin=math.nan),
                   dict(label_smoothing=-0.1), dict(label_smoothing=0.6), dict(kind=3), dict(kind=1, label_smoothing=0.1),
                   dict(kind=2, margin=0.5), dict(ref=3), dict(ref=1), dict(grad_scale=math.inf), dict(n=5), dict(n=1),
                   dict(n=0), dict(logp=0), dict(stats=0), dict(losses=0), dict(rewards=0), dict(d_logp=0)):
        assert call(**change) == BAD, change
    assert call(logp=P + 2) == MIS


def test_clip_list_is_checked():
    make = lambda *e: _status(A.adamw_clip_plan_create, e)
    f32, bf16 = A.DTYPE_FP32, A.DTYPE_BF16
    assert make((P, P + 4096, -1, f32, f32)) == BAD
    assert make((None, P, 10, f32, f32)) == BAD
    assert make((P, None, 10, 7, f32)) == BAD
    assert make((P, P + 4096, 10, f32, 7)) == BAD
    assert make((P + 2, None, 10, f32, f32)) == MIS
    assert make((P, P + 4097, 10, bf16, bf16)) == MIS
    assert make((P, P, 10, f32, bf16)) == BAD            # in place with two types
    assert make((P, P + 36, 10, f32, f32)) == BAD        # overlapping
    assert make((P + 18, P, 10, bf16, bf16)) == BAD
    assert make((P, None, (1 << 40) + 1, bf16, bf16)) == BIG
    lib = A.load()
    assert lib.adamw_clip_plan_create(None, 1, ctypes.byref(ctypes.c_void_p())) == BAD
    assert lib.adamw_clip_plan_create(None, 0, None) == BAD
    assert lib.adamw_clip_grads(None, 1.0, 0, P, None) == BAD
    assert lib.adamw_clip_plan_destroy(None) == 0


def test_python_refuses_host_tensors():
    x, t = torch.zeros(2, 5), torch.zeros(2, dtype=torch.int64)
    for f in (lambda: L.token_logprob(x, t), lambda: L.policy_loss(x, x, x), lambda: L.preference_loss(x),
              lambda: L.policy_loss_logits(x, t, x[:, 0], x[:, 0]), lambda: A.ClipPlan([x])):
        with pytest.raises(TypeError):
            f()


def test_logits_geometry():
    """Leading dimensions become at most two levels of strides."""
    x = torch.zeros(3, 5, 4, 7)
    assert L._geometry(x[0, 0]) == (4, 4, 0, 7)
    assert L._geometry(x[0]) == (20, 4, 28, 7)
    assert L._geometry(x[0, :, :-1]) == (15, 3, 28, 7)
    assert L._geometry(x) [0] == 60
    n, inner, outer, row = L._geometry(x[:, :, :-1])     # [3, 5, 3] rows: (15) x 3
    assert (n, inner, outer, row) == (45, 3, 28, 7)
    assert L._geometry(x[:, 0].transpose(0, 1)) == (12, 3, 7, 140)
    with pytest.raises(ValueError):
        L._geometry(x[:, :-1, :-1])
    assert L._geometry(torch.zeros(9)) == (1, 1, 0, 0)
