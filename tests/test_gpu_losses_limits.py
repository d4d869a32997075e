"""The fine-tuning operators at the limits of their inputs.

The definitions and tolerances are those of test_gpu_losses.py (in 64 bits, on
the CPU); what differs is derived at the test.
"""
import math

import pytest
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A
from adamw_optimizer_step_sm_gb300 import losses as L
from adamw_optimizer_step_sm_gb300.optim import AnyPrecisionAdamW, GlobalClip
from test_gpu_losses import (DEV, INF, ROUND, TYPES, _check_policy, _close_logp, _gen, _grad64,
                             _policy64, _policy_inputs, _preference64, _rows64)

pytestmark = pytest.mark.gpu


# ------------------------------------------------ tokens outside the sequences

@pytest.mark.parametrize("n,at", [(24, 0), (300, 124), (20000, 0), (20000, 16384)])
@pytest.mark.parametrize("reduce", ["token", "sequence", "fixed"])
def test_few_tokens_between_tokens_outside(n, at, reduce):
    """Tokens before the first and after the last sequence beside one another:
    every start and length up to five, at every phase of a group of four."""
    logp, old, ref, ent, _, _, g = _policy_inputs(n, 2, n + at, False)
    on = torch.ones(n, dtype=torch.bool)
    x = torch.randn(n, 8, generator=g)
    t = torch.randint(0, 8, (n,), generator=g)
    adv = torch.tensor([1.5, -0.7])
    d = lambda v: v.to(DEV)
    data = [d(v) for v in (logp, old, ref, ent, x, t, adv)]
    lp = L.token_logprob(data[4], data[5])
    for start in range(at, at + 8):
        for length in range(1, 6):
            for mid in {start, start + 1, start + length}:
                starts = [start, mid, start + length]
                off = torch.tensor(starts, device=DEV)
                o = dict(clip_low=0.2, clip_high=0.28, dual=0.0, kl="k3", kl_coef=0.05, entropy_coef=0.01,
                         reduce=reduce, divisor=3.0, per_token=False)
                args = dict(offsets=off, clip_low=0.2, clip_high=0.28, kl_coef=0.05, reduce=reduce, divisor=3.0)
                got = L.policy_loss(data[0], data[1], data[6], ref_logp=data[2], entropy=data[3],
                                    entropy_coef=0.01, **args)
                _check_policy(got, _policy64(logp, old, adv, ref, ent, on, starts, o), True)
                # from logits: the same counts and weights
                r = L.policy_loss_logits(data[4], data[5], data[1], data[6], ref_logp=data[2], **args)
                p = L.policy_loss(lp.logp, data[1], data[6], ref_logp=data[2], **args)
                assert r.counts.tolist() == got.counts.tolist()
                back = L.token_logprob_backward(data[4], data[5], lp, p.d_logp)
                assert torch.isfinite(back).all() and back.abs().max() > 0
                assert (r.d_logits - back).abs().max() <= 1e-6 * back.abs().max()


# ------------------------------------------------------- maxima along a row

@pytest.mark.parametrize("offset", [1000.0, -1000.0, 8000.0])
@pytest.mark.parametrize("n,v", [(3, 4096), (160, 50272)])
def test_maxima_that_rise_along_a_row(n, v, offset):
    """Every batch of a thread has a new maximum, far from 0: the products of
    maximum and scale round, and a record moves by what they rounded to."""
    x = torch.linspace(0, 8, v) + 0.1 * torch.rand(n, v, generator=_gen(v)) + offset
    t = torch.randint(0, v, (n,), generator=_gen(n))
    want = _rows64(x, t, 1.0)
    r = L.token_logprob(x.to(DEV), t.to(DEV), entropy=True)
    _close_logp(r.logp, want[0])
    _close_logp(r.entropy, want[1])


# -------------------------------------------------- masks by finite numbers

def _masked_rows(v, dtype, mask):
    """Rows masked by `mask`: throughout, in a leading stretch, all but a few,
    in isolated aligned groups, and not; with their targets."""
    x = (torch.randn(6, v, generator=_gen(v)) * 3).to(TYPES[dtype])
    t = torch.tensor([v // 2, v - 1, v - 2, v - 3, 1, v // 3])
    x[0] = mask
    x[1, : v * 3 // 4] = mask
    keep = x[2, v - 5:].clone()
    x[2] = mask
    x[2, v - 5:] = keep
    for k in range(0, v - 32, 64):
        x[3, k:k + 8] = mask
    x[4] = mask
    x[4, 2] = 2 * mask if mask > torch.finfo(TYPES[dtype]).min / 2 else mask   # one entry below the others
    return x, t


MASKS = [("fp32", 1.0, m) for m in (-1e8, -1e9, -1e10, -1e12, -1e30, -1e37)] + \
        [("fp32", 1.0, torch.finfo(torch.float32).min), ("fp32", 6.0, torch.finfo(torch.float32).min)] + \
        [("bf16", 1.0, m) for m in (-1e9, -1e10, -1e30, -1e32, -1e37)] + \
        [("bf16", 6.0, torch.finfo(torch.bfloat16).min), ("bf16", 0.7, -1e10), ("fp16", 1e-3, -60000.0)]


@pytest.mark.parametrize("dtype,temperature,mask", MASKS)
@pytest.mark.parametrize("v", [40, 1000, 3001, 9000, 50272])
def test_masks_by_large_finite_numbers(v, dtype, temperature, mask):
    x, t = _masked_rows(v, dtype, mask)
    n, scale = x.shape[0], 1 / temperature
    want = _rows64(x, t, scale)
    xd, td = x.to(DEV), t.to(DEV)
    _close_logp(L.token_logprob(xd, td, temperature=temperature).logp, want[0])
    r = L.token_logprob(xd, td, temperature=temperature, entropy=True)
    _close_logp(r.logp, want[0])
    _close_logp(r.entropy, want[1])
    g = _gen(1)
    dl, dh = torch.randn(n, generator=g), 0.3 * torch.randn(n, generator=g)
    for h in (None, dh):
        d = L.token_logprob_backward(xd, td, r, dl.to(DEV), None if h is None else h.to(DEV), temperature=temperature)
        w = _grad64(want, t, dl.double(), None if h is None else h.double(), scale)
        # as _close_grad, and where the target's probability is near 1 its
        # gradient is a difference of numbers of size scale |dl|: 4 u of that
        tol = 1e-5 * w.abs().amax(1, keepdim=True) + 2.4e-7 * scale * dl.abs()[:, None].double() \
            + ROUND[dtype] * w.abs() + (2.0 ** -25 if dtype == "fp16" else 1e-38)
        assert ((d.cpu().double() - w).abs() <= tol).all()
    # and from logits: ratio 1, so the gradient is that of -A logp - 0.1 entropy, a token's weight 1 / n
    old = r.logp
    adv = torch.randn(n, generator=g)
    p = L.policy_loss_logits(xd, td, old, adv.to(DEV), entropy_coef=0.1, temperature=temperature)
    _close_logp(p.logp, want[0])
    _close_logp(p.entropy, want[1])
    w = _grad64(want, t, -adv.double() / n, torch.full((n,), -0.1 / n, dtype=torch.float64), scale)
    # the ratio is 1 to within the difference of the two calls' logp, two ulps of each
    top = w.abs().amax(1, keepdim=True)
    tol = (3e-5 + 5e-7 * want[0].abs()[:, None]) * (top + scale / n) + ROUND[dtype] * w.abs() + (2.0 ** -25 if dtype == "fp16" else 1e-38)
    assert ((p.d_logits.cpu().double() - w).abs() <= tol).all()


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("v", [256, 4096, 50272])
@pytest.mark.parametrize("center,step,offset", [(46516320.0, 4, 2), (744261120.0, 64, 32)])
def test_logits_where_their_product_with_the_scale_is_coarse(v, sign, center, step, offset):
    """Rising logits around 2^26 / log2 e and 2^30 / log2 e, fp32's spacing there
    apart.  The row's largest element may have an exponent of its own, up to
    `offset`: what is added and taken off again for it costs 4 u of it."""
    steps = torch.linspace(-30, 0, v).round() + torch.randint(-3, 4, (5, v), generator=_gen(v)).float()
    x = sign * center + step * steps
    t = torch.randint(0, v, (5,), generator=_gen(3))
    want = _rows64(x, t, 1.0)
    r = L.token_logprob(x.to(DEV), t.to(DEV), entropy=True)
    for got, exact in ((r.logp, want[0]), (r.entropy, want[1])):
        tol = 4e-6 + 2e-6 * exact.abs() + 2.4e-7 * offset
        assert ((got.cpu().double() - exact).abs() <= tol).all()
    dl = torch.randn(5, generator=_gen(4))
    d = L.token_logprob_backward(x.to(DEV), t.to(DEV), r, dl.to(DEV))
    w = _grad64(want, t, dl.double(), None, 1.0)
    tol = 1e-5 * w.abs().amax(1, keepdim=True) + 2.4e-7 * dl.abs()[:, None].double()
    assert ((d.cpu().double() - w).abs() <= tol).all()


# ------------------------------------------------------ extreme temperatures

@pytest.mark.parametrize("temperature", [1e-19, 1e-12, 1e-9, 1e-7, 1e-5, 1e22, 1e32])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("v", [40, 3001, 9000])
def test_extreme_temperatures(v, dtype, temperature):
    x, t = _rows_with_masks(v, dtype)
    scale = 1 / temperature
    want = _rows64(x, t, scale)
    xd, td = x.to(DEV), t.to(DEV)
    r = L.token_logprob(xd, td, temperature=temperature, entropy=True)
    _close_logp(r.logp, want[0])
    _close_logp(r.entropy, want[1])
    one = torch.ones(4, device=DEV)
    d = L.token_logprob_backward(xd, td, r, one, 0.5 * one, temperature=temperature)
    w = _grad64(want, t, torch.ones(4).double(), torch.full((4,), 0.5).double(), scale)
    if dtype == "fp16":
        w = torch.where(w.abs() > 65504, w.sign() * INF, w)   # what does not fit the type
    got = d.cpu().double()
    big = torch.isinf(w)
    assert torch.equal(got[big], w[big])
    w[big], got[big] = 0.0, 0.0
    # as _close_grad, and 4 u of what is added and taken off again: the target's
    # own gradient (its p is 1), and up to 32 times the entropy's for the exponent
    # of the row's largest element, which is 0 where that is past 2^30
    slack = 2.4e-7 * scale * (1 + 32 * 0.5) if 15.0625 * 1.4427 * scale < 2 ** 30 else 0.0
    tol = 1e-5 * w.abs().amax(1, keepdim=True) + slack + ROUND[dtype] * w.abs() + (2.0 ** -25 if dtype == "fp16" else 1e-38)
    assert ((got - w).abs() <= tol).all()


def _rows_with_masks(v, dtype):
    """Four rows of distinct best logits with some entries masked by -inf (in
    one a whole leading stretch, in one everything but one)."""
    x = (torch.randn(4, v, generator=_gen(v)) * 3).to(TYPES[dtype])
    x[:, ::5] = -INF
    x[2, : v * 3 // 4] = -INF
    x[3] = -INF
    x[:, v - 2] = 15.0625    # the best, and the target
    return x, torch.full((4,), v - 2)


# --------------------------------------------------------- preference losses

def _long_pairs(pairs, length, seed):
    """Answers of about `length` tokens and their log-probabilities of about -2,
    on a grid of 2^-12 (sums are exact in 64 bits), the two sums of a pair close."""
    g = _gen(seed)
    grid = lambda v: (v * 4096).round() / 4096
    logp = -grid(torch.rand(2 * pairs, length, generator=g) * 4)
    logp[pairs:] = logp[:pairs][:, torch.randperm(length, generator=g)]
    for i in range(pairs):   # differences of 2^-12 and more, of either sign, and none
        logp[pairs + i, i % length] += [1, -1, 3, 0, -40, 4096][i % 6] / 4096
    return logp


@pytest.mark.parametrize("pairs,length", [(3, 2500), (12, 4096), (40, 8191), (2, 70001)])
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("average", [False, True])
def test_preference_sums_that_nearly_cancel(pairs, length, kind, average):
    """Long answers without a reference: D is the difference of the unrounded
    sums.  Their pairs of floats are good to some 2^-46 of the size of what they
    hold, over thousands of additions and a few joins to 2^-40; then one rounding."""
    logp = _long_pairs(pairs, length, length)
    rows = 2 * pairs
    starts = [i * length for i in range(rows + 1)]
    o = dict(ref=None, average=average, beta=0.1, margin=0.0, kind=kind, eps=0.0)
    losses, rewards, grad, D, h = _preference64(logp.reshape(-1), None, torch.ones(rows * length, dtype=torch.bool),
                                                starts, o)
    got = L.preference_loss(logp.to(DEV), beta=0.1, kind=kind, length_average=average)
    size = logp.double().abs().sum(1) / (length if average else 1)
    dD = 3e-7 * D.abs() + 2.0 ** -40 * (size[:pairs] + size[pairs:])
    assert ((got.rewards.cpu().double() - rewards).abs() <= 3e-7 * rewards.abs()).all()
    slope = 2 * (D - 5).abs() if kind == "ipo" else torch.full_like(D, 0.1)
    assert ((got.losses.cpu().double() - losses).abs() <= slope * dD + dD * dD + 1e-6 * losses.abs()).all()
    second = {"sigmoid": 0.0025, "hinge": 0.0, "ipo": 2.0}[kind]
    tol = (second * dD / pairs / (length if average else 1)).repeat(2).repeat_interleave(length)
    assert ((got.d_logp.cpu().double().reshape(-1) - grad).abs() <= 2e-6 * grad.abs() + tol + 1e-12).all()


@pytest.mark.parametrize("pairs,length", [(7, 1100), (40, 8191), (2, 70001)])
@pytest.mark.parametrize("average", [False, True])
def test_preference_statistics_of_close_pairs(pairs, length, average):
    """The share of pairs with D > 0 goes by D itself, and the mean of h is as
    good as D."""
    logp = _long_pairs(pairs, length, length + 1)
    S = logp.double().sum(1) / (length if average else 1)
    D = S[:pairs] - S[pairs:]
    got = L.preference_loss(logp.to(DEV), beta=0.1, margin=0.25, length_average=average)
    s = got.stats.cpu().double()
    share = (D > 0).double().mean()
    assert 0 < share < 1 and abs(float(s[1] - share)) <= 1e-7
    size = logp.double().abs().sum(1).max() / (length if average else 1)
    err = 4e-7 * (0.1 * D.abs() + 0.25).mean() + 0.1 * 2.0 ** -39 * size
    assert abs(float(s[2]) - float((0.1 * D - 0.25).mean())) <= err
    want = -torch.nn.functional.logsigmoid(0.1 * D - 0.25)
    assert abs(float(s[0] - want.mean())) <= 1e-6 * float(want.mean()) + err


def test_preference_order_of_a_pair():
    """The first half of the sequences is the preferred one."""
    r = L.preference_loss(torch.tensor([[2000.0], [-2000.0], [-2000.0], [2000.0]], device=DEV), beta=1.0)
    assert r.losses.tolist() == [0.0, 4000.0] and r.stats[1] == 0.5


# ------------------------------------------------- as many sequences as tokens

def test_advantages_where_both_readings_fit():
    """Three tokens, three sequences, one of them empty and one of two tokens."""
    z = torch.zeros(3, device=DEV)
    off = torch.tensor([0, 2, 2, 3], device=DEV)
    adv = torch.tensor([1.0, 50.0, 3.0], device=DEV)
    x, t = torch.zeros(3, 5, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    call = lambda **k: L.policy_loss(z, z, adv, offsets=off, reduce="fixed", **k).d_logp.tolist()
    rows = lambda **k: L.policy_loss_logits(x, t, torch.full((3,), -math.log(5), device=DEV), adv, offsets=off,
                                            reduce="fixed", **k).d_logits[:, 0]
    assert call(advantage_per_token=True) == [-1.0, -50.0, -3.0]
    assert call(advantage_per_token=False) == [-1.0, -1.0, -3.0]
    for per, want in ((True, (1.0, 50.0, 3.0)), (False, (1.0, 1.0, 3.0))):
        assert (rows(advantage_per_token=per).cpu() + 0.8 * torch.tensor(want)).abs().max() < 1e-4
    with pytest.raises(ValueError):
        call()
    with pytest.raises(ValueError):
        rows()
    # one reading only: as before, and the argument has to agree with the shape
    assert L.policy_loss(z, z, adv[:2], offsets=off[[0, 1, 3]], reduce="fixed").d_logp.tolist() == [-1.0, -1.0, -50.0]
    with pytest.raises(ValueError):
        L.policy_loss(z, z, adv[:2], offsets=off[[0, 1, 3]], advantage_per_token=True)
    with pytest.raises(ValueError):
        L.policy_loss(z, z, adv, offsets=off[[0, 1, 3]], advantage_per_token=False)
    # one token in one sequence: both readings are the same
    assert L.policy_loss(z[:1], z[:1], adv[:1], offsets=off[[0, 3]] // 3).d_logp.tolist() == [-1.0]


def test_reference_where_both_readings_fit():
    logp = torch.tensor([-1.0, -2.0], device=DEV)
    off = torch.tensor([0, 2, 2], device=DEV)     # two tokens preferred to an empty answer
    ref = torch.tensor([-0.5, -4.0], device=DEV)
    call = lambda **k: L.preference_loss(logp, ref, offsets=off, beta=0.5, **k).rewards.tolist()
    assert call(ref_per_token=True) == [0.75, 0.0]
    assert call(ref_per_token=False) == [-1.25, 2.0]
    with pytest.raises(ValueError):
        call()
    four = torch.zeros(4, device=DEV)
    for per, size in ((True, 2), (False, 4)):
        with pytest.raises(ValueError):
            L.preference_loss(four, torch.zeros(size, device=DEV), offsets=off, ref_per_token=per)


# ------------------------------------------------------- what autograd has to know

@pytest.mark.parametrize("which", ["backward", "policy"])
def test_a_graph_over_logits_that_were_overwritten_is_refused(which):
    x = torch.randn(4, 33, device=DEV).requires_grad_(True)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    y = x * 1.0
    r = L.token_logprob(y, t)
    d, z = y.detach(), torch.zeros(4, device=DEV)
    if which == "backward":
        L.token_logprob_backward(d, t, L.TokenLogprob(*(v if v is None else v.detach() for v in r)), z, out=d)
    else:
        L.policy_loss_logits(d, t, z, z, out=d)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        r.logp.sum().backward()


def test_a_graph_over_clipped_tensors_is_refused():
    a = torch.randn(100, device=DEV).requires_grad_(True)
    for in_place in (True, False):
        g, o = torch.randn(100, device=DEV), torch.zeros(100, device=DEV)
        y = (a * (g if in_place else o)).sum()
        A.ClipPlan([g], None if in_place else [o]).clip(0.1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    g = torch.randn(100, device=DEV)
    y = (a * g).sum()
    A.ClipPlan([g], norm_only=True).clip(0.1)     # writes no gradient
    y.backward()


def test_a_graph_over_an_optimizers_gradients_is_refused():
    p = torch.nn.Parameter(torch.randn(40, device=DEV).bfloat16())
    opt = AnyPrecisionAdamW([p], lr=1e-3)
    clip = GlobalClip(opt)
    opt.zero_grad()
    p.grad.fill_(1.0)
    x = torch.randn(40, device=DEV).bfloat16().requires_grad_(True)
    y = (x * p.grad).sum()
    clip(0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_forward_mode_is_refused():
    import torch.autograd.forward_ad as fwd
    x, t = torch.randn(4, 33, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    with fwd.dual_level():
        assert L.token_logprob(x, t).logp.shape == (4,)
        with pytest.raises(NotImplementedError):
            L.token_logprob(fwd.make_dual(x, torch.ones_like(x)), t)


# -------------------------------------------------------- ratios past fp32

@pytest.mark.parametrize("n", [6, 20000])
def test_ratios_past_fp32(n):
    """A token whose old log-probability is the type's lowest value or -inf has
    an infinite ratio: with advantage 0 it adds nothing."""
    old = torch.zeros(n, device=DEV)
    old[1], old[2], old[3] = -200.0, torch.finfo(torch.float32).min, -INF
    adv = torch.zeros(n, device=DEV)
    adv[4] = 1.0
    r = L.policy_loss(torch.zeros(n, device=DEV), old, adv, mask=torch.arange(n, device=DEV) < 5, reduce="fixed")
    assert r.stats[0] == -1.0 and r.stats[4] == 0.0
    assert r.d_logp[:5].tolist() == [0.0, 0.0, 0.0, 0.0, -1.0]
    x, t = torch.zeros(n, 3, device=DEV), torch.zeros(n, dtype=torch.int64, device=DEV)
    r = L.policy_loss_logits(x, t, old - math.log(3), adv, reduce="fixed")
    assert abs(float(r.stats[0]) + 1.0) < 1e-6
    assert (r.d_logits[:4] == 0).all() and (r.d_logits[4].cpu() - torch.tensor([-2 / 3, 1 / 3, 1 / 3])).abs().max() < 1e-5
    # a NaN is seen all the same
    nan = torch.full((2,), float("nan"), device=DEV)
    assert torch.isnan(L.policy_loss(nan, nan, torch.zeros(1, device=DEV)).stats[0])


@pytest.mark.parametrize("n", [12, 20000])
def test_kl_gradient_of_far_references(n):
    """d KL / d logp of k3 is 1 - exp(-k): exp is good to 2 ulps, the rest rounds."""
    k = torch.tensor([1e-3, 0.3, 0.69, 0.71, 1.0, 10.0, 1e3, 1e6, 1e8, 1e12, INF])
    logp, ref = torch.zeros(n), torch.zeros(n)
    ref[:11] = -k
    r = L.policy_loss(logp.to(DEV), logp.to(DEV), torch.zeros(1, device=DEV), ref_logp=ref.to(DEV), kl_coef=0.5,
                      mask=torch.arange(n, device=DEV) < 11, reduce="fixed")
    want = -0.5 * torch.expm1(-k.double())
    assert ((r.d_logp[:11].cpu().double() - want).abs() <= 1e-6 * want).all()


def test_kl_to_a_reference_that_the_policy_left():
    """logp -inf: the k3 estimate and the KL from the old policy are +inf, not NaN."""
    t = lambda *v: torch.tensor(v, device=DEV)
    r = L.policy_loss(t(-INF, 0.0), t(-1.0, 0.0), t(1.0), ref_logp=t(-1.0, 0.0))
    assert r.stats[2] == INF and r.stats[5] == INF
    r = L.policy_loss(t(0.0, 0.0), t(-INF, 0.0), t(1.0), ref_logp=t(0.0, 0.0))
    assert r.stats[5] == INF and r.stats[2] == 0


@pytest.mark.parametrize("v", [33, 3000, 450001])
def test_rows_outside_every_sequence_are_not_used(v):
    """Whatever they hold, in rows of a warp, a CTA, and too long for a cluster."""
    x = torch.randn(4, v, generator=_gen(v))
    x[0, v // 2] = float("nan")
    x[3] = INF
    t = torch.tensor([1, 2, 3, v])   # the last target is outside the vocabulary, too
    off = torch.tensor([1, 3], device=DEV)
    old = torch.full((4,), -10.0, device=DEV)
    r = L.policy_loss_logits(x.to(DEV), t.to(DEV), old, torch.ones(1, device=DEV), offsets=off, entropy_coef=0.1)
    assert r.counts.tolist() == [2, 1] and torch.isfinite(r.stats).all()
    d = r.d_logits
    assert (d[0] == 0).all() and (d[3] == 0).all()
    assert torch.isfinite(d[1:3]).all() and d[1].abs().max() > 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v", [40, 9000])
def test_log_probabilities_near_the_types_range(v, dtype):
    """A target of the lowest value beside the largest one: their difference is
    not a number of the type, its product with the scale is."""
    top = torch.finfo(TYPES[dtype]).max
    x = torch.full((6, v), -INF, dtype=TYPES[dtype])
    x[:, 0] = torch.tensor([top, top, top / 4, 0.0, -top / 2, -top])
    x[:, 1] = torch.tensor([-top, -top / 2, -top, -top, -top, -INF])
    t = torch.ones(6, dtype=torch.int64)
    for temperature in (1e-3, 0.7, 1.5, 6.0, 1e3):
        r = L.token_logprob(x.to(DEV), t.to(DEV), temperature=temperature)
        want = _rows64(x, t, 1 / temperature)[0]
        fits, over = want.abs() < 3.40e38, want.abs() > 3.41e38   # at the limit itself either
        got = r.logp.cpu().double()
        assert ((got - want).abs() <= 4e-7 * want.abs())[fits].all() and (got[over] == -INF).all()
