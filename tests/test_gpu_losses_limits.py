"""The fine-tuning operators at the limits of their inputs.

The definitions and tolerances are those of test_gpu_losses.py (in 64 bits, on
the CPU); what differs is derived at the test.
"""
import pytest
import torch

from adamw_optimizer_step_sm_gb300 import losses as L
from test_gpu_losses import DEV, _check_policy, _close_logp, _gen, _policy64, _policy_inputs, _rows64

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
