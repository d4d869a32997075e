"""What the global clip refuses of lists and optimizers on the GPU, and plans made
and used on different streams."""
import pytest
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A
from adamw_optimizer_step_sm_gb300.optim import AnyPrecisionAdamW, GlobalClip

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_a_tensor_or_an_optimizer_twice():
    g = torch.zeros(64, device=DEV)
    for grads, outs in (([g, g], None), ([g[:40], g[39:]], None), ([g, torch.zeros(64, device=DEV)], [g, g])):
        with pytest.raises(A.AdamWError) as e:
            A.ClipPlan(grads, outs)
        assert e.value.status == A.ADAMW_ERR_INVALID_ARG
    with pytest.raises(A.AdamWError):
        A.ClipPlan([g, g], norm_only=True)
    A.ClipPlan([g[:40], g[40:40], g[40:]]).close()
    opt = AnyPrecisionAdamW([torch.nn.Parameter(torch.zeros(8, device=DEV, dtype=torch.bfloat16))], lr=1e-3)
    with pytest.raises(ValueError):
        GlobalClip(opt, opt)


def test_plan_made_on_a_busy_stream():
    """A plan made while its stream has work queued, used on another stream."""
    g = torch.ones(64, device=DEV)
    torch.cuda.synchronize()
    busy, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(200_000_000)   # a tenth of a second
        plan = A.ClipPlan([g], norm_only=True)
    r = plan.clip(2.0, stream=other)
    torch.cuda.synchronize()
    assert float(r.norm) == 8.0 and abs(float(r.coef) - 0.25) < 1e-6 and int(r.nonfinite) == 0
