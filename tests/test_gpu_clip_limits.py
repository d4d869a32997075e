"""What the global clip refuses of lists and optimizers on the GPU."""
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
