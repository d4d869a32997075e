"""Lists that the global clip refuses because their buffers overlap.  No GPU:
they are refused before anything is allocated or looked up (addresses are never
dereferenced)."""
import pytest
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A

P = 1 << 40   # an address that is never read
F32, BF16 = A.DTYPE_FP32, A.DTYPE_BF16


def _status(*entries):
    with pytest.raises(A.AdamWError) as e:
        A.adamw_clip_plan_create(entries)
    return e.value.status


def _far(k):
    return P + (k << 30)


@pytest.mark.parametrize("entries", [
    # one gradient twice: in place, into two places, and for the norm alone
    [(P, P, 100, F32, F32), (P, P, 100, F32, F32)],
    [(P, _far(1), 100, F32, F32), (P, _far(2), 100, F32, BF16)],
    [(P, None, 100, F32, F32), (P, None, 100, F32, F32)],
    # two gradients into one place
    [(P, _far(2), 100, F32, F32), (_far(1), _far(2), 100, BF16, F32)],
    # by one element, at either end, and inside one another
    [(P, P, 100, F32, F32), (P + 396, P + 396, 100, F32, F32)],
    [(P + 396, P + 396, 100, F32, F32), (P, P, 100, F32, F32)],
    [(P, P, 100, F32, F32), (P + 200, None, 4, BF16, BF16)],
    # what one writes is what another reads
    [(P, _far(1), 100, F32, BF16), (_far(1) + 198, _far(2), 100, BF16, BF16)],
    # among others, with an empty tensor between them
    [(_far(5), _far(6), 9, F32, F32), (P, P, 100, F32, F32), (P, P, 0, F32, F32), (_far(7), None, 9, F32, F32),
     (P + 4, P + 4, 50, F32, F32)],
])
def test_overlapping_buffers_are_refused(entries):
    assert _status(*entries) == A.ADAMW_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="would make plans over addresses that hold nothing")
@pytest.mark.parametrize("entries", [
    [(P, P, 100, F32, F32), (P + 400, P + 400, 100, F32, F32)],           # one beside the other
    [(P + 400, _far(1), 100, F32, BF16), (P, _far(1) + 200, 100, F32, BF16)],
    [(P, P, 100, F32, F32), (P, None, 0, F32, F32), (P + 8, P + 8, 0, F32, F32)],
    [(P, _far(1), 100, F32, BF16), (P + 400, None, 1, F32, F32), (P + 404, P + 404, 3, F32, F32)],
])
def test_neighbouring_buffers_are_not(entries):
    """Refused here for want of a GPU or of the memory, not as overlapping."""
    assert _status(*entries) in (A.ADAMW_ERR_CUDA, A.ADAMW_ERR_NOT_ACCESSIBLE)
