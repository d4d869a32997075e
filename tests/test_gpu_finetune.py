"""The example runs: log-probabilities, both losses, the global clip and the
optimizer together train a small model toward its reward."""
import math
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_example_trains(kind):
    import finetune
    h = finetune.train(kind, steps=25, say=lambda *_: None)
    assert all(math.isfinite(v) for e in h for v in e.values())
    mean = lambda part: sum(e["reward"] for e in part) / len(part)
    # half of the tokens earn the reward by chance
    assert abs(h[0]["reward"] - 0.5) < 0.1
    assert mean(h[-5:]) > mean(h[:5]) + 0.1
    if kind == "preference":
        assert abs(h[0]["loss"] - math.log(2)) < 0.02   # the model starts as its reference
    else:
        assert all(e["tokens"] == 32 * finetune.ANSWER for e in h) and abs(h[0]["kl"]) < 1e-3
