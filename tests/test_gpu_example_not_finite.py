"""Choosing a token where the model's numbers have run away: no exception on the device, the other tokens as before."""

import pytest
import torch

from matrix_optimizer_update_gb300 import example_moe_lm as ex

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), 3e38])
def test_choices_without_finite_logits(value):
    model = ex.Model(vocab=300, dim=64, inner=96, experts=4, top=2, max_tokens=20)
    x = torch.arange(20, device="cuda")
    best = model.choose(x, top=1)
    with torch.no_grad():
        model.embedding[3] = value
    chosen = model.choose(x, top=5)
    keep = x != 3
    assert bool(((chosen >= -1) & (chosen < 300)).all()) and bool((chosen[keep] >= 0).all())
    assert torch.equal(model.choose(x, top=1)[keep], best[keep])
    with torch.no_grad():
        model.head_weight[:] = value
    chosen = model.choose(x, top=5)
    assert bool(((chosen >= -1) & (chosen < 300)).all())
    torch.cuda.synchronize()
