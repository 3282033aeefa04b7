"""What learning from its own choices sends back to the model's log probabilities and entropies."""

import pytest
import torch

from matrix_optimizer_update_gb300 import example_moe_lm as ex

pytestmark = pytest.mark.gpu


def test_the_advantage_is_over_the_tokens_that_count(monkeypatch):
    seen = []
    policy = ex.Model.policy

    def kept(self, tokens, chosen):
        logp, entropy = policy(self, tokens, chosen)
        logp.retain_grad()
        entropy.retain_grad()
        seen.append((chosen, logp, entropy))
        return logp, entropy

    monkeypatch.setattr(ex.Model, "policy", kept)
    history = ex.reinforce(steps=3, tokens=160, vocab=300, warm=4, bonus=0.01, log=None)
    assert len(history) == len(seen) == 3
    for chosen, logp, entropy in seen:
        counts = chosen >= 0
        n = int(counts.sum())
        assert n == 150
        assert not logp.grad[~counts].any() and not entropy.grad[~counts].any()
        # 150 terms of at most 1 / 150, each rounded to fp32
        assert abs(float(logp.grad.double().sum())) <= 1e-6
        assert torch.allclose(entropy.grad[counts], torch.full((n,), -0.01 / n, device="cuda"), rtol=1e-5)
