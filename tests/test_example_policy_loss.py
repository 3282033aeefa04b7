"""The example's policy loss, on the host: the baseline is that of the tokens that count, the others have no gradient."""

import pytest
import torch

from matrix_optimizer_update_gb300 import example_moe_lm as ex


@pytest.mark.parametrize("counts", [[True] * 6, [False, True, True, False, True, True], [False] * 6, [True] + [False] * 5])
@pytest.mark.parametrize("right", [[True] * 6, [False] * 6, [True, False, True, True, False, False]])
def test_gradients(counts, right):
    counts, right = torch.tensor(counts), torch.tensor(right)
    logp = torch.linspace(-3, -1, 6, dtype=torch.float64).requires_grad_()
    entropy = torch.linspace(1, 2, 6, dtype=torch.float64).requires_grad_()
    loss, average = ex.policy_loss(logp, entropy, right, counts, 0.01)
    loss.backward()
    n = max(1, int(counts.sum()))
    assert float(average) == pytest.approx(float((right & counts).sum()) / n)
    # as much pushes up as down, and nothing at all where all were right or none was
    assert abs(float(logp.grad.sum())) < 1e-6
    if bool((right == right[0]).all()):
        assert float(logp.grad.abs().max()) < 1e-6
    assert not logp.grad[~counts].any() and not entropy.grad[~counts].any()
    assert torch.allclose(entropy.grad[counts], torch.full((int(counts.sum()),), -0.01 / n, dtype=torch.float64))
    want = -(right.double() - average.double()) / n
    assert torch.allclose(logp.grad[counts], want[counts], atol=1e-7)


def test_masked_tokens_do_not_reach_the_loss():
    counts = torch.tensor([True, False, True])
    right = torch.tensor([True, True, False])
    logp, entropy = torch.tensor([-1.0, 0.0, -2.0]), torch.tensor([1.0, 5.0, 2.0])
    loss, average = ex.policy_loss(logp, entropy, right, counts, 0.5)
    assert float(average) == 0.5
    assert float(loss) == pytest.approx(-(0.5 * -1.0 - 0.5 * -2.0) / 2 - 0.5 * 3.0 / 2)
