"""The example's log probabilities on the host, with a stand-in for the head: both gradients come through, and second
derivatives are refused."""

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm
from matrix_optimizer_update_gb300 import example_moe_lm as ex


class Head:
    """Log probabilities and entropies of z = hidden weight^T, the gradients filled in by hand."""

    def logprobs(self, h, w, y):
        every = torch.log_softmax(h @ w.T, 1)
        logp = every.gather(1, y[:, None])[:, 0]
        return dm.Logprobs(logp, -(every.exp() * every).sum(1), torch.logsumexp(h @ w.T, 1), None, None)

    def logprobs_backward(self, h, w, y, scores, grad_logp, grad_entropy):
        every = torch.log_softmax(h @ w.T, 1)
        p = every.exp()
        dz = -p * (grad_logp[:, None] + grad_entropy[:, None] * (every + scores.entropy[:, None]))
        dz = dz + torch.nn.functional.one_hot(y, w.shape[0]) * grad_logp[:, None]
        out = torch.empty_like(h), torch.empty_like(w)
        out[0].copy_((dz @ w).detach())
        out[1].copy_((dz.T @ h).detach())
        return out


def leaf(*shape, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=torch.float64).requires_grad_()


def call(a, b):
    return ex.Logprob.apply(a, b, Head(), torch.tensor([1, 0, 4]))


def test_first_derivatives():
    a, b = leaf(3, 4), leaf(5, 4, seed=1)
    assert torch.autograd.gradcheck(call, (a, b))
    assert torch.autograd.gradcheck(lambda a, b: call(a, b)[1], (a, b))


@pytest.mark.parametrize("which", [0, 1])
def test_second_derivatives_are_refused(which):
    a, b = leaf(3, 4), leaf(5, 4, seed=1)
    loss = call(a, b)[which].sum()
    with pytest.raises(RuntimeError, match="second derivatives"):
        slope, = torch.autograd.grad(loss, a, create_graph=True)
        (loss + slope.square().sum()).backward()
