"""The example's autograd functions on the host, with stand-ins for router and head."""

import pytest
import torch

from matrix_optimizer_update_gb300 import example_moe_lm as ex


class Router:
    """Tokens to rows and back by a permutation."""

    order = torch.tensor([2, 0, 1])

    def dispatch(self, x, route):
        return x[self.order]

    def dispatch_backward(self, dxs, route):
        return torch.empty_like(dxs).index_copy(0, self.order, dxs)

    def combine(self, ys, weights, route):
        return ys * weights

    def combine_backward(self, dy, ys, weights, route):
        return dy * weights, (dy * ys).sum(1, keepdim=True)


class Head:
    """A loss of z = the sum over the weight of exp(hidden . row), the gradients filled in by hand."""

    def xent(self, h, w, y):
        z = (h @ w.T).exp().sum(1)
        return z.clone(), z.clone()

    def xent_backward(self, h, w, y, lse, grad, loss=None):
        e = (h @ w.T).exp() * grad[:, None]
        out = torch.empty_like(h), torch.empty_like(w)
        out[0].copy_((e @ w).detach())
        out[1].copy_((e.T @ h).detach())
        return out

    def distill(self, h, w, ids, logits, temperature):
        return self.xent(h, w, ids)

    def distill_backward(self, h, w, ids, logits, temperature, lse, grad):
        return self.xent_backward(h, w, ids, lse, grad)


def leaf(*shape, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * 0.3).requires_grad_()


CALLS = {
    "dispatch": lambda a, b: ex.Dispatch.apply(a, Router(), None).square(),
    "combine": lambda a, b: ex.Combine.apply(a, b[:, :1].clone(), Router(), None),
    "xent": lambda a, b: ex.Xent.apply(a, b, Head(), None),
    "distill": lambda a, b: ex.Distill.apply(a, b, Head(), torch.zeros(3, 1), torch.zeros(3, 1), 1.0),
}


@pytest.mark.parametrize("name", CALLS)
def test_first_derivatives(name):
    a, b = leaf(3, 4), leaf(3, 4, seed=1)
    assert torch.autograd.gradcheck(lambda a, b: CALLS[name](a, b), (a, b))


@pytest.mark.parametrize("name", CALLS)
def test_second_derivatives_are_refused(name):
    # a penalty on a gradient: without a refusal its part of the gradient would silently be missing
    a, b = leaf(3, 4), leaf(3, 4, seed=1)
    loss = CALLS[name](a, b).sum()
    with pytest.raises(RuntimeError, match="second derivatives"):
        slope, = torch.autograd.grad(loss, a, create_graph=True)
        (loss + slope.square().sum()).backward()
