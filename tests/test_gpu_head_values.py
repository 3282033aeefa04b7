"""GPU tests of values that are no ordinary numbers in the head's losses: gradients,
states and weights that are infinite or NaN show where the formulas have them, and
nowhere else."""

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu


def inputs(tokens, vocab, dim, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.randn(tokens, dim, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(vocab, dim, generator=g, device="cuda") / dim ** 0.5).to(torch.bfloat16)
    y = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    ids = torch.rand(tokens, vocab, generator=g, device="cuda").topk(5, 1).indices
    lists = torch.randn(tokens, 5, generator=g, device="cuda")
    return h, w, y, torch.randn(tokens, generator=g, device="cuda"), ids, lists


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("tokens", [20, 100, 200])
def test_a_gradient_that_is_not_finite_stays_in_its_row(tokens, value):
    h, w, y, g, ids, lists = inputs(tokens, 300, 64, 1)
    head = dm.Head.create(tokens, 300, 64, max_top=5)
    keep = torch.arange(tokens, device="cuda") != 5
    _, lse = head.xent(h, w, y)
    _, lse2 = head.distill(h, w, ids, lists, 2.0)
    both = [lambda: head.xent_backward(h, w, y, lse, g), lambda: head.distill_backward(h, w, ids, lists, 2.0, lse2, g)]
    g[5] = 0.0
    wants = [call()[0] for call in both]
    g[5] = value
    for call, want in zip(both, wants):
        dh, dw = call()
        # the other tokens' rows do not depend on it, the row itself and every row of dW (h times it) do
        assert torch.equal(dh[keep], want[keep])
        assert not torch.isfinite(dh[5]).any() and not torch.isfinite(dw).any()
