"""GPU tests of the gradients of tokens that are predicted with near certainty."""

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu


def sure(tokens, vocab, dim, height, seed):
    """Tokens of different targets whose logits are `height` above all others (of order 1)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = (torch.randn(vocab, dim, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    y = torch.randperm(vocab, generator=g, device="cuda")[:tokens]
    row = w[y].float()
    h = torch.randn(tokens, dim, generator=g, device="cuda") / (0.04 * dim ** 0.5)
    h = (h + row * (height / row.square().sum(1, keepdim=True))).to(torch.bfloat16)
    return h, w, y, torch.ones(tokens, device="cuda")


@pytest.mark.parametrize("height", [16, 20, 24, 28, 40])
@pytest.mark.parametrize("tokens", [1, 16, 100, 300])
def test_no_gradient_pushes_a_target_down(tokens, height):
    # dW[target] = (p - 1) h + what the other tokens have for this entry, p times h. Along h the first is never above 0.
    h, w, y, g = sure(tokens, 4000, 1024, height, tokens)
    head = dm.Head.create(tokens, 4000, 1024, max_top=1)
    _, lse = head.xent(h, w, y)
    dw = [head.xent_backward(h, w, y, lse, g)[1]]
    one = torch.zeros(tokens, 1, device="cuda")
    _, lse = head.distill(h, w, y[:, None].contiguous(), one, 1.0)
    dw.append(head.distill_backward(h, w, y[:, None].contiguous(), one, 1.0, lse, g)[1])
    hd = h.double()
    z = hd @ w.double().T
    p = torch.softmax(z, 1)[:, y]
    p.fill_diagonal_(0)
    others = (p * (hd @ hd.T).abs()).sum(0)  # of each target's row, along its token's state
    for d in dw:
        up = (d[y].double() * hd).sum(1)
        # one rounding of dz and one of dW to bf16 of the others' terms
        assert (up <= 1.02 * others).all()
