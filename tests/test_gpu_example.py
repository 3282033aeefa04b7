"""The example that runs every operator in one training step: it learns, and the
gradients it trains with are those of the same model in plain torch."""

import pytest
import torch

from matrix_optimizer_update_gb300 import example_moe_lm as ex

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("distill", [False, True])
def test_training_learns(distill):
    history = ex.train(steps=60, distill=distill, log=None)
    assert all(h == h for h in history)
    # untrained: ln(1000) = 6.9 nats of cross entropy; the map is learnt by heart from a thousand tokens
    assert sum(history[-5:]) / 5 < 0.5 * history[0]


def test_gradients_are_those_of_plain_torch():
    model = ex.Model(vocab=300, dim=64, inner=96, experts=4, top=2, max_tokens=200)
    x, y = next(ex.batches(300, 200))
    model.losses(x, y).sum().backward()
    # the same model in fp32 on the same weights, each expert over all tokens
    w = {n: getattr(model, n).detach().float().requires_grad_() for n in ("embedding", "head_weight", "router_weight")}
    up = [p.detach().float().requires_grad_() for p in model.up]
    down = [p.detach().float().requires_grad_() for p in model.down]
    h = w["embedding"][x]
    # the experts the model chose, from its own bf16 scores
    with torch.no_grad():
        ids = torch.softmax((model.embedding[x] @ model.router_weight.T).float(), 1).topk(2, dim=1).indices
    probs = torch.softmax(h @ w["router_weight"].T, 1)
    every = torch.stack([torch.nn.functional.silu(h @ u.T) @ d.T for u, d in zip(up, down)], 1)
    mix = torch.zeros(200, 4, device="cuda").scatter(1, ids, probs.gather(1, ids))
    out = h + (every * mix[:, :, None]).sum(1)
    out = out * torch.rsqrt(out.square().mean(1, keepdim=True) + 1e-6)
    keep = y >= 0
    torch.nn.functional.cross_entropy(out[keep] @ w["head_weight"].T, y[keep], reduction="sum").backward()
    pairs = [(getattr(model, n), w[n]) for n in w] + list(zip(model.up, up)) + list(zip(model.down, down))
    for got, want in pairs:
        # about ten roundings to bf16 (2^-8 each) between loss and weight, independent of each other
        off = torch.linalg.norm(got.grad.float() - want.grad) / torch.linalg.norm(want.grad)
        assert off < 10 * 2.0 ** -8
