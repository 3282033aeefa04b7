"""The alternatives' log probabilities follow their order, and the target's among them is its own."""

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu


def normal(*shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def falling(values):
    return bool((values[:, :-1] >= values[:, 1:]).all())


@pytest.mark.parametrize("tokens", [1, 40, 140, 500])
def test_values_follow_the_order(tokens):
    # logits that differ in their last places alone, and the target among them
    vocab, dim = 900, 512
    w = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 16.0
    w[:, 1:] = (normal(vocab, dim - 1, seed=9) * 2.0 ** -20).bfloat16()
    h = normal(tokens, dim, seed=10).bfloat16()
    h[:, 0] = 1.0
    best = (h.double() @ w.double().T).sort(dim=1, descending=True).indices
    head = dm.Head.create(tokens, vocab, dim)
    for y in (None, best[:, 0].contiguous(), best[:, 4].contiguous(), best[:, 700].contiguous()):
        got = head.logprobs(h, w, y, top=8)
        assert falling(got.top_logp)
        # (lse and z are 16 and 23: two roundings of 1e-6, and an exact logit)
        exact = (h.double() @ w.double().T).gather(1, got.top_ids) - got.lse.double()[:, None]
        at = torch.zeros_like(got.top_ids, dtype=torch.bool) if y is None else got.top_ids == y[:, None]
        assert bool(((got.top_logp - exact).abs()[~at] <= 4e-6).all())
        if y is not None:
            assert torch.equal(got.top_logp[at], got.logp[at.any(1)])


@pytest.mark.parametrize("tokens,vocab,dim,tau", [(1, 32000, 256, 1.0), (61, 5000, 1024, 0.8), (128, 20000, 64, 1.3),
                                                  (300, 20000, 64, 0.7), (2000, 3000, 16, 1.0)])
def test_values_fall_and_hold_the_targets(tokens, vocab, dim, tau):
    w = (normal(vocab, dim, seed=11) / dim ** 0.5).bfloat16()
    h = (2 * normal(tokens, dim, seed=12)).bfloat16()
    head = dm.Head.create(tokens, vocab, dim)
    best = head.logprobs(h, w, top=32, temperature=tau)
    assert falling(best.top_logp)
    for k in (0, 1, 31):
        y = best.top_ids[:, k].contiguous()
        got = head.logprobs(h, w, y, top=32, temperature=tau)
        assert torch.equal(got.top_ids, best.top_ids)
        assert torch.equal(got.top_logp[:, k], got.logp) and falling(got.top_logp)
