"""The alternatives' order where the tensor cores' sums do not tell neighbours apart."""

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu


def normal(*shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


@pytest.mark.parametrize("targets", [True, False])
@pytest.mark.parametrize("tokens,dim", [(5, 4096), (128, 4096), (140, 4096), (600, 2048)])
def test_order_where_large_terms_cancel(tokens, dim, targets):
    # Half of each sum is a part of about dim / 4 that all entries share, and the other half takes it back: the partial
    # sums are far above the logits (of order 1), and so is what the tensor cores truncate (up to 2.2e-9 * dim of them).
    vocab, half = 900, dim // 2
    h, w = 0.02 * normal(tokens, dim, seed=tokens), 0.02 * normal(vocab, dim, seed=dim)
    h += normal(tokens, dim, seed=3)
    h[:, :half] += 2.0
    h[:, half:] -= 2.0
    w += 0.25
    h, w = h.bfloat16(), w.bfloat16()
    y = torch.arange(tokens, device="cuda") % vocab if targets else None
    got = dm.Head.create(tokens, vocab, dim).logprobs(h, w, y, top=20)
    z = (h.double() @ w.double().T).gather(1, got.top_ids)
    # (which entries are held, some more than are asked for, is the tensor cores' business)
    assert bool((z[:, :-1] > z[:, 1:]).all())
