"""Entropies where one entry is nearly sure and is not the target: without targets, as a model generates, and with others.

As for a sure target, both terms of the entropy are sums over the other entries: off by er, their distances by ez (all
above 1) and some roundings; bounds as derived for the log probabilities' other tests."""

import numpy as np
import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm
from oracle import head_ref as ref
from test_gpu_logprobs import E, bounds, f64, inputs

pytestmark = pytest.mark.gpu


def rows(tokens, vocab, dim, low, high, seed):
    """Hidden states along one entry's row each: that entry's logit is `low` to `high`."""
    h, w, y, _, _ = inputs(tokens, vocab, dim, seed, sure=0.0)
    n = w[y].float()
    size = torch.linspace(low, high, tokens, device="cuda")[:, None]
    h.copy_(n * (size / n.square().sum(1, keepdim=True)))
    return h, w, y


@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("tokens,vocab", [(1, 500), (9, 500), (100, 3000), (200, 500), (700, 3000)])
def test_entropy_keeps_its_digits(tokens, vocab, top):
    h, w, y = rows(tokens, vocab, 64, 10, 40, 7)
    hn, wn = f64(h), f64(w)
    head = dm.Head.create(tokens, vocab, 64)
    other = (y + 1 + torch.arange(tokens, device="cuda") % (vocab - 1)) % vocab
    other[tokens // 2] = -1
    for targets in (None, torch.full_like(y, -100), other):
        got = head.logprobs(h, w, targets, top=top)
        r = ref.logprobs(hn, wn, None if targets is None else targets.cpu().numpy())
        ez, er = bounds(hn, wn, r, 1.0)
        assert np.all(r["entropy"] > 0)
        off = np.abs(f64(got.entropy) - r["entropy"])
        assert np.all(off <= r["entropy"] * (2 * er + ez + 16 * E) + vocab * 2.0 ** -120)
        assert np.all(np.abs(f64(got.lse) - r["lse"]) <= er + 2 * E * np.abs(r["lse"]))
        assert np.all(np.abs(f64(got.logp) - r["logp"]) <= er - 8 * E * r["logp"])


@pytest.mark.parametrize("tokens", [3, 150])
def test_one_far_above_others_that_are_equal(tokens):
    # every other logit is 0 exactly: entropy log1p(n e^-z) + n z e^-z / (1 + n e^-z). z is off by 1e-9 * dim of itself
    # (truncation) and a rounding, the sums by some roundings; e^-z moves as z does.
    vocab, dim = 500, 64
    w = torch.zeros(vocab, dim, device="cuda", dtype=torch.bfloat16)
    w[123, 0] = 1.0
    h = torch.zeros(tokens, dim, device="cuda", dtype=torch.bfloat16)
    h[:, 0] = torch.linspace(8, 60, tokens, device="cuda")
    z = f64(h[:, 0])
    ratio = (vocab - 1) * np.exp(-z)
    want = np.log1p(ratio) + ratio * z / (1 + ratio)
    move = z * (64e-9 + 4 * E)
    head = dm.Head.create(tokens, vocab, dim)
    y = torch.full((tokens,), 7, device="cuda")
    for targets in (None, y):
        got = f64(head.logprobs(h, w, targets).entropy)
        assert np.all(np.abs(got - want) <= want * (move + 64 * E))


@pytest.mark.parametrize("tokens", [3, 150])
def test_several_at_the_peak(tokens):
    # n entries of 20, the others 0: the entropy is log n and what the others add
    for n, at in ((2, (5, 6)), (2, (5, 400)), (3, (0, 130, 499)), (33, range(100, 133))):
        w = torch.zeros(500, 8, device="cuda", dtype=torch.bfloat16)
        w[list(at), 0] = 1.0
        h = torch.zeros(tokens, 8, device="cuda", dtype=torch.bfloat16)
        h[:, 0] = 20.0
        head = dm.Head.create(tokens, 500, 8)
        r = ref.logprobs(f64(h), f64(w), None)
        for y in (None, torch.full((tokens,), 77, device="cuda"), torch.full((tokens,), 5, device="cuda")):
            got = head.logprobs(h, w, y)
            assert np.all(np.abs(f64(got.entropy) - r["entropy"]) <= 1e-6 * r["entropy"])
            assert np.all(np.abs(f64(got.lse) - r["lse"]) <= 1e-6 * r["lse"])
