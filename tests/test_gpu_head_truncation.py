"""GPU tests of how exact the log sums are where the tensor cores form the logits.

Tensor cores truncate what they accumulate: each of the dim / 16 steps takes up
to a unit in the last place off the running sum, half a unit on average, which
is 0.36 * 2^-23 of it on average over its leading digits. Where the running sum
is the whole logit from the start on, that is 0.36 * 2^-23 * dim / 16 = 2.7e-9 *
dim of it; where it grows evenly, half of that; where the terms lie at the end,
or nothing is added any more, next to nothing. The library scales logits by
1 + c * dim with c = 1.0e-9. So what is left of c, measured here against 64
bits, is

 - within half of c where the terms are spread evenly: with no correction it
   would be all of it, with twice the correction as much the other way;
 - between -c and (2.7 - 1.0) c wherever the terms lie, 1.75 c with the roundings.

A log sum's own rounding (half a unit in its last place, at most 2^-21 here) is
5e-7 / sqrt(tokens) of the mean, against 1024 * 1e-9 for c at 1024 dims.
"""

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu

C = 1.0e-9


def left(tokens, dim, kind, scaled=0.0):
    """What is left of c, fitted over the tokens; ``scaled``: of an oracle whose logits are that much larger."""
    vocab = 1500
    g = torch.Generator(device="cuda")
    g.manual_seed(dim + tokens)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    h, w = normal(tokens, dim), normal(vocab, dim) * dim ** -0.5
    part, i = max(16, dim // 16), torch.arange(tokens, device="cuda")
    at = {"even": slice(0, dim), "planted": slice(0, dim), "early": slice(0, part), "late": slice(dim - part, dim),
          "only early": slice(0, part), "only late": slice(dim - part, dim)}[kind]
    if kind.startswith("only"):
        w.zero_()
    if kind != "even":
        w[i, at] += h[:, at] * (12.0 / (at.stop - at.start))
    h, w = h.to(torch.bfloat16), w.to(torch.bfloat16)
    _, lse = dm.Head.create(tokens, vocab, dim).xent(h, w, torch.full((tokens,), -100, device="cuda"))
    z = h.double() @ w.double().T * (1.0 + scaled)
    x = (torch.softmax(z, 1) * z).sum(1) * dim
    return float(((torch.logsumexp(z, 1) - lse.double()) * x).sum() / x.square().sum())


@pytest.mark.parametrize("tokens", [64, 200])
@pytest.mark.parametrize("kind", ["even", "planted"])
@pytest.mark.parametrize("dim", [1024, 2048, 4096, 8192, 16384, 65536])
def test_the_scale_makes_up_for_what_truncation_takes(tokens, dim, kind):
    assert abs(left(tokens, dim, kind)) < 0.5 * C
    # the bound notices a correction left out, or made twice
    assert abs(left(tokens, dim, kind, scaled=C * dim)) > 0.5 * C
    assert abs(left(tokens, dim, kind, scaled=-C * dim)) > 0.5 * C


@pytest.mark.parametrize("tokens", [64, 200])
@pytest.mark.parametrize("kind", ["early", "late", "only early", "only late"])
@pytest.mark.parametrize("dim", [256, 1024, 4096, 16384, 65536])
def test_wherever_the_terms_lie(tokens, dim, kind):
    assert abs(left(tokens, dim, kind)) < 1.75 * C
