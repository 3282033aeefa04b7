"""The example with more tokens than a call of the experts' serving form takes."""

import pytest
import torch

from matrix_optimizer_update_gb300 import example_moe_lm as ex

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,top", [(1025, 2), (2048, 2), (1500, 4), (1024, 2), (700, 3)])
def test_serving_and_training(tokens, top):
    model = ex.Model(vocab=300, dim=64, inner=96, experts=8, top=top, max_tokens=tokens)
    x, y = next(ex.batches(300, tokens))
    with torch.no_grad():
        want = model.hidden(x).float()
        got = model.serve(x)
    # both round x + y and the norm to bf16, the training form also u, h and each expert's rows: six roundings of 2^-8
    assert torch.linalg.norm(got.float() - want) <= 6 * 2.0 ** -8 * torch.linalg.norm(want)
    # a token's hidden state is the same among others, to one rounding of y, x + y and the norm each
    few = model.serve(x[-5:])
    assert torch.linalg.norm(few.float() - got[-5:].float()) <= 3 * 2.0 ** -8 * torch.linalg.norm(few.float())
    assert model.serve(x[:0]).shape == (0, 64)
    (model.losses(x, y).sum() / tokens).backward()
    model.step(max_norm=1.0)


def test_its_training_takes_any_number_of_tokens():
    assert len(ex.train(steps=1, tokens=2048, vocab=300, log=None)) == 1
    assert len(ex.reinforce(steps=1, tokens=1500, vocab=300, warm=1, log=None)) == 1
