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


@pytest.mark.parametrize("vocab", [300, 19457, 33000])
@pytest.mark.parametrize("tokens", [5, 128, 200])
def test_a_state_of_nan_shows_in_its_log_sum(tokens, vocab):
    h, w, y, _, ids, lists = inputs(tokens, vocab, 24, 2)
    head = dm.Head.create(tokens, vocab, 24, max_top=5)
    clean, lse = head.xent(h, w, y)
    keep = torch.arange(tokens, device="cuda") != 3
    h[3] = float("nan")
    for target in (7, -100):
        y[3] = target
        loss, lse2 = head.xent(h, w, y)
        assert torch.isnan(lse2[3]) and (torch.isnan(loss[3]) if target >= 0 else loss[3] == 0)
        assert torch.equal(loss[keep], clean[keep]) and torch.equal(lse2[keep], lse[keep])
    ids[3] = -1
    loss, lse2 = head.distill(h, w, ids, lists, 1.0)
    assert torch.isnan(lse2[3]) and loss[3] == 0 and torch.isfinite(lse2[keep]).all()


@pytest.mark.parametrize("tokens", [5, 200])
def test_rows_of_nan_in_the_weight_show_wherever_they_lie(tokens):
    # 32 entries at a time. Four of them 256 groups of 32 apart are summed by one thread of the few tokens' join
    # (152 tiles' halves of 72 entries, four groups each: 19457 entries on 76 pairs of SMs).
    vocab = 19457
    h, w, y, _, _, _ = inputs(tokens, vocab, 24, 3)
    y[:] = 1
    head = dm.Head.create(tokens, vocab, 24)
    for groups in ((100, 356, 612, 868), (100,), (356, 868), (0, 256, 512, 768)):
        bad = w.clone()
        for g in groups:
            at = g // 4 * 72 + g % 4 * 32
            bad[at + 2:at + 32] = float("nan")
            bad[at:at + 2] = float("nan") if at else w[:2]
        loss, lse = head.xent(h, bad, y)
        assert torch.isnan(lse).all() and torch.isnan(loss).all(), groups
