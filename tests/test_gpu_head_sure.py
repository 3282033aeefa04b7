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


@pytest.mark.parametrize("height", [8, 14, 18, 22, 26, 40])
@pytest.mark.parametrize("tokens", [1, 16, 100, 300])
def test_gradients_with_the_loss_given_keep_their_digits(tokens, height):
    # dz rounded to bf16 (U of it), and off by what its others' logits are: 2^-23 * (dim + 8) of the largest sum of
    # |h w| (below 60 here, from one of 40) and a few parts in 2^24 of lse, together below 0.02; the result rounded
    vocab, dim, U = 4000, 1024, 2.0 ** -8
    h, w, y, g = sure(tokens, vocab, dim, height, tokens + 1)
    head = dm.Head.create(tokens, vocab, dim)
    loss, lse = head.xent(h, w, y)
    dh, dw = head.xent_backward(h, w, y, lse, g, loss=loss)
    hd, wd = h.double(), w.double()
    p = torch.softmax(hd @ wd.T, 1)
    at = torch.arange(tokens, device="cuda")
    p[at, y] = 0
    dz = p.clone()
    dz[at, y] = -p.sum(1)
    for got, want, size in ((dh, dz @ wd, dz.abs() @ wd.abs()), (dw, dz.T @ hd, dz.abs().T @ hd.abs())):
        assert ((got.double() - want).abs() <= (U + 0.02) * size * (1 + U) + U * want.abs() + 1e-37).all()
        off = torch.linalg.norm(got.double() - want, dim=1) / torch.linalg.norm(want, dim=1).clamp(min=1e-37)
        # bf16's rounding errors of a row are independent: a hundredth holds ten times what they amount to
        if got is dh:
            assert (off < 0.01).all()


def test_tokens_of_every_kind_with_the_loss_given():
    # targets that do not count, and losses from 0 to 30: the same gradients up to what the loss's digits change
    h, w, y, g = sure(300, 900, 256, 9, 4)
    y[::7] = -100
    y[1::7] = torch.flip(y[1::7], (0,))  # others' targets: large losses
    g = torch.linspace(-1, 1, 300, device="cuda")
    head = dm.Head.create(300, 900, 256)
    loss, lse = head.xent(h, w, y)
    plain = head.xent_backward(h, w, y, lse, g)
    given = head.xent_backward(h, w, y, lse, g, loss=loss)
    for a, b in zip(plain, given):
        assert torch.linalg.norm(a.double() - b.double()) < 2.0 ** -8 * torch.linalg.norm(a.double())
    assert not given[0][::7].any()
    loss[::7] = float("nan")  # of tokens that do not count it may hold anything
    assert all(torch.equal(a, b) for a, b in zip(given, head.xent_backward(h, w, y, lse, g, loss=loss)))


def test_a_loss_that_is_no_such_tensor_is_refused():
    h, w, y, g = sure(8, 40, 24, 1, 5)
    head = dm.Head.create(8, 40, 24)
    loss, lse = head.xent(h, w, y)
    for bad in (loss[:7], loss.double(), loss.cpu(), torch.stack([loss, loss], 1)[:, 0]):
        with pytest.raises(dm.DmuonError) as e:
            head.xent_backward(h, w, y, lse, g, loss=bad)
        assert e.value.status == dm.ERR_INVALID_ARG
    args = (head._h, h.data_ptr(), 24, w.data_ptr(), 24, y.data_ptr(), 8, lse.data_ptr(), None, g.data_ptr(), None, 0,
            None, 0, None)
    assert dm.lib().dmuon_head_xent_backward_loss(*args) == dm.ERR_INVALID_ARG
