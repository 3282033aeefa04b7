"""Alternatives of a vocabulary whose logits do not fit the workspace at a time: the same as from one piece."""

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu


def inputs(tokens, vocab, dim, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = (torch.randn(vocab, dim, generator=g, device="cuda") / dim ** 0.5).to(torch.bfloat16)
    h = (2 * torch.randn(tokens, dim, generator=g, device="cuda")).to(torch.bfloat16)
    return h, w, torch.randint(0, vocab, (tokens,), generator=g, device="cuda")


def expected(h, w, y, top):
    z = h.double() @ w.double().T
    logp = z - torch.logsumexp(z, 1, keepdim=True)
    return logp, z.sort(dim=1, descending=True, stable=True).indices[:, :top]


# pieces in the smallest workspace, of z bytes: 128 tokens 2 (and few groups more than in one), 100: 2, 65: 2, 64: 1,
# 2048: 2, 2000 in the head for 2048: 3 by rounding; 600 and 77 in it: 1
@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("tokens,most,vocab,dim", [(128, 128, 70000, 24), (100, 128, 33000, 136), (65, 65, 200000, 16),
                                                   (64, 64, 5000, 64), (2048, 2048, 20011, 64), (2000, 2048, 33001, 136),
                                                   (600, 2048, 40000, 64), (77, 2048, 40000, 64), (129, 200, 700, 16),
                                                   (300, 300, 256, 64)])
def test_pieces(tokens, most, vocab, dim, room):
    h, w, y = inputs(tokens, vocab, dim, tokens)
    y[1] = -100
    y[2], y[3] = vocab - 1, 0
    head = dm.Head.create(most, vocab, dim, alternatives=room)
    past = -head.workspace.data_ptr() % 1024 + 1024
    head.workspace[past:].fill_(255)
    got = head.logprobs(h, w, y, top=32)
    logp, ids = expected(h, w, y, 32)
    assert torch.equal(got.top_ids, ids)
    # logits of order 10, sums of at most 136 terms of order 1 in fp32: 1e-5, and lse's rounding
    assert (got.top_logp - logp.gather(1, ids)).abs().max() < 1e-4
    at = y.clamp(min=0)[:, None]
    assert (got.logp - torch.where(y < 0, 0.0, logp.gather(1, at)[:, 0])).abs().max() < 1e-4
    assert (got.entropy + (logp.exp() * logp).sum(1)).abs().max() < 1e-3
    head.workspace[past:].fill_(255)
    again = head.logprobs(h, w, y, top=32)
    assert all(torch.equal(getattr(got, n), getattr(again, n)) for n in ("logp", "entropy", "lse", "top_ids", "top_logp"))
    assert head.read_device_status(torch.cuda.current_stream().cuda_stream) == 0


def test_gradients_and_losses_in_the_smallest_workspace():
    h, w, y = inputs(300, 40000, 72, 4)
    g = torch.linspace(-1, 1, 300, device="cuda")
    both = []
    for room in (False, True):
        head = dm.Head.create(300, 40000, 72, alternatives=room)
        head.workspace[-head.workspace.data_ptr() % 1024 + 1024:].fill_(255)
        scores = head.logprobs(h, w, y, top=3)
        loss, lse = head.xent(h, w, y)
        both.append([scores.logp, scores.entropy, scores.top_ids, loss, lse, *head.logprobs_backward(h, w, y, scores, g, g),
                     *head.xent_backward(h, w, y, lse, g)])
    assert all(torch.equal(a, b) for a, b in zip(*both))


def test_a_workspace_between_the_two_sizes():
    h, w, y = inputs(2048, 20000, 64, 6)
    whole = dm.Head.create(2048, 20000, 64)
    want = whole.logprobs(h, w, y, top=20)
    least, most = whole.workspace_bytes(), whole.workspace_bytes(alternatives=True)
    s = torch.cuda.current_stream().cuda_stream
    for nbytes in (least, least + 1, (least + most) // 2 + 4, most - 4, most):
        ws = torch.empty(nbytes + 1024 + 4096, dtype=torch.uint8, device="cuda").fill_(77)
        at = -ws.data_ptr() % 1024
        head = dm.Head.create(2048, 20000, 64)
        head.bind(ws.data_ptr() + at, nbytes, s)
        got = head.logprobs(h, w, y, top=20)
        assert torch.equal(got.top_ids, want.top_ids) and torch.equal(got.top_logp, want.top_logp)
        assert bool((ws[at + nbytes:] == 77).all()) and bool((ws[:at] == 77).all())
    with pytest.raises(dm.DmuonError) as e:
        whole.bind(ws.data_ptr() + at, least - 1, s)
    assert e.value.status == dm.ERR_WORKSPACE


def test_equal_logits_over_pieces_come_by_id():
    h, w, y = inputs(2048, 20000, 64, 5)
    head = dm.Head.create(2048, 20000, 64, alternatives=False)
    first = torch.arange(32, device="cuda").expand(2048, 32)
    assert torch.equal(head.logprobs(torch.zeros_like(h), w, y, top=32).top_ids, first)
    w.copy_(w[:50].repeat(400, 1))
    best = head.logprobs(h, w, top=1).top_ids
    assert torch.equal(head.logprobs(h, w, top=32).top_ids, best + 50 * torch.arange(32, device="cuda"))


def test_more_tokens_than_the_smallest_workspace_has_room_for():
    # 512 MB are the logits of 2^19 tokens for 256 entries
    h, w, y = inputs(1 << 20, 300, 8, 7)
    small = dm.Head.create(1 << 20, 300, 8, alternatives=False)
    with pytest.raises(dm.DmuonError) as e:
        small.logprobs(h, w, y, top=3)
    assert e.value.status == dm.ERR_WORKSPACE
    with pytest.raises(dm.DmuonError):
        small.logprobs(h[:(1 << 19) + 1], w, y[:(1 << 19) + 1], top=1)
    half = slice(0, 1 << 19)
    got, alone = small.logprobs(h[half], w, y[half], top=3), small.logprobs(h, w, y)
    want = dm.Head.create(1 << 20, 300, 8).logprobs(h, w, y, top=3)
    for name in ("logp", "entropy", "lse", "top_ids", "top_logp"):
        assert torch.equal(getattr(got, name), getattr(want, name)[half])
    assert torch.equal(alone.entropy, want.entropy) and torch.equal(alone.logp, want.logp)
