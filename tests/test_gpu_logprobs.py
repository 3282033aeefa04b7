"""GPU parity of log probabilities, entropies, alternatives and their gradients
(dmuon_head_logprobs, _backward) with the fp64 oracle.

Error bounds (e = 2^-24; ez and er of a token's logits and softmax sum as for the head's losses:
|dz| <= ez = (dim + 8) 2e A + 2e |z|max, er = 2 ez + 400 e + 4 e (1 + |z|max)):
 - log probability of a target: (1 - p) er + 8 e |logp| + vocab 2^-126, formed from the others' ratio to it;
 - entropy log S - U / S with S = sum exp(z - peak), U = sum exp(z - peak) (z - peak): log S is off by er, U and S
   by er of themselves, U by ez more for its factors: er (2 + 2 H) + 8 e (1 + H);
 - an alternative's log probability: its logit and lse, ez + er + 4 e (|z|max + |lse|);
 - ids are those of the logits in 64 bits, in their order;
 - dz: rounded to bf16 (U = 2^-8), and off by er p (|gl| + |ge| (|log p + H| + 3 + 2 H)); dH and dW sum that as
   the head's losses do."""

import numpy as np
import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm
from oracle import head_ref as ref

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = 2.0 ** -8


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def inputs(tokens, vocab, dim, seed, pitch=0, sure=12.0):
    """hidden and weight with logits of order 1 to 10, rows `pitch` elements further apart than they are long."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ld = -(-dim // 8) * 8 + pitch
    w = torch.full((vocab, ld), 7.0, device="cuda", dtype=torch.bfloat16)[:, :dim]
    h = torch.full((tokens, ld), 7.0, device="cuda", dtype=torch.bfloat16)[:, :dim]
    w.copy_(torch.randn(vocab, dim, generator=g, device="cuda") / dim ** 0.5)
    y = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    row = w[y].float()
    x = torch.randn(tokens, dim, generator=g, device="cuda")
    h.copy_(x + row * (sure * torch.rand(tokens, 1, generator=g, device="cuda") / row.square().sum(1, keepdim=True)))
    return h, w, y, torch.randn(tokens, generator=g, device="cuda"), torch.randn(tokens, generator=g, device="cuda")


def bounds(h, w, r, tau):
    a = (np.abs(h) @ np.abs(w).T).max(1) / tau
    ez = (h.shape[1] + 8) * 2 * E * a + 2 * E * np.abs(r["z"]).max(1)
    return ez, 2 * ez + 400 * E + 4 * E * (1 + np.abs(r["z"]).max(1))


def first_of(z, top):
    """Ids of the largest logits, ties by the lowest id."""
    return np.stack([np.lexsort((np.arange(z.shape[1]), -row))[:top] for row in z])


def check_scores(got, r, h, w, tau, top, ids=True):
    ez, er = bounds(h, w, r, tau)
    assert np.all(np.abs(f64(got.lse) - r["lse"]) <= er + 2 * E * np.abs(r["lse"]))
    assert np.all(np.abs(f64(got.logp) - r["logp"]) <= -np.expm1(r["logp"]) * er - 8 * E * r["logp"] +
                  w.shape[0] * 2.0 ** -126)
    assert np.all(np.abs(f64(got.entropy) - r["entropy"]) <= er * (2 + 2 * r["entropy"]) + 8 * E * (1 + r["entropy"]))
    if top == 0:
        assert got.top_ids is None and got.top_logp is None
        return
    want = first_of(r["z"], top)
    if ids:
        assert np.array_equal(got.top_ids.cpu().numpy(), want)
    zmax = np.abs(r["z"]).max(1) + np.abs(r["lse"])
    values = np.take_along_axis(r["every"], got.top_ids.cpu().numpy(), 1)
    assert np.all(np.abs(f64(got.top_logp) - values) <= (ez + er + 4 * E * zmax)[:, None])


def check_grads(dh, dw, r, h, w, gl, ge, tau, er):
    p = np.exp(r["every"])
    ent = r["entropy"][:, None]
    dz = np.abs(r["dz"]) / tau
    drift = er[:, None] * p * (np.abs(gl)[:, None] + np.abs(ge)[:, None] * (np.abs(r["every"] + ent) + 3 + 2 * ent)) / tau
    for got, want, left, right in ((dh, r["dhidden"], dz, w), (dw, r["dweight"], dz.T, h)):
        got = f64(got)
        off = drift if left is dz else drift.T
        total, moved = left @ np.abs(right), off @ np.abs(right)
        bound = (U * total + moved + (left.shape[1] + 8) * 2 * E * total) * (1 + 2.0 ** -8)
        bound += U * np.abs(want) + 1e-37
        assert np.all(np.isfinite(got))
        assert np.all(np.abs(got - want) <= bound)
        rms = np.sqrt(left ** 2 @ right ** 2)
        close = U * (np.linalg.norm(want) + np.linalg.norm(rms)) + np.linalg.norm(moved)
        assert np.linalg.norm(got - want) <= close + 1e-37


@pytest.mark.parametrize("tokens,vocab,dim,top,tau", [
    (1, 1, 8, 1, 1.0), (1, 2, 1, 2, 1.0), (1, 300, 64, 5, 0.7), (1, 33000, 1024, 20, 1.0), (3, 17, 24, 17, 1.0),
    (2, 128, 64, 32, 2.0), (64, 129, 72, 1, 1.0), (65, 5000, 136, 20, 1.3), (127, 255, 40, 32, 1.0),
    (128, 20000, 256, 10, 0.8), (129, 257, 264, 7, 1.0), (256, 512, 128, 20, 1.0), (257, 1000, 512, 32, 0.5),
    (300, 5003, 136, 20, 1.0), (40, 20000, 256, 0, 1.0), (1025, 640, 96, 3, 1.5), (4, 300, 65536, 5, 1.0),
    (5000, 50, 16, 8, 1.0), (129, 1, 8, 1, 1.0), (1000, 3, 1, 0, 1.0), (128, 70000, 24, 20, 1.0), (513, 257, 200, 0, 2.0),
    (200, 40000, 64, 32, 1.0)])
def test_logprobs(tokens, vocab, dim, top, tau):
    h, w, y, gl, ge = inputs(tokens, vocab, dim, tokens + vocab, pitch=16 if tokens % 2 else 0)
    if tokens > 2:
        y[tokens // 2] = -100
        y[tokens - 1] = vocab
        gl[0] = 0.0
        ge[1] = 0.0
    head = dm.Head.create(tokens + 5, vocab, dim)
    got = head.logprobs(h, w, y, top=top, temperature=tau)
    dh, dw = head.logprobs_backward(h, w, y, got, gl, ge, temperature=tau)
    hn, wn, gn, en = f64(h), f64(w), f64(gl), f64(ge)
    tau = float(np.float32(tau))
    r = ref.logprobs(hn, wn, y.cpu().numpy(), tau, gn, en)
    check_scores(got, r, hn, wn, tau, top, ids=dim > 1)  # one dim: equal logits in 64 bits all over
    check_grads(dh, dw, r, hn, wn, gn, en, tau, bounds(hn, wn, r, tau)[1])
    assert head.read_device_status(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("tokens", [6, 100, 300])
def test_each_gradient_alone_and_no_targets(tokens):
    h, w, y, gl, ge = inputs(tokens, 700, 72, 5)
    head = dm.Head.create(tokens, 700, 72)
    hn, wn, gn, en = f64(h), f64(w), f64(gl), f64(ge)
    got = head.logprobs(h, w, y)
    zero = np.zeros(tokens)
    for grads, a, b in (((gl, None), gn, zero), ((None, ge), zero, en)):
        r = ref.logprobs(hn, wn, y.cpu().numpy(), 1.0, a, b)
        check_grads(*head.logprobs_backward(h, w, y, got, *grads), r, hn, wn, a, b, 1.0, bounds(hn, wn, r, 1.0)[1])
    dh, dw = head.logprobs_backward(h, w, y, got)
    assert not dh.any() and not dw.any()
    none = head.logprobs(h, w, top=9)
    r = ref.logprobs(hn, wn, None, 1.0, gn, en)
    check_scores(none, r, hn, wn, 1.0, 9)
    assert not none.logp.any()
    check_grads(*head.logprobs_backward(h, w, None, none, gl, ge), r, hn, wn, zero, en, 1.0, bounds(hn, wn, r, 1.0)[1])


@pytest.mark.parametrize("tokens", [5, 128, 200])
def test_agrees_with_the_cross_entropy(tokens):
    h, w, y, g, _ = inputs(tokens, 3001, 264, 6, sure=30.0)
    y[2] = -1
    head = dm.Head.create(tokens, 3001, 264)
    got = head.logprobs(h, w, y)
    loss, lse = head.xent(h, w, y)
    _, er = bounds(f64(h), f64(w), ref.logprobs(f64(h), f64(w), None), 1.0)
    assert np.all(np.abs(f64(got.logp + loss)) <= 2 * er * -np.expm1(-f64(loss)) + 16 * E * f64(loss))
    mine = head.logprobs_backward(h, w, y, got, -g)
    theirs = head.xent_backward(h, w, y, lse, g, loss=loss)
    for a, b in zip(mine, theirs):
        assert torch.linalg.norm(a.double() - b.double()) <= 2 * U * torch.linalg.norm(b.double())


@pytest.mark.parametrize("tokens", [9, 200])
def test_sure_tokens_keep_their_digits(tokens):
    # targets up to 40 above the others: 1 - p from 1e-2 to 1e-14
    h, w, y, gl, ge = inputs(tokens, 500, 64, 7, sure=0.0)
    n = w[y].float()
    h.copy_(n * (torch.linspace(8, 40, tokens, device="cuda")[:, None] / n.square().sum(1, keepdim=True)))
    head = dm.Head.create(tokens, 500, 64)
    got = head.logprobs(h, w, y)
    hn, wn = f64(h), f64(w)
    r = ref.logprobs(hn, wn, y.cpu().numpy())
    ez, er = bounds(hn, wn, r, 1.0)
    assert np.all(np.abs(f64(got.logp) - r["logp"]) <= -r["logp"] * (er + 8 * E) + 500 * 2.0 ** -126)
    # both terms of the entropy are sums over the others: off by er, and the distances by ez (all above 1)
    assert np.all(np.abs(f64(got.entropy) - r["entropy"]) <= r["entropy"] * (2 * er + ez + 16 * E) + 500 * 2.0 ** -120)
    dh, _ = head.logprobs_backward(h, w, y, got, gl)
    want = ref.logprobs(hn, wn, y.cpu().numpy(), 1.0, f64(gl))["dhidden"]
    off = np.linalg.norm(f64(dh) - want, axis=1)
    assert np.all(off <= (4 * U + 2 * er) * np.linalg.norm(want, axis=1) + 1e-36)


@pytest.mark.parametrize("tokens,vocab", [(7, 3000), (200, 3000), (3, 100000), (300, 20000)])
def test_equal_logits_come_by_id(tokens, vocab):
    h, w, y, _, _ = inputs(tokens, vocab, 64, 8)
    head = dm.Head.create(tokens, vocab, 64)
    first = torch.arange(20, device="cuda").expand(tokens, 20)
    got = head.logprobs(torch.zeros_like(h), w, y, top=20)  # all logits 0
    assert torch.equal(got.top_ids, first)
    assert (got.top_logp + np.log(vocab)).abs().max() < 1e-4 and (got.entropy - np.log(vocab)).abs().max() < 1e-4
    # the same rows over and over: each logit comes vocab / 50 times
    w.copy_(w[:50].repeat(vocab // 50, 1))
    best = head.logprobs(h, w, y, top=1).top_ids
    got = head.logprobs(h, w, None, top=32).top_ids
    assert bool((best < 50).all())
    assert torch.equal(got, best + 50 * torch.arange(32, device="cuda"))


def test_neighbours_closer_than_fp32_are_in_the_order_of_64_bits():
    # logits that differ in their last places alone: sums of a large part that all share and small ones
    tokens, vocab, dim = 140, 900, 512
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    w = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 16.0
    w[:, 1:] = (torch.randn(vocab, dim - 1, generator=g, device="cuda") * 2.0 ** -20).to(torch.bfloat16)
    h = torch.randn(tokens, dim, generator=g, device="cuda").to(torch.bfloat16)
    h[:, 0] = 1.0
    for n in (tokens, 40):
        got = dm.Head.create(n, vocab, dim).logprobs(h[:n], w, top=3)
        z = h[:n].double() @ w.double().T
        # (the spread of all 900 is some 2e-5, so what 11 are held of is the tensor cores' business: of those held,
        # the order is exact)
        mine = z.gather(1, got.top_ids)
        assert bool((mine[:, :-1] > mine[:, 1:]).all())


@pytest.mark.parametrize("tokens", [3, 200])
def test_alternatives_that_lie_together_and_the_target_among_them(tokens):
    # all of the largest in one group of 128, at the vocabulary's end, across a border; the target is the n-th of them
    for start in (0, 100, 968):
        h, w, y, _, _ = inputs(tokens, 1000, 72, 10, sure=0.0)
        head = dm.Head.create(tokens, 1000, 72)
        w[start:start + 32] = h.float().mean(0).to(torch.bfloat16)
        w[start:start + 32] *= torch.linspace(0.5, 1.5, 32, device="cuda")[:, None]
        h[:] = h.float().mean(0).to(torch.bfloat16) * 8
        y[:] = start + torch.arange(tokens, device="cuda") % 32
        got = head.logprobs(h, w, y, top=32)
        hn, wn = f64(h), f64(w)
        check_scores(got, ref.logprobs(hn, wn, y.cpu().numpy()), hn, wn, 1.0, 32)
        at = (got.top_ids == y[:, None])
        assert torch.equal(got.top_logp[at], got.logp[at.any(1)])


def test_pieces_of_the_vocabulary():
    # room for 2^20 tokens holds the logits of 262144 tokens for 1024 entries, of 200 tokens for all: both ways
    h, w, y, _, _ = inputs(200, 5000, 64, 11)
    whole = dm.Head.create(200, 5000, 64).logprobs(h, w, y, top=20)
    many = dm.Head.create(300000, 5000, 64)
    rows = torch.arange(300000, device="cuda") % 200
    got = many.logprobs(h[rows].contiguous(), w, y[rows].contiguous(), top=20)
    assert torch.equal(got.top_ids, whole.top_ids[rows])
    for name in ("logp", "entropy", "lse"):
        assert torch.equal(getattr(got, name), getattr(whole, name)[rows])
    assert torch.equal(got.top_logp, whole.top_logp[rows])


def test_few_tokens_over_pieces():
    # 128 tokens of a vocabulary whose logits take more than 512 MB
    vocab = (1 << 20) + 4000
    h, w, y, _, _ = inputs(128, vocab, 16, 12)
    got = dm.Head.create(128, vocab, 16).logprobs(h, w, y, top=20)
    z = h.double() @ w.double().T
    lse = torch.logsumexp(z, 1)
    ids = z.sort(dim=1, descending=True, stable=True).indices[:, :20]
    assert torch.equal(got.top_ids, ids)
    assert (got.lse - lse).abs().max() < 1e-4
    logp = z - lse[:, None]
    assert (got.entropy + (logp.exp() * logp).sum(1)).abs().max() < 1e-3
    assert (got.top_logp - logp.gather(1, ids)).abs().max() < 1e-4


def test_gradient_agrees_with_differences():
    # as the cross entropy's: steps of 2^-5 are exact in bf16; a third derivative of log p and of the entropy along a
    # change c of the logits is at most 8 c^3 (1 + log vocab)
    h, w, y, gl, ge = inputs(40, 300, 64, 13, sure=0.0)
    h.copy_((h * 8).round().clamp(-16, 16) / 8)
    step = torch.where(torch.rand_like(h.float()) < 0.5, -1.0, 1.0).to(torch.bfloat16) * 2.0 ** -5
    head = dm.Head.create(40, 300, 64)
    got = head.logprobs(h, w, y)
    dh, _ = head.logprobs_backward(h, w, y, got, gl, ge)
    up, down = ((gl * s.logp).double() + (ge * s.entropy).double()
                for s in (head.logprobs(h + d * step, w, y) for d in (1, -1)))
    slope = (dh.double() * step.double()).sum(1)
    change = f64((step.double() @ w.double().T).abs().amax(1))
    size = np.abs(f64(gl)) + np.abs(f64(ge))
    rounding = f64(dh.float().abs().sum(1)) * 2.0 ** -5 * U + U * change * size * 4
    assert np.all(np.abs(f64((up - down) / 2 - slope)) <= 8 * 7 / 6 * size * change ** 3 + rounding + 1e-4)


@pytest.mark.parametrize("tokens", [5, 100, 200])
def test_values_that_are_no_numbers_stay_in_their_row(tokens):
    h, w, y, gl, ge = inputs(tokens, 300, 64, 14)
    head = dm.Head.create(tokens, 300, 64)
    keep = torch.arange(tokens, device="cuda") != 3
    clean = head.logprobs(h, w, y, top=8)
    grads = head.logprobs_backward(h, w, y, clean, gl, ge)[0]
    for which in (gl, ge):
        for value in (float("inf"), float("-inf"), float("nan")):
            old = which[3].clone()
            which[3] = value
            dh, dw = head.logprobs_backward(h, w, y, clean, gl, ge)
            # the scale of the others may change with the row that is left out of it
            assert torch.linalg.norm(dh[keep].double() - grads[keep].double()) <= 2 * U * torch.linalg.norm(
                grads[keep].double())
            assert not torch.isfinite(dh[3]).any() and not torch.isfinite(dw).any()
            which[3] = old
    bad = h.clone()
    for value in (float("nan"), float("inf")):
        bad[3] = value
        got = head.logprobs(bad, w, y, top=8)
        assert not torch.isfinite(got.lse[3]) and not torch.isfinite(got.logp[3])
        assert bool(((got.top_ids >= -1) & (got.top_ids < 300)).all())
        for name in ("logp", "entropy", "lse", "top_ids", "top_logp"):
            assert torch.equal(getattr(got, name)[keep], getattr(clean, name)[keep])
    # a vocabulary entry that nothing can choose
    w[7] = float("-inf")
    h.abs_()
    got = head.logprobs(h, w, y.clamp(min=8), top=8)
    assert torch.isfinite(got.entropy).all() and torch.isfinite(got.lse).all() and not (got.top_ids == 7).any()
    w[7] = float("inf")
    y[:] = 9
    got = head.logprobs(h, w, y)
    assert not torch.isfinite(got.lse).any()


@pytest.mark.parametrize("tokens,top", [(33, 20), (600, 20), (600, 0)])
def test_repeats_bit_for_bit_on_any_stream_and_in_a_graph(tokens, top):
    h, w, y, gl, ge = inputs(tokens, 3000, 256, 15)
    head = dm.Head.create(tokens, 3000, 256)

    def both(stream=None):
        s = head.logprobs(h, w, y, top=top, temperature=0.9, stream=stream)
        grads = head.logprobs_backward(h, w, y, s, gl, ge, temperature=0.9, stream=stream)
        return [s.logp, s.entropy, s.lse, *grads] + ([s.top_ids, s.top_logp] if top else [])

    first = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = both()
    for t in third:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, third))
    # nothing is read from a workspace that was not written, past the status and counters
    ws = head.workspace
    ws[-ws.data_ptr() % 1024 + 1024:].fill_(255)
    s = head.logprobs(h, w, y, top=top, temperature=0.9)
    assert torch.equal(s.entropy, first[1]) and (top == 0 or torch.equal(s.top_ids, first[5]))
    ws[-ws.data_ptr() % 1024 + 1024:].fill_(255)
    assert all(torch.equal(a, b) for a, b in zip(first[3:5], head.logprobs_backward(h, w, y, s, gl, ge, temperature=0.9)))
    assert head.read_device_status(torch.cuda.current_stream().cuda_stream) == 0


def test_nothing_to_do_and_given_outputs():
    h, w, y, gl, ge = inputs(150, 300, 72, 16, pitch=24)
    head = dm.Head.create(150, 300, 72)
    s = head.logprobs(h[:0], w, y[:0], top=4)
    assert s.logp.numel() == 0 and s.top_ids.shape == (0, 4)
    dw = torch.full_like(w, 3.0)
    head.logprobs_backward(h[:0], w, y[:0], s, gl[:0], ge[:0], dweight=dw)
    assert not dw.any()
    s = head.logprobs(h, w, y)
    dh, dw = head.logprobs_backward(h, w, y, s, gl, ge)
    big_h = torch.full((152, 96), 5.0, device="cuda", dtype=torch.bfloat16)
    big_w = torch.full((304, 112), 5.0, device="cuda", dtype=torch.bfloat16)
    head.logprobs_backward(h, w, y, s, gl, ge, dhidden=big_h[1:151, 8:80], dweight=big_w[2:302, 16:88])
    assert torch.equal(big_h[1:151, 8:80], dh) and torch.equal(big_w[2:302, 16:88], dw)
    big_h[1:151, 8:80] = 5.0
    big_w[2:302, 16:88] = 5.0
    assert (big_h == 5).all() and (big_w == 5).all()
    only_h, none = head.logprobs_backward(h, w, y, s, gl, ge, dweight=False)
    assert none is None and torch.equal(only_h, dh)


def test_bad_tensors_are_refused():
    h, w, y, gl, ge = inputs(8, 40, 24, 17)
    head = dm.Head.create(8, 40, 24)
    s = head.logprobs(h, w, y)
    bad = [lambda: head.logprobs(h, w, y, top=33), lambda: head.logprobs(h, w, y, top=-1),
           lambda: head.logprobs(h, w, y.int()), lambda: head.logprobs(h, w, y, temperature=0.0),
           lambda: head.logprobs(h, w, y, temperature=float("nan")), lambda: head.logprobs(h, w[:39], y),
           lambda: head.logprobs(torch.cat([h, h]), w), lambda: head.logprobs_backward(h, w, y, s, gl[:4]),
           lambda: head.logprobs_backward(h, w, y, s, gl, ge.half()),
           lambda: head.logprobs_backward(h, w, y, s, gl, ge, temperature=-1.0),
           lambda: dm.Head.create(8, 20, 24).logprobs(h, w[:20], y, top=21)]
    for call in bad:
        with pytest.raises(dm.DmuonError) as e:
            call()
        assert e.value.status == dm.ERR_INVALID_ARG


@pytest.mark.parametrize("tokens,vocab,dim", [(128, 200000, 16), (64, 200000, 16), (128, 200000, 64), (100, 400000, 40)])
def test_many_short_tiles(tokens, vocab, dim):
    # tiles of one K stage, more to a pair of SMs than the list between its warps holds
    h, w, y, gl, ge = inputs(tokens, vocab, dim, 18, sure=0.0)
    z = h.double() @ w.double().T
    logp = torch.log_softmax(z, 1)
    ids = z.sort(dim=1, descending=True, stable=True).indices[:, :20]
    head = dm.Head.create(tokens, vocab, dim)
    past = -head.workspace.data_ptr() % 1024 + 1024
    first = None
    for top in (0, 20) * 10:
        head.workspace[past:].fill_(255)
        got = head.logprobs(h, w, y, top=top)
        grads = head.logprobs_backward(h, w, y, got, gl, ge)
        assert head.read_device_status(torch.cuda.current_stream().cuda_stream) == 0
        assert (got.logp - logp.gather(1, y[:, None])[:, 0]).abs().max() < 1e-4
        assert (got.entropy + (logp.exp() * logp).sum(1)).abs().max() < 1e-4
        assert top == 0 or torch.equal(got.top_ids, ids)
        first = first or [got.logp, got.entropy, *grads]
        assert all(torch.equal(a, b) for a, b in zip(first, [got.logp, got.entropy, *grads]))


@pytest.mark.parametrize("tokens,vocab", [(1, 70000), (61, 140000), (2, 1 << 20), (2, 1500000)])
def test_few_tokens_of_large_vocabularies(tokens, vocab):
    # more groups than their finders' registers hold, and than shared memory does; one piece
    h, w, y, _, _ = inputs(tokens, vocab, 24, 19, sure=0.0)
    z = h.double() @ w.double().T
    for top in (1, 32):
        got = dm.Head.create(tokens, vocab, 24).logprobs(h, w, y, top=top)
        assert torch.equal(got.top_ids, z.sort(dim=1, descending=True, stable=True).indices[:, :top])
        logp = z - torch.logsumexp(z, 1, keepdim=True)
        assert (got.top_logp - logp.gather(1, got.top_ids)).abs().max() < 1e-4


@pytest.mark.parametrize("tokens,top", [(1, 0), (1, 5), (77, 0), (77, 3), (200, 0), (200, 5)])
@pytest.mark.parametrize("dim", [64, 1003])
def test_a_targets_logit_has_more_digits_than_fp32(tokens, top, dim):
    # every other entry's logit is 0 exactly, so that all that can be off is the target's, 16 to 56: half a unit in its
    # last place alone would be 1e-6 to 2e-6 of log p. Formed with twice the digits, with d = z + low: exp(d) (2 units,
    # and its factor's one), the sum's factor, log1p (2) and their roundings are within 10 E of log p; the entropy has d
    # and two sums more.
    vocab, tau, half = 600, np.float32(0.7), dim // 2
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens + dim)
    ld = -(-dim // 8) * 8
    h = torch.zeros(tokens, ld, device="cuda", dtype=torch.bfloat16)[:, :dim]
    w = torch.zeros(vocab, ld, device="cuda", dtype=torch.bfloat16)[:, :dim]
    w[:, half:] = torch.randn(vocab, dim - half, generator=g, device="cuda").to(torch.bfloat16)
    row = torch.randn(half, generator=g, device="cuda").to(torch.bfloat16)
    w[7], w[7, :half] = 0.0, row
    scale = torch.linspace(11.5, 39, tokens, device="cuda")[:, None] / row.double().square().sum()
    h[:, :half] = (row.double() * scale).to(torch.bfloat16)
    z = f64(h) @ f64(w[7]) / np.float64(tau)
    assert z.min() > 15 and z.max() < 58
    got = dm.Head.create(tokens, vocab, dim).logprobs(h, w, torch.full((tokens,), 7, device="cuda"), top=top,
                                                      temperature=float(tau))
    ratio = (vocab - 1) * np.exp(-z)
    logp = -np.log1p(ratio)
    entropy = -logp + ratio * z / (1 + ratio)
    assert np.all(np.abs(f64(got.logp) - logp) <= -10 * E * logp)
    assert np.all(np.abs(f64(got.entropy) - entropy) <= 14 * E * entropy)
    assert np.all(np.abs(f64(got.lse) - (z - logp)) <= 2 * E * z)
    if top:
        assert bool((got.top_ids[:, 0] == 7).all()) and torch.equal(got.top_logp[:, 0], got.logp)


@pytest.mark.parametrize("tokens", [1, 100, 300])
def test_a_vocabulary_of_one(tokens):
    h, w, _, gl, ge = inputs(tokens, 1, 40, 20)
    head = dm.Head.create(tokens, 1, 40)
    z = f64(h) @ f64(w).T
    for y in (torch.zeros(tokens, dtype=torch.int64, device="cuda"), None):
        got = head.logprobs(h, w, y, top=1)
        assert not got.logp.any() and not got.entropy.any()
        assert np.all(np.abs(f64(got.lse) - z[:, 0]) <= 1e-4) and not got.top_ids.any()
        assert got.top_logp.abs().max() <= 1e-5
        dh, dw = head.logprobs_backward(h, w, y, got, gl, ge)
        assert dh.abs().max() <= 1e-4 and dw.abs().max() <= 1e-2
