"""GPU parity of the head's losses (dmuon_head_*) with the fp64 oracle.

Error bounds, per call (e = 2^-24, the relative rounding error of fp32):
 - a logit z = sum_d h_d w_d: products of two bf16 are exact in fp32, and dim
   additions, each off by at most one part in 2^23 whatever the rounding mode,
   give |dz| <= ez = (dim + 8) * 2e * A, with A the largest sum_d |h_d w_d| of
   the token;
 - a share of the softmax sum: each exponential is off by its argument's error
   (twice ez, and 2e per unit of |z|) and a few e of its own, and the additions
   (128 in a group, then the groups over threads) by at most 400 e:
   rel <= er = 2 ez + 400 e + 4 e (1 + |z|max);
 - cross entropy, formed from the others' ratio to the target:
   |dloss| <= (1 - exp(-loss)) er + 8 e loss + vocab 2^-126 (an exponential
   below fp32's normal range may be 0), and where the target is not the
   larger share the difference of two numbers of size |z|max adds 4 e |z|max,
   which er holds;
 - distillation: |dloss| <= T^2 (er (2 + |log q|max) + 400 e (1 + |z|max));
 - dz: off by bf16's rounding, U = 2^-8 (8 significant bits, to nearest) times |dz|, and by |g| p er; dH and dW sum that
   against |W| and |H|, add at most (n + 8) * 2e of the sum of the absolute
   terms, and round once more to bf16.
The norm of the error is held closer: bf16's roundings are independent, so it
stays within U of the result's norm plus U of the root of the sum of the
squared terms (a rounding error's mean square is a third of its bound).
"""

import numpy as np
import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm
from oracle import head_ref as ref

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = 2.0 ** -8


def f64(t):
    return t.double().cpu().numpy()


def inputs(tokens, vocab, dim, seed, pitch=0, sure=True):
    """hidden and weight with logits of order 1 to 10, rows `pitch` elements further apart than they are long."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ld = -(-dim // 8) * 8 + pitch
    w = torch.full((vocab, ld), 7.0, device="cuda", dtype=torch.bfloat16)[:, :dim]
    h = torch.full((tokens, ld), 7.0, device="cuda", dtype=torch.bfloat16)[:, :dim]
    w.copy_(torch.randn(vocab, dim, generator=g, device="cuda") / dim ** 0.5)
    y = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    x = torch.randn(tokens, dim, generator=g, device="cuda")
    if sure:
        row = w[y].float()
        x += row * (12 * torch.rand(tokens, 1, generator=g, device="cuda") / row.square().sum(1, keepdim=True))
    h.copy_(x)
    grad = torch.randn(tokens, generator=g, device="cuda")
    return h, w, y, grad


def bounds(h, w, r, scale=1.0):
    """(ez, er) per token."""
    a = (np.abs(h) @ np.abs(w).T).max(1) * scale
    ez = (h.shape[1] + 8) * 2 * E * a + 2 * E * np.abs(r["z"]).max(1)
    return ez, 2 * ez + 400 * E + 4 * E * (1 + np.abs(r["z"]).max(1))


def check_grads(dh, dw, r, h, w, g, er):
    p = np.exp(r["z"] - r["lse"][:, None])
    dz = np.abs(r["dz"])
    drift = (np.abs(g) * er)[:, None] * p * (dz != 0)
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


SIZES = [(1, 1, 8), (1, 2, 1), (1, 300, 64), (3, 17, 24), (2, 128, 64), (64, 129, 72), (127, 255, 40), (129, 257, 264),
         (256, 512, 128), (257, 1000, 512), (300, 5003, 136), (40, 20000, 256), (1025, 640, 96), (1, 33000, 1024),
         (4, 300, 65536), (20000, 50, 16), (129, 1, 8), (1000, 3, 1), (128, 70000, 24), (513, 257, 200)]


@pytest.mark.parametrize("tokens,vocab,dim", SIZES)
def test_xent(tokens, vocab, dim):
    h, w, y, g = inputs(tokens, vocab, dim, tokens + vocab, pitch=16 if tokens % 2 else 0)
    if tokens > 2:
        y[tokens // 2] = -100
        y[tokens - 1] = vocab
        g[0] = 0.0
    head = dm.Head.create(tokens + 5, vocab, dim)
    loss, lse = head.xent(h, w, y)
    dh, dw = head.xent_backward(h, w, y, lse, g)
    hn, wn, gn = f64(h), f64(w), f64(g)
    r = ref.xent(hn, wn, y.cpu().numpy(), gn)
    ez, er = bounds(hn, wn, r)
    assert np.all(np.abs(f64(lse) - r["lse"]) <= er + 2 * E * np.abs(r["lse"]))
    assert np.all(np.abs(f64(loss) - r["loss"]) <= -np.expm1(-r["loss"]) * er + 8 * E * r["loss"] +
                  w.shape[0] * 2.0 ** -126)
    check_grads(dh, dw, r, hn, wn, gn, er)
    assert head.read_device_status(torch.cuda.current_stream().cuda_stream) == 0


def teacher(tokens, vocab, top, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ids = torch.stack([torch.randperm(vocab, generator=g, device="cuda")[:top] for _ in range(tokens)])
    lg = torch.randn(tokens, top, generator=g, device="cuda") * 3
    return ids, lg


def check_distill(h, w, ids, lg, tau, g, head):
    loss, lse = head.distill(h, w, ids, lg, tau)
    dh, dw = head.distill_backward(h, w, ids, lg, tau, lse, g)
    hn, wn, gn = f64(h), f64(w), f64(g)
    r = ref.distill(hn, wn, ids.cpu().numpy(), f64(lg), float(np.float32(tau)), gn)
    ez, er = bounds(hn, wn, r, 1 / tau)
    assert np.all(np.abs(f64(lse) - r["lse"]) <= er + 2 * E * np.abs(r["lse"]))
    zmax = np.abs(r["z"]).max(1)
    rows = ref.teacher(ids.cpu().numpy(), f64(lg), w.shape[0], tau)
    logq = np.array([max([abs(np.log(q)) for _, q in row if q > 0], default=0.0) for row in rows])
    assert np.all(np.abs(f64(loss) - r["loss"]) <= tau ** 2 * (er * (2 + logq) + 400 * E * (1 + zmax)))
    # q itself is off by a few parts in 2^24 (an exponential and a division) times its logits' range
    q_err = np.array([(64 + 4 * max([abs(x) for x in row_lg if np.isfinite(x) and abs(x) < 1e30], default=0.0) / tau) * E
                      for row_lg in f64(lg)])
    check_grads(dh, dw, r, hn, wn, gn * tau, er + q_err * 64)
    return f64(loss), r


@pytest.mark.parametrize("tokens,vocab,dim,top,tau", [
    (1, 5, 8, 1, 1.0), (1, 700, 64, 5, 2.0), (9, 64, 32, 64, 1.0), (65, 300, 48, 33, 0.5), (130, 1000, 264, 64, 1.5),
    (257, 4099, 128, 100, 4.0), (33, 2000, 72, 256, 2.0)])
def test_distill(tokens, vocab, dim, top, tau):
    h, w, _, g = inputs(tokens, vocab, dim, tokens + top, pitch=8 if tokens % 2 else 0, sure=False)
    ids, lg = teacher(tokens, vocab, top, tokens)
    if tokens > 8:
        lg[1, top // 2:] = -torch.inf      # a short list
        ids[2, 0] = -1                     # entries outside the vocabulary
        ids[3, top - 1] = vocab
        lg[4] = -torch.inf                 # empty rows
        ids[5] = -1
        lg[6] = torch.finfo(torch.float32).min  # all at the type's lowest: an even split
        lg[7, 0] = torch.finfo(torch.float32).min
    check_distill(h, w, ids, lg, tau, g, dm.Head.create(tokens, vocab, dim, max_top=top))


def test_distill_order_does_not_matter_and_equal_ids_add_up():
    h, w, _, g = inputs(20, 400, 64, 3, sure=False)
    ids, lg = teacher(20, 400, 31, 4)
    head = dm.Head.create(20, 400, 64, max_top=64)
    first = check_distill(h, w, ids, lg, 2.0, g, head)[0]
    order = torch.randperm(31, device="cuda")
    again, _ = head.distill(h, w, ids[:, order].contiguous(), lg[:, order].contiguous(), 2.0)
    # the same entries and the same sorted order: only the sums' order over equal logits could differ
    assert np.abs(f64(again) - first).max() <= 400 * E * (1 + np.abs(first).max())
    ids[:, 7] = ids[:, 8]
    check_distill(h, w, ids, lg, 2.0, g, head)


@pytest.mark.parametrize("tokens", [33, 200])
@pytest.mark.parametrize("places", ["first", "last", "ends"])
def test_lists_that_lie_together(tokens, places):
    # every entry of every list in the same 32 of the vocabulary, or at the ends of neighbouring 32s
    vocab, dim, top = 1000, 72, 30
    h, w, _, g = inputs(tokens, vocab, dim, 11, sure=False)
    ids, lg = teacher(tokens, vocab, top, 12)
    near = {"first": torch.arange(32), "last": torch.arange(968, 1000),
            "ends": torch.cat([torch.arange(31, 993, 32), torch.arange(32, 993, 32)])}[places].to(ids.dtype).cuda()
    order = torch.Generator(device="cuda")
    order.manual_seed(13)
    for t in range(tokens):
        ids[t] = near[torch.randperm(near.numel(), generator=order, device="cuda")[:top]]
    ids[3] = near[0]  # one id for the whole list
    check_distill(h, w, ids, lg, 2.0, g, dm.Head.create(tokens, vocab, dim, max_top=top))


def test_pieces_of_the_vocabulary():
    # room for 2^20 tokens leaves pieces of 256 entries: 1000 entries make 4 of them, the last ragged
    h, w, y, g = inputs(200, 1000, 64, 5)
    head = dm.Head.create(1 << 20, 1000, 64, max_top=4)
    whole = dm.Head.create(200, 1000, 64, max_top=4)
    loss, lse = head.xent(h, w, y)
    dh, dw = head.xent_backward(h, w, y, lse, g)
    hn, wn, gn = f64(h), f64(w), f64(g)
    r = ref.xent(hn, wn, y.cpu().numpy(), gn)
    check_grads(dh, dw, r, hn, wn, gn, bounds(hn, wn, r)[1])
    loss2, lse2 = whole.xent(h, w, y)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    ids, lg = teacher(200, 1000, 4, 6)
    check_distill(h, w, ids, lg, 1.5, g, head)


def test_no_tokens_and_tokens_that_do_not_count():
    h, w, y, g = inputs(70, 300, 64, 7)
    head = dm.Head.create(70, 300, 64)
    dw = torch.full_like(w, 3.0)
    head.xent_backward(h[:0], w, y[:0], g[:0], g[:0], dweight=dw)
    assert not dw.any()
    loss, lse = head.xent(h[:0], w, y[:0])
    assert loss.numel() == lse.numel() == 0
    y[:] = -100
    loss, lse = head.xent(h, w, y)
    assert not loss.any() and torch.isfinite(lse).all()
    dh, dw = head.xent_backward(h, w, y, lse, g)
    assert not dh.any() and not dw.any()


def test_a_token_that_does_not_count_may_have_any_logits():
    # hidden states far past the softmax's range: finite logits of order 1e30 in a masked row
    h, w, y, g = inputs(9, 300, 64, 8)
    h[4] = 1e30
    y[4] = -100
    head = dm.Head.create(9, 300, 64)
    loss, lse = head.xent(h, w, y)
    dh, dw = head.xent_backward(h, w, y, lse, g)
    keep = torch.arange(9, device="cuda") != 4
    loss2, lse2 = head.xent(h[keep].contiguous(), w, y[keep].contiguous())
    assert torch.equal(loss[keep], loss2) and loss[4] == 0
    assert not dh[4].any() and torch.isfinite(dw).all()


def test_large_logits_stay_finite():
    h, w, y, g = inputs(33, 500, 64, 9)
    h *= 64
    head = dm.Head.create(33, 500, 64)
    loss, lse = head.xent(h, w, y)
    dh, dw = head.xent_backward(h, w, y, lse, g)
    hn, wn, gn = f64(h), f64(w), f64(g)
    r = ref.xent(hn, wn, y.cpu().numpy(), gn)
    ez, er = bounds(hn, wn, r)
    assert np.abs(r["z"]).max() > 100
    assert np.all(np.abs(f64(loss) - r["loss"]) <= -np.expm1(-r["loss"]) * er + 8 * E * r["loss"] +
                  w.shape[0] * 2.0 ** -126)
    check_grads(dh, dw, r, hn, wn, gn, er)


def test_gradient_agrees_with_differences():
    # hidden on a grid of 2^-3 and steps of 2^-5 are exact in bf16. The sum of the losses along a direction:
    # truncation <= |E|^3/6 times the third derivative (at most the cube of a logit's change, about 0.35),
    # and fp32's rounding of the losses
    h, w, y, g = inputs(40, 300, 64, 10, sure=False)
    h.copy_((h * 8).round().clamp(-16, 16) / 8)
    step = torch.where(torch.rand_like(h.float()) < 0.5, -1.0, 1.0).to(torch.bfloat16) * 2.0 ** -5
    head = dm.Head.create(40, 300, 64)
    _, lse = head.xent(h, w, y)
    dh, _ = head.xent_backward(h, w, y, lse, torch.ones_like(g))
    up, down = (head.xent(h + s * step, w, y)[0].double() for s in (1, -1))
    slope = (dh.double() * step.double()).sum(1)
    change = (step.double() @ w.double().T).abs().amax(1)
    dz_norm = f64(dh.float().abs().sum(1)) * 2.0 ** -5 * 2.0 ** -8 + 2.0 ** -8 * f64(change)
    assert np.all(np.abs(f64((up - down) / 2 - slope)) <= f64(change) ** 3 + dz_norm + 1e-4)


def test_outputs_into_given_tensors_leave_the_rest_alone():
    h, w, y, g = inputs(150, 300, 72, 11, pitch=24)
    head = dm.Head.create(150, 300, 72)
    _, lse = head.xent(h, w, y)
    dh, dw = head.xent_backward(h, w, y, lse, g)
    big_h = torch.full((152, 96), 5.0, device="cuda", dtype=torch.bfloat16)
    big_w = torch.full((304, 112), 5.0, device="cuda", dtype=torch.bfloat16)
    head.xent_backward(h, w, y, lse, g, dhidden=big_h[1:151, 8:80], dweight=big_w[2:302, 16:88])
    assert torch.equal(big_h[1:151, 8:80], dh) and torch.equal(big_w[2:302, 16:88], dw)
    big_h[1:151, 8:80] = 5.0
    big_w[2:302, 16:88] = 5.0
    assert (big_h == 5).all() and (big_w == 5).all()
    only_h, none = head.xent_backward(h, w, y, lse, g, dweight=False)
    assert none is None and torch.equal(only_h, dh)
    none, only_w = head.xent_backward(h, w, y, lse, g, dhidden=False)
    assert none is None and torch.equal(only_w, dw)


def test_runs_repeat_bit_for_bit_on_any_stream_and_in_a_graph():
    h, w, y, g = inputs(600, 3000, 256, 12)
    ids, lg = teacher(600, 3000, 40, 13)
    head = dm.Head.create(600, 3000, 256, max_top=40)

    def both(stream=None):
        loss, lse = head.xent(h, w, y, stream=stream)
        a = head.xent_backward(h, w, y, lse, g, stream=stream)
        loss2, lse2 = head.distill(h, w, ids, lg, 2.0, stream=stream)
        b = head.distill_backward(h, w, ids, lg, 2.0, lse2, g, stream=stream)
        return [loss, lse, *a, loss2, lse2, *b]

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


def test_bad_tensors_are_refused():
    h, w, y, g = inputs(8, 40, 24, 14)
    head = dm.Head.create(8, 40, 24, max_top=4)
    ids, lg = teacher(8, 40, 5, 15)
    bad = [lambda: head.xent(h.float(), w, y), lambda: head.xent(h, w[:39], y), lambda: head.xent(h[:, :16], w, y),
           lambda: head.xent(h, w, y.int()), lambda: head.xent(h, w, y[:7]), lambda: head.xent(h.cpu(), w, y),
           lambda: head.xent(h, w.T.contiguous().T, y), lambda: head.xent(torch.cat([h, h]), w, torch.cat([y, y])),
           lambda: head.distill(h, w, ids, lg, 1.0), lambda: head.distill(h, w, ids[:, :4].contiguous(), lg, 1.0),
           lambda: head.distill(h, w, ids[:, :4].contiguous(), lg[:, :4].contiguous(), 0.0),
           lambda: head.distill(h, w, ids[:, :4].contiguous(), lg[:, :4].contiguous(), float("nan")),
           lambda: head.xent_backward(h, w, y, g, g[:4]),
           lambda: head.xent_backward(h, w, y, g, g, dhidden=torch.empty(8, 25, device="cuda", dtype=torch.bfloat16)
                                      [:, 1:])]
    for call in bad:
        with pytest.raises(dm.DmuonError) as e:
            call()
        assert e.value.status == dm.ERR_INVALID_ARG


@pytest.mark.parametrize("tokens,vocab,dim", [(1, 100, 40), (77, 1003, 72), (128, 5000, 64), (300, 1500, 136)])
def test_nothing_is_read_from_a_workspace_that_was_not_written(tokens, vocab, dim):
    # NaN everywhere before the bind, and again, past the status and counters, before each call
    h, w, y, g = inputs(tokens, vocab, dim, 16)
    ids, lg = teacher(tokens, vocab, 9, 17)
    head = dm.Head.create(tokens, vocab, dim, max_top=9)
    clean = head.xent(h, w, y)
    clean += head.xent_backward(h, w, y, clean[1], g)
    soft = head.distill(h, w, ids, lg, 2.0)
    soft += head.distill_backward(h, w, ids, lg, 2.0, soft[1], g)
    ws = head.workspace
    at = -ws.data_ptr() % 1024
    ws.fill_(255)
    head.bind(ws.data_ptr() + at, head.workspace_bytes(), torch.cuda.current_stream().cuda_stream)

    def poisoned(call):
        ws[at + 1024:].fill_(255)
        return call()

    again = poisoned(lambda: head.xent(h, w, y))
    again += poisoned(lambda: head.xent_backward(h, w, y, again[1], g))
    soft2 = poisoned(lambda: head.distill(h, w, ids, lg, 2.0))
    soft2 += poisoned(lambda: head.distill_backward(h, w, ids, lg, 2.0, soft2[1], g))
    assert all(torch.equal(a, b) for a, b in zip(clean + soft, again + soft2))
    assert head.read_device_status(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("tokens", [3, 200])
def test_a_weight_of_more_than_2_to_the_31_elements(tokens):
    vocab, dim = 540_000, 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w = torch.empty(vocab, dim, device="cuda", dtype=torch.bfloat16)
    for a in range(0, vocab, 60_000):
        w[a:a + 60_000].normal_(0, 0.02, generator=g)
    h = torch.randn(tokens, dim, generator=g, device="cuda").to(torch.bfloat16)
    y = vocab - 1 - torch.arange(tokens, device="cuda") * 7
    head = dm.Head.create(tokens, vocab, dim)
    loss, lse = head.xent(h, w, y)
    grad = torch.full((tokens,), 1.0 / tokens, device="cuda")
    dh, dw = head.xent_backward(h, w, y, lse, grad)
    hd = h.double()
    z = torch.cat([hd @ w[a:a + 30_000].double().T for a in range(0, vocab, 30_000)], 1)
    want = torch.logsumexp(z, 1)
    # |z| <= 8 and A <= 4096 * 0.02 * 3: the bound of test_xent with those, in round figures
    assert (lse - want).abs().max() < 4104 * 2 * E * 250 * 2
    assert (loss - (want - z[torch.arange(tokens), y])).abs().max() < 4104 * 2 * E * 250 * 2
    dz = torch.exp(z - want[:, None])
    dz[torch.arange(tokens), y] -= 1
    dz /= tokens
    for rows in (slice(0, 300), slice(524_200, 524_400), slice(vocab - 300, vocab)):  # 2^31 elements is row 524288
        assert torch.linalg.norm(dw[rows].double() - dz[:, rows].T @ hd) < 2 * U * torch.linalg.norm(dz[:, rows].T @ hd)
    want_h = sum(dz[:, a:a + 30_000] @ w[a:a + 30_000].double() for a in range(0, vocab, 30_000))
    assert torch.linalg.norm(dh.double() - want_h) < 2 * U * torch.linalg.norm(want_h)


@pytest.mark.parametrize("tokens", [20, 200])
def test_gradients_of_tokens_that_do_not_count_may_hold_anything(tokens):
    h, w, y, g = inputs(tokens, 300, 64, 18)
    y[3], y[11] = -100, 300
    head = dm.Head.create(tokens, 300, 64, max_top=3)
    loss, lse = head.xent(h, w, y)
    g[3] = g[11] = 0.0
    want = head.xent_backward(h, w, y, lse, g)
    g[3], g[11] = float("inf"), float("nan")
    assert all(torch.equal(a, b) for a, b in zip(want, head.xent_backward(h, w, y, lse, g)))
    ids, lg = teacher(tokens, 300, 3, 19)
    lg[3], ids[11] = -torch.inf, -1
    loss, lse = head.distill(h, w, ids, lg, 1.5)
    g[3] = g[11] = 0.0
    want = head.distill_backward(h, w, ids, lg, 1.5, lse, g)
    g[3], g[11] = float("inf"), float("nan")
    assert all(torch.equal(a, b) for a, b in zip(want, head.distill_backward(h, w, ids, lg, 1.5, lse, g)))


@pytest.mark.parametrize("tokens,vocab,dim", [(1, 3000, 264), (16, 3001, 256), (17, 5000, 72), (64, 2000, 200)])
def test_gradients_of_few_tokens_are_as_exact_as_their_type(tokens, vocab, dim):
    # The result's rounding is off by ulp / sqrt(12) in the root mean square, ulp = 2^-7 of the power of two below.
    # What else there is adds squares: dz to 2^-17, logits to 4 sqrt(dim) 2^-24 of 16, some 6e-5 against 1.7e-3.
    def near(got, want):
        ulp = 2.0 ** (np.floor(np.log2(np.abs(want) + 2.0 ** -120)) - 7)
        assert np.linalg.norm(f64(got) - want) <= 1.1 * np.linalg.norm(ulp) / np.sqrt(12)

    h, w, y, g = inputs(tokens, vocab, dim, 21)
    head = dm.Head.create(tokens, vocab, dim, max_top=12)
    _, lse = head.xent(h, w, y)
    dh, dw = head.xent_backward(h, w, y, lse, g)
    r = ref.xent(f64(h), f64(w), y.cpu().numpy(), f64(g))
    near(dh, r["dhidden"])
    near(dw, r["dweight"])
    ids, lg = teacher(tokens, vocab, 12, 22)
    _, lse = head.distill(h, w, ids, lg, 2.0)
    dh, dw = head.distill_backward(h, w, ids, lg, 2.0, lse, g)
    r = ref.distill(f64(h), f64(w), ids.cpu().numpy(), f64(lg), 2.0, f64(g))
    near(dh, r["dhidden"])
    near(dw, r["dweight"])


@pytest.mark.parametrize("tokens", [20, 200])
def test_a_nan_in_a_list_stays_in_its_row(tokens):
    h, w, _, _ = inputs(tokens, 300, 64, 20, sure=False)
    ids, lg = teacher(tokens, 300, 5, 21)
    head = dm.Head.create(tokens, 300, 64, max_top=5)
    clean, lse = head.distill(h, w, ids, lg, 2.0)
    lg[4, 2] = float("nan")
    loss, lse2 = head.distill(h, w, ids, lg, 2.0)
    keep = torch.arange(tokens, device="cuda") != 4
    assert torch.isnan(loss[4]) and torch.equal(loss[keep], clean[keep])
    # the student's sum is the teacher's business in no row: equal up to where its logits were formed
    assert torch.equal(lse2[keep], lse[keep]) and (lse2[4] - lse[4]).abs() < 1e-4
