"""GPU parity of the routing to experts (dmuon_route_*) with the fp64 oracle.

The sort's indices and the dispatched rows are exact. A combined row sums top
products in fp32: (top + 1) roundings of parts in 2^24 of the sum of absolute
terms, then one to the row's type. dys is one product, dweights a sum over dim."""

import numpy as np
import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm
from oracle import head_ref as ref

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def f64(t):
    return t.double().cpu().numpy()


def make(tokens, top, experts, dim, dtype, seed, dropped=0.1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ids = torch.randint(0, experts, (tokens, top), generator=g, device="cuda")
    gone = torch.rand(tokens, top, generator=g, device="cuda") < dropped
    ids = torch.where(gone, torch.where(ids % 2 == 0, -1, experts), ids)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (ids, torch.softmax(r(tokens, top), 1), r(tokens, dim).to(dtype), r(tokens * top, dim).to(dtype),
            r(tokens, dim).to(dtype), r(tokens * top, dim).to(dtype))


@pytest.mark.parametrize("tokens,top,experts,dim,dtype,dropped", [
    (1, 1, 1, 1, "bf16", 0.0), (1, 8, 64, 64, "bf16", 0.0), (5, 3, 4, 24, "bf16", 0.4), (33, 2, 7, 5, "bf16", 0.1),
    (257, 6, 64, 72, "bf16", 0.05), (1030, 8, 16, 40, "bf16", 0.02), (700, 4, 300, 17, "f32", 0.1),
    (300, 2, 4096, 36, "f32", 0.1), (2100, 1, 3, 12, "f32", 0.0), (100, 64, 80, 8, "f32", 0.3),
    (64, 2, 8, 32, "bf16", 1.0), (6, 2, 8, 4200, "bf16", 0.2)])
def test_route(tokens, top, experts, dim, dtype, dropped):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    ids, wts, x, ys, dy, dxs = make(tokens, top, experts, dim, dt, tokens + dim, dropped)
    router = dm.Router.create(tokens, top, experts)
    route = router.sort(ids)
    dest, source, offsets = ref.route(ids.cpu().numpy(), experts)
    assert np.array_equal(route.dest.cpu().numpy(), dest)
    assert np.array_equal(route.source.cpu().numpy(), source)
    assert np.array_equal(route.offsets.cpu().numpy(), offsets)
    # rows that are not in use may hold anything: it must not show
    ys[int(offsets[-1]):] = float("nan")
    dxs[int(offsets[-1]):] = float("nan")
    assert np.array_equal(f64(router.dispatch(x, route)), ref.dispatch(f64(x), source, top))
    ysn, wn, dyn, dxsn = f64(ys), f64(wts), f64(dy), f64(dxs)

    def near(got, want, absolute, adds, rounding):
        got = f64(got)
        assert np.all(np.abs(got - want) <= (adds + 2) * E * absolute * (1 + rounding) + rounding * np.abs(want)
                      + 1e-37)

    near(router.combine(ys, wts, route), ref.combine(ysn, wn, dest), ref.combine(np.abs(ysn), np.abs(wn), dest), top,
         ROUND[dt])
    near(router.dispatch_backward(dxs, route), ref.combine(dxsn, None, dest), ref.combine(np.abs(dxsn), None, dest),
         top, ROUND[dt])
    dys, dw = router.combine_backward(dy, ys, wts, route)
    want, want_w = ref.combine_backward(dyn, np.nan_to_num(ysn), wn, dest)
    near(dys, want, np.abs(want), 1, ROUND[dt])
    near(dw, want_w, ref.combine_backward(np.abs(dyn), np.abs(np.nan_to_num(ysn)), wn, dest)[1], dim, 0.0)


def test_long_lists_take_several_blocks():
    tokens, top, experts = 40001, 3, 130
    ids = make(tokens, top, experts, 1, torch.float32, 1)[0]
    route = dm.Router.create(tokens, top, experts).sort(ids)
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    n = int((key < experts).sum())
    assert torch.equal(route.source[:n].long(), order[:n]) and (route.source[n:] == -1).all()
    assert int(route.offsets[-1]) == n
    assert torch.equal(route.dest.reshape(-1)[order[:n]].long(), torch.arange(n, device="cuda"))
    assert int((route.dest >= 0).sum()) == n


def test_one_expert_takes_all():
    ids = torch.full((3000, 2), 5, device="cuda", dtype=torch.int64)
    route = dm.Router.create(3000, 2, 9).sort(ids)
    assert torch.equal(route.source, torch.arange(6000, device="cuda", dtype=torch.int32))
    assert route.offsets.tolist() == [0] * 6 + [6000] * 4


def test_pitches_and_unaligned_rows():
    ids, wts, x, ys, dy, _ = make(50, 2, 6, 40, torch.bfloat16, 3)
    router = dm.Router.create(64, 2, 6)
    route = router.sort(ids)
    for pad, off in ((8, 0), (1, 1), (8, 4)):
        wide = torch.zeros(50, 40 + pad + off, device="cuda", dtype=torch.bfloat16)
        view = wide[:, off:off + 40]
        view.copy_(x)
        assert torch.equal(router.dispatch(view, route), router.dispatch(x, route))
        view.copy_(dy)
        for a, b in zip(router.combine_backward(view, ys, wts, route), router.combine_backward(dy, ys, wts, route)):
            # the vector and the element path add a dot product's terms in different orders
            assert torch.allclose(a.float(), b.float(), rtol=0, atol=40 * 2 * E * 200)


def test_no_tokens_side_stream_and_graph():
    router = dm.Router.create(300, 2, 6)
    none = torch.empty(0, 2, device="cuda", dtype=torch.int64)
    route = router.sort(none)
    assert route.offsets.tolist() == [0] * 7
    x0 = torch.empty(0, 16, device="cuda")
    assert router.dispatch(x0, route).shape == (0, 16) and router.combine(x0, None, route).shape == (0, 16)
    ids, wts, x, ys, dy, dxs = make(300, 2, 6, 64, torch.bfloat16, 4)

    def all_of(stream=None):
        r = router.sort(ids, stream=stream)
        return [r.dest, r.source, r.offsets, router.dispatch(x, r, stream=stream),
                router.combine(ys, wts, r, stream=stream), *router.combine_backward(dy, ys, wts, r, stream=stream),
                router.dispatch_backward(dxs, r, stream=stream)]

    first = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = all_of(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = all_of()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, third))


def test_bad_tensors_are_refused():
    ids, wts, x, ys, dy, dxs = make(20, 2, 6, 16, torch.bfloat16, 5)
    router = dm.Router.create(20, 2, 6)
    route = router.sort(ids)
    bad = [lambda: router.sort(ids.int()), lambda: router.sort(torch.cat([ids, ids])), lambda: router.sort(ids[:, :1]),
           lambda: router.sort(ids.T.contiguous().T), lambda: router.dispatch(x.half(), route),
           lambda: router.dispatch(x[:10], route), lambda: router.dispatch(x.T.contiguous().T, route),
           lambda: router.combine(ys[:10], wts, route), lambda: router.combine(ys, wts.double(), route),
           lambda: router.combine_backward(dy.float(), ys, wts, route),
           lambda: router.combine(ys, wts[:, :1], route)]
    for call in bad:
        with pytest.raises(dm.DmuonError) as e:
            call()
        assert e.value.status == dm.ERR_INVALID_ARG


@pytest.mark.parametrize("n,experts", [(255, 7), (257, 1), (8192, 64), (8193, 64), (40000, 1024), (65536, 1024), (65537, 1025),
                                       (131072, 130), (131073, 3), (33000, 4096), (1100000, 300)])
def test_sort_of_every_launch_shape(n, experts):
    # one block, clusters of 2 to 8, and three launches
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    ids = (torch.rand(n, 1, generator=g, device="cuda") ** 3 * experts).long()
    ids[torch.rand(n, 1, generator=g, device="cuda") < 0.03] = -5
    route = dm.Router.create(n, 1, experts).sort(ids)
    key = torch.where(ids[:, 0] < 0, experts, ids[:, 0])
    order = torch.argsort(key, stable=True)
    used = int((key < experts).sum())
    assert route.offsets.tolist() == [0] + torch.bincount(key, minlength=experts + 1)[:experts].cumsum(0).tolist()
    assert torch.equal(route.source[:used].long(), order[:used]) and (route.source[used:] == -1).all()
    assert torch.equal(route.dest[order[:used], 0].long(), torch.arange(used, device="cuda"))
    assert (route.dest[order[used:], 0] == -1).all()


def test_rows_of_more_than_2_to_the_31_elements():
    tokens, top, experts, dim = 70_000, 8, 16, 4096  # 2.3e9 elements of expert rows
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    ids = torch.randint(0, experts, (tokens, top), generator=g, device="cuda")
    x = torch.randn(tokens, dim, generator=g, device="cuda").to(torch.bfloat16)
    router = dm.Router.create(tokens, top, experts)
    route = router.sort(ids)
    xs = router.dispatch(x, route)
    src = route.source.long() // top
    for a in range(0, tokens * top, 56_000):
        assert torch.equal(xs[a:a + 56_000], x[src[a:a + 56_000]])
    wts = torch.full((tokens, top), 0.125, device="cuda")
    assert torch.equal(router.combine(xs, wts, route), x)  # eight eighths, exact
    dys, dw = router.combine_backward(x, xs, wts, route)
    assert torch.equal(dys[-1], xs[-1] * 0.125) and torch.equal(dys[-40_000], xs[-40_000] * 0.125)
    norm = x.double().square().sum(1)
    assert ((dw.double() - norm[:, None]).abs() <= dim * E * norm[:, None]).all()
