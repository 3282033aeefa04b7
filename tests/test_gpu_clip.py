"""The gradients' global norm and their clipping (dmuon_grad_norm, dmuon_grad_clip) against 64 bits.

The norm: a vector's squares are summed in fp32 (at most 10 roundings), a thread's vectors of a unit too (at most
64, as a unit has 16 turns of 4), the rest in 64 bits; squares are positive, so the sum is off by at most
80 * 2^-24, its root by half of that, and the result is rounded once. Clipped elements: the scale (the norm's
error and one rounding), one product, one rounding to the type."""

import math

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu

NORM = 42 * 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def exact(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def make(sizes, seed, scale=1.0):
    """Tensors of (elements, dtype, offset): views that start `offset` elements into their memory."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = []
    for n, dtype, offset in sizes:
        base = torch.randn(n + offset + 3, generator=g, device="cuda") * scale
        out.append(base.to(torch.bfloat16 if dtype == "b" else torch.float32)[offset:offset + n])
    return out


SETS = {
    "one": [(1, "b", 0)],
    "odd": [(1, "b", 1), (7, "b", 3), (8, "f", 1), (9, "f", 0), (0, "b", 0), (2047, "b", 5), (4099, "f", 3), (3, "f", 2)],
    "aligned": [(4096, "b", 0), (1024, "f", 0)],
    "vectors": [(1536, "f", i % 4) for i in range(40)],
    "many": [(100 + i, "bf"[i % 2], i % 8) for i in range(1500)],
    "large": [(3000001, "b", 1), (2000003, "f", 2), (5, "b", 0)],
    "hundred": [(50000, "b", 0)] * 100,
    "few": [(65536, "b", 0), (65536, "f", 1), (7, "f", 3), (60000, "f", 0)],               # just what one launch holds
    "more": [(65536, "b", 0), (65536, "f", 1), (65537, "b", 3)],          # and a little more
    "rows": [(2048 * (1 + i % 3), "bf"[i % 2], i % 5) for i in range(128)],
}


@pytest.mark.parametrize("name", SETS)
def test_norm_and_clip(name):
    grads = make(SETS[name], len(name))
    clip = dm.GradClip.create()
    clip.workspace.fill_(255)
    want = exact(grads)
    norm = clip.norm(grads)
    assert norm.shape == () and norm.dtype == torch.float32
    assert abs(float(norm) - want) <= NORM * want
    before = [g.clone() for g in grads]
    for limit in (want / 3.0, want * 2.0, 0.0, math.inf):
        scale = min(1.0, limit / want) if want else 1.0
        out = [torch.full_like(g, 7.0) for g in grads]
        place = [g.clone() for g in grads]
        assert torch.equal(clip.clip(grads, limit, out=out), norm)
        assert torch.equal(clip.clip(place, limit), norm)
        for g, b, o, p in zip(grads, before, out, place):
            assert torch.equal(g, b) and torch.equal(o, p)
            exactly = b.double() * scale
            off = (NORM + 3 * 2.0 ** -24 + half_step(b.dtype)) * exactly.abs() + 1e-38
            assert bool(((o.double() - exactly).abs() <= off).all())
            if scale == 1.0:
                assert torch.equal(o, b)


def test_neighbours_stay():
    """What lies around a tensor is left as it was, wherever it starts."""
    clip = dm.GradClip.create()
    for dtype in (torch.bfloat16, torch.float32):
        for offset in range(9):
            for n in (1, 5, 8, 17, 300):
                memory = torch.full((n + 32,), 3.0, dtype=dtype, device="cuda")
                clip.clip([memory[offset:offset + n]], 1.0)
                assert bool((memory[:offset] == 3.0).all()) and bool((memory[offset + n:] == 3.0).all())
                assert abs(float(memory[offset]) - n ** -0.5) <= 2 * half_step(dtype) * n ** -0.5


def test_out_lies_otherwise():
    """A result whose start is not that of its gradient's."""
    clip = dm.GradClip.create()
    for dtype in (torch.bfloat16, torch.float32):
        g = torch.randn(1000, device="cuda").to(dtype)
        want = [g.clone()]
        clip.clip(want, 1.0)
        for offset in range(9):
            memory = torch.zeros(1040, dtype=dtype, device="cuda")
            clip.clip([g], 1.0, out=[memory[offset:offset + 1000]])
            assert torch.equal(memory[offset:offset + 1000], want[0])
            assert not bool(memory[:offset].any()) and not bool(memory[offset + 1000:].any())


@pytest.mark.parametrize("dtype", ["b", "f"])
@pytest.mark.parametrize("scale", [1e-36, 1e-30, 1e-25, 1e-20, 1e-16, 1e15, 1e18, 1e19, 1e25, 1e33])
def test_far_from_one(dtype, scale):
    """Squares that leave the range of fp32."""
    grads = make([(5000, dtype, 1), (77, dtype, 0)], 3, scale)
    want = exact(grads)
    clip = dm.GradClip.create()
    assert abs(float(clip.norm(grads)) - want) <= NORM * want
    mixed = grads + make([(3000, dtype, 0)], 4)
    want = exact(mixed)
    assert abs(float(clip.norm(mixed)) - want) <= NORM * want


def test_not_finite():
    clip = dm.GradClip.create()
    for bad in (math.inf, -math.inf, math.nan):
        for where in (0, 4, 999):
            grads = make([(1000, "b", 0), (1000, "f", 0)], 5)
            grads[1][where] = bad
            before = [g.clone() for g in grads]
            norm = float(clip.clip(grads, 0.5))
            assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
            assert all(torch.equal(g.view(torch.uint8), b.view(torch.uint8)) for g, b in zip(grads, before))
    assert float(clip.norm([torch.full((4,), 3e38, device="cuda")] * 4)) == math.inf  # above what fp32 holds


def test_nothing_and_zeros():
    clip = dm.GradClip.create()
    assert float(clip.norm([])) == 0.0 and float(clip.clip([], 1.0)) == 0.0
    empty = torch.empty(0, 5, device="cuda")
    zeros = torch.zeros(3000, dtype=torch.bfloat16, device="cuda")
    assert float(clip.clip([empty, zeros], 0.0)) == 0.0
    assert float(clip.norm([zeros, -zeros])) == 0.0
    one = torch.ones(100, device="cuda")
    assert abs(float(clip.norm([one, one])) - 200 ** 0.5) < 1e-5  # twice, so it counts twice


def test_past_32_bits():
    """A tensor of more than 2^32 bytes and 2^31 elements."""
    n = (1 << 31) + 12345
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    g[-1] = 2.0 ** 20
    want = math.sqrt(n - 1 + 2.0 ** 40)
    clip = dm.GradClip.create()
    assert abs(float(clip.clip([g], want / 4)) - want) <= NORM * want
    assert bool((g[:-1] == 0.25).all()) and float(g[-1]) == 2.0 ** 18


def test_repeats_bit_for_bit_and_captured():
    grads = make(SETS["many"] + SETS["large"], 9)
    clip = dm.GradClip.create()
    first = clip.norm(grads)
    assert all(torch.equal(clip.norm(grads), first) for _ in range(10))
    out = [torch.empty_like(g) for g in grads]
    limit = float(first) / 2
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = clip.clip(grads, limit, out=out)
    for k in (1.0, 3.0):
        for g in grads:
            g *= k
        graph.replay()
        plain = dm.GradClip.create()
        want = [g.clone() for g in grads]
        assert torch.equal(plain.clip(want, limit), norm)
        assert all(torch.equal(o, w) for o, w in zip(out, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = clip.norm(grads, stream=side)
    side.synchronize()
    assert torch.equal(got, norm)


def test_refusals_reach_python():
    clip = dm.GradClip.create()
    a = torch.ones(64, device="cuda")
    for call in (lambda: clip.clip([a, a], 1.0), lambda: clip.clip([a[:40], a[39:]], 1.0),
                 lambda: clip.clip([a[:32], a[32:]], 1.0, out=[a[32:], a[:32]]), lambda: clip.clip([a], -1.0),
                 lambda: clip.clip([a], math.nan), lambda: clip.clip([a], 1.0, out=[a[:32]]),
                 lambda: clip.norm([a.cpu()]), lambda: clip.norm([a.half()]), lambda: clip.norm([a.view(8, 8).T])):
        with pytest.raises(dm.DmuonError):
            call()
    assert bool((a == 1.0).all())


def test_a_tensor_named_twice_counts_twice():
    clip = dm.GradClip.create()
    for n in (1000, 1 << 20):
        a = torch.ones(n, device="cuda", dtype=torch.bfloat16)
        assert float(clip.norm([a, a, a[:n // 2]])) == pytest.approx((2.5 * n) ** 0.5, rel=1e-6)


@pytest.mark.parametrize("size", [500, 1 << 20])
def test_limits_of_zero_and_infinity(size):
    clip = dm.GradClip.create()
    grads = [torch.randn(size, device="cuda"), torch.randn(size, device="cuda").to(torch.bfloat16)]
    before = [g.clone() for g in grads]
    clip.clip(grads, math.inf)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    assert float(clip.clip(grads, 0.0)) > 0.0 and not any(g.any() for g in grads)
    assert float(clip.clip(grads, 0.0)) == 0.0 and not any(g.any() for g in grads)  # 0 / 0 is not asked for
