"""GPU parity of a mixture's experts for a few tokens (dmuon_experts_forward) with the fp64 oracle,
element by element within the oracle's bound on what rounding may do."""

import numpy as np
import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm
from oracle import experts_ref as ref

pytestmark = pytest.mark.gpu


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(tokens, top, experts, dim, inner, gated, seed, dropped=0.1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(0, experts, (tokens, top), generator=g, device="cuda")
    gone = torch.rand(tokens, top, generator=g, device="cuda") < dropped
    ids = torch.where(gone, torch.where(ids % 2 == 0, -1, experts + 5), ids)
    bf16 = lambda t: t.to(torch.bfloat16)  # noqa: E731
    return dict(x=bf16(r(tokens, dim)), expert_ids=ids, weights=torch.softmax(r(tokens, top), 1),
                up=bf16(r(experts, inner, dim) * dim ** -0.5), down=bf16(r(experts, dim, inner) * inner ** -0.5),
                gate=bf16(r(experts, inner, dim) * dim ** -0.5) if gated else None)


def check(layer, s, y=None):
    got = f64(layer.forward(**s) if y is None else y)
    want, off = ref.forward(f64(s["x"]), s["expert_ids"].cpu().numpy(), f64(s["weights"]), f64(s["up"]), f64(s["down"]),
                            f64(s["gate"]))
    assert layer.read_device_status(torch.cuda.current_stream().cuda_stream) == 0
    assert np.all(np.abs(got - want) <= off), np.max(np.abs(got - want) / off)


@pytest.mark.parametrize("tokens,top,experts,dim,inner,gated,dropped", [
    (1, 1, 1, 8, 8, True, 0.0), (1, 1, 1, 1, 1, False, 0.0), (1, 2, 4, 64, 48, True, 0.0), (1, 8, 64, 256, 136, True, 0.0),
    (2, 3, 5, 40, 24, False, 0.2), (3, 2, 8, 33, 17, True, 0.1), (7, 2, 8, 200, 72, False, 0.0),
    (8, 4, 6, 512, 264, True, 0.1), (9, 1, 2, 136, 1000, True, 0.0), (13, 2, 3, 15, 520, False, 0.1),
    (16, 8, 16, 72, 64, True, 0.0), (31, 6, 60, 264, 104, True, 0.05), (33, 1, 1, 88, 80, True, 0.0),
    (64, 8, 64, 128, 88, True, 0.0), (70, 2, 2, 104, 40, False, 0.0), (100, 3, 200, 24, 56, True, 0.3),
    (32, 64, 70, 16, 24, True, 0.0), (2048, 1, 3, 8, 16, False, 0.1), (5, 2, 4096, 16, 8, True, 0.1),
    (6, 2, 4, 4096, 8, True, 0.0), (2, 1, 2, 8, 8960, False, 0.0),
    (40, 3, 3, 1000, 4000, True, 0.0), (300, 1, 2, 1032, 520, False, 0.1), (12, 4, 5, 520, 5000, False, 0.0)])
def test_experts(tokens, top, experts, dim, inner, gated, dropped):
    check(dm.Experts.create(tokens, top, experts, dim, inner), make(tokens, top, experts, dim, inner, gated,
                                                                    tokens + dim + inner, dropped))


@pytest.mark.parametrize("gated", [True, False])
def test_the_same_expert_again_and_nobody(gated):
    s = make(6, 4, 9, 48, 40, gated, 3, 0.0)
    s["expert_ids"][0] = 4
    s["expert_ids"][2] = -1
    s["expert_ids"][3] = torch.tensor([2, 2, 9, 2 ** 40], device="cuda")
    s["expert_ids"][5] = torch.tensor([-2 ** 62, 8, 8, 0], device="cuda")
    layer = dm.Experts.create(6, 4, 9, 48, 40)
    y = layer.forward(**s)
    check(layer, s, y)
    assert torch.equal(y[2], torch.zeros_like(y[2]))
    s["expert_ids"][:] = -1
    assert torch.equal(layer.forward(**s), torch.zeros_like(y))


def test_all_tokens_to_one_expert():
    s = make(64, 2, 8, 72, 56, True, 4, 0.0)
    s["expert_ids"][:, 0], s["expert_ids"][:, 1] = 5, 6
    check(dm.Experts.create(64, 2, 8, 72, 56), s)


def test_larger_layer_than_tokens_and_strided_rows():
    s = make(5, 2, 4, 64, 40, True, 5)
    wide = torch.zeros(5, 80, dtype=torch.bfloat16, device="cuda")
    layer = dm.Experts.create(40, 2, 4, 64, 40)
    for at in (0, 8, 3):  # pitch 80; the last does not start on 16 bytes
        wide[:, at:at + 64] = s["x"]
        check(layer, {**s, "x": wide[:, at:at + 64]})
    assert layer.forward(**{**s, "x": s["x"][:0], "expert_ids": s["expert_ids"][:0],
                            "weights": s["weights"][:0]}).shape == (0, 64)


def test_what_is_not_named_is_not_read():
    s = make(4, 2, 6, 64, 48, True, 6, 0.0)
    s["expert_ids"] %= 5
    want = dm.Experts.create(4, 2, 6, 64, 48).forward(**s)
    for m in ("up", "gate", "down"):
        s[m][5] = float("nan")
    layer = dm.Experts.create(4, 2, 6, 64, 48)
    layer.workspace.fill_(255)  # NaN
    assert torch.equal(layer.forward(**s), want)
    s["weights"][1] = 0.0
    s["up"][s["expert_ids"][1, 0], 0] = float("inf")  # a weight of 0 does not hide it
    assert not torch.isfinite(layer.forward(**s)[1]).any()


def test_repeats_bit_for_bit_and_on_a_stream():
    s = make(23, 5, 12, 256, 136, True, 7)
    layer = dm.Experts.create(23, 5, 12, 256, 136)
    want = layer.forward(**s)
    side = torch.cuda.Stream()
    for _ in range(20):
        assert torch.equal(layer.forward(**s), want)
    side.wait_stream(torch.cuda.current_stream())
    got = layer.forward(**s, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_captured():
    s = make(9, 3, 8, 128, 72, True, 8)
    layer = dm.Experts.create(9, 3, 8, 128, 72)
    layer.forward(**s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(**s)
    for seed in (9, 10):  # other routing and other values in the same places
        other = make(9, 3, 8, 128, 72, True, seed, 0.3)
        for k, v in other.items():
            s[k].copy_(v)
        graph.replay()
        check(layer, s, y)


@pytest.mark.parametrize("tokens", [1, 7, 20])
def test_call_after_call_without_a_wait(tokens):
    """A call's launches are set up while those before still run, its own and the last call's, in the same workspace."""
    layer = dm.Experts.create(tokens, 3, 10, 1100, 2000)
    calls = [make(tokens, 3, 10, 1100, 2000, gated, 50 + k, 0.05) for k, gated in enumerate([True, False, True])]
    first = []
    for s in calls:
        first.append(layer.forward(**s))
        torch.cuda.synchronize()
    later = [[layer.forward(**s) for s in calls] for _ in range(40)]
    for s, y in zip(calls, first):
        check(layer, s, y)
    for ys in later:
        for y, again in zip(first, ys):
            assert torch.equal(y, again)


@pytest.mark.parametrize("which", ["up", "gate", "down", "all"])
def test_matrices_that_do_not_start_on_16_bytes(which):
    s = make(6, 2, 4, 64, 48, True, 11)

    def shifted(t):
        flat = torch.full((t.numel() + 8,), float("nan"), dtype=t.dtype, device="cuda")
        flat[1:t.numel() + 1] = t.flatten()
        return flat[1:t.numel() + 1].view(t.shape)

    names = ("up", "gate", "down") if which == "all" else (which,)
    check(dm.Experts.create(6, 2, 4, 64, 48), {**s, **{k: shifted(s[k]) for k in names}})


@pytest.mark.parametrize("gated", [True, False])
def test_few_tokens_that_name_the_same_experts_over_and_over(gated):
    # 256 assignments each to two experts, and 8 to one
    s = make(8, 64, 3, 72, 56, gated, 12, 0.0)
    s["expert_ids"][:, 0] = 1
    s["expert_ids"][:, 1:] = torch.arange(63, device="cuda") % 2 * 2
    check(dm.Experts.create(8, 64, 3, 72, 56), s)


@pytest.mark.parametrize("dim,inner", [(1 << 20, 8), (8, 1 << 20), ((1 << 20) - 1, 3)])
def test_the_widest_layers(dim, inner):
    check(dm.Experts.create(2, 1, 2, dim, inner), make(2, 1, 2, dim, inner, True, 13, 0.0))


@pytest.mark.parametrize("inner", [48, 43])
def test_values_that_are_no_numbers_stay_in_their_token(inner):
    s = make(12, 3, 5, 64, inner, True, 14, 0.0)
    layer = dm.Experts.create(12, 3, 5, 64, inner)
    want = layer.forward(**s)
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = s["x"].clone()
        x[7, 5] = bad
        y = layer.forward(**{**s, "x": x})
        assert torch.equal(y[:7], want[:7]) and torch.equal(y[8:], want[8:])
        assert not torch.isfinite(y[7]).any()
    # an assignment that adds nothing does so whatever its weight is
    s["expert_ids"][4, 1] = -1
    want = layer.forward(**s)
    s["weights"][4, 1] = float("nan")
    assert torch.equal(layer.forward(**s), want)
