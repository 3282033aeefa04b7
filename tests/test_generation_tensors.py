"""What the Python calls of the experts' layer, the log probabilities and the clipping check and record of their
tensors, with stand-ins for CUDA tensors, devices and streams. No GPU, and nothing reaches the library."""

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm
from test_operator_tensors import World, stand, stream


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def objects():
    head = dm.Head(None, 6, 40, 16, 4)
    head.workspace, head.device = stand(64, dtype=torch.uint8), 0
    return dict(head=head, layer=dm.Experts(6, 2, 8, 16, 24, stand(64, dtype=torch.uint8)),
                clip=dm.GradClip(stand(64, dtype=torch.uint8)))


def tensors():
    bf16, i64 = torch.bfloat16, torch.int64
    return dict(h=stand(6, 16, dtype=bf16), w=stand(40, 16, dtype=bf16), y=stand(6, dtype=i64), logp=stand(6),
                entropy=stand(6), lse=stand(6), gl=stand(6), ge=stand(6), dh=stand(6, 16, dtype=bf16),
                dw=stand(40, 16, dtype=bf16), x=stand(6, 16, dtype=bf16), ids=stand(6, 2, dtype=i64), wts=stand(6, 2),
                up=stand(8, 24, 16, dtype=bf16), gate=stand(8, 24, 16, dtype=bf16), down=stand(8, 16, 24, dtype=bf16),
                g0=stand(5, 3), g1=stand(7, dtype=bf16), o0=stand(5, 3), o1=stand(7, dtype=bf16))


def scores(t):
    return dm.Logprobs(t["logp"], t["entropy"], t["lse"], None, None)


CALLS = {
    "logprobs": (("h", "w", "y"), lambda o, t, s: o["head"].logprobs(t["h"], t["w"], t["y"], stream=s)),
    "logprobs_backward": (("h", "w", "y", "logp", "entropy", "lse", "gl", "ge", "dh", "dw"),
                          lambda o, t, s: o["head"].logprobs_backward(
                              t["h"], t["w"], t["y"], scores(t), t["gl"], t["ge"], dhidden=t["dh"], dweight=t["dw"],
                              stream=s)),
    "forward": (("x", "ids", "wts", "up", "gate", "down"),
                lambda o, t, s: o["layer"].forward(t["x"], t["ids"], t["wts"], t["up"], t["down"], gate=t["gate"],
                                                   stream=s)),
    "norm": (("g0", "g1"), lambda o, t, s: o["clip"].norm([t["g0"], t["g1"]], stream=s)),
    "clip": (("g0", "g1", "o0", "o1"), lambda o, t, s: o["clip"].clip([t["g0"], t["g1"]], 1.0,
                                                                        out=[t["o0"], t["o1"]], stream=s)),
}
OWNER = {"logprobs": "head", "logprobs_backward": "head", "forward": "layer", "norm": "clip", "clip": "clip"}
EACH = [(call, name) for call, (names, _) in CALLS.items() for name in names]


@pytest.fixture(autouse=True)
def results_on_the_host(monkeypatch):
    # results are made on the stand-ins' device, the host
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **{**k, "device": "cpu"}))


def test_calls_reach_the_library_once(world):
    for call in CALLS:
        CALLS[call][1](objects(), tensors(), None)
    assert world.library.calls == ["dmuon_head_logprobs", "dmuon_head_logprobs_backward", "dmuon_experts_forward",
                                   "dmuon_grad_norm", "dmuon_grad_clip"]


@pytest.mark.parametrize("call,name", EACH)
def test_a_tensor_of_another_device_is_refused(world, call, name):
    t = tensors()
    t[name].place = 1
    with pytest.raises(dm.DmuonError) as e:
        CALLS[call][1](objects(), t, None)
    assert e.value.status == dm.ERR_INVALID_ARG and "cuda:1" in str(e.value)
    assert not world.library.calls


@pytest.mark.parametrize("call,name", EACH)
def test_a_tensor_of_the_host_is_refused(world, call, name):
    t = tensors()
    t[name] = torch.zeros(t[name].shape, dtype=t[name].dtype)
    with pytest.raises(dm.DmuonError) as e:
        CALLS[call][1](objects(), t, None)
    assert e.value.status == dm.ERR_INVALID_ARG and not world.library.calls


@pytest.mark.parametrize("call,name", EACH)
def test_other_types_and_shapes_are_refused(world, call, name):
    for other in (lambda a: a.to(torch.float16), lambda a: a[:-1]):
        t = tensors()
        place = t[name]
        t[name] = other(place).as_subclass(type(place))
        t[name].place = 0
        if name in ("g0", "g1") and t[name].dtype == place.dtype and call == "norm":
            continue  # any shape has a norm
        if name in ("h", "x") and t[name].dtype == place.dtype and call == "logprobs":
            t["y"] = stand(6, dtype=torch.int64)
        with pytest.raises(dm.DmuonError) as e:
            CALLS[call][1](objects(), t, None)
        assert e.value.status == dm.ERR_INVALID_ARG and not world.library.calls


@pytest.mark.parametrize("call", CALLS)
def test_another_current_device_and_streams_of_another_device_are_refused(world, call):
    with pytest.raises(dm.DmuonError) as e:
        CALLS[call][1](objects(), tensors(), stream(0, device=1))
    assert e.value.status == dm.ERR_INVALID_ARG
    o = objects()
    world.device = 1
    with pytest.raises(dm.DmuonError) as e:
        CALLS[call][1](o, tensors(), None)
    assert e.value.status == dm.ERR_INVALID_ARG and not world.library.calls
    CALLS[call][1](o, tensors(), stream(7))  # a stream of the object's device brings its device
    assert len(world.library.calls) == 1 and world.device == 1


@pytest.mark.parametrize("call", CALLS)
def test_every_tensor_of_a_call_and_the_workspace_are_recorded_on_its_stream(world, call):
    t, o = tensors(), objects()
    CALLS[call][1](o, t, stream(7))
    for name in CALLS[call][0]:
        assert 7 in getattr(t[name], "seen", ()), name
    assert 7 in o[OWNER[call]].workspace.seen


@pytest.mark.parametrize("call", CALLS)
def test_a_workspace_is_recorded_on_the_current_stream_where_that_is_another(world, call):
    o = objects()
    CALLS[call][1](o, tensors(), None)
    assert not hasattr(o[OWNER[call]].workspace, "seen")
    world.current = stream(7)
    CALLS[call][1](o, tensors(), None)
    assert 7 in o[OWNER[call]].workspace.seen


def test_more_tokens_than_the_layer_was_made_for_are_refused(world):
    t = tensors()
    layer = dm.Experts(5, 2, 8, 16, 24, stand(64, dtype=torch.uint8))
    with pytest.raises(dm.DmuonError):
        layer.forward(t["x"], t["ids"], t["wts"], t["up"], t["down"])
    assert not world.library.calls


def test_gradients_out_of_order_and_parts_are_refused(world):
    o, t = objects(), tensors()
    wide = stand(8, 8)
    for call in (lambda: o["clip"].norm([wide.T[:, 1:]]), lambda: o["clip"].clip([t["g0"]], 1.0, out=[t["o1"]]),
                 lambda: o["clip"].clip([t["g0"]], 1.0, out=[]), lambda: o["clip"].clip([t["g0"]], 1.0, out=[stand(3, 5)])):
        with pytest.raises(dm.DmuonError) as e:
            call()
        assert e.value.status == dm.ERR_INVALID_ARG
    assert not world.library.calls
