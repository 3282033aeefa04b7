"""What the Python calls of the head's losses and of the routing check and record of
their tensors, with stand-ins for CUDA tensors, devices and streams. No GPU, and
nothing reaches the library."""

import contextlib
import types

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm


class Stand(torch.Tensor):
    """A CPU tensor that says it lies on a CUDA device, and notes the streams it is recorded on."""

    is_cuda = True

    def get_device(self):
        return getattr(self, "place", 0)

    def record_stream(self, stream):
        self.__dict__.setdefault("seen", []).append(stream.cuda_stream)


def stand(*shape, dtype=torch.float32, place=0):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(Stand)
    t.place = place
    return t


class Library:
    """Notes the calls that get past the checks."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if not name.endswith("_destroy"):
                self.calls.append(name)
            return dm.OK
        return call


def stream(handle, device=0):
    return types.SimpleNamespace(cuda_stream=handle, device_index=device)


class World:
    """Which device and stream are current, and the library."""

    def __init__(self, monkeypatch):
        self.device, self.current, self.library = 0, stream(0), Library()

        @contextlib.contextmanager
        def on(s):
            before, self.current, self.device = (self.current, self.device), s, s.device_index
            yield
            self.current, self.device = before

        monkeypatch.setattr(dm, "lib", lambda: self.library)
        monkeypatch.setattr(dm, "_current_device", lambda: self.device)
        monkeypatch.setattr(dm, "_here", lambda device: self.current.cuda_stream)
        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)

    def objects(self):
        head = dm.Head(None, 6, 40, 16, 4)
        head.workspace, head.device = stand(64, dtype=torch.uint8), 0
        return head, dm.Router(6, 2, 8, stand(64, dtype=torch.uint8))


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def tensors():
    bf16, i64, i32 = torch.bfloat16, torch.int64, torch.int32
    return dict(h=stand(6, 16, dtype=bf16), w=stand(40, 16, dtype=bf16), y=stand(6, dtype=i64), lse=stand(6),
                loss=stand(6), g=stand(6), ids=stand(6, 4, dtype=i64), lg=stand(6, 4), dh=stand(6, 16, dtype=bf16),
                dw=stand(40, 16, dtype=bf16), experts=stand(6, 2, dtype=i64), x=stand(6, 16, dtype=bf16),
                ys=stand(12, 16, dtype=bf16), wts=stand(6, 2), dest=stand(6, 2, dtype=i32),
                source=stand(12, dtype=i32))


def route(t):
    return dm.Route(t["dest"], t["source"], None)


# each call, and the tensors it takes
CALLS = {
    "xent": (("h", "w", "y"), lambda o, t, s: o[0].xent(t["h"], t["w"], t["y"], stream=s)),
    "xent_backward": (("h", "w", "y", "lse", "g", "dh", "dw"),
                      lambda o, t, s: o[0].xent_backward(t["h"], t["w"], t["y"], t["lse"], t["g"], dhidden=t["dh"],
                                                         dweight=t["dw"], stream=s)),
    "xent_backward_loss": (("h", "w", "y", "lse", "g", "loss"),
                           lambda o, t, s: o[0].xent_backward(t["h"], t["w"], t["y"], t["lse"], t["g"],
                                                              loss=t["loss"], stream=s)),
    "distill": (("h", "w", "ids", "lg"), lambda o, t, s: o[0].distill(t["h"], t["w"], t["ids"], t["lg"], 2.0,
                                                                      stream=s)),
    "distill_backward": (("h", "w", "ids", "lg", "lse", "g", "dh", "dw"),
                         lambda o, t, s: o[0].distill_backward(t["h"], t["w"], t["ids"], t["lg"], 2.0, t["lse"],
                                                               t["g"], dhidden=t["dh"], dweight=t["dw"], stream=s)),
    "sort": (("experts",), lambda o, t, s: o[1].sort(t["experts"], stream=s)),
    "dispatch": (("x", "dest", "source"), lambda o, t, s: o[1].dispatch(t["x"], route(t), stream=s)),
    "combine": (("ys", "wts", "dest"), lambda o, t, s: o[1].combine(t["ys"], t["wts"], route(t), stream=s)),
    "combine_backward": (("x", "ys", "wts", "dest", "source"),
                         lambda o, t, s: o[1].combine_backward(t["x"], t["ys"], t["wts"], route(t), stream=s)),
    "dispatch_backward": (("ys", "dest"), lambda o, t, s: o[1].dispatch_backward(t["ys"], route(t), stream=s)),
}
EACH = [(call, name) for call, (names, _) in CALLS.items() for name in names]


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_the_objects_device_are_taken(world, call):
    for s in (None, stream(0), stream(7)):
        CALLS[call][1](world.objects(), tensors(), s)
    assert len(world.library.calls) == 3


@pytest.mark.parametrize("call,name", EACH)
def test_a_tensor_of_another_device_is_refused(world, call, name):
    t = tensors()
    t[name].place = 1
    with pytest.raises(dm.DmuonError) as e:
        CALLS[call][1](world.objects(), t, None)
    assert e.value.status == dm.ERR_INVALID_ARG and "cuda:1" in str(e.value)
    assert not world.library.calls


@pytest.mark.parametrize("call", CALLS)
def test_another_current_device_and_streams_of_another_device_are_refused(world, call):
    with pytest.raises(dm.DmuonError) as e:
        CALLS[call][1](world.objects(), tensors(), stream(0, device=1))
    assert e.value.status == dm.ERR_INVALID_ARG
    world.device = 1
    with pytest.raises(dm.DmuonError) as e:
        CALLS[call][1](world.objects(), tensors(), None)
    assert e.value.status == dm.ERR_INVALID_ARG
    assert not world.library.calls
    CALLS[call][1](world.objects(), tensors(), stream(7))  # a stream of the object's device brings its device
    assert len(world.library.calls) == 1 and world.device == 1


@pytest.mark.parametrize("call", CALLS)
def test_every_tensor_of_a_call_is_recorded_on_its_stream(world, call):
    t, objects = tensors(), world.objects()
    CALLS[call][1](objects, t, stream(7))
    for name in CALLS[call][0]:
        assert 7 in getattr(t[name], "seen", ()), name


@pytest.mark.parametrize("want", [True, False, None])
def test_gradients_that_are_not_given_are_nothing_to_record(world, want):
    t, (head, _) = tensors(), world.objects()
    head.xent_backward(t["h"], t["w"], t["y"], t["lse"], t["g"], dhidden=want, dweight=want, stream=stream(7))
    assert len(world.library.calls) == 1


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_that_is_current_is_recorded_all_the_same(world, call):
    t, objects = tensors(), world.objects()
    world.current = stream(7)
    CALLS[call][1](objects, t, stream(7))
    for name in CALLS[call][0]:
        assert 7 in getattr(t[name], "seen", ()), name


@pytest.mark.parametrize("call", ["xent", "xent_backward", "distill", "distill_backward", "sort"])
@pytest.mark.parametrize("given", [None, stream(7)])
def test_a_workspace_is_recorded_on_the_streams_that_use_it(world, call, given):
    # allocated on stream 0, used while stream 7 is current: only the object can record it
    objects = world.objects()
    scratch = objects[call == "sort"].workspace
    CALLS[call][1](objects, tensors(), None)
    assert not hasattr(scratch, "seen")
    world.current = stream(7)
    CALLS[call][1](objects, tensors(), given)
    assert 7 in scratch.seen


@pytest.mark.parametrize("name", ["dh", "dw"])
def test_given_gradients_are_looked_at_before_they_are_recorded(world, name):
    t = tensors()
    t[name] = torch.zeros(t[name].shape, dtype=torch.bfloat16)  # of the host
    with pytest.raises(dm.DmuonError) as e:
        CALLS["xent_backward"][1](world.objects(), t, stream(7))
    assert e.value.status == dm.ERR_INVALID_ARG and not world.library.calls
    assert not any(hasattr(x, "seen") for x in t.values())


def test_calls_before_a_bind_are_refused(world):
    head = dm.Head(None, 6, 40, 16, 4)
    for name in ("xent", "xent_backward", "distill", "distill_backward"):
        with pytest.raises(dm.DmuonError) as e:
            CALLS[name][1]((head, None), tensors(), None)
        assert e.value.status == dm.ERR_NOT_BOUND
