"""Which sets are one launch: those whose 16-byte vectors fit 128 units of 256, whatever their tensors' number up to 128.
A tensor of n elements from a 16-byte boundary has n / 4 (fp32) or n / 8 (bf16) vectors and begins a unit of its own."""

import ctypes
import math

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu

UNIT = {torch.float32: 1024, torch.bfloat16: 2048}  # elements
F, B = torch.float32, torch.bfloat16

# sets, and whether they fit
SETS = {
    "toy": ([(128 * 256, F)] * 4, True),
    "full fp32": ([(128 * UNIT[F], F)], True),
    "full bf16": ([(128 * UNIT[B], B)], True),
    "full of tensors": ([(UNIT[F] if i % 2 else UNIT[B], F if i % 2 else B) for i in range(128)], True),
    "full, uneven": ([(50 * UNIT[F], F), (77 * UNIT[B], B), (5, F)], True),
    "a unit more": ([(128 * UNIT[F], F), (1, F)], False),
    "a vector more": ([(128 * UNIT[F] + 4, F)], False),
    "a tensor more": ([(8, B)] * 129, False),
}


def launches(call):
    """Kernels that a call captures."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    n = ctypes.c_size_t()
    assert ctypes.CDLL("libcudart.so.13").cudaGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None,
                                                            ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("name", SETS)
def test_sets_that_fit_are_one_launch(name):
    sizes, fits = SETS[name]
    g = torch.Generator(device="cuda")
    g.manual_seed(len(name))
    grads = [torch.randn(n, generator=g, device="cuda").to(dtype) for n, dtype in sizes]
    want = math.sqrt(sum(float(x.double().square().sum()) for x in grads))
    clip = dm.GradClip.create()
    clip.workspace.fill_(255)
    before = [x.clone() for x in grads]
    for limit in (want / 7, want * 2):
        out = [torch.full_like(x, 3.0) for x in grads]
        norm = clip.clip(grads, limit, out=out)
        assert abs(float(norm) - want) <= 42 * 2.0 ** -24 * want  # as derived for other sets
        assert torch.equal(clip.norm(grads), norm)
        scale = min(1.0, limit / want)
        for o, b in zip(out, before):
            exactly = b.double() * scale
            off = (46 * 2.0 ** -24 + torch.finfo(b.dtype).eps / 2) * exactly.abs()
            assert bool(((o.double() - exactly).abs() <= off).all())
            assert scale < 1.0 or torch.equal(o, b)
    place = [x.clone() for x in grads]
    clip.clip(place, want / 7)
    clip.clip(grads, want / 7, out=out)
    assert all(torch.equal(p, o) for p, o in zip(place, out))
    assert all(torch.equal(x, b) for x, b in zip(grads, before))
    assert launches(lambda: clip.norm(grads)) == (1 if fits else 2)
    assert launches(lambda: clip.clip(grads, 1.0, out=out)) == (1 if fits else 2)
