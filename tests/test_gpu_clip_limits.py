"""What is clipped goes by the norm that the caller gets: one that is infinite in fp32 clips nothing, even where the sum
in 64 bits is finite."""

import math

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu

FEW, MANY = 1000, 400000  # elements of a tensor: the set in one launch, and in two


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("size", [4, FEW, MANY])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_norm_above_fp32_clips_nothing(size, dtype):
    # each element is finite, and so is the sum of their squares in 64 bits: 3e38 * sqrt(4 * size) is above 3.4028e38
    grads = [torch.full((size,), 3e38, device="cuda", dtype=dtype) for _ in range(4)]
    grads[1][size // 2] = -1.0
    before = [g.clone() for g in grads]
    clip = dm.GradClip.create()
    for limit in (0.0, 1.0, 1e38):
        out = [torch.zeros_like(g) for g in grads]
        assert float(clip.clip(grads, limit, out=out)) == math.inf
        assert all(same(o, b) for o, b in zip(out, before))
        assert float(clip.clip(grads, limit)) == math.inf
        assert all(same(g, b) for g, b in zip(grads, before))
    assert float(clip.norm(grads)) == math.inf


@pytest.mark.parametrize("size", [4, FEW, MANY])
def test_a_norm_just_inside_fp32_clips(size):
    # 4 * size elements of 1.6e38 / sqrt(size) have the norm 3.2e38. Scale, element and product are rounded once each,
    # and the norm (at most 42 * 2^-24 off) goes into the scale.
    grads = [torch.full((size,), 1.6e38 / math.sqrt(size), device="cuda") for _ in range(4)]
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    clip = dm.GradClip.create()
    before = [g.double() for g in grads]
    norm = float(clip.clip(grads, 1e30))
    assert abs(norm - want) <= 42 * 2.0 ** -24 * want
    for g, b in zip(grads, before):
        exactly = b * (1e30 / want)
        assert bool(((g.double() - exactly).abs() <= 46 * 2.0 ** -24 * exactly).all())
