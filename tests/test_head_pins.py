"""The oracle of the head's losses and of expert routing, pinned by differences
and closed forms, and the refusals of the library's calls. No GPU."""

import ctypes

import numpy as np
import pytest

from matrix_optimizer_update_gb300 import dmuon as dm
from oracle import head_ref as ref


def rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def central(f, x, eps=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


def test_xent_gradient_is_the_derivative():
    h, w, y, g = rand(4, 6), rand(9, 6, seed=1), np.array([3, -100, 8, 0]), rand(4, seed=2)
    r = ref.xent(h, w, y, g)
    # central differences: truncation ~ eps^2 times third derivatives of order 1, rounding ~ 1e-16 / eps
    assert np.abs(r["dhidden"] - central(lambda a: g @ ref.xent(a, w, y)["loss"], h)).max() < 1e-8
    assert np.abs(r["dweight"] - central(lambda a: g @ ref.xent(h, a, y)["loss"], w)).max() < 1e-8
    assert r["loss"][1] == 0 and not r["dhidden"][1].any()


def test_distill_gradient_is_the_derivative():
    h, w, g = rand(3, 5), rand(8, 5, seed=1), rand(3, seed=2)
    ids = np.array([[7, 0, 3], [2, -1, 5], [1, 1, 1]])
    lg = np.array([[1.0, 0.5, -2.0], [3.0, 9.0, -np.inf], [-np.inf] * 3])
    r = ref.distill(h, w, ids, lg, 1.7, g)
    assert np.abs(r["dhidden"] - central(lambda a: g @ ref.distill(a, w, ids, lg, 1.7)["loss"], h)).max() < 1e-8
    assert np.abs(r["dweight"] - central(lambda a: g @ ref.distill(h, a, ids, lg, 1.7)["loss"], w)).max() < 1e-8
    assert r["loss"][2] == 0 and not r["dhidden"][2].any()


def test_distill_of_one_entry_is_cross_entropy():
    h, w = rand(5, 4), rand(11, 4, seed=1)
    y = np.array([0, 10, 5, 5, 2])
    a = ref.xent(h, w, y)
    b = ref.distill(h, w, y[:, None], np.full((5, 1), 3.0), 1.0)
    assert np.abs(a["loss"] - b["loss"]).max() < 1e-14


def test_distill_from_oneself_is_zero():
    h, w = rand(5, 4), rand(11, 4, seed=1)
    z = h @ w.T
    ids = np.tile(np.arange(11), (5, 1))
    assert np.abs(ref.distill(h, w, ids, z, 2.5)["loss"]).max() < 1e-13


def test_route_gradients_are_the_derivatives():
    ids = np.array([[2, 0], [0, -1], [1, 0]])
    dest, source, offsets = ref.route(ids, 3)
    assert offsets.tolist() == [0, 3, 4, 5]
    assert dest.tolist() == [[4, 0], [1, -1], [3, 2]] and source.tolist() == [1, 2, 5, 4, 0, -1]
    ys, w, dy = rand(6, 4), rand(3, 2, seed=1), rand(3, 4, seed=2)
    dys, dw = ref.combine_backward(dy, ys, w, dest)
    assert np.abs(dys - central(lambda a: (dy * ref.combine(a, w, dest)).sum(), ys)).max() < 1e-8
    assert np.abs(dw - central(lambda a: (dy * ref.combine(ys, a, dest)).sum(), w)).max() < 1e-8
    x, dxs = rand(3, 4, seed=3), rand(6, 4, seed=4)
    dx = ref.combine(dxs, None, dest)
    assert np.abs(dx - central(lambda a: (dxs * ref.dispatch(a, source, 2)).sum(), x)).max() < 1e-8


# ---------------------------------------------------------------- refusals

def refused(status, fn, *args):
    with pytest.raises(dm.DmuonError) as e:
        dm._check(fn(*args))
    assert e.value.status == status
    assert str(e.value).split(": ", 1)[1]


def make_head(*sizes):
    h = ctypes.c_void_p()
    dm._check(dm.lib().dmuon_head_create(*sizes, ctypes.byref(h)))
    return h


@pytest.mark.parametrize("sizes", [(0, 10, 8, 0), (1 << 21, 10, 8, 0), (4, 0, 8, 0), (4, (1 << 22) + 1, 8, 0),
                                   (4, 10, 0, 0), (4, 10, (1 << 16) + 1, 0), (4, 10, 8, -1), (4, 10, 8, 257)])
def test_head_sizes_are_refused(sizes):
    refused(dm.ERR_INVALID_ARG, dm.lib().dmuon_head_create, *sizes, ctypes.byref(ctypes.c_void_p()))


def test_head_create_refuses_no_handle():
    refused(dm.ERR_INVALID_ARG, dm.lib().dmuon_head_create, 4, 10, 8, 0, None)


def test_head_workspace_does_not_hold_the_logits():
    # 64k tokens of a 128k vocabulary: 17 GB of bf16 logits; the workspace's dz stays within 512 MB
    def bytes_of(*sizes):
        n = ctypes.c_size_t()
        h = make_head(*sizes)
        dm._check(dm.lib().dmuon_head_workspace_bytes(h, ctypes.byref(n)))
        dm.lib().dmuon_head_destroy(h)
        return n.value
    tokens, vocab, dim = 65536, 128000, 1024
    parts, acc = 8 * -(-vocab // 128) * tokens, 4 * tokens * dim
    assert bytes_of(tokens, vocab, dim, 0) <= (512 << 20) + parts + 2 * acc


def test_head_calls_are_refused_before_a_bind():
    L, h = dm.lib(), make_head(4, 10, 8, 2)
    refused(dm.ERR_NOT_BOUND, L.dmuon_head_xent, h, 16, 8, 16, 8, 16, 4, 16, 16, None)
    refused(dm.ERR_NOT_BOUND, L.dmuon_head_xent_backward, h, 16, 8, 16, 8, 16, 4, 16, 16, 16, 8, 16, 8, None)
    refused(dm.ERR_NOT_BOUND, L.dmuon_head_distill, h, 16, 8, 16, 8, 16, 16, 2, 1.0, 4, 16, 16, None)
    refused(dm.ERR_NOT_BOUND, L.dmuon_head_distill_backward, h, 16, 8, 16, 8, 16, 16, 2, 1.0, 4, 16, 16, 16, 8, 16, 8,
            None)
    bits = ctypes.c_uint32()
    refused(dm.ERR_NOT_BOUND, L.dmuon_head_read_device_status, h, None, ctypes.byref(bits))
    refused(dm.ERR_INVALID_ARG, L.dmuon_head_xent, h, 16, 8, 16, 8, 16, 5, 16, 16, None)  # tokens > max_tokens
    refused(dm.ERR_INVALID_ARG, L.dmuon_head_xent, None, 16, 8, 16, 8, 16, 4, 16, 16, None)
    for ws, n in ((None, 1 << 40), (1024 * 7 + 16, 1 << 40), (1024 * 1024, 16)):
        refused(dm.ERR_WORKSPACE, L.dmuon_head_bind, h, ws, n, None)
    L.dmuon_head_destroy(h)
    L.dmuon_head_destroy(None)


def test_route_sizes_and_pointers_are_refused():
    L, n = dm.lib(), ctypes.c_size_t()
    for sizes in ((-1, 2, 4), (4, 0, 4), (4, 65, 4), (1 << 30, 2, 4), (4, 2, 0), (4, 2, 4097)):
        refused(dm.ERR_INVALID_ARG, L.dmuon_route_workspace_bytes, *sizes, ctypes.byref(n))
    refused(dm.ERR_INVALID_ARG, L.dmuon_route_workspace_bytes, 4, 2, 4, None)
    dm._check(L.dmuon_route_workspace_bytes(0, 1, 1, ctypes.byref(n)))
    dm._check(L.dmuon_route_workspace_bytes(4, 2, 4, ctypes.byref(n)))
    refused(dm.ERR_INVALID_ARG, L.dmuon_route_sort, None, 4, 2, 4, 256, 256, 256, 256, n.value, None)
    refused(dm.ERR_INVALID_ARG, L.dmuon_route_sort, 260, 4, 2, 4, 256, 256, 256, 256, n.value, None)
    for ws, b in ((None, n.value), (128, n.value), (256, n.value - 1)):
        refused(dm.ERR_WORKSPACE, L.dmuon_route_sort, 256, 4, 2, 4, 256, 256, 256, ws, b, None)
    refused(dm.ERR_INVALID_ARG, L.dmuon_route_dispatch, 256, 7, 256, 256, 4, 2, 8, dm.BF16, 256, None)  # pitch < dim
    refused(dm.ERR_INVALID_ARG, L.dmuon_route_dispatch, None, 8, 256, 256, 4, 2, 8, dm.BF16, 256, None)
    refused(dm.ERR_INVALID_ARG, L.dmuon_route_dispatch, 256, 8, 256, 256, 4, 2, 0, dm.BF16, 256, None)
    refused(dm.ERR_UNSUPPORTED, L.dmuon_route_dispatch, 256, 8, 256, 256, 4, 2, 8, 7, 256, None)
    refused(dm.ERR_INVALID_ARG, L.dmuon_route_combine, 256, None, None, 4, 2, 8, dm.F32, 256, 8, None)
    refused(dm.ERR_INVALID_ARG, L.dmuon_route_combine_backward, 256, 8, 256, None, 256, 256, 4, 2, 8, dm.F32, 256, 256,
            None)
