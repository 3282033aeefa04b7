"""The oracle of log probabilities and of the experts' layer, pinned by differences and closed forms, and the refusals
of the library's calls. No GPU: every refusal comes before anything is launched."""

import ctypes

import numpy as np
import pytest

from matrix_optimizer_update_gb300 import dmuon as dm
from oracle import experts_ref, head_ref as ref


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


@pytest.mark.parametrize("tau", [1.0, 0.6])
def test_logprobs_gradient_is_the_derivative(tau):
    h, w, y = rand(4, 6), rand(9, 6, seed=1), np.array([3, -100, 8, 0])
    gl, ge = rand(4, seed=2), rand(4, seed=3)
    r = ref.logprobs(h, w, y, tau, gl, ge)

    def total(h, w):
        s = ref.logprobs(h, w, y, tau)
        return gl @ s["logp"] + ge @ s["entropy"]

    # central differences: truncation ~ eps^2 times third derivatives of order 1 to 10, rounding ~ 1e-16 / eps
    assert np.abs(r["dhidden"] - central(lambda a: total(a, w), h)).max() < 1e-8
    assert np.abs(r["dweight"] - central(lambda a: total(h, a), w)).max() < 1e-8
    assert r["logp"][1] == 0


def test_logprobs_closed_forms():
    h, w = rand(5, 4), rand(11, 4, seed=1)
    y = np.array([0, 10, 5, 5, 2])
    r = ref.logprobs(h, w, y)
    assert np.abs(r["logp"] + ref.xent(h, w, y)["loss"]).max() < 1e-13
    assert np.abs(ref.logprobs(np.zeros((2, 4)), w, None)["entropy"] - np.log(11)).max() < 1e-14
    # one entry 40 above the rest: H = (1 - p) (1 + 40) and a little
    sure = ref.logprobs(np.array([[40.0]]), np.array([[1.0], [0.0], [0.0]]), np.array([0]))
    rest = 2 * np.exp(-40.0)
    assert abs(sure["logp"][0] + rest) < 1e-9 * rest
    assert abs(sure["entropy"][0] - rest * 41) < 1e-9 * rest


def test_experts_closed_forms():
    x, up, down = rand(3, 5), rand(4, 6, 5, seed=1), rand(4, 5, 6, seed=2)
    ids, weights = np.array([[0, 2], [3, 3], [-1, 4]]), rand(3, 2, seed=3)
    y, off = experts_ref.forward(x, ids, weights, up, down)

    def one(e, v):
        h = up[e] @ v
        return down[e] @ (h / (1 + np.exp(-h)))

    want = np.stack([weights[0, 0] * one(0, x[0]) + weights[0, 1] * one(2, x[0]), weights[1].sum() * one(3, x[1]),
                     np.zeros(5)])
    assert np.abs(y - want).max() < 1e-14 and np.all(off > 0) and np.all(off < 0.2 * (1 + np.abs(y)))
    # a gate of 40 everywhere is the identity times 40
    gate = np.zeros((4, 6, 5))
    gate[:, :, 0] = 40.0
    x[:, 0] = 1.0
    y, _ = experts_ref.forward(x, ids, weights, up, down, gate)
    assert np.abs(y[0] - 40 * sum(weights[0, k] * down[ids[0, k]] @ (up[ids[0, k]] @ x[0]) for k in range(2))).max() < 1e-12


# ------------------------------------------------------------------ refusals
def refused(status, call, *words):
    st = call()
    assert st == status, dm.lib().dmuon_last_error()
    message = dm.lib().dmuon_last_error().decode()
    assert message and all(w in message for w in words), message


A, B = 1 << 20, 1 << 21  # addresses that nothing looks at


def norm(ptrs, counts, types, n=None, norm=A, ws=A, bytes_=1 << 20):
    n = len(ptrs) if n is None else n
    arr = lambda t, v: (t * max(1, len(v)))(*v)  # noqa: E731
    return dm.lib().dmuon_grad_norm(arr(ctypes.c_uint64, ptrs), arr(ctypes.c_int64, counts), arr(ctypes.c_int32, types), n,
                                    norm, ws, bytes_, 0)


def clip(ptrs, out, counts, types, max_norm=1.0):
    arr = lambda t, v: (t * max(1, len(v)))(*v)  # noqa: E731
    return dm.lib().dmuon_grad_clip(arr(ctypes.c_uint64, ptrs), arr(ctypes.c_uint64, out), arr(ctypes.c_int64, counts),
                                    arr(ctypes.c_int32, types), len(ptrs), max_norm, A, A, 1 << 20, 0)


def test_clip_refusals():
    bad = dm.ERR_INVALID_ARG
    refused(bad, lambda: norm([A], [4], [0], norm=0), "norm")
    refused(bad, lambda: norm([A], [4], [0], norm=A + 2), "norm")
    refused(bad, lambda: norm([A], [4], [0], n=-1), "n must")
    refused(bad, lambda: norm([A], [-1], [0]), "count")
    refused(bad, lambda: norm([A], [(1 << 40) + 1], [0]), "count")
    refused(bad, lambda: norm([0], [4], [0]), "gradient")
    refused(bad, lambda: norm([A + 2], [4], [0]), "gradient")
    refused(bad, lambda: norm([A + 1], [4], [1]), "gradient")
    refused(dm.ERR_UNSUPPORTED, lambda: norm([A], [4], [2]), "dtypes")
    for ws, n in ((0, 1 << 20), (A + 128, 1 << 20), (A, 64)):
        refused(dm.ERR_WORKSPACE, lambda: norm([A], [4], [0], ws=ws, bytes_=n), "workspace")
    for limit in (-1.0, float("nan")):
        refused(bad, lambda: clip([A], [A], [4], [0], limit), "max_norm")
    refused(bad, lambda: clip([A], [0], [4], [0]), "result")
    refused(bad, lambda: clip([A], [B + 2], [4], [0]), "result")


@pytest.mark.parametrize("grads,out,counts", [
    ([A, A], [A, A], [4, 4]),                     # a tensor twice
    ([A, A + 12], [A, A + 12], [4, 4]),           # partly over another
    ([A, B], [B, A], [4, 4]),                     # each into the other's place
    ([A, B], [A + 4, B], [4, 4]),                 # a shifted place of one's own
    ([A, B, B + 64], [A, B + 32, B + 100], [4, 16, 4]),
    ([A, B], [B + 1024, B + 1024], [4, 4]),       # one place for two
    ([A, A + 1000, B], [A, A + 1000, A + 4], [2000, 10, 1])])
def test_results_that_overlap_are_refused(grads, out, counts):
    refused(dm.ERR_INVALID_ARG, lambda: clip(grads, out, counts, [0] * len(counts)), "overlaps")


def experts(x=A, ld=16, ids=A, w=A, tokens=4, top=2, n=8, dim=16, inner=24, up=A, gate=A, down=A, y=B, ld_y=16, ws=A,
            bytes_=1 << 30):
    return dm.lib().dmuon_experts_forward(x, ld, ids, w, tokens, top, n, dim, inner, up, gate, down, y, ld_y, ws, bytes_, 0)


def test_experts_refusals():
    bad = dm.ERR_INVALID_ARG
    for kw in (dict(top=0), dict(top=65), dict(tokens=-1), dict(tokens=1025, top=2), dict(n=0), dict(n=4097), dict(dim=0),
               dict(inner=0), dict(dim=(1 << 20) + 1), dict(n=4096, dim=1 << 19), dict(tokens=1 << 40), dict(x=0), dict(ids=0),
               dict(w=0), dict(up=0), dict(down=0), dict(y=0), dict(ids=A + 4), dict(w=A + 2), dict(x=A + 1), dict(up=A + 1),
               dict(gate=A + 1), dict(down=A + 1), dict(y=B + 1), dict(ld=15), dict(ld_y=15)):
        refused(bad, lambda: experts(**kw))
    for kw in (dict(ws=0), dict(ws=A + 16), dict(bytes_=100)):
        refused(dm.ERR_WORKSPACE, lambda: experts(**kw), "workspace")
    assert experts(tokens=0, x=0, y=0) == dm.OK
    n = ctypes.c_size_t()
    assert dm.lib().dmuon_experts_workspace_bytes(0, 1, 1, 1, 1, ctypes.byref(n)) == dm.OK
    refused(bad, lambda: dm.lib().dmuon_experts_workspace_bytes(4, 2, 8, 16, 24, None))
    refused(bad, lambda: dm.lib().dmuon_clip_workspace_bytes(None))


def test_logprobs_refusals_before_a_bind():
    h = ctypes.c_void_p()
    assert dm.lib().dmuon_head_create(4, 10, 8, 0, ctypes.byref(h)) == dm.OK
    L = dm.lib()
    call = lambda tokens=2: L.dmuon_head_logprobs(h, A, 8, A, 8, A, 1.0, 3, tokens, A, A, A, A, A, 0)  # noqa: E731
    refused(dm.ERR_NOT_BOUND, call)
    refused(dm.ERR_INVALID_ARG, lambda: call(5), "tokens")
    refused(dm.ERR_INVALID_ARG, lambda: L.dmuon_head_logprobs(None, A, 8, A, 8, A, 1.0, 3, 2, A, A, A, A, A, 0))
    refused(dm.ERR_INVALID_ARG, lambda: L.dmuon_head_logprobs_backward(h, A, 8, A, 8, A, 1.0, 2, None, A, A, A, A, A, 8, A, 8,
                                                                       0), "logp")
    refused(dm.ERR_NOT_BOUND, lambda: L.dmuon_head_logprobs_backward(h, A, 8, A, 8, A, 1.0, 2, A, A, A, A, A, A, 8, A, 8, 0))
    L.dmuon_head_destroy(h)
