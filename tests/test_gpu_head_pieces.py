"""GPU parity of the head's losses on few tokens where the vocabulary takes several pieces."""

import numpy as np
import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm
from oracle import head_ref as ref
from test_gpu_head import bounds, check_distill, check_grads, f64, inputs, teacher

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [1000, 1283])
@pytest.mark.parametrize("tokens", [1, 40, 64, 65, 128])
def test_few_tokens_over_several_pieces(tokens, vocab):
    # room for 2^20 tokens leaves pieces of 256 entries: 4 or 6 of them, the last ragged. dH's sums are added to, and
    # the two parts of dz are written anew for each piece.
    h, w, y, g = inputs(tokens, vocab, 72, tokens, pitch=8)
    if tokens > 2:
        y[1] = -100
    head = dm.Head.create(1 << 20, vocab, 72, max_top=9)
    loss, lse = head.xent(h, w, y)
    dh, dw = head.xent_backward(h, w, y, lse, g)
    hn, wn, gn = f64(h), f64(w), f64(g)
    r = ref.xent(hn, wn, y.cpu().numpy(), gn)
    check_grads(dh, dw, r, hn, wn, gn, bounds(hn, wn, r)[1])
    # dW alone is the same
    only = head.xent_backward(h, w, y, lse, g, dhidden=False)[1]
    assert torch.equal(only, dw)
    # as one piece has it: losses bit for bit, gradients up to the order of dH's sums over the pieces
    whole = dm.Head.create(tokens, vocab, 72, max_top=9)
    assert all(torch.equal(a, b) for a, b in zip((loss, lse), whole.xent(h, w, y)))
    assert torch.equal(dw, whole.xent_backward(h, w, y, lse, g)[1])
    ids, lg = teacher(tokens, vocab, 9, tokens + 1)
    check_distill(h, w, ids, lg, 1.5, g, head)
    assert np.isfinite(f64(dh)).all()
    assert head.read_device_status(torch.cuda.current_stream().cuda_stream) == 0
