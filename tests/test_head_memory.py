"""What a head's workspace holds: room for a scoring call's logits is a size of its own, beside what the losses need. No
GPU."""

import ctypes

import pytest

from matrix_optimizer_update_gb300 import dmuon as dm

MB = 1 << 20
SIZES = [(1, 32000, 2048), (64, 128000, 4096), (65, 50257, 1024), (128, 128000, 4096), (128, 1 << 22, 64),
         (512, 32000, 2048), (2048, 32000, 2048), (4096, 32000, 2048), (1024, 128000, 4096), (4096, 128000, 4096),
         (8192, 128000, 512), (1 << 18, 32000, 64), (1 << 19, 70000, 8), (1 << 20, 50000, 64), (77, 33, 8), (5000, 17, 16)]


def workspace(tokens, vocab, dim):
    """(least bytes, bytes with room for logits)"""
    head, n, m = ctypes.c_void_p(), ctypes.c_size_t(), ctypes.c_size_t()
    assert dm.lib().dmuon_head_create(tokens, vocab, dim, 0, ctypes.byref(head)) == 0
    assert dm.lib().dmuon_head_workspace_bytes(head, ctypes.byref(n)) == 0
    assert dm.lib().dmuon_head_scores_workspace_bytes(head, ctypes.byref(m)) == 0
    dm.lib().dmuon_head_destroy(head)
    return n.value, m.value


@pytest.mark.parametrize("tokens,vocab,dim", SIZES)
def test_the_losses_pay_for_their_gradients_alone(tokens, vocab, dim):
    padded = -(-vocab // 256) * 256
    piece = min(padded, max(256, (1 << 28) // tokens // 256 * 256))
    few = min(tokens, 128)
    # dz (held twice for few tokens), or one block of 256 entries' logits where the vocabulary is hardly longer
    dz = max(2 * max(tokens, min(2 * tokens, 128)) * piece, min(1024 * tokens, 512 * MB))
    logits = 4 * few
    pieces = -(-vocab // (dz // logits // 256 * 256))
    groups = max(-(-vocab // 128) * tokens, (-(-vocab // 32) + 1024 * pieces) * few)
    row = 4 * (dim + 64) * tokens
    sums = max(row, min(256 * row, 64 * MB), 4 * groups + 320 * tokens + 1024)
    least, most = workspace(tokens, vocab, dim)
    assert least <= 8 * groups + 4 * tokens + dz + sums + 16 * 1024
    # with the logits in place of dz
    whole = max(dz, min(4 * tokens * padded, 512 * MB), 1024 * tokens)
    assert most == max(least, least - dz + whole) or most - (least - dz + whole) in range(-1024, 1025)


@pytest.mark.parametrize("tokens,vocab", [(512, 32000), (2048, 32000), (4096, 32000), (1024, 128000)])
def test_room_for_logits_is_what_makes_the_difference(tokens, vocab):
    least, most = workspace(tokens, vocab, 2048)
    assert most - least == 2 * tokens * vocab


def test_refusals():
    n = ctypes.c_size_t()
    assert dm.lib().dmuon_head_scores_workspace_bytes(None, ctypes.byref(n)) == dm.ERR_INVALID_ARG
