"""Sizes whose products pass 64 bits are refused. No GPU."""

import ctypes

import pytest

from matrix_optimizer_update_gb300 import dmuon as dm


@pytest.mark.parametrize("tokens", [2049, 1 << 31, 1 << 58, 1 << 62, (1 << 63) - 1, -1, -(1 << 63)])
@pytest.mark.parametrize("top", [1, 2, 64])
def test_experts_tokens(tokens, top):
    n = ctypes.c_size_t()
    assert dm.lib().dmuon_experts_workspace_bytes(tokens, top, 8, 64, 64, ctypes.byref(n)) == dm.ERR_INVALID_ARG
    assert dm.lib().dmuon_experts_forward(256, 64, 256, 256, tokens, top, 8, 64, 64, 256, 256, 256, 256, 64, 256, 1 << 30,
                                          None) == dm.ERR_INVALID_ARG
