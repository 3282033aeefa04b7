"""A mixture's experts in 64 bits, one assignment at a time, and what rounding may do to them."""

import numpy as np


def silu(v):
    return v / (1.0 + np.exp(-v))


def forward(x, ids, weights, up, down, gate=None):
    """y [tokens, dim], and the bound of its error: sums of K terms in fp32, in any order and truncated, are off by
    at most (K + 16) * 2^-23 of the terms' absolute sum; silu's slope is at most 1.1; exp and the division add 2^-20
    of h, and h as the sum of two 8-bit significands 2^-16; y is rounded to bf16 once (half a step: 2^-8)."""
    tokens, top = ids.shape
    experts, inner, dim = up.shape
    y, off = np.zeros((tokens, dim)), np.zeros((tokens, dim))
    size = np.zeros((tokens, dim))
    for t in range(tokens):
        for k in range(top):
            e = int(ids[t, k])
            if not 0 <= e < experts:
                continue
            w = float(weights[t, k])
            u = up[e] @ x[t]
            u_off = (dim + 16) * 2.0 ** -23 * (np.abs(up[e]) @ np.abs(x[t]))
            if gate is None:
                h = silu(u)
                h_off = 1.1 * u_off
            else:
                g = gate[e] @ x[t]
                g_off = (dim + 16) * 2.0 ** -23 * (np.abs(gate[e]) @ np.abs(x[t]))
                h = silu(g) * u
                h_off = 1.1 * g_off * (np.abs(u) + u_off) + np.abs(silu(g)) * u_off
            h_off = h_off + (2.0 ** -16 + 2.0 ** -20) * np.abs(h)
            y[t] += w * (down[e] @ h)
            terms = np.abs(down[e]) @ np.abs(h)
            off[t] += abs(w) * (np.abs(down[e]) @ h_off + (inner + 16) * 2.0 ** -23 * terms)
            size[t] += abs(w) * terms
    off += (top + 2) * 2.0 ** -23 * size
    return y, off + 2.0 ** -8 * (np.abs(y) + off) + 1e-37
