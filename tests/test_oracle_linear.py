"""Pins of the linear-attention oracle: closed forms that the recurrence fixes."""

import numpy as np
import pytest

from oracle.linear import linear_attention


def _inputs(B, T, H, Hk, dk, dv, seed=0):
    r = np.random.default_rng(seed)
    return (r.normal(size=(B, T, Hk, dk)), r.normal(size=(B, T, Hk, dk)),
            r.normal(size=(B, T, H, dv)), -r.random((B, T, H)), r.normal(size=(B, H, dk, dv)))


def test_quadratic_form():
    q, k, v, g, h0 = _inputs(2, 7, 4, 2, 3, 5)
    o, hT = linear_attention(q, k, v, g, h0)
    for b in range(2):
        for h in range(4):
            G = np.cumsum(g[b, :, h])
            D = np.tril(np.exp(G[:, None] - G[None, :]))
            P = (q[b, :, h // 2] @ k[b, :, h // 2].T) * D
            ref = P @ v[b, :, h] + np.exp(G)[:, None] * (q[b, :, h // 2] @ h0[b, h])
            np.testing.assert_allclose(o[b, :, h], ref, rtol=1e-12, atol=1e-12)
            end = np.exp(G[-1]) * h0[b, h] + (k[b, :, h // 2] * np.exp(G[-1] - G)[:, None]).T @ v[b, :, h]
            np.testing.assert_allclose(hT[b, h], end, rtol=1e-12, atol=1e-12)


def test_head_gate_is_a_constant_token_gate():
    q, k, v, g, h0 = _inputs(1, 6, 3, 3, 4, 2)
    one = g[0, 0]
    a = linear_attention(q, k, v, one, h0)
    b = linear_attention(q, k, v, np.broadcast_to(one, (1, 6, 3)), h0)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_documents_are_separate_and_empty_ones_keep_their_state():
    q, k, v, g, _ = _inputs(1, 9, 2, 1, 3, 2)
    h0 = np.random.default_rng(1).normal(size=(4, 2, 3, 2))
    cu = [0, 4, 4, 5, 9]
    o, hT = linear_attention(q, k, v, g, h0, cu)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        on, hn = linear_attention(q[:, a:b], k[:, a:b], v[:, a:b], g[:, a:b], h0[n:n + 1])
        assert np.array_equal(o[:, a:b], on) and np.array_equal(hT[n], hn[0])
    assert np.array_equal(hT[1], h0[1])


def test_reset_gate_clears_the_state():
    q, k, v, g, h0 = _inputs(1, 5, 1, 1, 2, 2)
    g[0, 3] = -np.inf
    o, hT = linear_attention(q, k, v, g, h0)
    o2, h2 = linear_attention(q[:, 3:], k[:, 3:], v[:, 3:], g[:, 3:])
    np.testing.assert_allclose(o[:, 3:], o2, rtol=0, atol=0)
    np.testing.assert_allclose(hT, h2, rtol=0, atol=0)


@pytest.mark.parametrize("cu", [[1, 5], [0, 4], [0, 3, 2, 5]])
def test_malformed_offsets(cu):
    q, k, v, g, _ = _inputs(1, 5, 1, 1, 2, 2)
    with pytest.raises(ValueError):
        linear_attention(q, k, v, g, None, cu)
