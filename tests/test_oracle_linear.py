"""Pins of the fp64 oracle of linear attention with one decay per head and of the block norm:
closed forms, exact small numbers and invariants."""

import math

import numpy as np
import pytest

from oracle import block_norm, linear_recurrent


def _case(lens, H=2, H_k=1, d_k=3, d_v=4, seed=0):
    r = np.random.default_rng(seed)
    T = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    return (r.normal(size=(T, H_k, d_k)), r.normal(size=(T, H_k, d_k)), r.normal(size=(T, H, d_v)),
            -np.abs(r.normal(size=(T, H))), cu, r.normal(size=(len(lens), H, d_k, d_v)))


def test_small_numbers_by_hand():
    # d = 1, decay 1/2: S = 10 -> 5 + 2*3 = 11 -> 5.5 + 1*4 = 9.5; read out with q = 1, 2
    q, k, v = np.array([[[1.0]], [[2.0]]]), np.array([[[2.0]], [[1.0]]]), np.array([[[3.0]], [[4.0]]])
    out, fin = linear_recurrent(q, k, v, np.full((2, 1), -math.log(2)), [0, 2], np.full((1, 1, 1, 1), 10.0), scale=3.0)
    assert np.allclose(out.ravel(), [33.0, 57.0], rtol=1e-14) and np.allclose(fin.ravel(), [9.5], rtol=1e-14)


def test_masked_quadratic_form():
    """o_i = scale (e^{G_i} S0^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j), written with products."""
    q, k, v, g, cu, s0 = _case([7])
    out, fin = linear_recurrent(q, k, v, g, cu, s0, scale=0.5)
    G = np.cumsum(g, 0)
    for h in range(2):
        D = np.tril(np.exp(G[:, None, h] - G[None, :, h]))
        want = 0.5 * ((q[:, 0] @ k[:, 0].T * D) @ v[:, h] + np.exp(G[:, h])[:, None] * (q[:, 0] @ s0[0, h]))
        assert np.allclose(out[:, h], want, rtol=1e-12)
        end = np.exp(G[-1, h]) * s0[0, h] + (k[:, 0] * np.exp(G[-1, h] - G[:, h])[:, None]).T @ v[:, h]
        assert np.allclose(fin[0, h], end, rtol=1e-12)


def test_packing_splitting_and_empty_sequences():
    q, k, v, g, cu, s0 = _case([5, 0, 3])
    out, fin = linear_recurrent(q, k, v, g, cu, s0)
    assert np.array_equal(fin[1], s0[1])
    a, fa = linear_recurrent(q[:2], k[:2], v[:2], g[:2], [0, 2], s0[:1])
    b, fb = linear_recurrent(q[2:5], k[2:5], v[2:5], g[2:5], [0, 3], fa)
    assert np.allclose(out[:5], np.concatenate([a, b]), rtol=1e-13) and np.allclose(fin[0], fb[0], rtol=1e-13)


def test_heads_share_queries_and_keys_and_constant_decay():
    q, k, v, g, cu, s0 = _case([4], H=4, H_k=2)
    const = np.array([-0.1, -0.2, 0.0, -math.inf])
    out, fin = linear_recurrent(q, k, v, const, cu, s0)
    for h in range(4):
        o, f = linear_recurrent(q[:, h // 2:h // 2 + 1], k[:, h // 2:h // 2 + 1], v[:, h:h + 1],
                                np.full((4, 1), const[h]), cu, s0[:, h:h + 1])
        assert np.array_equal(out[:, h], o[:, 0]) and np.array_equal(fin[:, h], f[:, 0])
    # decay -inf forgets everything before the token
    assert np.allclose(fin[0, 3], np.outer(k[3, 1], v[3, 3]), rtol=1e-15)


def test_block_norm_by_hand():
    # y = (3, 4): rms^2 = 12.5; gate logits 0 and ln 3 (factors 1/2, 3/4); weight (2, 1); scale 2
    x, h = block_norm(np.array([[1.0, -1.0]]), np.array([[3.0, 4.0]]), gate=np.array([[0.0, math.log(3)]]),
                      post_norm=True, post_weight=np.array([2.0, 1.0]), scale=2.0, eps=0.0)
    r = math.sqrt(12.5)
    assert np.allclose(x, [[1 + 6 / r, -1 + 6 / r]], rtol=1e-14)
    assert np.allclose((h ** 2).mean(), 1.0, rtol=1e-14) and np.allclose(h[0, 0] / h[0, 1], x[0, 0] / x[0, 1])
    x, h = block_norm(np.array([[3.0, 4.0]]), pre_weight=np.array([5.0, 10.0]), eps=0.0)
    assert np.allclose(h, [[15 / r, 40 / r]], rtol=1e-14) and np.array_equal(x, [[3.0, 4.0]])


@pytest.mark.parametrize("rows", [1, 3])
def test_block_norm_row_gate_and_eps(rows):
    r = np.random.default_rng(1)
    x, y, gate, c = r.normal(size=(rows, 5)), r.normal(size=(rows, 5)), r.normal(size=rows), r.normal(size=5)
    a, _ = block_norm(x, y, gate=gate, channel_scale=c, scale=0.5)
    b, _ = block_norm(x, y, gate=np.repeat(gate[:, None], 5, 1), channel_scale=c, scale=0.5)
    assert np.allclose(a, b, rtol=1e-14)
    assert np.allclose(a - x, 0.5 * c * y / (1 + np.exp(-gate))[:, None], rtol=1e-10)
    # a row far below eps: h ~ x' / sqrt(eps)
    _, h = block_norm(1e-9 * x, eps=1e-4)
    assert np.allclose(h, 1e-7 * x, rtol=1e-6)
