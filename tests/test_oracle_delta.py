"""Pins of the fp64 oracle of the gated delta rule with one decay per head and of the norm and rotation
of queries and keys: closed forms, exact small numbers, the other oracles and invariants."""

import math

import numpy as np
import pytest

from oracle import delta_recurrent, kda_recurrent, linear_recurrent, norm_rotate


def _case(lens, H=2, H_k=1, d_k=3, d_v=4, seed=0):
    r = np.random.default_rng(seed)
    T = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    return (unit(r.normal(size=(T, H_k, d_k))), unit(r.normal(size=(T, H_k, d_k))), r.normal(size=(T, H, d_v)),
            -np.abs(r.normal(size=(T, H))), r.uniform(size=(T, H)), cu, r.normal(size=(len(lens), H, d_k, d_v)))


def test_small_numbers_by_hand():
    # d = 1, decay 1/2, beta 1/2: S = 10 -> 5, u = (3 - 10) / 2, S = 5 + 2 (-3.5) = -2; -> -1,
    # u = (4 + 1) / 2, S = -1 + 2.5 = 1.5; read out with q = 1, 2
    q, k, v = np.array([[[1.0]], [[2.0]]]), np.array([[[2.0]], [[1.0]]]), np.array([[[3.0]], [[4.0]]])
    out, fin = delta_recurrent(q, k, v, np.full((2, 1), -math.log(2)), np.full((2, 1), 0.5), [0, 2],
                               np.full((1, 1, 1, 1), 10.0), scale=3.0)
    assert np.allclose(out.ravel(), [-6.0, 9.0], rtol=1e-14) and np.allclose(fin.ravel(), [1.5], rtol=1e-14)


def test_equals_the_channel_wise_rule_with_equal_channels():
    q, k, v, g, beta, cu, s0 = _case([7, 0, 12], H=3, H_k=3)
    g = np.maximum(g, -4.9)  # above that rule's bound
    out, fin = delta_recurrent(q, k, v, g, beta, cu, s0, scale=0.5)
    wide = np.broadcast_to(g[..., None], k.shape).copy()
    o, f = kda_recurrent(q, k, v, wide, beta, cu, init_state=s0, scale=0.5)
    assert np.allclose(out, o, rtol=1e-12, atol=1e-14) and np.allclose(fin, f, rtol=1e-12, atol=1e-14)


def test_orthogonal_keys_are_linear_attention_and_a_key_overwrites():
    _, _, v, g, _, _, _ = _case([3], H=1, d_k=3)
    eye = np.eye(3)[:, None, :]
    out, fin = delta_recurrent(eye, eye, v, g, np.ones((3, 1)), [0, 3])
    o, f = linear_recurrent(eye, eye, v, g, [0, 3])
    assert np.allclose(out, o, rtol=1e-13, atol=1e-15) and np.allclose(fin, f, rtol=1e-13, atol=1e-15)
    same = np.broadcast_to(eye[:1], (3, 1, 3))  # beta = 1, one key: the last value stands
    out, fin = delta_recurrent(same, same, v, g, np.ones((3, 1)), [0, 3])
    assert np.allclose(out, v, rtol=1e-13) and np.allclose(fin[0, 0, 0], v[2, 0], rtol=1e-13)


def test_packing_splitting_and_empty_sequences():
    q, k, v, g, beta, cu, s0 = _case([5, 0, 3])
    out, fin = delta_recurrent(q, k, v, g, beta, cu, s0)
    assert np.array_equal(fin[1], s0[1])
    a, fa = delta_recurrent(q[:2], k[:2], v[:2], g[:2], beta[:2], [0, 2], s0[:1])
    b, fb = delta_recurrent(q[2:5], k[2:5], v[2:5], g[2:5], beta[2:5], [0, 3], fa)
    assert np.allclose(out[:5], np.concatenate([a, b]), rtol=1e-13) and np.allclose(fin[0], fb[0], rtol=1e-13)


def test_heads_share_queries_and_keys_and_constant_decay():
    q, k, v, _, beta, cu, s0 = _case([4], H=4, H_k=2)
    const = np.array([-0.1, -0.2, 0.0, -math.inf])
    out, fin = delta_recurrent(q, k, v, const, beta, cu, s0)
    for h in range(4):
        o, f = delta_recurrent(q[:, h // 2:h // 2 + 1], k[:, h // 2:h // 2 + 1], v[:, h:h + 1],
                               np.full((4, 1), const[h]), beta[:, h:h + 1], cu, s0[:, h:h + 1])
        assert np.allclose(out[:, h], o[:, 0], rtol=1e-13) and np.allclose(fin[:, h], f[:, 0], rtol=1e-13)
    assert np.allclose(fin[0, 3], beta[3, 3] * np.outer(k[3, 1], v[3, 3]), rtol=1e-13)


@pytest.mark.parametrize("C", [1, 4, 16])
def test_chunked_form(C):
    """(I + A) U = diag(beta) (V - diag(e^G) K S0), O = diag(e^G) Q S0 + P U, S = e^{G_C} S0 + (e^{G_C - G} K)^T U."""
    q, k, v, g, beta, cu, s0 = _case([16], H=1, d_k=5)
    out, fin = delta_recurrent(q, k, v, g, beta, cu, s0)
    S, got = s0[0, 0], []
    for t in range(0, 16, C):
        Q, K, V, b, G = q[t:t + C, 0], k[t:t + C, 0], v[t:t + C, 0], beta[t:t + C], np.cumsum(g[t:t + C, 0])
        D = np.exp(G[:, None] - G)
        A = np.tril(b * (K @ K.T) * D, -1)
        U = np.linalg.solve(np.eye(C) + A, b * (V - np.exp(G)[:, None] * (K @ S)))
        got.append(np.exp(G)[:, None] * (Q @ S) + np.tril(Q @ K.T * D) @ U)
        S = np.exp(G[-1]) * S + (np.exp(G[-1] - G)[:, None] * K).T @ U
    assert np.allclose(np.concatenate(got), out[:, 0], rtol=1e-11, atol=1e-13) and np.allclose(S, fin[0, 0], rtol=1e-11)


def test_rotation_by_hand():
    # a quarter turn: (1, 2) -> (-2, 1); halves pair channels 0, 2 and 1, 3, neighbours 0, 1 and 2, 3
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    f = np.array([math.pi / 2, math.pi], dtype=np.float64)
    assert np.allclose(norm_rotate(x, [1], f), [[[-3, -2, 1, -4, 5]]], atol=1e-14)
    assert np.allclose(norm_rotate(x, [1], f, interleaved=True), [[[-2, 1, -3, -4, 5]]], atol=1e-14)
    assert np.allclose(norm_rotate(x, [[1], [2]], f, pair_axis=[0, 1]), [[[-3, 2, 1, 4, 5]]], atol=1e-14)
    y = norm_rotate(x, None, None, norm="l2", eps=0.0)
    assert np.allclose(y, x / math.sqrt(55), rtol=1e-15)
    y = norm_rotate(x, None, None, norm="rms", weight=np.arange(5.0), eps=4.0)
    assert np.allclose(y, x * np.arange(5) / math.sqrt(15), rtol=1e-15)


def test_rotation_keeps_norms_relative_positions_and_far_angles():
    r = np.random.default_rng(1)
    q, k, f = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8)), np.float32(10.0) ** -np.arange(4)
    dot = lambda m, n: float((norm_rotate(q, [m], f) * norm_rotate(k, [n], f)).sum())  # noqa: E731
    assert math.isclose(dot(5, 3), dot(1002, 1000), rel_tol=1e-10) and not math.isclose(dot(5, 3), dot(3, 5), rel_tol=1e-3)
    assert math.isclose(dot(5, 3), dot((1 << 62) + 2, 1 << 62), rel_tol=1e-10)
    assert math.isclose(dot(5, 3), dot(-1, -3), rel_tol=1e-10)
    assert np.allclose((norm_rotate(q, [77], f) ** 2).sum(), (q ** 2).sum(), rtol=1e-14)
    # angles that a double holds
    assert np.allclose(norm_rotate(q, [12345], f)[0, 0, :4], q[0, 0, :4] * np.cos(12345 * f.astype(float))
                       - q[0, 0, 4:] * np.sin(12345 * f.astype(float)), atol=1e-11)
