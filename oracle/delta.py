"""The gated delta rule with one decay per head, and the norm and rotation of queries and keys, in
numpy fp64.

``delta_recurrent`` runs the defining recurrence a token at a time, per sequence and value head
``h`` with query/key head ``h // (H // H_k)``:

    S' = e^{g_t} S_{t-1},   S_t = S' + beta_t k_t (v_t - S'^T k_t)^T,   o_t = scale S_t^T q_t.

``norm_rotate`` is one formula per head row: n = w x / sqrt(mean(x^2) + eps), x / sqrt(sum(x^2) + eps)
or x, then channel pair i turned by positions[axis(i)] * inv_freq[i].
"""

from __future__ import annotations

import numpy as np

from .linear import _f64


def delta_recurrent(q, k, v, log_decay, beta, cu_seqlens, init_state=None, scale: float = 1.0):
    """(out [T, H, d_v], final states [N, H, d_k, d_v]); log_decay [T, H] or [H], beta [T, H]."""
    q, k, v, g, beta, init = _f64(q), _f64(k), _f64(v), _f64(log_decay), _f64(beta), _f64(init_state)
    cu = [int(x) for x in cu_seqlens]
    T, H, d_v = v.shape
    group = np.arange(H) // (H // q.shape[1])
    g = np.broadcast_to(g, (T, H))
    out = np.zeros((T, H, d_v))
    final = np.zeros((len(cu) - 1, H, q.shape[2], d_v)) if init is None else init.copy()
    for n in range(len(cu) - 1):
        S = final[n]
        for t in range(cu[n], cu[n + 1]):
            S = np.exp(g[t])[:, None, None] * S
            kt = k[t, group]
            u = beta[t][:, None] * (v[t] - np.einsum("hk,hkv->hv", kt, S))
            S = S + kt[:, :, None] * u[:, None, :]
            out[t] = scale * np.einsum("hk,hkv->hv", q[t, group], S)
        final[n] = S
    return out, final


def norm_rotate(x, positions, inv_freq, *, norm=None, weight=None, eps=1e-6, interleaved=False, pair_axis=None):
    """x [T, heads, d] normed and turned; positions [T] or [A, T] with pair_axis."""
    x, f, w = _f64(x), _f64(inv_freq), _f64(weight)
    if norm is not None:
        power = (x * x).sum(-1, keepdims=True)
        x = x / np.sqrt((power / x.shape[-1] if norm == "rms" else power) + eps)
    if w is not None:
        x = x * w
    if f is None:
        return x
    half = f.shape[0]
    positions = np.asarray(positions, dtype=np.int64)
    positions = positions.reshape(-1, x.shape[0])
    axis = np.zeros(half, dtype=int) if pair_axis is None else np.asarray(pair_axis)
    angle = _angles(positions[axis].T, f)
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    y = x.copy()
    cos, sin = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _angles(pos, f):
    """pos [T, half] * f [half] modulo 2 pi in integers of 2^-300, for positions whose product with f a
    double does not resolve. pi by Machin's formula, 16 atan(1/5) - 4 atan(1/239)."""
    bits = 300

    def atan_inverse(n):
        total, term, k, sign = 0, (1 << bits) // n, 1, 1
        while term:
            total += sign * (term // k)
            term //= n * n
            k, sign = k + 2, -sign
        return total

    two_pi = 2 * (16 * atan_inverse(5) - 4 * atan_inverse(239))
    out = np.zeros(pos.shape)
    for i, x in enumerate(f):
        if not np.isfinite(x):
            out[:, i] = np.nan
            continue
        num, den = float(x).as_integer_ratio()
        for t in range(pos.shape[0]):
            scaled = (int(pos[t, i]) * num << bits) // den  # the angle in units of 2^-bits
            out[t, i] = float(scaled % two_pi) / 2.0 ** bits
    return out
