"""Linear attention with one decay per head, and the block norm, in numpy fp64.

``linear_recurrent`` runs the defining recurrence a token at a time, per sequence and value head
``h`` with query/key head ``h // (H // H_k)``:

    S_t = e^{g_t} S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t.

``block_norm`` is one row-wise formula: n = w_post y / sqrt(mean(y^2) + eps) (or y),
x' = x + scale c Sigmoid(r) n, h = w_pre x' / sqrt(mean(x'^2) + eps).
"""

from __future__ import annotations

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x.double().numpy() if hasattr(x, "double") else x, dtype=np.float64)


def linear_recurrent(q, k, v, log_decay, cu_seqlens, init_state=None, scale: float = 1.0):
    """(out [T, H, d_v], final states [N, H, d_k, d_v]); log_decay [T, H] or [H]."""
    q, k, v, g, init = _f64(q), _f64(k), _f64(v), _f64(log_decay), _f64(init_state)
    cu = [int(x) for x in cu_seqlens]
    T, H, d_v = v.shape
    group = np.arange(H) // (H // q.shape[1])
    g = np.broadcast_to(g, (T, H))
    out = np.zeros((T, H, d_v))
    final = np.zeros((len(cu) - 1, H, q.shape[2], d_v)) if init is None else init.copy()
    for n in range(len(cu) - 1):
        S = final[n]
        for t in range(cu[n], cu[n + 1]):
            S = np.exp(g[t])[:, None, None] * S + k[t, group][:, :, None] * v[t][:, None, :]
            out[t] = scale * np.einsum("hk,hkv->hv", q[t, group], S)
        final[n] = S
    return out, final


def block_norm(x, y=None, *, gate=None, post_norm=False, post_weight=None, scale=1.0, channel_scale=None,
               pre_weight=None, eps=1e-6, post_eps=None):
    """(x', h) of the block norm, fp64."""
    x, y, gate = _f64(x), _f64(y), _f64(gate)
    one = lambda w: 1.0 if w is None else _f64(w)  # noqa: E731
    if y is not None:
        if post_norm:
            y = one(post_weight) * y / np.sqrt(np.mean(y * y, -1, keepdims=True) + (eps if post_eps is None else post_eps))
        if gate is not None:
            y = y / (1.0 + np.exp(-(gate if gate.ndim == 2 else gate[:, None])))
        x = x + scale * one(channel_scale) * y
    return x, one(pre_weight) * x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
