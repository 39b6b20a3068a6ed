"""Inputs, bounds and calls shared by the tests of the gated delta rule.

Bounds. With unit keys (off by a bf16 rounding at most) and 0 <= beta <= 1 a token's transition
(I - beta k k^T) e^g shrinks every column, so an error made at one token is carried on by e^g at most,
in the column's 2-norm. ``bounds`` follows three numbers per column and token:

    n_t = e^{g_t} n_{t-1} + 1.01 beta_t |k_t| |v_t|         (above the column's norm)
    E_t = e^{g_t} E_{t-1} + (what the step's own roundings come to)

where 1.01 covers keys that bf16 rounding left a little longer than one. fp32, per token: the decay
and its factor (3 roundings of n), the sum S^T k (d_k + 8 roundings of |k| n), u and k u (4 of
|u| <= beta (|v| + |k| n)), the sum's rounding (2 of n): (d_k + 20) 2^-24 (n + beta |v|), doubled for
what four tokens at a time share (the products k.k, their decays).

The tensor cores work in chunks of 64 tokens on operands that are pairs of bf16, off by at most
p = 2^-16 of themselves (the pair's own rounding and the product of two low parts that is left out).
Of a chunk's u: the state's pair, |K| |S|; the residual's and the inverse's pairs, each |T'| |r| entry
by entry with |r| <= |v| + |k| n; u's own pair. fp32 accumulation adds (128 + 64) 2^-24 of the same
sums, less than p. |T'_ti| <= beta_t |k_t| beta_i |k_i| for unit keys, so a chunk makes at most

    p n + 3 p sum_i |k_i| beta_i R_i (1 + sum over the chunk of beta)

with R_i = |v_i| + n: that is how ``bounds`` adds it, at each chunk's end. An output reads a column with
|q|; its own sums over the chunk have the same terms."""

from __future__ import annotations

import numpy as np
import torch

from kimi_delta_attention_02_gb300 import binding
from oracle import delta_recurrent


def make(lens, H=2, H_k=None, d_k=128, d_v=128, dtype=torch.bfloat16, per_token=True, decay=0.1, init=True, seed=0,
         device="cuda", alike=0.0):
    """Packed inputs on ``device``: unit-norm q, k, normal v, g = -decay softplus(normal), beta in (0, 1).
    ``alike``: how much of a common direction the keys share."""
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    H_k = H if H_k is None else H_k
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    ld = -decay * torch.nn.functional.softplus(rn(T, H) if per_token else rn(H))
    c = dict(q=unit(rn(T, H_k, d_k) + alike).to(dtype), k=unit(rn(T, H_k, d_k) + alike).to(dtype), v=rn(T, H, d_v).to(dtype),
             log_decay=ld, beta=torch.sigmoid(rn(T, H)),
             cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32),
             init_state=0.5 * rn(N, H, d_k, d_v) if init else None)
    return {n: None if t is None else t.to(device) for n, t in c.items()}


def cpu(c):
    return {n: None if t is None else t.cpu() for n, t in c.items()}


def f64(t):
    return t.detach().double().cpu().numpy()


P = 2.0 ** -16  # a pair of bf16


def bounds(c, scale=1.0, pairs=False, read=0.0, chunk=64, n0=None, E0=None):
    """(bound of out [T, H, d_v], bound of a final column [N, H, 1, d_v], the column norms at the end):
    fp32 token by token, or with ``pairs`` the tensor cores' chunks. ``read``: what rounds the
    read-out's operands (2^-8 where they are single bf16)."""
    c = cpu(c)
    k, q, v, beta = (f64(c[n]) for n in ("k", "q", "v", "beta"))
    T, H, d_v = v.shape
    d_k = k.shape[2]
    group = np.arange(H) // (H // k.shape[1])
    nk, nq = np.linalg.norm(k, axis=-1)[:, group], np.linalg.norm(q, axis=-1)[:, group]
    g = np.exp(np.broadcast_to(f64(c["log_decay"]), (T, H)))
    cu = [int(x) for x in c["cu_seqlens"]]
    N = len(cu) - 1
    n = np.zeros((N, H, d_v)) if c["init_state"] is None else np.linalg.norm(f64(c["init_state"]), axis=2)
    n = n if n0 is None else n0.copy()
    E = np.zeros((N, H, d_v)) if E0 is None else E0.copy()
    out = np.zeros((T, H, d_v))
    unit = (d_k + 20) * 2.0 ** -23
    for s in range(N):
        for t in range(cu[s], cu[s + 1]):
            a, b, kt = g[t][:, None], beta[t][:, None], nk[t][:, None]
            if pairs and (t - cu[s]) % chunk == 0:
                bsum, terms, start = np.zeros((H, 1)), np.zeros((H, d_v)), n[s].copy()
            w = b * kt * (np.abs(v[t]) + kt * n[s])
            n[s] = a * n[s] + 1.01 * b * kt * np.abs(v[t])
            if pairs:
                bsum, terms = bsum + b, terms + w
                own = P * start + 3 * P * terms * (1 + bsum) * 1.01
                e_here = E[s] + own
                if t + 1 == cu[s + 1] or (t + 1 - cu[s]) % chunk == 0:
                    total = np.exp(np.log(np.maximum(g[cu[s] + (t - cu[s]) // chunk * chunk:t + 1], 1e-300)).sum(0))[:, None]
                    E[s] = total * E[s] + own + 2.0 ** -22 * n[s]
            else:
                E[s] = a * E[s] + unit * (n[s] + w)
                e_here = E[s]
            level = (start + terms * 1.01) if pairs else n[s]
            out[t] = abs(scale) * nq[t][:, None] * (e_here + (unit + (2 * P if pairs else 0) + read) * level)
    return out, E[:, :, None, :], n


def reference(c, scale=1.0):
    return delta_recurrent(**cpu(c), scale=scale)


def check(got, want, bound, what):
    d = np.abs(f64(got) - want)
    bad = ~(d <= bound + 1e-37)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(d / (bound + 1e-30))), bool(np.isnan(f64(got)).any()))


def half_step(want, dtype):
    """What rounding the result to dtype may add: half a step."""
    return np.abs(want) * (torch.finfo(dtype).eps / 2)


def run(c, **kw):
    out, fin = binding.delta_prefill(**c, **kw)
    binding.check_device_error()
    return out, fin
