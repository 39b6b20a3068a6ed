"""Inputs, bounds and calls shared by the linear-attention tests."""

from __future__ import annotations

import numpy as np
import torch

from kimi_delta_attention_02_gb300 import binding
from oracle import linear_recurrent


def make(lens, H=2, H_k=None, d_k=128, d_v=128, dtype=torch.bfloat16, per_token=True, decay=0.1, init=True, seed=0,
         device="cuda"):
    """Packed inputs on ``device``: unit-norm q, k, normal v, g = -decay softplus(normal)."""
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    H_k = H if H_k is None else H_k
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    ld = -decay * torch.nn.functional.softplus(rn(T, H) if per_token else rn(H))
    c = dict(q=unit(rn(T, H_k, d_k)).to(dtype), k=unit(rn(T, H_k, d_k)).to(dtype), v=rn(T, H, d_v).to(dtype),
             log_decay=ld, cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32),
             init_state=0.5 * rn(N, H, d_k, d_v) if init else None)
    return {n: None if t is None else t.to(device) for n, t in c.items()}


def cpu(c):
    return {n: None if t is None else t.cpu() for n, t in c.items()}


def reference(c, scale=1.0):
    """(out, final) of the oracle and their magnitudes: the same sums over absolute values, which
    every rounding error below is a multiple of."""
    c = cpu(c)
    out, fin = linear_recurrent(**c, scale=scale)
    m = {n: (t if n in ("log_decay", "cu_seqlens") or t is None else t.abs()) for n, t in c.items()}
    mo, mf = linear_recurrent(**m, scale=abs(scale))
    return out, fin, mo, mf


def f64(t):
    return t.detach().double().cpu().numpy()


def fp32_factor(longest, d_k):
    """Error of the fp32 recurrence relative to the magnitude: per token of a term's life one
    rounding of the decay's product and one of the write's sum, and e^g - 1 off by an ulp or two
    (4 x 2^-24 together); d_k products summed for a read-out; a few more for inputs and scale."""
    return (4 * longest + d_k + 32) * 2.0 ** -24


def check(got, want, magnitude, factor, what):
    d = np.abs(f64(got) - want)
    bad = d > factor * magnitude + 1e-37
    assert not bad.any() and not np.isnan(f64(got)).any(), (what, int(bad.sum()), float((d / (magnitude + 1e-30)).max()),
                                                            factor)


def run(c, **kw):
    out, fin = binding.linear_prefill(**c, **kw)
    binding.check_device_error()
    return out, fin
