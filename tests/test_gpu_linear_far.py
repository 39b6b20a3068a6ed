"""Decays between tokens of one block of 32 on the tensor-core kernel with an fp32 output, where the block
as a whole decays by much: an entry's decay is then the difference of two long sums over the block.

q k = 1 everywhere and v is 1 at one token of a block, so an output is one decay. Sums of up to 32 terms
formed in five levels are off by at most 5 x 2^-24 of their size, plus 2^-24 for the terms' own roundings:
differences of two sums of up to 32 (log2 units) are off by 11 x 32 x 2^-24 x ln 2 < 2^-16, and blocks that
decay by more take a sum of each entry's own, token by token: 32 x 2^-24 of a sum, which at 10 (decays of
2^-10, the smallest looked at here) is 10 x 32 x 2^-24 x ln 2 < 2^-16 as well. The entry's pair of bf16
adds 2^-16, the exponential 2^-22, and 8 x 2^-24 are the scale's and the products' sums."""

import numpy as np
import pytest
import torch

from linear_cases import f64, reference, run

pytestmark = pytest.mark.gpu


def _sums(v):
    """Inclusive sums of 32 fp32 terms in five levels, each rounded."""
    p, o = v.copy(), 1
    while o < 32:
        q = p.copy()
        q[:, o:] = p[:, o:] + p[:, :-o]
        p, o = q, 2 * o
    return p


def _worst_blocks(total, count, seed):
    """Blocks whose log2-decays sum to `total`, and for each a token whose decay to a later one suffers most
    from the difference of the sums: (natural log-decays [count, 32], tokens [count])."""
    r = np.random.default_rng(seed)
    x = r.exponential(size=(20000, 32)) ** 2
    x[:, 20:] *= 0.02  # tokens that lose little behind those that lose much
    g = (-np.log(2) * total * x / x.sum(-1, keepdims=True)).astype(np.float32)
    v = g * np.float32(1.4426950408889634)
    a, exact = _sums(v).astype(np.float64), np.cumsum(v.astype(np.float64), -1)
    off, token = np.zeros(len(x)), np.zeros(len(x), dtype=int)
    for j in range(31):
        d = np.abs((a[:, j + 1:] - a[:, j:j + 1]) - (exact[:, j + 1:] - exact[:, j:j + 1]))
        d = np.where(exact[:, j + 1:] - exact[:, j:j + 1] > -10, d, 0).max(-1)
        token, off = np.where(d > off, j, token), np.maximum(off, d)
    best = np.argsort(off)[-count:]
    return g[best], token[best]


@pytest.mark.parametrize("total", [10, 25, 31, 33, 60, 100, 200, 255, 257, 1000])
def test_uneven_decays_within_a_block(total):
    H, blocks = 32, 16
    T = 32 * blocks
    g, token = _worst_blocks(total, H * blocks, total)
    ld = g.reshape(blocks, H, 32).transpose(0, 2, 1).reshape(T, H)
    v = torch.zeros(blocks, 32, H, 64)
    for n, t in enumerate(token):
        v[n // H, t, n % H] = 1
    q = torch.zeros(T, 1, 64)
    q[..., 0] = 1
    c = dict(q=q.bfloat16(), k=q.bfloat16(), v=v.reshape(T, H, 64).bfloat16(), log_decay=torch.from_numpy(ld.copy()),
             cu_seqlens=torch.tensor([0, T], dtype=torch.int32), init_state=None)
    c = {n: None if t is None else t.cuda() for n, t in c.items()}
    out, _ = run(c, out_dtype=torch.float32, workspace=None)
    o = reference(c)[0]
    seen = o > 2.0 ** -10
    err = float((np.abs(f64(out) - o)[seen] / o[seen]).max())
    assert err <= 2 * 2.0 ** -16 + 2.0 ** -22 + 8 * 2.0 ** -24, err
