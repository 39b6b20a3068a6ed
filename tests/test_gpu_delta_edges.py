"""The gated delta rule where two of its ways meet: padded head sizes with several cut sequences or with the
longest-first list, growth across cuts, beta above one, cut fp32 sequences of many segments."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from delta_cases import bounds, check, f64, make, reference, run
from delta_precision import check_pairs, off

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("d_k,d_v", [(100, 72), (65, 127), (128, 61), (33, 128)])
def test_padded_and_several_cut(d_k, d_v, out_dtype):
    lens = [1500, 0, 1, 3000, 511, 1536]
    c = make(lens, H=2, d_k=d_k, d_v=d_v, decay=0.01, seed=d_k)
    up = lambda d: (d + 7) // 8 * 8  # noqa: E731
    copies = sum(lens) * 2 * 2 * ((2 * up(d_k) if d_k % 8 else 0) + (up(d_v) if d_v % 8 else 0))
    n = binding.delta_workspace_size(sum(lens), len(lens), 2, d_k, d_v, B16, out_dtype)
    assert n > copies + 2 * 4 * up(d_k) * up(d_v)  # copies and segments
    ref = reference(c)
    ws = torch.full((n // 4,), float("nan"), device="cuda").view(torch.uint8)
    out, fin = run(c, out_dtype=out_dtype, workspace=ws)
    check_pairs(c, out, fin, ref)


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("d_k,d_v", [(68, 36), (64, 33), (100, 128)])
def test_padded_and_longest_first(d_k, d_v, out_dtype):
    lens = [30 + 17 * i % 190 for i in range(40)] + [0, 900, 1]
    c = make(lens, H=32, H_k=4, d_k=d_k, d_v=d_v, seed=12)
    n = binding.delta_workspace_size(sum(lens), len(lens), 32, d_k, d_v, B16, out_dtype, H_k=4)
    assert n % 256 == 0 and n > 256
    ref = reference(c)
    out, fin = run(c, out_dtype=out_dtype)
    check_pairs(c, out, fin, ref)
    ws = torch.empty(n - 256, dtype=torch.uint8, device="cuda")  # the copies without the list
    o, f = run(c, out_dtype=out_dtype, workspace=ws)
    assert torch.equal(out, o) and torch.equal(fin, f)


@pytest.mark.parametrize("dtype,out_dtype,H,T", [(B16, B16, 2, 3000), (B16, F32, 2, 3000), (F32, F32, 1, 3000)])
def test_growth_across_cuts(dtype, out_dtype, H, T):
    """60 tokens that grow by 0.3, 40 that decay by 0.45, over and over: no run of tokens sums above 18, and
    segments begin and end anywhere in it. With G_t the sums from the start, e^{-G_t} S_t follows the recurrence
    without a decay, so both sides are compared times e^{-G_t}."""
    c = make([T], H=H, d_k=128, d_v=64, dtype=dtype, seed=5)
    t = torch.arange(T, device="cuda") % 100
    c["log_decay"] = torch.where(t < 60, 0.3, -0.45).float()[:, None].expand(T, H).contiguous()
    n = binding.delta_workspace_size(T, 1, H, 128, 64, dtype, out_dtype)
    assert n >= 3 * H * 128 * (128 + 64) * 4
    out, fin = run(c, out_dtype=out_dtype)
    o, f = reference(c)
    G = np.cumsum(f64(c["log_decay"]), 0)
    shrunk = np.exp(-G)[:, :, None]
    err = np.linalg.norm((f64(out) - o) * shrunk) / np.linalg.norm(o * shrunk)
    end = np.linalg.norm(f64(fin) - f) / np.linalg.norm(f)
    if dtype == F32:
        # as without growth 1e-6 (a state remembers some 256 tokens by its keys alone), and each decay of a block,
        # up to 1.8 in the exponent, off by 2^-24 of it: 1e-6 more over 64 blocks one way
        assert err < 2e-6 and end < 2e-6, (err, end)
        return
    # pairs as elsewhere, and decays off by up to 26 2^-24 in the exponent of two, 1e-6 each way for three factors
    if out_dtype == B16:
        rounded = torch.from_numpy(o).to(B16).double().numpy()
        own = np.linalg.norm((rounded - o) * shrunk) / np.linalg.norm(o * shrunk)
        assert err < own + 6e-5, (err, own)
    else:
        assert err < 3e-5, err
    assert end < 3e-5, end


@pytest.mark.parametrize("dtype,out_dtype", [(B16, B16), (B16, F32), (F32, F32)])
@pytest.mark.parametrize("lens", [[400], [70, 0, 1, 200, 64], [3000]])
def test_beta_above_one(lens, dtype, out_dtype):
    """1 < beta < 2, transitions with a negative eigenvalue: |1 - beta |k|^2| stays below one (bf16 keys are off
    by 2^-9 in length), so the bounds hold, with terms up to twice as large."""
    c = make(lens, H=2, d_k=128, d_v=72, dtype=dtype, decay=0.01, seed=6)
    c["beta"] = 1 + 0.98 * c["beta"]
    ref = reference(c)
    out, fin = run(c, out_dtype=out_dtype)
    if dtype == B16 and sum(lens) / len(lens) > 44:
        check_pairs(c, out, fin, ref, tolerance=4e-5)
    else:
        bo, bf, _ = bounds(c)
        assert off(out, ref[0]) < 2e-6 and off(fin, ref[1]) < 2e-6, (off(out, ref[0]), off(fin, ref[1]))
        if lens != [3000]:
            check(out, ref[0], bo, "out")
            check(fin, ref[1], bf, "final")


@pytest.mark.parametrize("T,d_k,d_v,H", [(16384, 128, 128, 1), (9000, 128, 64, 2), (8000, 64, 64, 3), (5000, 40, 128, 2), (3333, 16, 16, 4)])
def test_cut_on_the_token_kernel_is_as_exact(T, d_k, d_v, H):
    """fp32 in one long sequence: a joined state is M S + B, whose M and B are as exact as a sequence's own states
    and whose sum over the key rows is one fp32 sum more, so the error is that of the uncut sequence, below 1e-6 in
    the 2-norm, for each of the two."""
    c = make([T], H=H, d_k=d_k, d_v=d_v, dtype=F32, decay=0.003, seed=T)
    assert binding.delta_workspace_size(T, 1, H, d_k, d_v, F32, F32) > 0
    o, f = reference(c)
    for kw in ({}, {"recurrent": True}):
        out, fin = run(c, **kw)
        assert off(out, o) < 1e-6 and off(fin, f) < 1e-6, (kw, off(out, o), off(fin, f))
