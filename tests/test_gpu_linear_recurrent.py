"""kda_linear_prefill on the token-recurrent kernel, and its segments and scan, against the fp64
oracle. Bounds: see linear_cases.fp32_factor; a bf16 output adds half a step, 2^-8 of the value."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from linear_cases import check, f64, fp32_factor, make, reference, run

pytestmark = pytest.mark.gpu


def _check(c, lens, scale=1.0, out_dtype=torch.float32, **kw):
    out, fin = run(c, scale=scale, recurrent=True, out_dtype=out_dtype, **kw)
    o, f, mo, mf = reference(c, scale)
    fac = fp32_factor(max(lens), c["q"].shape[2])
    half = 2.0 ** -8 if out_dtype == torch.bfloat16 else 0.0
    check(out, o, mo * fac + half * np.abs(o), 1.0, "out")
    if fin is not None:
        check(fin, f, mf, fac, "final")
    return out, fin


@pytest.mark.parametrize("d_k,d_v", [(128, 128), (64, 64), (1, 1), (100, 72), (5, 128), (128, 3), (65, 65), (17, 33)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_head_sizes(d_k, d_v, dtype):
    lens = [37, 0, 1, 16, 70]
    _check(make(lens, H=3, d_k=d_k, d_v=d_v, dtype=dtype, seed=d_k), lens, scale=0.3)


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [64], [65], [200], [0, 0, 3], [3, 0], [0]])
@pytest.mark.parametrize("per_token", [True, False])
def test_lengths(lens, per_token):
    _check(make(lens, H=2, d_k=40, d_v=24, dtype=torch.float32, per_token=per_token, seed=sum(lens)), lens)


@pytest.mark.parametrize("H,H_k", [(6, 1), (6, 2), (6, 6), (1, 1)])
def test_shared_heads_and_output_types(H, H_k):
    lens = [33, 90]
    for dtype in (torch.float32, torch.bfloat16):
        for out_dtype in (torch.float32, torch.bfloat16):
            _check(make(lens, H=H, H_k=H_k, d_k=32, d_v=48, dtype=dtype, seed=H), lens, out_dtype=out_dtype)


@pytest.mark.parametrize("lens", [[1000], [500, 0, 1, 700, 63, 64, 65]])
@pytest.mark.parametrize("decay", [0.0, 1e-3, 5.0])
def test_segments_join(lens, decay):
    """Long sequences are cut (the workspace is not empty); without one they run end to end."""
    c = make(lens, H=2, d_k=128, d_v=72, dtype=torch.float32, decay=decay, seed=9)
    assert binding.linear_workspace_size(sum(lens), len(lens), 2, 128, 72, torch.float32) > 0
    _check(c, lens)
    _check(c, lens, workspace=None)


def test_final_state_over_the_initial_one_and_none():
    lens = [130, 5]
    c = make(lens, d_k=64, d_v=64, dtype=torch.float32)
    o, f, mo, mf = reference(c)
    state = c["init_state"]
    out, fin = run(c, recurrent=True, final_state=state)
    assert fin is state
    check(fin, f, mf, fp32_factor(130, 64), "in place")
    out, fin = run(make(lens, d_k=64, d_v=64, dtype=torch.float32), recurrent=True, want_final=False)
    assert fin is None
    check(out, o, mo, fp32_factor(130, 64), "out")
    _check(make(lens, d_k=64, d_v=64, dtype=torch.float32, init=False), lens)


def test_infinite_decay_forgets_and_nan_propagates():
    lens = [40, 40]
    c = make(lens, H=2, d_k=32, d_v=32, dtype=torch.float32)
    c["log_decay"][7, 0] = -float("inf")
    c["log_decay"][8, 0] = -float("inf")
    _check(c, lens)
    c["log_decay"][20, 1] = float("nan")
    out, fin = run(c, recurrent=True)
    nan = torch.isnan(out)
    assert nan[20:40, 1].all() and not nan[:20].any() and not nan[:, 0].any() and not nan[40:].any()
    assert torch.isnan(fin[0, 1]).all() and not torch.isnan(fin[1]).any()


def test_long_constant_decay_stays_exact():
    """A memory of thousands of tokens: rounding e^g itself would drift by 2^-25 per token in one
    direction; the kernel's e^g - 1 must not. Against the fp64 closed form of a constant input
    k = q = 1 (d = 1), v = 1: S_T = (1 - a^T) / (1 - a)."""
    T, g = 20000, -3e-4
    one = torch.ones(T, 1, 1, device="cuda")
    ld = torch.full((1,), g, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out, fin = binding.linear_prefill(one, one, one, ld, cu, recurrent=True)
    gd = float(ld.double())
    want = np.expm1(gd * np.arange(1, T + 1)) / np.expm1(gd)
    # each step rounds the sum twice: 2 x 2^-24 per token of the memory (about 1 / |g| tokens), and
    # e^g - 1 is off by at most 2^-23 of itself
    assert np.all(np.abs(f64(out).ravel() - want) <= (2 * 2.0 ** -24 / -gd + 2.0 ** -22 + 2.0 ** -23) * want)


def test_rows_behind_the_last_sequence_stay():
    lens = [20, 30]
    c = make(lens, d_k=32, d_v=32, dtype=torch.float32)
    big = {n: torch.cat([c[n], torch.full_like(c[n][:10], float("nan"))]) for n in ("q", "k", "v", "log_decay")}
    out = torch.full((60, 2, 32), 7.0, device="cuda")
    binding.linear_prefill(big["q"], big["k"], big["v"], big["log_decay"], c["cu_seqlens"], c["init_state"], out=out,
                           recurrent=True)
    o, _, mo, _ = reference(c)
    check(out[:50], o, mo, fp32_factor(30, 32), "out")
    assert (out[50:] == 7.0).all()
