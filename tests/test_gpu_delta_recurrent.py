"""kda_delta_prefill on the fp32 token kernel, against the fp64 oracle. Bounds: delta_cases."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from delta_cases import bounds, check, f64, half_step, make, reference, run

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


def _check(c, scale=1.0, out_dtype=F32, **kw):
    out, fin = run(c, scale=scale, out_dtype=out_dtype, recurrent=True, **kw)
    o, f = reference(c, scale)
    bo, bf, _ = bounds(c, scale)
    check(out, o, bo + half_step(o, out_dtype), "out")
    if fin is not None:
        check(fin, f, bf, "final")
    return out, fin


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (B16, B16), (B16, F32), (F32, B16)])
@pytest.mark.parametrize("lens", [[1], [2], [3], [4], [5], [15], [16], [17], [64, 0, 33], [0, 1, 0, 2, 130]])
def test_lengths(lens, dtype, out_dtype):
    _check(make(lens, H=2, d_k=32, d_v=24, dtype=dtype, seed=sum(lens)), out_dtype=out_dtype)


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("d_k,d_v", [(128, 128), (64, 64), (1, 1), (100, 72), (5, 33), (128, 6), (65, 127), (16, 17)])
def test_head_sizes(d_k, d_v, dtype):
    _check(make([37, 20], H=3, d_k=d_k, d_v=d_v, dtype=dtype, seed=d_k + d_v), scale=0.25)


@pytest.mark.parametrize("H,H_k,N", [(6, 1, 2), (6, 3, 2), (8, 2, 2), (64, 4, 3), (48, 48, 30)])
@pytest.mark.parametrize("per_token", [True, False])
def test_shared_heads_and_column_widths(H, H_k, N, per_token):
    """Few chains take 16 columns per CTA, more 32, many 64."""
    _check(make([11] * N, H=H, H_k=H_k, d_k=24, d_v=80, per_token=per_token, seed=H))


@pytest.mark.parametrize("decay", [0.0, 1e-3, 0.3, 3.0, 30.0])
def test_decays(decay):
    _check(make([150], decay=decay, d_k=64, d_v=16, dtype=F32, seed=7))


def test_keys_alike():
    _check(make([200], d_k=64, d_v=16, dtype=F32, seed=8, alike=3.0))
    c = make([200], d_k=64, d_v=16, dtype=F32, seed=8, decay=0.0)
    c["k"] = c["k"][:1].expand(200, -1, -1).contiguous()  # one key over and over
    c["beta"].fill_(1.0)
    _check(c)


def test_states():
    lens = [90, 0, 40]
    c = make(lens, d_k=64, d_v=64, dtype=F32)
    o, f = reference(c)
    bo, bf, _ = bounds(c)
    state = c["init_state"]
    out, fin = run(c, recurrent=True, final_state=state)
    assert fin is state
    check(fin, f, bf, "in place")
    check(out, o, bo, "out")
    out, fin = run(make(lens, d_k=64, d_v=64, dtype=F32), recurrent=True, want_final=False)
    assert fin is None
    check(out, o, bo, "out")
    _check(make(lens, d_k=64, d_v=64, dtype=F32, init=False))


def test_infinite_decay_forgets_and_nan_stays_where_it_belongs():
    lens = [40, 40]
    c = make(lens, H=2, d_k=32, d_v=32, dtype=F32)
    c["log_decay"][7, 0] = -float("inf")
    c["log_decay"][8, 0] = -float("inf")
    _check(c)
    c["log_decay"][21, 1] = float("nan")
    out, fin = run(c, recurrent=True)
    nan = torch.isnan(out)
    assert nan[21:40, 1].all() and not nan[:21].any() and not nan[:, 0].any() and not nan[40:].any()
    assert torch.isnan(fin[0, 1]).all() and not torch.isnan(fin[1]).any()
    c = make(lens, H=2, d_k=32, d_v=32, dtype=F32)
    want, _ = run(c, recurrent=True)
    c["v"][22, 1, 5] = float("inf")
    out, fin = run(c, recurrent=True)
    bad = ~torch.isfinite(out)
    assert bad[22:40, 1, 5].all() and int(bad.sum()) == 18 and torch.equal(out[:22], want[:22])
    assert torch.equal(out[40:], want[40:]) and bool(torch.isfinite(fin[1]).all())


def test_growth():
    """Positive log-decays while no run of tokens sums above 40."""
    c = make([60], H=2, d_k=32, d_v=16, dtype=F32, decay=0.0)
    c["log_decay"][10:50] = 0.9
    _check(c)


def test_long_constant_decay_stays_exact():
    """A memory of thousands of tokens, k = q = 1 (d = 1), beta = 1/2: S_t = a' S_{t-1} + v / 2 with
    a' = e^g / 2 forgets fast, so the decay is seen with k = 0: S_T = e^{g T} S_0."""
    T, g = 20000, -3e-4
    zero = torch.zeros(T, 1, 1, device="cuda")
    ld = torch.full((1,), g, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    s0 = torch.full((1, 1, 1, 1), 3.0, device="cuda")
    _, fin = binding.delta_prefill(zero, zero, zero, ld, torch.full((T, 1), 0.5, device="cuda"), cu, s0, recurrent=True)
    want = 3.0 * np.exp(float(ld.double()) * T)
    # 5000 steps of four tokens: each rounds the product, 2^-24 either way (bounded here by all one way),
    # and the factors stay within an ulp, 2^-23, of e to the sum of every 4096 steps
    assert abs(float(fin.double()) - want) <= (5000 * 2.0 ** -24 + 4 * 2.0 ** -23) * want


def test_rows_behind_the_last_sequence_stay():
    lens = [20, 30]
    c = make(lens, d_k=32, d_v=32, dtype=F32)
    big = {n: torch.cat([c[n], torch.full_like(c[n][:10], float("nan"))]) for n in ("q", "k", "v", "log_decay", "beta")}
    out = torch.full((60, 2, 32), 7.0, device="cuda")
    binding.delta_prefill(big["q"], big["k"], big["v"], big["log_decay"], big["beta"], c["cu_seqlens"], c["init_state"],
                          out=out, recurrent=True)
    o, _ = reference(c)
    bo, _, _ = bounds(c)
    check(out[:50], o, bo, "out")
    assert (out[50:] == 7.0).all()
    assert not np.isnan(f64(out)).any()


@pytest.mark.parametrize("T,d_k,d_v,H,H_k", [(3000, 128, 128, 2, 1), (3500, 100, 72, 2, 1), (1500, 33, 7, 2, 2), (2111, 64, 65, 1, 1),
                                             (4100, 5, 127, 1, 1), (1900, 128, 128, 1, 1)])
@pytest.mark.parametrize("dtype", [F32, B16])
def test_one_long_sequence_in_segments(T, d_k, d_v, H, H_k, dtype):
    """Cut into segments that are joined by their transition maps, with a workspace full of NaN; without one, from
    end to end. Errors are roundings of 2^-24 with random signs, some four a token, of which a state
    remembers d_k / beta tokens, 256 or so: 4 sqrt(256) 2^-24 = 4e-6 in the 2-norm, and as much again from the
    maps; bf16 prompts are on the tensor cores, where ten roundings of pairs make it 2e-5."""
    c = make([T], H=H, H_k=H_k, d_k=d_k, d_v=d_v, dtype=dtype, decay=0.003, seed=T)
    assert binding.delta_workspace_size(T, 1, H, d_k, d_v, F32, F32, H_k=H_k) > 0  # (bf16: cut from 1536 tokens on)
    o, f = reference(c)
    wide = {x: torch.cat([c[x], torch.full_like(c[x][:20], float("nan"))]) for x in ("q", "k", "v", "log_decay", "beta")}
    n = binding.delta_workspace_size(T + 20, 1, H, d_k, d_v, dtype, F32, H_k=H_k)
    ws = torch.full((n // 4,), float("nan"), device="cuda").view(torch.uint8) if n else None
    out = torch.full((T + 20, H, d_v), 7.0, device="cuda")
    _, fin = run({**c, **wide}, out=out, workspace=ws)
    assert (out[T:] == 7).all()
    tolerance = 1e-5 if dtype == F32 else 2e-5
    for got, want in ((out[:T], o), (fin, f)):
        err = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
        assert err < tolerance, err
    if dtype == F32:
        out, fin = run(c, workspace=None)
        again, end = run(c, recurrent=True)
        assert torch.equal(out, again) and torch.equal(fin, end)
        state = c["init_state"].clone()
        a, b = run({**c, "init_state": state}, final_state=state)
        x, y = run(c)
        assert torch.equal(a, x) and torch.equal(b, y) and not torch.equal(y, end)
