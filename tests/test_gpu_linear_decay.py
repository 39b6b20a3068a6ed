"""What a strong decay leaves of a state: decode, the token-recurrent kernel, the tensor-core kernel
and the scan between segments against fp64, relative to the state that is left.

Bounds, relative to the decayed value. One step of a token: e^g (or e^g - 1, at most 1/2 in size, on
the value) is off by one ulp, 2^-23, its product is rounded, 2^-24: 3 x 2^-24. Behind the first token
the token-recurrent kernel rounds a factor above one half either way, by up to one ulp of 2^-24: with e^g
- 1 off by 2^-25, and the rounded product, 4 x 2^-24. The tensor-core kernel
takes e to a chunk's sum of log2-decays: each term rounded once, five levels of additions within 32
tokens and three across, so off by 9 x 2^-24 of the sum of their sizes; 2 ulps of the power (2^-22)
and one rounding of the product. A segment's sum is rounded once more on its way to the scan."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from linear_cases import check, f64, fp32_factor, make, reference, run

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32
STEP, LATER_STEP = 3 * 2.0 ** -24, 4 * 2.0 ** -24
DECAYS = [-0.3, -0.6931, -0.6932, -1.0, -4.0, -6.0, -8.0, -10.0, -14.0, -17.0, -18.0, -30.0, -60.0, -70.0]


def _still(lens, H=2, d=64, dtype=B16, seed=0, **kw):
    """A case that writes nothing (v = 0) over states of size 10^4, without decay as yet."""
    c = make(lens, H=H, d_k=d, d_v=d, dtype=dtype, seed=seed, **kw)
    c["v"].zero_(), c["log_decay"].zero_(), c["init_state"].mul_(2e4)
    return c


def _left(c):
    """The states in fp64; log-decays as the kernels get them."""
    g = c["log_decay"].double()
    S = c["init_state"].double() * torch.exp(g.sum(0))[None, :, None, None]
    return S.cpu().numpy()


def _relative(got, want, bound):
    d = np.abs(f64(got) - want)
    assert not (d > bound * np.abs(want)).any(), (float((d / np.abs(want).clip(1e-300)).max()), bound)


@pytest.mark.parametrize("d_k,d_v", [(64, 64), (33, 53), (128, 128)])
@pytest.mark.parametrize("per_token", [True, False])
def test_one_step(d_k, d_v, per_token):
    """Every head another decay; the read-out sums d_k products."""
    H = len(DECAYS)
    c = make([1] * 3, H=H, H_k=1, d_k=d_k, d_v=d_v, seed=d_k)
    c["v"].zero_(), c["init_state"].mul_(2e4)
    g = torch.tensor(DECAYS, device="cuda")
    c["log_decay"] = g.expand(3, H).contiguous() if per_token else g
    want = c["init_state"].double() * torch.exp(g.double())[None, :, None, None]
    q = c["q"].double()[:, 0, None, :, None]
    o, mo = (q * want).sum(-2), (q.abs() * want.abs()).sum(-2)
    for dt in (B16, F32):
        c = {n: t.to(dt) if n in ("q", "k", "v") else t for n, t in c.items()}
        state = c["init_state"].clone()
        out = binding.linear_decode(c["q"], c["k"], c["v"], c["log_decay"], state)
        _relative(state, want.cpu().numpy(), STEP)
        assert ((out.double() - o).abs() <= fp32_factor(1, d_k) * mo).all()
        out, fin = run(c, recurrent=True)
        _relative(fin, want.cpu().numpy(), STEP)
        assert ((out.double() - o).abs() <= fp32_factor(1, d_k) * mo).all()


@pytest.mark.parametrize("dtype", [B16, F32])
def test_writes_beside_a_large_state(dtype):
    """Ordinary tokens after a head that summed to 10^4 forgets most of it."""
    for g in (-6.0, -10.0, -17.0):
        lens = [170, 30]
        c = make(lens, H=3, d_k=40, d_v=24, dtype=dtype, decay=1e-3, seed=3)
        c["init_state"].mul_(2e4)
        c["log_decay"][5, 0], c["log_decay"][20, 1], c["log_decay"][171, 2] = g, g, g
        o, f, mo, mf = reference(c)
        out, fin = run(c, recurrent=True)
        check(out, o, mo, fp32_factor(170, 40), "out")
        check(fin, f, mf, fp32_factor(170, 40), "final")
        if dtype == B16:
            out, fin = run(c, out_dtype=F32)
            check(out, o, mo, 2.0 ** -15 + fp32_factor(130, 40), "out")
            check(fin, f, mf, 2.0 ** -15 + fp32_factor(130, 40), "final")


@pytest.mark.parametrize("total", [-0.3, -0.7, -2.0, -6.0, -10.0, -17.0, -18.0, -30.0, -60.0])
@pytest.mark.parametrize("d,out_dtype", [(128, B16), (64, F32)])
def test_chunks(total, d, out_dtype):
    """A chunk's decays sum to `total`: evenly, and in one token; the state passes through further
    chunks that keep it, and through none."""
    for T in (100, 300):
        c = _still([T], H=3, d=d, seed=T)
        c["log_decay"][:100, 0] = total / 100
        c["log_decay"][40, 1] = total
        want = _left(c)
        out, fin = run(c, out_dtype=out_dtype)
        _relative(fin, want, 9 * 2.0 ** -24 * -total + 2.0 ** -22 + 3 * 2.0 ** -24)
        o, _, mo, _ = reference(c)
        half = 2.0 ** -7 if out_dtype == B16 else 2.0 ** -15  # the state's and the output's own roundings
        check(out, o, mo, half + 9 * 2.0 ** -24 * -total + fp32_factor(8, d), "out")


@pytest.mark.parametrize("total", [-0.3, -0.7, -2.0, -6.0, -10.0, -17.0, -18.0, -30.0, -60.0])
@pytest.mark.parametrize("recurrent", [False, True])
@pytest.mark.parametrize("d_v", [64, 65])
def test_across_a_cut(total, recurrent, d_v):
    """The same in one of many segments, which pass 2 chains (four entries at a time, or one)."""
    T = 2500
    c = make([T], H=2, d_k=64, d_v=d_v, seed=1)
    c["v"].zero_(), c["log_decay"].zero_(), c["init_state"].mul_(2e4)
    assert binding.linear_workspace_size(T, 1, 2, 64, d_v, B16, F32, recurrent) > 0
    c["log_decay"][600:700, 0] = total / 100
    c["log_decay"][1030, 1] = total
    want = _left(c)
    fin = run(c, recurrent=recurrent)[1]
    # the token kernel: sums of 16 log-decays one after the other; a hundred decaying tokens at most
    _relative(fin, want, 18 * 2.0 ** -24 * -total + 2.0 ** -22 + 101 * LATER_STEP)


@pytest.mark.parametrize("g", [15.0, 18.0, 30.0, -15.0, -18.0, -30.0])
def test_growth_and_decay_cancel(g):
    """e^g and e^-g one after the other leave the state, within a chunk, across chunks and across a cut."""
    for first, second in ((3, 7), (3, 100), (100, 140), (5, 2000)):
        c = _still([2500], H=2, seed=2)
        c["log_decay"][first], c["log_decay"][second] = g, -g
        want = f64(c["init_state"])
        bound = 20 * 2.0 ** -24 * abs(g) + 2.0 ** -20
        for recurrent in (False, True):
            for workspace in ("auto", None):
                _relative(run(c, recurrent=recurrent, workspace=workspace)[1], want, bound)
    c = make([1] * 2, H=2, d_k=64, d_v=64, dtype=F32)
    c["v"].zero_()
    state = c["init_state"].clone()
    for x in (g, -g):
        binding.linear_decode(c["q"], c["k"], c["v"], torch.full((2, 2), x, device="cuda"), state)
    _relative(state, f64(c["init_state"]), 2 * STEP)


@pytest.mark.parametrize("per_token", [True, False])
def test_a_constant_decay_does_not_drift(per_token):
    """3000 tokens of one decay, nothing written: the mean relative error over a head's 4096 entries.
    What they share: factors that together stay within an ulp (2^-23) of e to the sum, e^g - 1 off by an
    ulp of itself at every token; each entry's own roundings (at most 2^-24, without a bias: a standard
    deviation below 2^-24 / sqrt(3)) shrink with the number of entries. e^g rounded to nearest at every
    token would be off by up to 3000 x 2^-25, a hundred times as much."""
    T, g = 3000, torch.tensor([-1e-5, -3e-4, -1e-3, -2.7e-3, -7e-3, -1.1e-2, -0.0201, 1e-3], device="cuda")
    H = g.numel()
    c = make([T], H=H, H_k=1, d_k=64, d_v=64, dtype=F32, seed=4)
    c["v"].zero_()
    c["log_decay"] = g.expand(T, H).contiguous() if per_token else g
    want = c["init_state"].double() * torch.exp(T * g.double())[None, :, None, None]
    fin = run(c, recurrent=True, workspace=None)[1]
    mean = ((fin.double() - want) / want).mean((0, 2, 3)).abs().cpu()
    bound = 2.0 ** -23 + T * g.abs().cpu() * 2.0 ** -23 + 6 * (T / 3 / 4096) ** 0.5 * 2.0 ** -24
    assert (mean <= bound).all(), (mean, bound)


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("recurrent", [False, True])
def test_growth_among_decays(out_dtype, recurrent):
    """Log-decays of either sign, whose runs all sum to between -18 and 18 (26 in log2 units), cut and
    uncut. On the tensor-core kernel a sum over a block passes 31 additions and 32 roundings of its terms,
    each of at most 26, and an entry takes a difference of two: 126 x 26 x 2^-24 x ln 2 < 2^-12."""
    T, H = 1500, 4
    c = make([T], H=H, d_k=64, d_v=64, seed=6)
    g = torch.Generator().manual_seed(6)
    level = 6 * torch.sin(torch.arange(T + 1)[:, None] * torch.tensor([0.01, 0.11, 0.7, 3.0])) + 6 * torch.rand(T + 1, H, generator=g) - 3
    c["log_decay"] = (level[1:] - level[:-1]).float().cuda()
    o, f, mo, mf = reference(c)
    fine = 2.0 ** -12 + 2.0 ** -15 + fp32_factor(T, 64)
    half = 2.0 ** -8 if out_dtype == B16 else 0.0
    for workspace in ("auto", None):
        out, fin = run(c, out_dtype=out_dtype, recurrent=recurrent, workspace=workspace)
        check(out, o, mo * (half + fine) + half * np.abs(o), 1.0, "out")
        check(fin, f, mf, fine, "final")


@pytest.mark.parametrize("recurrent", [False, True])
def test_what_a_long_decay_forgets_stays_forgotten(recurrent):
    """Growth by up to e^40 behind tokens that forget brings back e^-48 of the state at most."""
    for where, then in ((5, 9), (5, 100), (5, 1000), (130, 2300)):
        for g in (-float("inf"), -1e4, -88.0):
            c = _still([2500], H=2, seed=2)
            c["log_decay"][where], c["log_decay"][then] = g, 40.0
            most = float(np.exp(-48.0)) * float(c["init_state"].abs().max())
            for workspace in ("auto", None):
                out, fin = run(c, recurrent=recurrent, workspace=workspace)
                assert float(fin.abs().max()) <= 1.0001 * most
