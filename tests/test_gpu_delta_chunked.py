"""kda_delta_prefill on the tensor-core kernel (bf16), its segments and its order, against the fp64
oracle. Bounds: delta_cases (pairs); a bf16 output has P, U and the state rounded to bf16 for the
read-out, 2^-8, and its own half step."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from delta_cases import bounds, check, f64, half_step, make, reference, run

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


def _check_against(c, out, fin, scale=1.0, ref=None):
    o, f = ref or reference(c, scale)
    bo, bf, n = bounds(c, scale, pairs=True, read=2.0 ** -8 * 2 if out.dtype == B16 else 0.0)
    check(out, o, bo + half_step(o, out.dtype), "out")
    # In 2-norm over the tensor, where the errors' signs are random, a pair is off by 2^-18 / sqrt(3) of the
    # value; some ten of them meet on the way through a chunk, and 2e-5 is 9 x 2^-18 / sqrt(3) with room
    # for the read-out's cancellation. bf16 read-outs are held by the bound above alone.
    if out.dtype == F32:
        err = np.linalg.norm(f64(out) - o) / max(np.linalg.norm(o), 1e-30)
        assert err < 2e-5, err
    if fin is not None:
        check(fin, f, bf, "final")
        err = np.linalg.norm(f64(fin) - f) / max(np.linalg.norm(f), 1e-30)
        assert err < 2e-5, err


def _check(c, scale=1.0, out_dtype=B16, **kw):
    out, fin = run(c, scale=scale, out_dtype=out_dtype, **kw)
    _check_against(c, out, fin, scale)
    return out, fin


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("lens", [[64], [63], [65], [128], [40], [200], [31, 32, 33], [0, 300, 0, 5], [640], [1, 1, 1, 2, 250],
                                  [127, 129, 1, 64, 192]])
def test_lengths(lens, out_dtype):
    _check(make(lens, H=2, seed=sum(lens)), out_dtype=out_dtype)


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("d_k,d_v", [(128, 64), (64, 128), (64, 64), (8, 8), (16, 128), (120, 72), (128, 8), (72, 104), (56, 40)])
def test_head_sizes(d_k, d_v, out_dtype):
    _check(make([150, 40], H=3, d_k=d_k, d_v=d_v, seed=d_k + d_v), scale=0.25, out_dtype=out_dtype)


def _on_tensor_cores(c, out, fin, **kw):
    """Whether a result is not the token kernel's (they differ in the last bits)."""
    o, f = run(c, out_dtype=out.dtype, recurrent=True, **kw)
    return not torch.equal(o, out) and not torch.equal(f, fin)


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("d_k,d_v", [(100, 72), (72, 100), (33, 40), (127, 127), (65, 1), (1, 128), (3, 3), (128, 61), (17, 17)])
def test_padded_head_sizes(d_k, d_v, out_dtype):
    c = make([150, 0, 140, 1], H=6, H_k=2, d_k=d_k, d_v=d_v, seed=d_k + d_v)
    c = c if d_k > 64 or d_v > 64 else make([150, 140], H=6, H_k=2, d_k=d_k, d_v=d_v, seed=d_k + d_v)
    out, fin = _check(c, scale=0.25, out_dtype=out_dtype)
    assert d_k <= (8 if out_dtype == B16 else 16) or _on_tensor_cores(c, out, fin, scale=0.25)
    o, f = run(c, scale=0.25, out_dtype=out_dtype, workspace=None)  # no room for the copies
    assert not _on_tensor_cores(c, o, f, scale=0.25)


@pytest.mark.parametrize("d_k,d_v", [(100, 72), (128, 33), (65, 127)])
def test_padded_segments_and_rows_behind(d_k, d_v):
    """Cut sequences of odd head sizes, a workspace full of NaN, rows behind the last sequence."""
    lens = [2600]
    c = make(lens, H=2, d_k=d_k, d_v=d_v, decay=0.01, seed=13)
    wide = {n: torch.cat([c[n], torch.full_like(c[n][:40], float("nan"))]) for n in ("q", "k", "v", "log_decay", "beta")}
    n = binding.delta_workspace_size(2640, 1, 2, d_k, d_v, B16, F32)
    assert n > 2 * 2640 * 2 * d_v
    ws = torch.full((n // 4,), float("nan"), device="cuda").view(torch.uint8)
    for out_dtype in (B16, F32):
        out = torch.full((2640, 2, d_v), 7.0, device="cuda", dtype=out_dtype)
        o, fin = run({**c, **wide}, out=out, workspace=ws)
        assert (out[2600:] == 7).all()
        _check_against(c, out[:2600].contiguous(), fin)


@pytest.mark.parametrize("d_k", [5, 8, 9, 16, 17, 24])
@pytest.mark.parametrize("d_v", [16, 128])
def test_few_key_channels_stay_exact(d_k, d_v):
    """Keys that are far from orthogonal make the terms of a chunk's U larger than U itself. Up to 16 channels
    the token kernel takes them (2^-24 a rounding, under 1e-6 in the 2-norm as elsewhere); from 17 on the terms
    are at most some 1 + 64 / d_k times as large in power, and the ten pairs' 2^-18 / sqrt(3), 7e-6 together, stay
    below 1e-5. With a bf16 output the state alone is fp32, and 9 channels are enough."""
    c = make([270, 497], H=4, H_k=2, d_k=d_k, d_v=d_v, decay=0.02, seed=d_k)
    out, fin = run(c, scale=4 * d_k ** -0.5)
    o, f = reference(c, 4 * d_k ** -0.5)
    for got, want in ((out, o), (fin, f)):
        err = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
        assert err < (1e-6 if d_k <= 16 else 1e-5), err
    _, fin = run(c, scale=4 * d_k ** -0.5, out_dtype=B16)
    err = np.linalg.norm(f64(fin) - f) / np.linalg.norm(f)
    assert err < (1e-6 if d_k <= 8 else 1e-5), err


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("lens", [[40, 0], [31, 32, 33], [6, 6, 7], [63, 1, 5], [8, 64, 10]])
def test_short_sequences_of_many_heads(lens, out_dtype):
    c = make(lens, H=104, H_k=8, seed=sum(lens))
    out, fin = _check(c, out_dtype=out_dtype)
    assert _on_tensor_cores(c, out, fin)


@pytest.mark.parametrize("H,H_k", [(6, 1), (6, 3), (8, 2)])
@pytest.mark.parametrize("per_token", [True, False])
def test_shared_heads(H, H_k, per_token):
    for out_dtype in (B16, F32):
        _check(make([70, 200], H=H, H_k=H_k, d_v=64, per_token=per_token, seed=H), out_dtype=out_dtype)


@pytest.mark.parametrize("decay", [0.0, 1e-3, 0.3, 3.0, 30.0])
@pytest.mark.parametrize("out_dtype", [B16, F32])
def test_decays(decay, out_dtype):
    _check(make([400], decay=decay, seed=7), out_dtype=out_dtype)


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("lens,first,g", [([64], 3, 0.6), ([150], 5, 0.3)])
def test_growth(lens, first, g, out_dtype):
    """Positive log-decays while no run of tokens sums above 40: entries of the inverse reach e^36. With
    G_t the sums from the start, e^{-G_t} S_t follows the recurrence without a decay and with e^{-G_t} v_t,
    and every rounding is relative to its entry, so the bound is that of this one times e^{G_t}. (An
    entry's decay is off by 2^-19 of it more, a sum of up to 58 in units of ln 2 held in fp32; the bound counts
    each pair, at most 2^-17 off, as 2^-16.)"""
    c = make(lens, decay=0.0, seed=9)
    c["log_decay"][first:first + int(36 / g)] = g
    out, fin = run(c, out_dtype=out_dtype)
    o, f = reference(c)
    G = torch.cumsum(c["log_decay"].double(), 0)[:, :, None]
    still = {**c, "v": c["v"].double() * torch.exp(-G), "log_decay": torch.zeros_like(c["log_decay"])}
    bo, bf, _ = bounds(still, pairs=True, read=2.0 ** -8 * 2 if out_dtype == B16 else 0.0)
    grown = f64(torch.exp(G))
    check(out, o, bo * grown + half_step(o, out_dtype), "out")
    check(fin, f, bf * grown[-1][None, :, None], "final")


@pytest.mark.parametrize("out_dtype", [B16, F32])
def test_keys_alike(out_dtype):
    """Keys with a common direction, and one key over and over: the inverse of I + A is then far from
    I - A, and powers of A would grow like binomials."""
    _check(make([300], seed=8, alike=2.0), out_dtype=out_dtype)
    c = make([300], seed=8, decay=0.0)
    c["k"] = c["k"][:1].expand(300, -1, -1).contiguous()
    _check(c, out_dtype=out_dtype)


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("lens", [[3000], [1600], [5121], [1500, 0, 1, 7000, 511, 1536]])
@pytest.mark.parametrize("d_v", [128, 64])
def test_segments_join(lens, d_v, out_dtype):
    c = make(lens, H=2, d_v=d_v, decay=0.01, seed=11)
    assert binding.delta_workspace_size(sum(lens), len(lens), 2, 128, d_v, B16, out_dtype) > 1 << 16
    ref = reference(c)
    for ws in ("auto", None):
        out, fin = run(c, out_dtype=out_dtype, workspace=ws)
        _check_against(c, out, fin, ref=ref)


def test_longest_first():
    lens = [30 + 17 * i % 190 for i in range(40)] + [0, 900, 1]
    c = make(lens, H=32, H_k=4, d_k=64, d_v=32, seed=12)
    assert 0 < binding.delta_workspace_size(sum(lens), len(lens), 32, 64, 32, B16, B16) <= 256
    out, fin = _check(c)
    o, f = run(c, out_dtype=B16, workspace=None)
    assert torch.equal(out, o) and torch.equal(fin, f)


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("init", [True, False])
@pytest.mark.parametrize("lens", [[900, 300, 130] + [0] * 40, [0, 64, 0, 1] * 10 + [700], [70] * 30 + [0] * 7 + [1] * 9,
                                  [1] * 25 + [500, 400]])
def test_many_sequences_and_heads(lens, init, out_dtype):
    """Several times more (sequence, head)s than SMs: long ones, some of one token, empty ones in a row."""
    c = make(lens, H=24, H_k=2, d_k=64, d_v=72, init=init, seed=sum(lens))
    assert binding.delta_workspace_size(sum(lens), len(lens), 24, 64, 72, B16, out_dtype) == 256
    out, fin = _check(c, out_dtype=out_dtype)
    o, f = run(c, out_dtype=out_dtype, workspace=None)
    assert torch.equal(out, o) and torch.equal(fin, f)
    if init:
        state = c["init_state"].clone()
        o, f = run({**c, "init_state": state}, out_dtype=out_dtype, final_state=state)
        assert torch.equal(out, o) and torch.equal(fin, f)


@pytest.mark.parametrize("T", [200, 2500])
def test_states(T):
    lens = [T, 0, 60]
    _check(make(lens, init=False))
    c = make(lens, decay=0.02)
    o, f = reference(c)
    state = c["init_state"].clone()
    out, fin = run({**c, "init_state": state}, out_dtype=B16, final_state=state)
    assert fin is state
    _check_against(c, out, fin, ref=(o, f))
    out, fin = run(c, out_dtype=B16, want_final=False)
    assert fin is None
    _check_against(c, out, None, ref=(o, f))


def test_neighbours_and_rows_behind_stay_out():
    """NaN in another sequence's tokens and behind the last one; output rows behind stay as they were."""
    lens = [100, 90, 70]
    c = make(lens, H=4, H_k=2, d_v=64, seed=4)
    o, f = reference(c)
    for n in ("q", "k", "v", "beta"):
        c[n][100:190] = float("nan")
    wide = {n: torch.cat([c[n], torch.full_like(c[n][:40], float("nan"))]) for n in ("q", "k", "v", "log_decay", "beta")}
    keep = np.r_[0:100, 190:260]
    out = torch.full((300, 4, 64), 7.0, device="cuda", dtype=F32)
    state = c["init_state"].clone()
    binding.delta_prefill(wide["q"], wide["k"], wide["v"], wide["log_decay"], wide["beta"], c["cu_seqlens"], state,
                          out=out, final_state=state)
    binding.check_device_error()
    assert (out[260:] == 7.0).all()
    assert np.abs(f64(out[:260])[keep] - o[keep]).max() < 1e-3 and np.abs(f64(state)[[0, 2]] - f[[0, 2]]).max() < 1e-3


def test_infinite_decay_forgets_and_nan_goes_on():
    c = make([200, 100], H=2)
    c["log_decay"][70, 0] = c["log_decay"][71, 0] = c["log_decay"][130, 0] = -float("inf")
    finite = {**c, "log_decay": c["log_decay"].clamp(min=-88.0)}
    o, f = reference(finite)
    for out_dtype in (B16, F32):
        out, fin = run(c, out_dtype=out_dtype)
        _check_against(finite, out, fin, ref=(o, f))
    c["log_decay"][150, 1] = float("nan")
    out, fin = run(c, out_dtype=F32)
    bad = torch.isnan(out)
    assert bad[150:200, 1].all() and not bad[:128].any() and not bad[:, 0].any() and not bad[200:].any()
    assert torch.isnan(fin[0, 1]).all() and torch.isfinite(fin[1]).all() and torch.isfinite(fin[0, 0]).all()
    c = make([200, 100], H=2)
    c["v"][140, 1, 5] = float("inf")  # its channel alone, from its chunk on
    out, fin = run(c, out_dtype=F32)
    bad = ~torch.isfinite(out)
    assert bad[140:200, 1, 5].all() and not bad[:128].any() and not bad[200:].any()
    bad[:, 1, 5] = False
    assert not bad.any()


def test_causal():
    """What comes later changes nothing before its chunk, bit by bit."""
    c = make([400], H=2, seed=9)
    out, _ = run(c, out_dtype=F32, workspace=None)
    for n in ("q", "k", "v", "log_decay", "beta"):
        c[n][320:] = c[n][320:].flip(0)
    again, _ = run(c, out_dtype=F32, workspace=None)
    assert torch.equal(out[:320], again[:320]) and not torch.equal(out[320:], again[320:])


def test_unaligned_outputs():
    c = make([140, 30], H=2, d_k=64, d_v=72, seed=5)
    for out_dtype in (B16, F32):
        per = 8 if out_dtype == B16 else 4
        flat = torch.full((170 * 2 * 72 + 2 * per,), 7.0, device="cuda", dtype=out_dtype)
        out = flat[per:-per].view(170, 2, 72)
        states = torch.full((2 * 2 * 64 * 72 + 8,), 7.0, device="cuda")
        fin = states[4:-4].view(2, 2, 64, 72)
        fin.copy_(c["init_state"])
        run({**c, "init_state": fin}, out=out, final_state=fin)
        _check_against(c, out, fin)
        assert (flat[:per] == 7).all() and (flat[-per:] == 7).all() and (states[:4] == 7).all() and (states[-4:] == 7).all()


@pytest.mark.parametrize("lens,H", [([700, 40], 2), ([2600], 2)])
def test_captured_and_replayed(lens, H):
    """Two captured calls with a workspace each replay together on two streams."""
    cs = [make(lens, H=H, d_v=64, decay=0.02, seed=s) for s in (1, 2)]
    size = max(16, binding.delta_workspace_size(sum(lens), len(lens), H, 128, 64, B16, B16))
    refs = [run(c, out_dtype=B16) for c in cs]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in cs]
    for c, st in zip(cs, streams):
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        out, fin = torch.empty_like(refs[0][0]), torch.empty_like(refs[0][1])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            binding.delta_prefill(**c, out=out, final_state=fin, workspace=ws)
        graphs.append(graph)
        outs.append((out, fin, ws))
    for _ in range(3):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for (o, f, _), (out, fin) in zip(outs, refs):
            assert torch.equal(o, out) and torch.equal(f, fin)
            o.fill_(3), f.fill_(3)
    binding.check_device_error()


def test_norm_and_rotation_then_prompt_then_tokens():
    """The operators as a layer uses them: raw queries and keys normed and turned, the prompt, then tokens
    at the following positions, against the oracle's run over all of them."""
    from oracle import delta_recurrent, norm_rotate
    g = torch.Generator().manual_seed(3)
    T, H, H_k, d = 210, 4, 2, 128
    raw = torch.randn(T, 2 * H_k * d, generator=g).to(B16).cuda()
    q, k = raw[:, :H_k * d].view(T, H_k, d), raw[:, H_k * d:].view(T, H_k, d)
    f = torch.exp(-torch.arange(32) * 0.3).cuda()
    pos = torch.arange(T, device="cuda") + 100000
    c = make([T], H=H, H_k=H_k, d_k=d, d_v=64, seed=3)
    rot = lambda x, y, p: binding.norm_rotate(x, y, p, f, norm="l2")  # noqa: E731
    n = 200
    qn, kn = rot(q[:n], k[:n], pos[:n])
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, state = binding.delta_prefill(qn, kn, c["v"][:n], c["log_decay"][:n], c["beta"][:n], cu, c["init_state"])
    outs, qs, ks = [out], [qn], [kn]
    for t in range(n, T):
        qt, kt = rot(q[t:t + 1], k[t:t + 1], pos[t:t + 1])
        qs.append(qt), ks.append(kt)
        outs.append(binding.delta_decode(qt, kt, c["v"][t:t + 1], c["log_decay"][t:t + 1], c["beta"][t:t + 1], state))
    binding.check_device_error()
    c = {**c, "q": torch.cat(qs), "k": torch.cat(ks)}
    for x, y in ((q, c["q"]), (k, c["k"])):
        want = norm_rotate(x.cpu(), pos.cpu(), f.cpu(), norm="l2")
        assert np.all(np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + 1e-6)
    _check_against(c, torch.cat(outs), state)
    o, _ = delta_recurrent(**{n_: None if t is None else t.cpu() for n_, t in c.items()})
    assert np.linalg.norm(f64(torch.cat(outs)) - o) < 2e-5 * np.linalg.norm(o)
