"""kda_linear_prefill on the tensor-core kernel (bf16), its segments and its pass of state sums,
against the fp64 oracle.

Bounds, relative to the magnitude (the same sums over absolute values). The state: its terms'
decayed values enter as bf16 pairs, off by at most 2^-16; the decay of a term is 2 to a sum of at
most 32 log-decays per factor, each sum at most 32 x 5 x 1.45 = 231 in these tests and so off by
231 x 2^-24 x ln 2 < 2^-16; fp32 accumulation as in linear_cases.fp32_factor over a chunk (128
tokens) and two roundings per chunk. An fp32 output is made of the same (P and the state enter as
pairs). A bf16 output has P and the state rounded to bf16, 2^-8, and its own half step, 2^-8."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from linear_cases import check, fp32_factor, make, reference, run

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


def _check(c, lens, scale=1.0, out_dtype=B16, **kw):
    return _check_against(c, lens, out_dtype, *run(c, scale=scale, out_dtype=out_dtype, **kw), scale=scale)


def _check_against(c, lens, out_dtype, out, fin, scale=1.0):
    o, f, mo, mf = reference(c, scale)
    fine = 2.0 ** -15 + fp32_factor(128 + max(lens) // 64, c["q"].shape[2])
    if out_dtype == B16:
        check(out, o, mo * (2.0 ** -8 + fine) + 2.0 ** -8 * np.abs(o), 1.0, "out")
    else:
        check(out, o, mo, fine, "out")
    if fin is not None:
        check(fin, f, mf, fine, "final")
    return out, fin


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("lens", [[128], [1], [127], [129], [256], [31, 32, 33], [0, 300, 0, 5], [640], [1, 1, 1, 2, 250]])
def test_lengths(lens, out_dtype):
    _check(make(lens, H=2, seed=sum(lens)), lens, out_dtype=out_dtype)


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("d_k,d_v", [(128, 64), (64, 128), (64, 64), (8, 8), (16, 128), (120, 72), (128, 8), (72, 104)])
def test_head_sizes(d_k, d_v, out_dtype):
    lens = [150, 40]
    _check(make(lens, H=3, d_k=d_k, d_v=d_v, seed=d_k + d_v), lens, scale=0.25, out_dtype=out_dtype)


@pytest.mark.parametrize("out_dtype", [B16, F32])
@pytest.mark.parametrize("d_k,d_v", [(1, 1), (127, 127), (13, 128), (128, 13), (65, 66), (100, 4), (7, 121), (128, 124)])
def test_padded_head_sizes(d_k, d_v, out_dtype):
    """Head sizes that are no multiple of 8 pass through a padded copy in the workspace; without
    one the token-recurrent kernel runs them."""
    lens = [350, 0, 1, 140]
    c = make(lens, H=4, H_k=2, d_k=d_k, d_v=d_v, seed=d_k + d_v)
    assert binding.linear_workspace_size(491, 4, 4, d_k, d_v, B16, out_dtype, H_k=2) > 0
    _check(c, lens, scale=0.25, out_dtype=out_dtype)
    _check(c, lens, scale=0.25, out_dtype=out_dtype, workspace=None)
    long = [1300]  # padded and cut into segments
    _check(make(long, H=2, d_k=d_k, d_v=d_v, seed=d_k), long, out_dtype=out_dtype)


@pytest.mark.parametrize("lens", [[15], [16], [17], [14, 0, 34], [23, 24], [25, 23], [47, 48], [50, 46], [95, 96], [99, 93]])
@pytest.mark.parametrize("d,out_dtype", [(128, B16), (128, F32), (64, F32), (60, B16)])
def test_either_side_of_the_length_rule(lens, d, out_dtype):
    """Sequences short on average take the token-recurrent kernel, the same as when it is asked for."""
    c = make(lens, H=2, d_k=d, d_v=d, seed=sum(lens))
    out, fin = _check(c, lens, out_dtype=out_dtype)
    if sum(lens) < {60: 96, 64: 48, 128: 16 if out_dtype == B16 else 24}[d] * len(lens):
        o, f = run(c, out_dtype=out_dtype, recurrent=True)
        assert torch.equal(out, o) and torch.equal(fin, f)


def test_padded_states_and_rows_behind():
    """Through the padded copies: no initial or final states, states in place, rows behind the last
    sequence left as they were, NaN there and in another sequence kept out."""
    lens = [100, 90, 70]
    c = make(lens, H=4, H_k=2, d_k=75, d_v=37, seed=4)
    o, f, mo, mf = reference(c)
    fine = 2.0 ** -15 + fp32_factor(130, 64)
    for n in ("q", "k", "v"):
        c[n][100:190] = float("nan")
    wide = {n: torch.cat([c[n], torch.full_like(c[n][:40], float("nan"))]) for n in ("q", "k", "v", "log_decay")}
    keep = np.r_[0:100, 190:260]
    out = torch.full((300, 4, 37), 7.0, device="cuda", dtype=F32)
    state = c["init_state"].clone()
    binding.linear_prefill(wide["q"], wide["k"], wide["v"], wide["log_decay"], c["cu_seqlens"], state, out=out,
                           final_state=state)
    binding.check_device_error()
    check(out[:260][keep], o[keep], mo[keep], fine, "out")
    check(state[[0, 2]], f[[0, 2]], mf[[0, 2]], fine, "final")
    assert (out[260:] == 7.0).all()
    _check(make(lens, H=4, H_k=2, d_k=75, d_v=37, init=False), lens)
    assert run(make(lens, H=4, H_k=2, d_k=75, d_v=37), want_final=False)[1] is None


def test_unaligned_views():
    """States and outputs that start 16 bytes off a 32-byte boundary, and packed rows behind them."""
    lens = [140, 30]
    c = make(lens, H=2, d_k=64, d_v=72, seed=5)
    o, f, mo, mf = reference(c)
    fine = 2.0 ** -15 + fp32_factor(130, 64)
    for out_dtype in (B16, F32):
        per = 8 if out_dtype == B16 else 4
        flat = torch.full((170 * 2 * 72 + 2 * per,), 7.0, device="cuda", dtype=out_dtype)
        out = flat[per:-per].view(170, 2, 72)
        states = torch.full((2 * 2 * 64 * 72 + 8,), 7.0, device="cuda")
        fin = states[4:-4].view(2, 2, 64, 72)
        fin.copy_(c["init_state"])
        run({**c, "init_state": fin}, out=out, final_state=fin)
        if out_dtype == B16:
            check(out, o, mo * (2.0 ** -8 + fine) + 2.0 ** -8 * np.abs(o), 1.0, "out")
        else:
            check(out, o, mo, fine, "out")
        check(fin, f, mf, fine, "final")
        assert (flat[:per] == 7).all() and (flat[-per:] == 7).all() and (states[:4] == 7).all() and (states[-4:] == 7).all()


@pytest.mark.parametrize("H,H_k", [(6, 1), (6, 3), (8, 2)])
@pytest.mark.parametrize("per_token", [True, False])
def test_shared_heads(H, H_k, per_token):
    lens = [70, 200]
    for out_dtype in (B16, F32):
        _check(make(lens, H=H, H_k=H_k, d_v=64, per_token=per_token, seed=H), lens, out_dtype=out_dtype)


@pytest.mark.parametrize("decay", [0.0, 1e-3, 0.3, 3.0])
@pytest.mark.parametrize("out_dtype", [B16, F32])
def test_decays(decay, out_dtype):
    lens = [400]
    _check(make(lens, decay=decay, seed=7), lens, out_dtype=out_dtype)


@pytest.mark.parametrize("lens", [[3000], [1500, 0, 1, 2600, 511, 512, 513, 1025]])
@pytest.mark.parametrize("d_v,out_dtype", [(128, B16), (64, B16), (128, F32)])
def test_segments_join(lens, d_v, out_dtype):
    c = make(lens, H=2, d_v=d_v, decay=0.01, seed=11)
    assert binding.linear_workspace_size(sum(lens), len(lens), 2, 128, d_v, B16, out_dtype) > 0
    _check(c, lens, out_dtype=out_dtype)
    _check(c, lens, out_dtype=out_dtype, workspace=None)


def test_states():
    lens = [200, 0, 60]
    _check(make(lens, init=False), lens)
    c = make(lens)
    o, f, mo, mf = reference(c)
    state = c["init_state"]
    out, fin = run(c, final_state=state)
    assert fin is state
    check(fin, f, mf, 2.0 ** -15 + fp32_factor(130, 128), "in place")
    assert run(make(lens), want_final=False)[1] is None


@pytest.mark.parametrize("H,d_v,out_dtype", [(77, 16, B16), (96, 16, F32), (120, 24, B16), (48, 72, F32), (96, 72, B16)])
@pytest.mark.parametrize("init", [True, False])
def test_one_sequence_on_many_heads(H, d_v, out_dtype, init):
    """About as many chains as SMs, kept whole or cut in few segments; heads that forget everything."""
    lens = [2500]
    c = make(lens, H=H, H_k=1, d_k=16, d_v=d_v, decay=0.01, init=init, seed=H)
    _check(c, lens, out_dtype=out_dtype)
    c["log_decay"][300:1400, ::3] = -float("inf")
    c["log_decay"][:, 1::3] = -0.2  # pass 1 stops early
    out, fin = _check(c, lens, out_dtype=out_dtype)
    again = run(c, out_dtype=out_dtype)
    assert torch.equal(out, again[0]) and torch.equal(fin, again[1])
    if init:  # in place
        state = c["init_state"].clone()
        _check_against(c, lens, out_dtype, *run({**c, "init_state": state}, out_dtype=out_dtype, final_state=state))


@pytest.mark.parametrize("end", [2500, 2049, 900, 130, 0])
@pytest.mark.parametrize("H", [8, 96])
def test_a_sequence_shorter_than_the_rows(end, H):
    """The sequence may end before the rows do, also inside the first of the planned segments."""
    lens = [2500]
    c = make(lens, H=H, H_k=2, d_k=16, d_v=16, decay=0.01, seed=2)
    c["cu_seqlens"] = torch.tensor([0, end], dtype=torch.int32, device="cuda")
    short = {n: t[:end] if n in ("q", "k", "v", "log_decay") else t for n, t in c.items()}
    for n in ("q", "k", "v"):
        c[n][end:] = float("nan")
    out = torch.full((2500, H, 16), 7.0, device="cuda")
    _, fin = run(c, out=out)
    assert (out[end:] == 7.0).all()
    o, f, mo, mf = reference(short)
    fine = 2.0 ** -15 + fp32_factor(128 + 40, 16)
    check(out[:end], o, mo, fine, "out")
    check(fin, f, mf, fine, "final")


@pytest.mark.parametrize("recurrent", [False, True])
@pytest.mark.parametrize("lens", [[1300], [1025, 0, 1, 700, 1537]])
def test_states_in_place_of_cut_sequences(lens, recurrent):
    """The last segment's final state takes the initial state's place, which the first segment reads:
    with many heads, so that segments of one sequence run at different times."""
    c = make(lens, H=24, H_k=1, d_k=32, d_v=32, decay=0.01, seed=6)
    want = run({**c, "init_state": c["init_state"].clone()}, out_dtype=F32, recurrent=recurrent, final_state=None)
    got = run(c, out_dtype=F32, recurrent=recurrent, final_state=c["init_state"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_forgetting_and_nan():
    lens = [300]
    c = make(lens, H=2, seed=3)
    for t in (5, 6, 31, 32, 127, 128, 200, 201, 202):
        c["log_decay"][t, 0] = -float("inf")
    _check(c, lens, out_dtype=F32)
    c["log_decay"][150, 1] = float("nan")
    out, fin = run(c, out_dtype=F32)
    nan = torch.isnan(out)
    assert nan[150:, 1].all() and not nan[:150].any() and not nan[:, 0].any()
    assert torch.isnan(fin[0, 1]).all() and not torch.isnan(fin[0, 0]).any()


@pytest.mark.parametrize("decay", [-float("inf"), -90.0, -12.0])
def test_accuracy_behind_many_forgetting_tokens(decay):
    """Runs of tokens that forget all or most, which end inside a block: what follows is as exact as ever."""
    lens = [500]
    c = make(lens, H=3, seed=17)
    c["log_decay"][10:60, 0] = decay
    c["log_decay"][64:95, 1] = decay
    c["log_decay"][130:447:2, 2] = decay
    _check(c, lens, out_dtype=F32)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_sequences_infinities_stay_there(bad):
    """Tiles reach into the next sequence and behind the last one: nothing of theirs may arrive."""
    lens = [100, 90, 70]
    c = make(lens, H=2, seed=4)
    o, f, mo, mf = reference(c)
    for n in ("q", "k", "v"):
        c[n][100:190] = bad
    pad = {n: torch.cat([c[n], torch.full_like(c[n][:40], bad)]) for n in ("q", "k", "v", "log_decay")}
    out = torch.full((300, 2, 128), 7.0, device="cuda", dtype=F32)
    _, fin = binding.linear_prefill(pad["q"], pad["k"], pad["v"], pad["log_decay"], c["cu_seqlens"], c["init_state"],
                                    out=out)
    binding.check_device_error()
    keep = np.r_[0:100, 190:260]
    fine = 2.0 ** -15 + fp32_factor(130, 128)
    check(out[:260][keep], o[keep], mo[keep], fine, "out")
    check(fin[[0, 2]], f[[0, 2]], mf[[0, 2]], fine, "final")
    assert (out[260:] == 7.0).all()


def test_agrees_with_the_token_kernel_on_a_long_memory():
    lens = [5000]
    c = make(lens, H=4, H_k=1, decay=1e-3, per_token=False, seed=8)
    o, f = run(c, recurrent=True)
    _, _, mo, mf = reference(c)
    out, fin = run(c, out_dtype=F32)
    fine = 2.0 ** -15 + 2 * fp32_factor(5000, 128)
    check(out, o.double().cpu().numpy(), mo, fine, "out")
    check(fin, f.double().cpu().numpy(), mf, fine, "final")


def test_prompt_of_the_packed_layer_then_block_norm_and_tokens():
    """The operators together: a packed prompt, its output through the block norm, then tokens."""
    lens = [130, 61]
    c = make(lens, H=4, H_k=2, d_v=64, seed=12)
    out, state = run(c, out_dtype=B16)
    x = torch.randn(sum(lens), 4 * 64, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x2, h = binding.block_norm(x, out.reshape(sum(lens), -1), post_norm=True, scale=0.5, out_dtype=B16)
    want = x.double() + 0.5 * out.reshape(sum(lens), -1).double() * torch.rsqrt(
        out.reshape(sum(lens), -1).double().square().mean(-1, keepdim=True) + 1e-6)
    assert torch.allclose(x2.double(), want, rtol=1e-5, atol=1e-5)
    n = make([1, 1], H=4, H_k=2, d_v=64, seed=13)
    n["init_state"] = state.clone()
    o, f, mo, mf = reference(n)
    tok = binding.linear_decode(n["q"], n["k"], n["v"], n["log_decay"], state)
    check(tok, o, mo, fp32_factor(1, 128), "token")
    check(state, f, mf, fp32_factor(1, 128), "state")


def test_captured_prefill_replays_on_new_inputs_beside_another():
    """Two captured graphs with a workspace each, replayed on two streams at once."""
    lens = [2600]
    graphs, cases, results = [], [], []
    for i in range(2):
        c = make(lens, H=2, seed=20 + i)
        ws = torch.empty(binding.linear_workspace_size(2600, 1, 2, 128, 128, B16, F32), dtype=torch.uint8, device="cuda")
        out, fin = torch.empty(2600, 2, 128, device="cuda"), torch.empty(1, 2, 128, 128, device="cuda")
        run(c, out=out, final_state=fin, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.linear_prefill(**c, out=out, final_state=fin, workspace=ws)
        graphs.append(g), cases.append((c, ws)), results.append((out, fin))
    refs = []
    for i in range(2):
        new = make(lens, H=2, seed=30 + i)
        for n in ("q", "k", "v", "log_decay", "init_state"):
            cases[i][0][n].copy_(new[n])
        refs.append(reference(new))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    binding.check_device_error()
    fine = 2.0 ** -15 + fp32_factor(128 + 40, 128)
    for (out, fin), (o, f, mo, mf) in zip(results, refs):
        check(out, o, mo, fine, "out")
        check(fin, f, mf, fine, "final")


def test_where_a_nan_goes():
    """One in q stays in its row, one in k reaches its token and later ones, one in v its chunk of 128
    and later ones."""
    lens = [300]
    for name, first, rows in (("q", 150, 1), ("k", 150, 150), ("v", 128, 172)):
        c = make(lens, H=2, H_k=2, seed=21)
        good, _ = run(c, out_dtype=F32)
        c[name][150, 0, 5] = float("nan")
        out, fin = run(c, out_dtype=F32)
        nan = torch.isnan(out).any(-1)
        assert nan[first:first + rows, 0].any() and not nan[:, 1].any()
        assert not nan[:first].any() and not nan[first + rows:].any()
        assert nan[150, 0] and torch.equal(out[:first], good[:first]) and torch.equal(out[:, 1], good[:, 1])
        assert torch.isnan(fin[0, 0]).any() == (name != "q") and not torch.isnan(fin[0, 1]).any()


def test_eager_calls_on_two_streams():
    """Segmented calls that overlap, each with the workspace that its call allocates."""
    lens = [3000]
    cases = [make(lens, H=2, decay=0.01, seed=50 + i) for i in range(4)]
    want = [run(c, out_dtype=F32) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [binding.linear_prefill(**c, out_dtype=F32, stream=streams[i % 2]) for i, c in enumerate(cases)]
    torch.cuda.synchronize()
    binding.check_device_error()
    for (o, f), (wo, wf) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(f, wf)


@pytest.mark.parametrize("recurrent", [False, True])
def test_offsets_past_32_bits(recurrent):
    """140000 tokens x 128 heads x 128 channels: the last sequence is where it belongs."""
    T, H, tail = 140000, 128, 200
    g = torch.Generator("cuda").manual_seed(1)
    q = torch.randn(T, 1, 64, device="cuda", generator=g).to(B16)
    k = (0.1 * torch.randn(T, 1, 64, device="cuda", generator=g)).to(B16)
    v = torch.empty(T, H, 128, device="cuda", dtype=B16).normal_(generator=g)
    ld = -torch.rand(T, H, device="cuda", generator=g)
    cut = T - tail
    # sequences of 400 tokens, then the tail: nothing is cut, so a sequence does not depend on its place
    ends = list(range(0, cut, 400)) + [cut, T]
    cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out, _ = binding.linear_prefill(q, k, v, ld, cu, out_dtype=B16, want_final=False, workspace=None, recurrent=recurrent)
    one = torch.tensor([0, tail], dtype=torch.int32, device="cuda")
    want, _ = binding.linear_prefill(q[cut:].contiguous(), k[cut:].contiguous(), v[cut:].contiguous(),
                                     ld[cut:].contiguous(), one, out_dtype=B16, want_final=False, workspace=None,
                                     recurrent=recurrent)
    binding.check_device_error()
    assert torch.equal(out[cut:], want)


@pytest.mark.parametrize("recurrent", [False, True])
def test_thousand_sequences_and_a_long_one(recurrent):
    """1201 sequences, empty ones among them, of which one is cut: the pieces are found among them all."""
    lens = [0] * 400 + [40] * 500 + [2000] + [45] * 300
    c = make(lens, H=2, H_k=1, d_k=72, d_v=72, decay=0.02, seed=9)
    assert binding.linear_workspace_size(sum(lens), len(lens), 2, 72, 72, B16, F32, recurrent, H_k=1) > 0
    _check(c, lens, out_dtype=F32, recurrent=recurrent)
