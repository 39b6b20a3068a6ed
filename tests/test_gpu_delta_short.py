"""Prompts of a few tokens beside many others, which the decode kernel takes one token after the other,
against the fp64 oracle within the bound of fp32 token by token (delta_cases), and what stands beside them."""

import pytest
import torch

from delta_cases import bounds, check, half_step, make, reference, run

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


def _check(c, out_dtype=F32, scale=1.0, **kw):
    out, fin = run(c, scale=scale, out_dtype=out_dtype, **kw)
    o, f = reference(c, scale)
    bo, bf, _ = bounds(c, scale)
    check(out, o, bo + (half_step(o, B16) if out.dtype == B16 else 0), "out")
    if fin is not None:
        check(fin, f, bf, "final")
    return out, fin


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (B16, B16), (B16, F32), (F32, B16)])
@pytest.mark.parametrize("lens", [[1] * 30, [0, 1, 2, 3, 4, 5] * 4, [5, 0] * 10, [0] * 20 + [1]])
def test_lengths(lens, dtype, out_dtype):
    _check(make(lens, H=16, H_k=4, d_k=24, d_v=20, dtype=dtype, seed=len(lens)), out_dtype, scale=0.3)


@pytest.mark.parametrize("d_k,d_v", [(128, 128), (64, 64), (1, 1), (100, 72), (5, 33), (128, 6), (31, 127), (128, 16)])
@pytest.mark.parametrize("dtype", [F32, B16])
def test_head_sizes(d_k, d_v, dtype):
    _check(make([1, 3, 0, 2] * 3, H=14, d_k=d_k, d_v=d_v, dtype=dtype, seed=d_k + d_v))


@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("decay", [0.0, 0.3, 30.0])
def test_decays(per_token, decay):
    _check(make([4, 5, 1, 2] * 3, H=15, H_k=5, d_k=40, d_v=36, dtype=F32, per_token=per_token, decay=decay))


def test_states():
    c = make([3, 0, 5, 1] * 10, H=5, d_k=32, d_v=24, dtype=F32, init=False)
    _check(c)
    _check(c, want_final=False)
    c = make([3, 0, 5, 1] * 10, H=5, d_k=32, d_v=24, dtype=F32)
    want, end = _check(c)
    state = c["init_state"].clone()
    out, fin = run({**c, "init_state": state}, final_state=state)
    assert fin is state and torch.equal(out, want) and torch.equal(state, end)


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("lens", [[1, 700] + [2] * 60, [6, 5, 13, 12] * 12, [0, 300, 1, 64, 5] * 8])
def test_beside_longer_ones(lens, dtype):
    """Short sequences are as exact as alone, and where the call's mean length lets the decode kernel take them
    (below 64 tokens) they give the same bits."""
    c = make(lens, H=8, H_k=2, d_k=64, d_v=72, dtype=dtype, seed=sum(lens))
    out, fin = run(c)
    short = [i for i, n in enumerate(lens) if n <= 5]
    rows = torch.cat([torch.arange(sum(lens[:i]), sum(lens[:i + 1])) for i in short]).cuda()
    part = {n: c[n][rows].contiguous() for n in ("q", "k", "v", "log_decay", "beta")}
    part["cu_seqlens"] = torch.tensor([0] + [lens[i] for i in short]).cumsum(0).int().cuda()
    part["init_state"] = c["init_state"][short].contiguous()
    got, end = _check(part)
    if len(short) * 8 > 152 and sum(lens) < 64 * len(lens):
        assert torch.equal(out[rows], got) and torch.equal(fin[short], end)
    o, f = reference(c)
    bo, bf, _ = bounds(c)
    bp, bg, _ = bounds(c, pairs=True)
    check(out, o, bo + bp, "out")
    check(fin, f, bf + bg, "final")


@pytest.mark.parametrize("N,H", [(3, 2), (40, 8)])
@pytest.mark.parametrize("init", [True, False])
def test_no_tokens_at_all(N, H, init):
    c = make([0] * N, H=H, d_k=24, d_v=20, dtype=B16, init=init)
    out, fin = run(c)
    assert out.shape == (0, H, 20) and torch.equal(fin, c["init_state"] if init else torch.zeros_like(fin))


def test_rows_behind_and_nan_stay():
    c = make([2, 1, 4] * 20, H=8, d_k=16, d_v=12, dtype=F32)
    T = c["q"].shape[0]
    want, end = run(c)
    wide = {n: torch.cat([c[n], torch.full_like(c[n][:3], float("nan"))]) for n in ("q", "k", "v", "log_decay", "beta")}
    out = torch.full((T + 3, 8, 12), 7.0, device="cuda")
    run({**c, **wide}, out=out)
    assert torch.equal(out[:T], want) and (out[T:] == 7).all()
    c["v"][4, 3, 5] = float("inf")  # the second of the third sequence's tokens 3 to 6
    c["k"][8, 2, 1] = float("nan")  # the last of the fourth's, 7 and 8
    out, fin = run(c)
    bad = ~torch.isfinite(out)
    assert bad[4:7, 3, 5].all() and bad[8, 2].all() and int(bad.sum()) == 3 + 12
    keep = [i for i in range(60) if i not in (2, 3)]
    assert torch.equal(fin[keep], end[keep])


def test_captured_and_replayed():
    c = make([1, 2, 0, 5] * 16, H=8, d_k=64, d_v=64, dtype=B16)
    want, end = run(c)
    out, fin = torch.empty_like(want), torch.empty_like(end)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run(c, out=out, final_state=fin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    from kimi_delta_attention_02_gb300 import binding
    with torch.cuda.graph(graph, stream=s):
        binding.delta_prefill(**c, out=out, final_state=fin)
    for _ in range(2):
        out.fill_(7), fin.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(fin, end)
