"""Refusals of the linear-attention and block-norm entry points, on the host with fake addresses
(validation comes before any CUDA call), and of their binding, and the segment slots' arithmetic."""

import ctypes

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding as B
from linear_cases import make

INV, UNS = B.KDA_ERR_INVALID_ARG, B.KDA_ERR_UNSUPPORTED


def _prefill(**over):
    f = dict(struct_size=ctypes.sizeof(B.LinearPrefillParams), in_dtype=1, out_dtype=0, num_seqs=1, H=4, H_k=2, d_k=128,
             d_v=128, decay_per_token=1, force_recurrent=0, total_tokens=4, q=0x100000, k=0x200000, v=0x300000,
             log_decay=0x400000, cu_seqlens=0x500000, init_state=None, out=0x600000, final_state=0x700000,
             workspace=None, workspace_bytes=0, scale=1.0)
    f.update(over)
    return B.lib().kda_linear_prefill(ctypes.byref(B.LinearPrefillParams(**f)), None)


@pytest.mark.parametrize("over,expect", [
    (dict(struct_size=8), INV), (dict(in_dtype=2), INV), (dict(out_dtype=-1), INV), (dict(H=0), INV), (dict(H_k=0), INV),
    (dict(H_k=3), INV), (dict(H_k=8), INV), (dict(d_k=0), INV), (dict(d_v=129), UNS), (dict(d_k=129), UNS),
    (dict(num_seqs=-1), INV), (dict(num_seqs=0), INV), (dict(total_tokens=-1), INV), (dict(total_tokens=1 << 31), UNS),
    (dict(num_seqs=1 << 29), UNS), (dict(decay_per_token=2), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(log_decay=None), INV), (dict(cu_seqlens=None), INV), (dict(out=None), INV),
    (dict(q=0x100008), INV), (dict(out=0x600004), INV), (dict(final_state=0x700008), INV), (dict(init_state=0x800004), INV),
    (dict(log_decay=0x400002), INV), (dict(cu_seqlens=0x500001), INV),
    (dict(out=0x200000), INV), (dict(final_state=0x300000), INV), (dict(final_state=0x600000), INV),
    (dict(init_state=0x700000 + 4096), INV), (dict(out=0x500000), INV),
    (dict(workspace=0x900000), INV), (dict(workspace_bytes=64), INV), (dict(workspace=0x900008, workspace_bytes=64), INV),
    (dict(workspace=0x600000, workspace_bytes=64), INV), (dict(workspace=0x500000 - 16, workspace_bytes=32), INV),
])
def test_prefill_rejects(over, expect):
    assert _prefill(**over) == expect


def test_empty_work_needs_no_gpu():
    assert _prefill(num_seqs=0, total_tokens=0, q=None, k=None, v=None, log_decay=None, out=None, final_state=None) == B.KDA_OK
    assert _prefill(num_seqs=3, total_tokens=0, q=None, k=None, v=None, log_decay=None, out=None, final_state=None) == B.KDA_OK
    assert B.lib().kda_linear_prefill(None, None) == INV and B.lib().kda_linear_decode(None, None) == INV
    assert B.lib().kda_block_norm(None, None) == INV
    assert _norm(rows=0, x=None, y=None, gate=None, residual_out=None, out=None, post_weight=None, channel_scale=None,
                 pre_weight=None, post_norm=0) == B.KDA_OK


def _decode(**over):
    f = dict(struct_size=ctypes.sizeof(B.LinearDecodeParams), in_dtype=1, out_dtype=0, B=2, H=4, H_k=2, d_k=128, d_v=128,
             decay_per_token=1, scale=1.0, q=0x100000, k=0x200000, v=0x300000, log_decay=0x400000, state=0x1000000,
             out=0x600000)
    f.update(over)
    return B.lib().kda_linear_decode(ctypes.byref(B.LinearDecodeParams(**f)), None)


@pytest.mark.parametrize("over,expect", [
    (dict(struct_size=0), INV), (dict(in_dtype=5), INV), (dict(out_dtype=5), INV), (dict(B=0), INV), (dict(H_k=3), INV),
    (dict(d_k=200), UNS), (dict(d_v=0), INV), (dict(decay_per_token=-1), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(log_decay=None), INV), (dict(state=None), INV), (dict(out=None), INV),
    (dict(state=0x1000004), INV), (dict(q=0x100002), INV), (dict(state=0x300000), INV), (dict(out=0x400000), INV),
    (dict(out=0x1000000 + 65536), INV), (dict(B=1 << 30), UNS),
])
def test_decode_rejects(over, expect):
    assert _decode(**over) == expect


def _norm(**over):
    f = dict(struct_size=ctypes.sizeof(B.BlockNormParams), x_dtype=0, y_dtype=1, out_dtype=1, gate_form=1, post_norm=1,
             D=64, scale=1.0, rows=4, x=0x100000, y=0x200000, gate=0x300000, post_weight=0x400000, channel_scale=0x500000,
             pre_weight=0x600000, residual_out=0x700000, out=0x800000, post_eps=1e-6, pre_eps=1e-6)
    f.update(over)
    return B.lib().kda_block_norm(ctypes.byref(B.BlockNormParams(**f)), None)


@pytest.mark.parametrize("over,expect", [
    (dict(struct_size=1), INV), (dict(x_dtype=2), INV), (dict(y_dtype=2), INV), (dict(out_dtype=2), INV),
    (dict(gate_form=3), INV), (dict(gate_form=0), INV), (dict(gate=None), INV), (dict(post_norm=2), INV),
    (dict(post_norm=0), INV), (dict(D=0), INV), (dict(D=16385), UNS), (dict(rows=-1), INV), (dict(rows=1 << 31), UNS),
    (dict(x=None), INV), (dict(y=None), INV), (dict(out=None), INV), (dict(out=None, pre_weight=None, residual_out=None), INV),
    (dict(x=0x100004), INV), (dict(pre_weight=0x600004), INV), (dict(gate=0x300002), INV),
    (dict(residual_out=0x100000 + 64), INV), (dict(out=0x100000), INV), (dict(out=0x200000), INV),
    (dict(out=0x700000), INV), (dict(residual_out=0x600000), INV),
    (dict(pre_eps=-1.0), INV), (dict(post_eps=float("nan")), INV), (dict(pre_eps=float("inf")), INV),
])
def test_block_norm_rejects(over, expect):
    assert _norm(**over) == expect


def test_binding_refuses():
    c = make([5, 2], H=4, H_k=2, d_k=16, d_v=8, device="cpu")
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        B.linear_prefill(**c)
    with pytest.raises(ValueError, match=r"\[T, H_k, d_k\]"):
        B.linear_prefill(**{**c, "k": c["k"][:, :, :8]})
    with pytest.raises(ValueError, match="multiple"):
        B.linear_prefill(**{**c, "v": c["v"][:, :3]})
    with pytest.raises(TypeError, match="one dtype"):
        B.linear_prefill(**{**c, "v": c["v"].float()})
    with pytest.raises(TypeError, match="log_decay"):
        B.linear_prefill(**{**c, "log_decay": c["log_decay"].double()})
    with pytest.raises(ValueError, match="log_decay"):
        B.linear_prefill(**{**c, "log_decay": c["log_decay"][:, :2]})
    with pytest.raises(TypeError, match="cu_seqlens"):
        B.linear_prefill(**{**c, "cu_seqlens": c["cu_seqlens"].long()})
    st = torch.zeros(7, 4, 16, 8)
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        B.linear_decode(c["q"], c["k"], c["v"], c["log_decay"], st)
    x = torch.zeros(3, 8)
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        B.block_norm(x, x)
    with pytest.raises(ValueError, match=r"\[rows, D\]"):
        B.block_norm(x, x[:2])
    with pytest.raises(ValueError, match="belong to y"):
        B.block_norm(x, gate=x)
    with pytest.raises(ValueError, match="belong to y"):
        B.block_norm(x, post_norm=True)
    with pytest.raises(TypeError, match="gate"):
        B.block_norm(x, x, gate=x.bfloat16())
    with pytest.raises(ValueError, match="gate must be"):
        B.block_norm(x, x, gate=x[:, :4])
    with pytest.raises(ValueError, match="weight"):
        B.block_norm(x, x, pre_weight=torch.zeros(7))
    with pytest.raises(TypeError, match="weight"):
        B.block_norm(x, x, pre_weight=torch.zeros(8).double())


def _piece(cu, L, index):
    """The kernels' way from a piece to (sequence, place, first token, end, first, last), or None if
    idle: pieces below total // L find a segment that has a successor, the others last segments."""
    inner = cu[-1] // L
    if index >= inner:
        n = index - inner
        j = 0 if cu[n + 1] == cu[n] else (cu[n + 1] - cu[n] - 1) // L
        return n, cu[n] // L + n + j, cu[n] + j * L, cu[n + 1], j == 0, True
    mark = (index + 1) * L
    n = max(m for m in range(len(cu) - 1) if cu[m] < mark)
    j = index - cu[n] // L
    t0 = cu[n] + j * L
    return (n, cu[n] // L + n + j, t0, t0 + L, j == 0, False) if t0 + L < cu[n + 1] else None


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("L", [16, 64, 128, 1000])
def test_pieces_cover_every_token_once(seed, L):
    r = np.random.default_rng(seed)
    lens = [int(x) for x in r.integers(0, [3, 40, 300, 5000][seed % 4], size=1 + seed * 3)]
    if seed == 3:
        lens = [0, 0, L, 0, 2 * L, L - 1, 1, L + 1, 0]
    cu = [0] + [int(x) for x in np.cumsum(lens)]
    got = [_piece(cu, L, i) for i in range(cu[-1] // L + len(lens))]
    got = [g for g in got if g is not None]
    places = [g[1] for g in got]
    assert len(set(places)) == len(places) and max(places) < cu[-1] // L + len(lens)
    for n, length in enumerate(lens):
        mine = sorted((g for g in got if g[0] == n), key=lambda g: g[2])
        assert len(mine) == max(1, -(-length // L))
        assert [g[1] for g in mine] == list(range(mine[0][1], mine[0][1] + len(mine)))
        assert [g[4] for g in mine] == [True] + [False] * (len(mine) - 1)
        assert [g[5] for g in mine] == [False] * (len(mine) - 1) + [True]
        edge = cu[n]
        for _, _, a, b, _, _ in mine:
            assert a == edge
            edge = b
        assert edge == cu[n + 1]


def test_workspace_query():
    q = B.lib().kda_linear_prefill_workspace_size
    for args in [(4096, 1, 96, 96, 128, 128, 1, 1, 0), (65536, 1, 16, 4, 128, 128, 1, 1, 0),
                 (1000, 7, 2, 1, 100, 72, 0, 0, 0), (50, 1, 4, 2, 13, 7, 1, 1, 0)]:
        assert q(*args) == q(*args) and q(*args) % 256 == 0
    assert q(65536, 1, 16, 4, 128, 128, 1, 1, 0) > 0
    # bf16 head sizes that are no multiple of 8: q and k [128, 2, 16], v and out [128, 4, 8], the states
    # [1, 4, 13, 8] in fp32, each rounded up to 256 bytes; nothing for
    # the token-recurrent kernel, which also runs short sequences
    assert q(128, 1, 4, 2, 13, 7, 1, 1, 0) == 2 * 8192 + 2 * 8192 + 1792
    assert q(128, 1, 4, 2, 13, 7, 1, 0, 0) == 2 * 8192 + 8192 + 16384 + 1792
    assert q(128, 1, 4, 2, 13, 8, 1, 1, 0) == 2 * 8192 and q(128, 1, 4, 2, 16, 7, 1, 1, 0) == 2 * 8192 + 2048
    assert q(48, 1, 4, 2, 13, 7, 1, 1, 0) == q(48, 1, 4, 2, 13, 7, 1, 1, 1) == q(48, 1, 4, 2, 13, 7, 0, 0, 0) == 0
    # invalid or empty sizes ask for nothing
    for args in [(0, 1, 1, 1, 64, 64, 1, 1, 0), (10, 0, 1, 1, 64, 64, 1, 1, 0), (10, 1, 0, 1, 64, 64, 1, 1, 0),
                 (10, 1, 1, 1, 129, 64, 1, 1, 0), (10, 1, 1, 1, 64, 64, 3, 1, 0), (-5, 1, 1, 1, 64, 64, 1, 1, 0),
                 (10, 1, 4, 3, 64, 64, 1, 1, 0), (2**31 - 1, 1, 2**28, 1, 63, 63, 1, 1, 0)]:
        assert q(*args) == 0


def test_the_most_tokens():
    """2^31 - 128: token indexes rounded up to a chunk of 128 stay below 2^31."""
    most = 2**31 - 128
    for T in (most + 1, 2**31 - 1):
        assert _prefill(total_tokens=T, H=1, H_k=1, d_k=8, d_v=8) == UNS
        assert B.linear_workspace_size(T, 1, 1, 8, 8) == 0
    assert B.linear_workspace_size(most, 1, 1, 8, 8) > 0
    # up to there the plan's segments, and what the kernels form of a length, fit in 32 bits
    seg = -(-(-(-most // 152)) // 128) * 128
    assert (most + 127) // 128 * 128 < 2**31 and (most - 1) // seg + 1 == 152
    # rounding a length up to whole segments would not: that is why the count is formed without it
    assert most + seg - 1 >= 2**31
