"""Refusals of the gated delta rule's and the norm and rotation's entry points, on the host with fake
addresses (validation comes before any CUDA call), and of their binding."""

import ctypes

import pytest
import torch

from kimi_delta_attention_02_gb300 import binding as B
from delta_cases import make

INV, UNS = B.KDA_ERR_INVALID_ARG, B.KDA_ERR_UNSUPPORTED


def _prefill(**over):
    f = dict(struct_size=ctypes.sizeof(B.DeltaPrefillParams), in_dtype=1, out_dtype=0, num_seqs=1, H=4, H_k=2, d_k=128,
             d_v=128, decay_per_token=1, force_recurrent=0, total_tokens=4, q=0x100000, k=0x200000, v=0x300000,
             log_decay=0x400000, beta=0x480000, cu_seqlens=0x500000, init_state=None, out=0x600000, final_state=0x700000,
             workspace=None, workspace_bytes=0, scale=1.0)
    f.update(over)
    return B.lib().kda_delta_prefill(ctypes.byref(B.DeltaPrefillParams(**f)), None)


@pytest.mark.parametrize("over,expect", [
    (dict(struct_size=8), INV), (dict(in_dtype=2), INV), (dict(out_dtype=-1), INV), (dict(H=0), INV), (dict(H_k=0), INV),
    (dict(H_k=3), INV), (dict(H_k=8), INV), (dict(d_k=0), INV), (dict(d_v=129), UNS), (dict(d_k=129), UNS),
    (dict(num_seqs=-1), INV), (dict(num_seqs=0), INV), (dict(total_tokens=-1), INV), (dict(total_tokens=1 << 31), UNS),
    (dict(num_seqs=1 << 29), UNS), (dict(decay_per_token=2), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(log_decay=None), INV), (dict(beta=None), INV), (dict(cu_seqlens=None), INV),
    (dict(out=None), INV), (dict(q=0x100008), INV), (dict(out=0x600004), INV), (dict(final_state=0x700008), INV),
    (dict(init_state=0x800004), INV), (dict(log_decay=0x400002), INV), (dict(beta=0x480002), INV),
    (dict(cu_seqlens=0x500001), INV), (dict(out=0x200000), INV), (dict(final_state=0x300000), INV),
    (dict(final_state=0x600000), INV), (dict(out=0x480000), INV), (dict(final_state=0x480000), INV),
    (dict(init_state=0x700000 + 4096), INV), (dict(out=0x500000), INV),
    (dict(workspace=0x900000), INV), (dict(workspace_bytes=64), INV), (dict(workspace=0x900008, workspace_bytes=64), INV),
    (dict(workspace=0x600000, workspace_bytes=64), INV), (dict(workspace=0x480000, workspace_bytes=32), INV),
])
def test_prefill_rejects(over, expect):
    assert _prefill(**over) == expect


def test_empty_work_needs_no_gpu():
    none = dict(q=None, k=None, v=None, log_decay=None, beta=None, out=None, final_state=None)
    assert _prefill(num_seqs=0, total_tokens=0, **none) == B.KDA_OK
    assert _prefill(num_seqs=3, total_tokens=0, **none) == B.KDA_OK
    assert B.lib().kda_delta_prefill(None, None) == INV and B.lib().kda_delta_decode(None, None) == INV
    assert B.lib().kda_norm_rotate(None, None) == INV
    assert _rotate(tokens=0, q=None, k=None, q_out=None, k_out=None, positions=None, inv_freq=None) == INV  # k without H_k = 0
    assert _rotate(tokens=0, positions=None, inv_freq=None) == B.KDA_OK


def _decode(**over):
    f = dict(struct_size=ctypes.sizeof(B.DeltaDecodeParams), in_dtype=1, out_dtype=0, B=2, H=4, H_k=2, d_k=128, d_v=128,
             decay_per_token=1, scale=1.0, q=0x100000, k=0x200000, v=0x300000, log_decay=0x400000, beta=0x480000,
             state=0x1000000, out=0x600000)
    f.update(over)
    return B.lib().kda_delta_decode(ctypes.byref(B.DeltaDecodeParams(**f)), None)


@pytest.mark.parametrize("over,expect", [
    (dict(struct_size=0), INV), (dict(in_dtype=5), INV), (dict(out_dtype=5), INV), (dict(B=0), INV), (dict(H_k=3), INV),
    (dict(d_k=200), UNS), (dict(d_v=0), INV), (dict(decay_per_token=-1), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(log_decay=None), INV), (dict(beta=None), INV), (dict(state=None), INV), (dict(out=None), INV),
    (dict(state=0x1000004), INV), (dict(q=0x100002), INV), (dict(beta=0x480001), INV), (dict(state=0x300000), INV),
    (dict(out=0x400000), INV), (dict(out=0x480000), INV), (dict(state=0x480000), INV),
    (dict(out=0x1000000 + 65536), INV), (dict(B=1 << 30), UNS),
])
def test_decode_rejects(over, expect):
    assert _decode(**over) == expect


def _rotate(axis=(), **over):
    f = dict(struct_size=ctypes.sizeof(B.NormRotateParams), in_dtype=1, out_dtype=1, norm=1, H_q=4, H_k=2, d=64, rot_dim=32,
             interleaved=0, num_axes=1, position_bytes=8, eps=1e-6, tokens=10, q_stride=256, k_stride=128,
             q_out_stride=256, k_out_stride=128, q=0x100000, k=0x200000, q_weight=0x300000, k_weight=0x310000,
             positions=0x320000, inv_freq=0x330000, q_out=0x400000, k_out=0x500000)
    f.update(over)
    p = B.NormRotateParams(**f)
    for i, x in enumerate(axis):
        p.pair_axis[i] = x
    return B.lib().kda_norm_rotate(ctypes.byref(p), None)


@pytest.mark.parametrize("over,expect", [
    (dict(struct_size=8), INV), (dict(in_dtype=2), INV), (dict(out_dtype=2), INV), (dict(norm=3), INV), (dict(norm=-1), INV),
    (dict(norm=2), INV), (dict(norm=0), INV), (dict(H_q=0), INV), (dict(H_k=-1), INV), (dict(H_k=0), INV), (dict(d=0), INV),
    (dict(d=264, q_stride=2000, k_stride=2000, q_out_stride=2000, k_out_stride=2000), UNS), (dict(rot_dim=-2), INV),
    (dict(rot_dim=3), INV), (dict(rot_dim=66), INV), (dict(interleaved=2), INV), (dict(num_axes=0), INV),
    (dict(num_axes=5), UNS), (dict(position_bytes=2), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(tokens=-1), INV), (dict(tokens=1 << 31), UNS), (dict(q_stride=255), INV), (dict(k_out_stride=127), INV),
    (dict(q_stride=1 << 60), UNS), (dict(q=None), INV), (dict(q_out=None), INV), (dict(k=None), INV), (dict(k_out=None), INV),
    (dict(positions=None), INV), (dict(inv_freq=None), INV), (dict(q=0x100001), INV), (dict(k_out=0x500001), INV),
    (dict(positions=0x320004), INV), (dict(inv_freq=0x330002), INV), (dict(q_weight=0x300002), INV),
    (dict(axis=[0] * 15 + [1]), INV), (dict(num_axes=2, axis=[0, 2]), INV),
    # outputs over inputs, each other and the small tensors
    (dict(q_out=0x100010), INV), (dict(q_out=0x200000), INV), (dict(k_out=0x100000), INV), (dict(k_out=0x400000), INV),
    (dict(q_out=0x300000 - 64), INV), (dict(k_out=0x320000), INV), (dict(q_out=0x330000), INV), (dict(k_out=0x310040), INV),
    # in place with another stride or dtype
    (dict(q_out=0x100000, q_out_stride=512), INV), (dict(q_out=0x100000, out_dtype=0, q_out_stride=256), INV),
    # parts of one buffer of 640-element rows: q and k there, q_out over k's part
    (dict(q=0x100000, q_stride=640, k=0x100000 + 512, k_stride=640, q_out=0x100000 + 256, q_out_stride=640), INV),
    (dict(q=0x100000, q_stride=640, k=0x100000 + 512, k_stride=640, q_out=0x100000 + 1024 - 64, q_out_stride=640), INV),
])
def test_norm_rotate_rejects(over, expect):
    assert _rotate(**over) == expect


def test_norm_rotate_head_counts():
    wide = dict(q_stride=65536 * 64, k_stride=65536 * 64, q_out_stride=65536 * 64, k_out_stride=65536 * 64, d=1, rot_dim=0)
    assert _rotate(**{**wide, "H_q": 65536}) == UNS and _rotate(**{**wide, "H_k": 65536}) == UNS
    assert _rotate(**{**wide, "H_q": 65535, "H_k": 65535, "tokens": 0}) == 0


def test_workspace_sizes():
    size = B.delta_workspace_size
    f32, bf16 = torch.float32, torch.bfloat16
    for T in (1, 63, 380):  # the token kernel
        assert size(T, 1, 8, dtype=f32) == size(T, 1, 8, recurrent=True) == size(T, 1, 8, dtype=f32, d_k=68) == 0
    assert size(100000, 1, 8, recurrent=True) == size(100000, 1, 8, d_k=68, recurrent=True) == size(100000, 2, 8, dtype=f32) == 0
    # .. which cuts one long sequence too, where SMs are idle (in its workspace sizes are padded to multiples of 8)
    n = size(16384, 1, 4, dtype=f32)
    assert n > 0 and n % (4 * 128 * 128 * 8) == 0 and size(4096, 1, 96, dtype=f32) == 0
    n = size(16384, 1, 8, dtype=f32, d_k=68, d_v=5)
    assert n > 0 and n % 256 == 0
    # copies of q and k, of v, or of all, with head sizes padded to multiples of 8; segments behind them
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    assert size(100, 1, 8, d_k=68, H_k=2) == 2 * up(100 * 2 * 72 * 2) and size(100, 1, 8, d_v=5) == up(100 * 8 * 8 * 2)
    assert size(100, 1, 8, d_k=68, d_v=5, H_k=2) == 2 * up(100 * 2 * 72 * 2) + up(100 * 8 * 8 * 2)
    assert size(43, 1, 8, d_k=68) == 0
    cut = size(65536, 1, 16, d_k=128, d_v=120)
    assert size(65536, 1, 16, d_k=128, d_v=117) == cut + 65536 * 16 * 120 * 2
    assert size(0, 0, 8) == size(0, 3, 8) == size(100, 1, 0) == size(-1, 1, 8) == size(100, 1, 8, H_k=3) == 0
    # one long sequence that leaves SMs idle is cut: an end state and a map for each segment
    n = size(65536, 1, 16)
    assert n > 0 and n % (16 * 128 * 128 * 8) == 0
    assert size(65536, 1, 16, d_v=64) == n * 3 // 4
    assert size(65536, 1, 152) == 0 and size(600, 1, 4) == 0
    # more chains than SMs, of lengths that are not known: an order
    assert size(40 * 200, 40, 32) == 256 and size(40 * 60, 40, 3) == 0
    # .. or segments, where the tokens would make long ones and SMs are idle
    assert size(40 * 200, 40, 3) % (3 * 128 * 128 * 8) == 0
    assert size(9000 * 10, 9000, 32) == 0
    # short sequences go to the token kernel, by head sizes
    for n, d_k, d_v in ((6, 128, 128), (16, 64, 128), (24, 128, 64), (44, 64, 64)):
        assert size(40 * n - 1, 40, 32, d_k=d_k, d_v=d_v) == 0 and size(40 * n, 40, 32, d_k=d_k, d_v=d_v) == 256
    for T in (2**31 - 128, 2**30):  # the largest
        for N, H in ((1, 1), (1, 64), (7, 3), (1000, 64)):
            assert size(T, N, H) < 1 << 33
            assert size(T, N, H) == size(T, N, H)


def test_binding_refuses():
    c = make([5, 2], H=4, H_k=2, d_k=16, d_v=8, device="cpu")
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        B.delta_prefill(**c)
    with pytest.raises(ValueError, match="beta"):
        B.delta_prefill(**{**c, "beta": c["beta"][:, :2]})
    with pytest.raises(TypeError, match="beta"):
        B.delta_prefill(**{**c, "beta": c["beta"].double()})
    with pytest.raises(ValueError, match="multiple"):
        B.delta_prefill(**{**c, "v": c["v"][:, :3]})
    with pytest.raises(TypeError, match="one dtype"):
        B.delta_prefill(**{**c, "v": c["v"].float()})
    with pytest.raises(TypeError, match="cu_seqlens"):
        B.delta_prefill(**{**c, "cu_seqlens": c["cu_seqlens"].long()})
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        B.delta_decode(c["q"], c["k"], c["v"], c["log_decay"], c["beta"], torch.zeros(7, 4, 16, 8))
    q, k, pos, f = torch.zeros(3, 4, 8), torch.zeros(3, 2, 8), torch.zeros(3, dtype=torch.int64), torch.ones(4)
    with pytest.raises(ValueError, match="CUDA"):
        B.norm_rotate(q, k, pos, f)
    for bad, error, match in [
            (lambda: B.norm_rotate(q, k[:2], pos, f), ValueError, r"\[T, H_k, d\]"),
            (lambda: B.norm_rotate(q, k.double(), pos, f), TypeError, "one dtype"),
            (lambda: B.norm_rotate(q, k, pos, f, norm="layer"), ValueError, "norm"),
            (lambda: B.norm_rotate(q, k, pos, None), ValueError, "together"),
            (lambda: B.norm_rotate(q, k, pos.float(), f), TypeError, "positions"),
            (lambda: B.norm_rotate(q, k, pos[:2], f), ValueError, "positions"),
            (lambda: B.norm_rotate(q, k, pos[None], f), ValueError, "positions"),
            (lambda: B.norm_rotate(q, k, pos, f.double()), TypeError, "inv_freq"),
            (lambda: B.norm_rotate(q, k, pos, torch.ones(5)), ValueError, "pairs"),
            (lambda: B.norm_rotate(q, k, pos[None], f, pair_axis=[0, 0, 0]), ValueError, "pair_axis"),
            (lambda: B.norm_rotate(q, k, pos[None], f, pair_axis=[0, 0, 0, 1]), ValueError, "axis"),
            (lambda: B.norm_rotate(q, k, pos[None], f, pair_axis=[0, 0, 0, -1]), ValueError, "axis"),
            (lambda: B.norm_rotate(q, k, pos[None], f, pair_axis=[0, 0, 0, 256]), ValueError, "axis"),
            (lambda: B.norm_rotate(q, k, pos, f, q_weight=torch.ones(7)), ValueError, "weight"),
            (lambda: B.norm_rotate(q, None, pos, f, k_weight=torch.ones(8)), ValueError, "belong")]:
        with pytest.raises(error, match=match):
            bad()
