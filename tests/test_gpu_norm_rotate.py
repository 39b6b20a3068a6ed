"""kda_norm_rotate against the fp64 oracle.

Bounds, relative to the pair's magnitude m = |n_a| + |n_b| (n the normed channels): an angle is off by
2^-32 of a turn and the conversion to fp32 (2^-25 of half a turn, pi 2^-25 < 2^-23) with fp64's 2^-53
of position * inv_freq before, sine and cosine by two ulps (2^-22); the products, their sum, the
weights and the norm's factor round eight times more, the sum of squares d / 2 + 8 times at most (half
of it counts, under the root): (2^-23 + 2^-22 + (8 + d / 4) 2^-24) m + 2^-52 |position inv_freq| m."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from oracle import norm_rotate

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


def _inputs(T, Hq, Hk, d, rot, dtype=B16, axes=1, far=100, seed=0, fused=False, pos_dtype=torch.int64, weights=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    if fused:
        rows = rn(T, (Hq + 2 * Hk) * d).to(dtype).cuda()
        q, k = rows[:, :Hq * d].view(T, Hq, d), rows[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    else:
        q, k = rn(T, Hq, d).to(dtype).cuda(), (rn(T, Hk, d).to(dtype).cuda() if Hk else None)
    pos = torch.randint(0, far, (axes, T) if axes > 1 else (T,), generator=g).to(pos_dtype).cuda()
    f = torch.exp(-torch.arange(rot // 2) * (9.0 / max(1, rot // 2))).cuda() if rot else None
    axis = [i % axes for i in range(rot // 2)] if axes > 1 else None
    w = [(1 + 0.1 * rn(d)).cuda() if weights else None for _ in range(2)]
    return q, k, pos if rot else None, f, axis, w


def _compare(got, x, pos, f, axis, w, norm, interleaved, eps):
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    kw = dict(norm=norm, weight=cpu(w), eps=eps)
    want = norm_rotate(cpu(x), cpu(pos), cpu(f), interleaved=interleaved, pair_axis=axis, **kw)
    n = np.abs(norm_rotate(cpu(x), None, None, **kw))
    m, d = n.copy(), x.shape[2]
    far = np.zeros(x.shape[0])
    if f is not None:
        half = f.shape[0]
        a = np.arange(half) * 2 if interleaved else np.arange(half)
        b = a + 1 if interleaved else a + half
        m[..., a] = m[..., b] = n[..., a] + n[..., b]
        far = np.abs(pos.cpu().double().numpy()).reshape(-1, x.shape[0]).max(0) * float(f.abs().max())
    rel = 2.0 ** -23 + 2.0 ** -22 + (8 + d / 4) * 2.0 ** -24 + 2.0 ** -52 * far
    bound = m * rel[:, None, None] + np.abs(want) * (torch.finfo(got.dtype).eps / 2 if got.dtype == B16 else 0)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound + 1e-37).all(), float((err / (bound + 1e-30)).max())


def _check(T, Hq, Hk, d, rot, norm="rms", interleaved=False, out_dtype=None, eps=1e-6, **kw):
    q, k, pos, f, axis, w = _inputs(T, Hq, Hk, d, rot, weights=norm == "rms", **kw)
    qo, ko = binding.norm_rotate(q, k, pos, f, norm=norm, q_weight=w[0], k_weight=w[1] if Hk else None, eps=eps,
                                 interleaved=interleaved, pair_axis=axis, out_dtype=out_dtype)
    assert qo.dtype == (out_dtype or q.dtype) and qo.shape == q.shape and (ko is None) == (k is None)
    for got, x, weight in ((qo, q, w[0]), (ko, k, w[1])):
        if x is not None:
            _compare(got, x, pos, f, axis, weight, norm, interleaved, eps)


SIZES = [(128, 128), (128, 32), (64, 64), (256, 256), (72, 72), (96, 48), (80, 20), (8, 8), (16, 2), (200, 104), (248, 124),
         (1, 0), (2, 2), (3, 2), (5, 4), (63, 62), (100, 36), (127, 126), (255, 254), (128, 0), (250, 250)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", ["rms", "l2", None])
@pytest.mark.parametrize("d,rot", SIZES)
def test_head_sizes(d, rot, norm, interleaved):
    _check(5, 3, 2, d, rot, norm=norm, interleaved=interleaved, seed=d)


@pytest.mark.parametrize("dtype,out_dtype", [(B16, B16), (B16, F32), (F32, B16), (F32, F32)])
@pytest.mark.parametrize("d,rot", [(128, 128), (72, 40), (33, 20)])
def test_types(d, rot, dtype, out_dtype):
    for interleaved in (False, True):
        _check(9, 4, 1, d, rot, dtype=dtype, out_dtype=out_dtype, interleaved=interleaved)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 0), (1, 96, 96), (1, 224, 32), (3, 1, 1), (700, 8, 2), (5000, 2, 1), (2, 300, 3)])
@pytest.mark.parametrize("d,rot", [(128, 64), (60, 60)])
def test_tokens_and_heads(T, Hq, Hk, d, rot):
    _check(T, Hq, Hk, d, rot, seed=T)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("d,rot", [(128, 128), (72, 60), (30, 30)])
def test_axes(axes, d, rot):
    for interleaved in (False, True):
        _check(40, 4, 2, d, rot, axes=axes, far=3000, interleaved=interleaved, pos_dtype=torch.int32, fused=True)


@pytest.mark.parametrize("d,rot", [(128, 128), (36, 20)])
def test_far_and_negative_positions(d, rot):
    q, k, _, f, _, w = _inputs(7, 2, 2, d, rot, dtype=F32)
    for pos in ([0, 1, -1, (1 << 22) + 1, -(1 << 22), (1 << 31) + 5, 1 << 40], [-(1 << 31), 2 ** 31 - 1, 3, -7, 1 << 24, 16777217, 9]):
        for dt in (torch.int64, torch.int32):
            p = torch.tensor([x if dt == torch.int64 else max(-2 ** 31, min(2 ** 31 - 1, x)) for x in pos], dtype=dt, device="cuda")
            qo, ko = binding.norm_rotate(q, k, p, f, q_weight=w[0], k_weight=w[1])
            _compare(qo, q, p, f, None, w[0], "rms", False, 1e-6)
            _compare(ko, k, p, f, None, w[1], "rms", False, 1e-6)


@pytest.mark.parametrize("d,rot", [(128, 128), (64, 24), (30, 20), (72, 72)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_in_a_fused_projection(d, rot, interleaved):
    """q and k are turned where they are; the values between them, and rows of other tokens, stay."""
    q, k, pos, f, _, w = _inputs(33, 5, 2, d, rot, fused=True, seed=3)
    rows = q._base
    was = rows.clone()
    want = binding.norm_rotate(q, k, pos, f, q_weight=w[0], k_weight=w[1], interleaved=interleaved)
    qo, ko = binding.norm_rotate(q, k, pos, f, q_weight=w[0], k_weight=w[1], interleaved=interleaved, q_out=q, k_out=k)
    assert qo is q and ko is k and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(rows[:, 7 * d:], was[:, 7 * d:]) and not torch.equal(rows[:, :7 * d], was[:, :7 * d])


@pytest.mark.parametrize("dtype,out_dtype", [(B16, B16), (F32, F32), (B16, F32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 20), (128, 6), (72, 70), (200, 106), (24, 22), (256, 252), (40, 2)])
def test_pieces_that_turn_in_part(d, rot, interleaved, dtype, out_dtype):
    """rot is no multiple of 8, so that a piece of 8 channels turns in part; also in place, and beside an infinity
    in the first channel that does not turn."""
    for T, H in ((70, 3), (3, 40)):
        _check(T, H, 2, d, rot, "rms", interleaved, dtype=dtype, out_dtype=out_dtype)
    q, k, pos, f, _, w = _inputs(37, 5, 2, d, rot, dtype=dtype, seed=3)
    q[4, 1, rot] = float("inf")
    want, _ = binding.norm_rotate(q, k, pos, f, norm=None, interleaved=interleaved)
    assert want[4, 1, rot] == float("inf") and int((~torch.isfinite(want)).sum()) == 1
    qo, _ = binding.norm_rotate(q, k, pos, f, norm=None, interleaved=interleaved, q_out=q)
    assert qo is q and torch.equal(q, want)


def test_views_off_16_byte_boundaries():
    flat = torch.randn(4 * 3 * 64 + 3, device="cuda").to(B16)
    pos, f = torch.arange(4, device="cuda"), torch.rand(32, device="cuda")
    for off in (0, 1, 3):
        q = flat[off:off + 768].view(4, 3, 64)
        out = torch.full((4 * 3 * 64 + 8,), 7.0, device="cuda", dtype=B16)
        qo = out[off:off + 768].view(4, 3, 64)
        binding.norm_rotate(q, None, pos, f, norm="l2", q_out=qo)
        _compare(qo, q, pos, f, None, None, "l2", False, 1e-6)
        assert (out[:off] == 7).all() and (out[off + 768:] == 7).all()
    # tokens an odd number of elements apart
    q = torch.randn(6, 200, device="cuda")[:, 3:195].view(6, 3, 64)
    qo, _ = binding.norm_rotate(q, None, torch.arange(6, device="cuda"), f)
    _compare(qo, q, torch.arange(6), f, None, None, "rms", False, 1e-6)


def test_nan_infinity_and_zero_rows_keep_to_themselves():
    for d, rot in ((128, 64), (33, 20)):
        q = torch.randn(4, 3, d, device="cuda")
        pos, f = torch.arange(4, device="cuda"), torch.rand(rot // 2, device="cuda")
        want, _ = binding.norm_rotate(q, None, pos, f, norm=None)
        q[1, 1, 2], q[2, 0, d - 1], q[3, 2] = float("nan"), float("inf"), 0.0
        out, _ = binding.norm_rotate(q, None, pos, f, norm=None)
        same = torch.ones_like(out, dtype=torch.bool)
        same[1, 1, 2] = same[1, 1, 2 + rot // 2] = same[2, 0, d - 1] = False
        same[3, 2] = False
        assert torch.equal(out[same], want[same]) and out[2, 0, d - 1] == float("inf")
        assert torch.isnan(out[1, 1, 2]) and torch.isnan(out[1, 1, 2 + rot // 2]) and (out[3, 2] == 0).all()
        out, _ = binding.norm_rotate(q, None, pos, f, norm="rms")
        assert torch.isnan(out[1, 1]).all() and (out[3, 2] == 0).all() and torch.isfinite(out[0]).all()
        out, _ = binding.norm_rotate(q, None, pos, f, norm="l2", eps=0.0)
        assert torch.isnan(out[3, 2]).all() and torch.isfinite(out[0]).all()
    f[1] = float("inf")  # its pair alone
    out, _ = binding.norm_rotate(q[:1], None, pos[:1], f, norm=None)
    assert torch.isnan(out[0, :, 1]).all() and torch.isfinite(out[0, :, 2]).all()


def test_captured_and_replayed():
    q, k, pos, f, _, w = _inputs(3, 8, 2, 128, 64)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    call = lambda: binding.norm_rotate(q, k, pos, f, q_weight=w[0], k_weight=w[1], q_out=qo, k_out=ko)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    pos += 1
    graph.replay()
    torch.cuda.synchronize()
    got = qo.clone()
    call()
    assert torch.equal(got, qo)
