"""kda_norm_rotate at positions as far as 64 bits reach, against the oracle's exact angles.

Bound of an angle: 2^-32 of a turn for the integers, 2^-28 for what fp32 rounds of an eighth of a turn, so
2 pi (2^-28 + 2^-32) < 2^-25 rad; sine and cosine two ulps of at most one, 2^-22. Products, their sum and the final
rounding: 3 roundings of the pair's magnitude m = |a| + |b|. In all (2^-25 + 2^-22 + 3 2^-24) m, whatever the position."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from oracle import norm_rotate

pytestmark = pytest.mark.gpu
FAR = [0, 1, -1, (1 << 31) + 5, -(1 << 33) - 7, (1 << 40) + 12345, -(1 << 45) + 3, (1 << 48) + 1, (1 << 53) + 1, -(1 << 56) - 11,
       1_765_000_000_123_456_789, -(1 << 62) + 1, (1 << 63) - 1, -(1 << 63), -(1 << 63) + 1]


def _check(pos, f, d, interleaved=False, axis=None, dtype=torch.float32):
    T, half = pos.shape[-1], f.shape[0]
    g = torch.Generator().manual_seed(d)
    q = torch.randn(T, 2, d, generator=g).to(dtype).cuda()
    out, _ = binding.norm_rotate(q, None, pos.cuda(), f.cuda(), norm=None, interleaved=interleaved, pair_axis=axis,
                                 out_dtype=torch.float32)
    want = norm_rotate(q.cpu(), pos, f, interleaved=interleaved, pair_axis=axis)
    x = np.abs(q.double().cpu().numpy())
    m = x.copy()
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    m[..., a] = m[..., b] = x[..., a] + x[..., b]
    err = np.abs(out.double().cpu().numpy() - want)
    bound = (2.0 ** -25 + 2.0 ** -22 + 3 * 2.0 ** -24) * m
    assert (err <= bound).all(), (float((err / (m + 1e-30)).max()), np.argwhere(err > bound)[:4].tolist())


@pytest.mark.parametrize("d,half", [(128, 64), (72, 36), (30, 15), (33, 16), (256, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_of_64_bits(d, half, interleaved):
    f = torch.exp(-torch.arange(half) * (14.0 / half))
    _check(torch.tensor(FAR), f, d, interleaved)


@pytest.mark.parametrize("d", [128, 31])
def test_frequencies(d):
    """From denormal ones to 2^24, negative ones among them."""
    half = 15
    f = torch.tensor([1.0, -1.0, 3.14159274, 1e-3, -1e-6, 1e-12, 1e-20, 1e-38, 1e-45, 0.0, 6.2831855, 1e3, 1e6, 16777214.0, -123456.789],
                     dtype=torch.float32)
    assert f.shape[0] == half
    _check(torch.tensor(FAR), f, d)
    small = torch.tensor([0, 1, -1, 2, 12345, -(1 << 31), (1 << 31) - 1], dtype=torch.int32)
    _check(small, f, d)


def test_all_eighths_of_a_turn():
    """Angles on and beside the borders between eighths, where sine and cosine change places."""
    f = torch.full((1,), 0.78539819)  # pi / 4, rounded up by 2^-24.6: position n is n eighths and a little
    f = torch.cat([f, torch.nextafter(f, torch.zeros(1)), -f, 3 * f])
    pos = torch.cat([torch.arange(-20, 21), 8 * torch.arange(100000, 100009), torch.arange(5) + (1 << 50)])
    _check(pos, f, 16)
    _check(pos, f, 9)


def test_far_axes():
    f = torch.exp(-torch.arange(30) * 0.3)
    pos = torch.stack([torch.tensor(FAR), torch.tensor(FAR).flip(0), torch.arange(len(FAR))])
    axis = [i % 3 for i in range(30)]
    _check(pos, f, 72, True, axis, torch.bfloat16)
    _check(pos, f, 61, False, axis)
