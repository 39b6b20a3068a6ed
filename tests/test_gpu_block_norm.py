"""kda_block_norm against the fp64 oracle.

Bounds, relative to the fp32 steps of one channel. n: y w rstd, the mean of D squares is off by at
most (D / 8 + 16) roundings of 2^-24 however it is summed here (each thread's run of at most 32,
then shuffles: fewer), half of that reaches the root; sigmoid about 2^-21; a handful of products:
c_n = 2^-18 covers them for every D. x' = x + s n then errs by at most 2^-24 |x'| + c_n |s n|, and h
by c_n |h| + |w| rstd |dx'|, with the change of rstd from dx' (a mean over the row) below
max |dx'| rstd. Storage in bf16 adds half a step, 2^-8 of the value, and fp32 2^-24."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from linear_cases import f64
from oracle import block_norm

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32
HALF = {B16: 2.0 ** -8, F32: 2.0 ** -24}


def _make(rows, D, x=F32, y=B16, gate="channel", post=True, weights=True, seed=0):
    g = torch.Generator().manual_seed(seed + D)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = dict(x=(3 * rn(rows, D)).to(x), y=None if y is None else rn(rows, D).to(y),
             gate=None if gate is None else rn(*((rows, D) if gate == "channel" else (rows,))).to(y),
             post_norm=post, post_weight=1 + 0.1 * rn(D) if post and weights else None,
             channel_scale=rn(D) if weights and y is not None else None, pre_weight=1 + 0.1 * rn(D) if weights else None)
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in c.items()}


def _check(c, out_dtype=B16, scale=0.7, eps=1e-6, post_eps=None, **kw):
    x2, h = binding.block_norm(**c, scale=scale, eps=eps, post_eps=post_eps, out_dtype=out_dtype, **kw)
    host = {n: t.cpu() if isinstance(t, torch.Tensor) else t for n, t in c.items()}
    rx, rh = block_norm(**host, scale=scale, eps=eps, post_eps=post_eps)
    sn = np.abs(rx - f64(c["x"]))
    dx = 2.0 ** -24 * np.abs(rx) + 2.0 ** -18 * sn
    gain = np.abs(rh) / np.maximum(np.abs(rx), 1e-300)  # |w| rstd per channel
    rstd = 1 / np.sqrt((rx * rx).mean(-1, keepdims=True) + eps)
    dh = 2.0 ** -18 * np.abs(rh) + gain * dx + np.abs(rh) * rstd * dx.max(-1, keepdims=True)
    assert x2.dtype == c["x"].dtype and h.dtype == out_dtype
    assert np.all(np.abs(f64(x2) - rx) <= dx + HALF[x2.dtype] * np.abs(rx) + 1e-37)
    bad = np.abs(f64(h) - rh) > dh + HALF[out_dtype] * np.abs(rh) + 1e-37
    assert not bad.any(), (int(bad.sum()), float(np.abs(f64(h) - rh).max()))
    return x2, h


@pytest.mark.parametrize("D", [1, 7, 8, 31, 64, 255, 256, 257, 264, 511, 512, 1000, 1001, 1024, 1025, 1032, 4096, 7168,
                               8184, 8192, 8193, 8200, 16384, 16383])
@pytest.mark.parametrize("rows", [1, 5])
def test_row_lengths(D, rows):
    _check(_make(rows, D))


@pytest.mark.parametrize("rows", [153, 400])
@pytest.mark.parametrize("D", [40, 1001, 2048, 7168])
def test_many_rows(rows, D):
    _check(_make(rows, D))


@pytest.mark.parametrize("rows", [1, 2, 3, 33, 6000])
@pytest.mark.parametrize("D", [1, 9, 63, 64, 65, 120, 127, 128, 129])
def test_several_rows_per_warp(rows, D):
    """8, 16 and 32 lanes a row; rows past the last one in a warp, more rows than one pass takes."""
    _check(_make(rows, D, x=B16))
    _check(_make(rows, D, y=F32, gate="row"), out_dtype=F32)


@pytest.mark.parametrize("x", [F32, B16])
@pytest.mark.parametrize("y", [F32, B16])
@pytest.mark.parametrize("out", [F32, B16])
def test_types(x, y, out):
    for D in (72, 1100, 75):
        _check(_make(4, D, x=x, y=y), out_dtype=out)


@pytest.mark.parametrize("gate", ["channel", "row", None])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("weights", [True, False])
def test_options(gate, post, weights):
    for D in (96, 1025, 3000):
        _check(_make(3, D, gate=gate, post=post, weights=weights), scale=-1.5, eps=1e-3, post_eps=0.1)


def test_norm_before_alone():
    for D in (96, 1025, 3000):
        c = _make(3, D, y=None, gate=None, post=False)
        x2, h = _check(c)
        assert x2 is c["x"]


def test_parts():
    c = _make(6, 512)
    x2, h = binding.block_norm(**c)
    a, none = binding.block_norm(**{**c, "pre_weight": None}, want_out=False)
    assert none is None and torch.equal(a, x2)
    none, b = binding.block_norm(**c, want_residual=False)
    assert none is None and torch.equal(b, h)
    inplace = c["x"].clone()
    r, hh = binding.block_norm(**{**c, "x": inplace}, residual_out=inplace)
    assert r is inplace and torch.equal(inplace, x2) and torch.equal(hh, h)


def test_saturated_gates_infinities_and_zero_rows():
    c = _make(4, 64, y=F32)
    c["gate"][0] = -1e30
    c["gate"][1] = 1e30
    c["gate"][2] = float("-inf")
    x2, h = binding.block_norm(**c, scale=1.0)
    assert torch.equal(x2[0], c["x"][0]) and torch.equal(x2[2], c["x"][2])
    want, _ = block_norm(**{n: t.cpu() if isinstance(t, torch.Tensor) else t for n, t in c.items() if n != "gate"})
    assert np.allclose(f64(x2[1]), want[1], rtol=1e-5, atol=1e-6)
    c = _make(3, 64, y=F32)
    c["x"][1], c["y"][1] = 0.0, 0.0
    c["y"][2, 5] = float("nan")
    x2, h = binding.block_norm(**c)
    assert (h[1] == 0).all() and (x2[1] == 0).all()
    assert torch.isnan(h[2]).all() and not torch.isnan(h[:2]).any()


def test_empty_and_neighbouring_rows_untouched():
    c = _make(0, 64)
    x2, h = binding.block_norm(**c)
    assert x2.shape == (0, 64) and h.shape == (0, 64)
    for D in (64, 65):
        c = _make(3, D)
        out = torch.full((8, D), 3.0, device="cuda", dtype=B16)
        res = torch.full((8, D), 3.0, device="cuda")
        binding.block_norm(**c, out=out[:3], residual_out=res[:3])
        assert (out[3:] == 3).all() and (res[3:] == 3).all()


def test_offsets_past_32_bits():
    """300001 rows of 7200 channels, and 2400001 of 901: the last row is where it belongs."""
    for rows, D in ((300001, 7200), (2400001, 901)):
        x = torch.zeros(rows, D, device="cuda", dtype=B16)
        y = torch.zeros(rows, D, device="cuda", dtype=B16)
        x[-1].normal_(), y[-1].normal_()
        r, h = binding.block_norm(x, y, post_norm=True)
        r1, h1 = binding.block_norm(x[-1:].clone(), y[-1:].clone(), post_norm=True)
        assert torch.equal(r[-1:], r1) and torch.equal(h[-1:], h1)
        assert not r[:-1].any() and not h[:-1].any()
        del x, y, r, h


@pytest.mark.parametrize("D", [64, 777, 2048, 7168, 12288])
@pytest.mark.parametrize("size", [1e17 / 6, 1e-18])
def test_rows_of_the_largest_and_smallest_values(D, size):
    """Squares stay within fp32: 16384 x (10^17)^2 = 1.6 x 10^38, and those of 10^-18 are normal numbers."""
    for c in (_make(3, D, x=F32, y=F32), _make(3, D, x=F32, y=F32, post=False, weights=False)):
        c["x"], c["y"] = (size / 3 * c["x"]).clamp(-1e17, 1e17), (size * c["y"]).clamp(-1e17, 1e17)
        if not c["post_norm"]:
            c["y"] = c["y"] / 3
        _check(c, eps=0.0, out_dtype=F32)
