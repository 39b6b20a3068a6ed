"""The transition maps of a cut sequence on the token kernel: M has d_k columns, padded to a multiple of 8, and
all of them enter the joining of the segments, whatever d_v is and however few columns a CTA has."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from delta_cases import f64, make, reference, run

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T,d_k,d_v,H,dtype", [
    (1600, 100, 100, 1, F32), (1891, 100, 100, 1, F32), (1600, 60, 60, 1, F32), (1891, 60, 60, 1, F32), (1700, 33, 33, 1, F32),
    (1600, 65, 65, 1, F32), (1891, 65, 66, 1, F32), (1600, 20, 20, 1, F32), (2500, 25, 25, 1, F32), (1700, 9, 10, 1, F32),
    (1600, 3, 3, 1, F32), (1600, 1, 1, 1, F32), (1777, 97, 98, 1, F32), (1800, 12, 12, 4, B16), (1700, 9, 11, 2, B16)])
def test_every_column_of_the_maps(T, d_k, d_v, H, dtype):
    """d_k <= d_v with fewer columns of d_v, in whole CTAs, than M has, and a workspace full of NaN: what the maps'
    pass leaves unwritten would reach the outputs from the third segment on. Roundings of 2^-24 with random
    signs, 2^-24 / sqrt(6) in the mean: a block of four tokens makes five of the state, which remembers some 100
    blocks at a decay of 0.003, sqrt(500) 2^-24 / sqrt(6) = 6e-7, and 8e-7 with the maps' own."""
    c = make([T], H=H, d_k=d_k, d_v=d_v, dtype=dtype, decay=0.003, seed=T + d_k)
    n = binding.delta_workspace_size(T, 1, H, d_k, d_v, dtype, F32)
    assert n > 0  # cut
    o, f = reference(c)
    ws = torch.full((n // 4,), float("nan"), device="cuda").view(torch.uint8)
    out, fin = run(c, workspace=ws)
    for got, want in ((out, o), (fin, f)):
        assert bool(torch.isfinite(got).all())
        err = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
        assert err < 1e-6, err
    zero, end = run(c, workspace=torch.zeros_like(ws))  # nothing depends on what the workspace held
    assert torch.equal(out, zero) and torch.equal(fin, end)
