"""bf16 outputs of the gated delta rule's tensor-core kernel are off by their own rounding, like the fp32 ones that
they are rounded from: every operand of the read-out is a pair. With one of them a single bf16 they would be off by
0.0023 where keys are random and 0.0065 where keys share a direction, in place of 0.0017."""

import pytest
import torch

from delta_cases import make, reference, run
from delta_precision import check_pairs, off

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("d_k,d_v,H", [(128, 128, 4), (64, 128, 4), (128, 40, 4), (24, 64, 4), (100, 72, 4), (9, 128, 4)])
@pytest.mark.parametrize("lens", [[500], [200, 333, 64], [1700]])
def test_random_keys(lens, d_k, d_v, H):
    c = make(lens, H=H, H_k=2, d_k=d_k, d_v=d_v, decay=0.02, seed=sum(lens) + d_k)
    out, fin = run(c, out_dtype=B16)
    check_pairs(c, out, fin, reference(c))


@pytest.mark.parametrize("alike", [1.0, 5.0, 1e4])
@pytest.mark.parametrize("d_k", [17, 128])
@pytest.mark.parametrize("out_dtype", [B16, F32])
def test_keys_that_share_a_direction(alike, d_k, out_dtype):
    """The terms of P U then nearly cancel: up to 64 of them, each with up to four pairs' roundings, 2^-18 / sqrt(3) with
    random signs, sqrt(64 4) 2^-18 / sqrt(3) = 3.5e-5 together."""
    c = make([500], H=4, d_k=d_k, d_v=64, decay=0.02, seed=d_k, alike=alike)
    out, fin = run(c, out_dtype=out_dtype)
    check_pairs(c, out, fin, reference(c), tolerance=3.5e-5)
    if out_dtype == B16:  # and the nearest bf16 to the fp32 output, up to the ties that the two calls' roundings cross
        wide, _ = run(c, out_dtype=F32)
        assert off(out, wide.to(B16).double().cpu().numpy()) < 1e-3
