"""The linear-attention prefill at sizes whose indexes pass 31 or 32 bits."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from linear_cases import check, fp32_factor, reference

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


def test_the_longest_sequence():
    """2^31 - 128 tokens of one head of 8, cut into 152 segments: the tokens around some cuts and the last
    ones against the oracle. A constant decay of e^-0.02 leaves e^-60 of what lies 3000 tokens back.
    Bounds as in test_gpu_linear_chunked.py. q, k and v are one tensor (34 GB), read only."""
    T = 2**31 - 128
    x = torch.empty(T, 1, 8, device="cuda", dtype=B16)
    g = torch.Generator("cuda").manual_seed(3)
    for part in x.split(1 << 27):
        part.normal_(generator=g).mul_(0.25)
    ld = torch.tensor([-0.02], device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out, fin = binding.linear_prefill(x, x, x, ld, cu, out_dtype=B16)
    binding.check_device_error()
    seg = -(-(-(-T // 152)) // 128) * 128
    fine = 2.0 ** -15 + fp32_factor(128 + 3000 // 64, 8)
    for at, n in ((0, 200), (seg, 200), (2 * seg, 200), (76 * seg, 200), (151 * seg, 200), (T - 200, 200)):
        first = max(0, at - 3000)
        w = x[first:at + n].contiguous()
        c = dict(q=w, k=w, v=w, log_decay=ld, cu_seqlens=torch.tensor([0, w.shape[0]], dtype=torch.int32), init_state=None)
        o, f, mo, mf = (r[at - first:] if i in (0, 2) else r for i, r in enumerate(reference(c)))
        check(out[at:at + n], o, mo * (2.0 ** -8 + fine) + 2.0 ** -8 * np.abs(o), 1.0, at)
    check(fin, f, mf, fine, "final")  # of the last window


@pytest.mark.parametrize("recurrent", [False, True])
def test_segment_places_past_32_bits(recurrent):
    """A cut sequence behind 2200 others on 64 heads: its segments' states lie past 2^31 entries of the
    workspace (2200 x 64 x 128 x 128 = 2.3 x 10^9), the final states too; with rows behind it."""
    short, T, H = 2200, 4000, 64
    g = torch.Generator("cuda").manual_seed(1)
    rows = 30 * short + T + 5
    q = torch.randn(rows, 1, 128, device="cuda", generator=g).to(B16)
    k = (0.1 * torch.randn(rows, 1, 128, device="cuda", generator=g)).to(B16)
    v = torch.randn(rows, H, 128, device="cuda", generator=g).to(B16)
    ld = -0.01 * torch.rand(rows, H, device="cuda", generator=g)
    ends = list(range(0, 30 * short + 1, 30)) + [30 * short + T]
    cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
    first, last = 30 * short, 30 * short + T
    state = torch.zeros(short + 1, H, 128, 128, device="cuda")
    state[-1].normal_(generator=g)
    init = state[-1:].clone()
    assert binding.linear_workspace_size(rows, short + 1, H, 128, 128, B16, B16, recurrent, H_k=1) > 4 * 2**31
    out, fin = binding.linear_prefill(q, k, v, ld, cu, state, final_state=state, out_dtype=B16, recurrent=recurrent)
    binding.check_device_error()
    heads = [0, H - 1]
    c = dict(q=q[first:last], k=k[first:last], v=v[first:last, heads], log_decay=ld[first:last, heads],
             cu_seqlens=torch.tensor([0, T], dtype=torch.int32), init_state=init[:, heads])
    o, f, mo, mf = reference(c)
    fine = 2.0 ** -15 + fp32_factor(T if recurrent else 128 + T // 64, 128)
    half = 0.0 if recurrent else 2.0 ** -8
    check(out[first:last][:, heads], o, mo * (half + fine) + 2.0 ** -8 * np.abs(o), 1.0, "out")
    check(fin[-1:][:, heads], f, mf, fine, "final")
