"""kda_linear_decode against the fp64 oracle: B one-token sequences per step. Bounds: see
linear_cases.fp32_factor with the steps as the tokens of a term's life."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from linear_cases import check, cpu, fp32_factor, make, reference

pytestmark = pytest.mark.gpu


def _steps(B, H, H_k, d_k, d_v, dtype, per_token, out_dtype=torch.float32, steps=3, scale=0.7):
    first = make([1] * B, H=H, H_k=H_k, d_k=d_k, d_v=d_v, dtype=dtype, seed=100)
    state = first["init_state"].clone()
    ref, mag = first["init_state"].cpu(), None
    for s in range(steps):
        c = make([1] * B, H=H, H_k=H_k, d_k=d_k, d_v=d_v, dtype=dtype, per_token=per_token, seed=s)
        out = binding.linear_decode(c["q"], c["k"], c["v"], c["log_decay"], state, out_dtype=out_dtype, scale=scale)
        c["init_state"] = ref
        o, ref64, mo, mf = reference(c, scale)
        if mag is not None:  # magnitudes chain like the values
            c["init_state"] = mag
            _, _, mo, mf = reference(c, scale)
        fac = fp32_factor(s + 1, d_k)
        half = 2.0 ** -8 if out_dtype == torch.bfloat16 else 0.0
        check(out, o, mo * fac + half * np.abs(o), 1.0, "out")
        check(state, ref64, mf, fac, "state")
        ref, mag = torch.from_numpy(ref64), torch.from_numpy(mf)
    binding.check_device_error()


@pytest.mark.parametrize("d_k,d_v", [(128, 128), (64, 128), (128, 64), (1, 1), (100, 72), (5, 33), (128, 6), (17, 127)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_head_sizes(d_k, d_v, dtype):
    _steps(3, 4, 2, d_k, d_v, dtype, True)


@pytest.mark.parametrize("B,H,H_k", [(1, 1, 1), (1, 96, 96), (7, 24, 8), (700, 3, 1)])
@pytest.mark.parametrize("per_token", [True, False])
def test_batches_and_shared_heads(B, H, H_k, per_token):
    _steps(B, H, H_k, 32, 32, torch.bfloat16, per_token, out_dtype=torch.bfloat16, steps=2)


@pytest.mark.parametrize("B", [2, 80])
@pytest.mark.parametrize("d_k,d_v", [(16, 16), (128, 32), (64, 33), (33, 64), (48, 72), (128, 60), (31, 53), (65, 31),
                                     (53, 53), (100, 53), (9, 127), (33, 118), (118, 118), (16, 128), (128, 100)])
def test_every_tile(d_k, d_v, B):
    """Tiles of 32, 64 and 128 columns with 64, 128 and 256 threads, four columns per thread or one;
    8 and 320 states, so that few states take narrower tiles."""
    _steps(B, 4, 2, d_k, d_v, torch.bfloat16, True, steps=2)


def test_on_another_stream():
    """With ``stream=`` the call runs there, behind what that stream has been given."""
    side = torch.cuda.Stream()
    c = make([1] * 2, H=2, d_k=64, d_v=64)
    state = torch.zeros_like(c["init_state"])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        state.copy_(c["init_state"])
    out = binding.linear_decode(c["q"], c["k"], c["v"], c["log_decay"], state, stream=side)
    side.synchronize()
    o, f, mo, mf = reference(c)
    check(out, o, mo, fp32_factor(1, 64), "out")
    check(state, f, mf, fp32_factor(1, 64), "state")


def test_prompt_then_tokens_equals_a_longer_prompt():
    """Prefill of 50 tokens, then five decode steps, against the oracle's 55 tokens."""
    c = make([55], H=4, H_k=2, d_k=128, d_v=64)
    o, f, mo, mf = reference(c)
    cut = {n: (t[:50] if n in ("q", "k", "v", "log_decay") else t) for n, t in c.items()}
    cut["cu_seqlens"] = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    out, state = binding.linear_prefill(**cut, recurrent=True)
    outs = [out] + [binding.linear_decode(c["q"][t:t + 1], c["k"][t:t + 1], c["v"][t:t + 1], c["log_decay"][t:t + 1],
                                          state) for t in range(50, 55)]
    check(torch.cat(outs), o, mo, fp32_factor(55, 128), "out")
    check(state, f, mf, fp32_factor(55, 128), "state")


def test_forgetting_and_nan():
    c = make([1] * 2, H=2, d_k=16, d_v=16, dtype=torch.float32)
    c["log_decay"][0, 0], c["log_decay"][1, 1] = -float("inf"), float("nan")
    want = c["k"][0, 0][:, None] * c["v"][0, 0][None, :]
    state = c["init_state"].clone()
    out = binding.linear_decode(c["q"], c["k"], c["v"], c["log_decay"], state)
    # s + (-1) s is exactly 0 for every finite s, so the state is the fp32 product
    assert torch.equal(state[0, 0], want)
    assert torch.isnan(state[1, 1]).all() and torch.isnan(out[1, 1]).all()
    assert not torch.isnan(state[0]).any() and not torch.isnan(out[0]).any() and not torch.isnan(out[1, 0]).any()


def test_captured_step_replays_on_new_inputs():
    c = make([1] * 3, H=2, d_k=64, d_v=64)
    state, out = c["init_state"].clone(), torch.empty(3, 2, 64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        binding.linear_decode(c["q"], c["k"], c["v"], c["log_decay"], state, out=out)
    new = make([1] * 3, H=2, d_k=64, d_v=64, seed=5)
    for n in ("q", "k", "v", "log_decay"):
        c[n].copy_(new[n])
    state.copy_(new["init_state"])
    graph.replay()
    torch.cuda.synchronize()
    o, f, mo, mf = reference(new)
    check(out, o, mo, fp32_factor(1, 64), "out")
    check(state, f, mf, fp32_factor(1, 64), "state")
    assert cpu(c)["q"].shape == (3, 2, 64)


def test_offsets_past_32_bits():
    """1100 sequences x 128 heads x 128 x 128 states: the last one is where it belongs."""
    B, H, d = 1100, 128, 128
    g = torch.Generator("cuda").manual_seed(1)
    q, k = (torch.randn(B, 1, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    v = torch.randn(B, H, d, device="cuda", generator=g).to(torch.bfloat16)
    ld = -torch.rand(B, H, device="cuda", generator=g)
    state = torch.zeros(B, H, d, d, device="cuda")
    state[-1].normal_(generator=g)
    last = state[-1:].clone()
    out = binding.linear_decode(q, k, v, ld, state)
    want = binding.linear_decode(q[-1:].contiguous(), k[-1:].contiguous(), v[-1:].contiguous(), ld[-1:].contiguous(), last)
    # the one sequence takes narrower tiles, whose read-out sums in another order
    assert torch.equal(state[-1:], last)
    assert ((out[-1:] - want).abs() <= 2.0 ** -14 * (q[-1:].float().abs() @ last[0].abs()).transpose(0, 1)).all()
