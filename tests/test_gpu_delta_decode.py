"""kda_delta_decode against the fp64 oracle: B one-token sequences per step. Bounds: delta_cases."""

import numpy as np
import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from delta_cases import bounds, check, half_step, make, reference

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


def _steps(B, H, H_k, d_k, d_v, dtype, per_token, out_dtype=F32, steps=3, scale=0.7):
    first = make([1] * B, H=H, H_k=H_k, d_k=d_k, d_v=d_v, dtype=dtype, seed=100)
    state = first["init_state"].clone()
    ref, n, E = first["init_state"].cpu(), None, None
    for s in range(steps):
        c = make([1] * B, H=H, H_k=H_k, d_k=d_k, d_v=d_v, dtype=dtype, per_token=per_token, seed=s)
        out = binding.delta_decode(c["q"], c["k"], c["v"], c["log_decay"], c["beta"], state, out_dtype=out_dtype,
                                   scale=scale)
        c["init_state"] = ref
        o, ref64 = reference(c, scale)
        bo, bf, n = bounds(c, scale, n0=n, E0=E)
        check(out, o, bo + half_step(o, out_dtype), "out")
        check(state, ref64, bf, "state")
        ref, E = torch.from_numpy(ref64), bf[:, :, 0]
    binding.check_device_error()


@pytest.mark.parametrize("d_k,d_v", [(128, 128), (64, 128), (128, 64), (1, 1), (100, 72), (5, 33), (128, 6), (17, 127)])
@pytest.mark.parametrize("dtype", [F32, B16])
def test_head_sizes(d_k, d_v, dtype):
    _steps(3, 4, 2, d_k, d_v, dtype, True)


@pytest.mark.parametrize("B,H,H_k", [(1, 1, 1), (1, 96, 96), (7, 24, 8), (700, 3, 1)])
@pytest.mark.parametrize("per_token", [True, False])
def test_batches_and_shared_heads(B, H, H_k, per_token):
    _steps(B, H, H_k, 32, 32, B16, per_token, out_dtype=B16, steps=2)


@pytest.mark.parametrize("B", [2, 80])
@pytest.mark.parametrize("d_k,d_v", [(16, 16), (128, 32), (64, 33), (33, 64), (48, 72), (128, 60), (31, 53), (65, 31),
                                     (100, 53), (9, 127), (33, 118), (32, 16), (64, 16), (65, 15), (40, 9), (32, 30)])
def test_every_tile(d_k, d_v, B):
    """Tiles of 16, 32 and 64 columns, 32, 64 and 128 key rows, four columns per thread or one; 8 and 320
    states, so that few states take narrower tiles."""
    _steps(B, 4, 2, d_k, d_v, B16, True, steps=2)


def test_on_another_stream():
    """With ``stream=`` the call runs there, behind what that stream has been given."""
    side = torch.cuda.Stream()
    c = make([1] * 2, H=2, d_k=64, d_v=64)
    state = torch.zeros_like(c["init_state"])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        state.copy_(c["init_state"])
    out = binding.delta_decode(c["q"], c["k"], c["v"], c["log_decay"], c["beta"], state, stream=side)
    side.synchronize()
    o, f = reference(c)
    bo, bf, _ = bounds(c)
    check(out, o, bo, "out")
    check(state, f, bf, "state")


def test_prompt_then_tokens_equals_a_longer_prompt():
    """Prefill of 50 tokens, then five decode steps, against the oracle's 55 tokens."""
    c = make([55], H=4, H_k=2, d_k=128, d_v=64)
    o, f = reference(c)
    bo, bf, _ = bounds(c)
    names = ("q", "k", "v", "log_decay", "beta")
    cut = {n: (t[:50] if n in names else t) for n, t in c.items()}
    cut["cu_seqlens"] = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    out, state = binding.delta_prefill(**cut, recurrent=True)
    outs = [out] + [binding.delta_decode(*(c[n][t:t + 1] for n in names), state) for t in range(50, 55)]
    check(torch.cat(outs), o, bo, "out")
    check(state, f, bf, "state")


def test_forgetting_and_nan():
    c = make([1] * 2, H=2, d_k=16, d_v=16, dtype=F32)
    c["log_decay"][0, 0], c["log_decay"][1, 1] = -float("inf"), float("nan")
    state = c["init_state"].clone()
    out = binding.delta_decode(c["q"], c["k"], c["v"], c["log_decay"], c["beta"], state)
    # 0 times every finite state is 0, so beta v k^T is left, rounded twice
    want = (c["beta"][0, 0] * c["v"][0, 0])[None, :] * c["k"][0, 0][:, None]
    assert torch.allclose(state[0, 0], want, rtol=2.0 ** -22, atol=0)
    assert torch.isnan(state[1, 1]).all() and torch.isnan(out[1, 1]).all()
    assert torch.isfinite(state[0]).all() and torch.isfinite(state[1, 0]).all() and torch.isfinite(out[0]).all()


def test_captured_and_replayed():
    c = make([1] * 5, H=4, H_k=2, d_k=128, d_v=64)
    args = [c[n] for n in ("q", "k", "v", "log_decay", "beta")]
    state, twin = c["init_state"].clone(), c["init_state"].clone()
    out = torch.empty(5, 4, 64, device="cuda")
    binding.delta_decode(*args, state.clone(), out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.delta_decode(*args, state, out=out)
    for _ in range(3):
        graph.replay()
        want = binding.delta_decode(*args, twin)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(state, twin)
    assert not np.isnan(float(out.sum()))
