"""The gated delta rule, its decode and the norm with rotation as a server calls them: on another stream
beside pending work, two calls at once, tensors of more than 2^31 elements, more of everything."""

import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
from delta_cases import make, run
from test_gpu_streams import _check_beside_pending_work

pytestmark = pytest.mark.gpu
B16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("recurrent", [False, True])
def test_prefill_beside_pending_work(recurrent):
    c = make([3000], H=2, d_k=64, d_v=72, decay=0.01, seed=1)
    assert binding.delta_workspace_size(3000, 1, 2, 64, 72) > 0
    _check_beside_pending_work(lambda s: binding.delta_prefill(**c, stream=s, recurrent=recurrent))


def test_decode_beside_pending_work():
    c = make([1] * 64, H=8, d_k=64, d_v=64, seed=1)
    states = iter([c["init_state"].clone() for _ in range(3)])
    _check_beside_pending_work(lambda s: [binding.delta_decode(c["q"], c["k"], c["v"], c["log_decay"], c["beta"],
                                                               next(states), stream=s)])


def test_norm_rotate_beside_pending_work():
    q, k = torch.randn(300, 8, 64, device="cuda"), torch.randn(300, 2, 64, device="cuda")
    pos, f = torch.arange(300, device="cuda"), torch.rand(32, device="cuda")
    _check_beside_pending_work(lambda s: binding.norm_rotate(q, k, pos, f, stream=s))


def test_two_prompts_at_once():
    """Two streams, each with the workspace that its own call allocates, the same inputs on both."""
    c = make([2600, 0, 300], H=2, decay=0.02, seed=3)
    want = run(c, out_dtype=B16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [binding.delta_prefill(**c, out_dtype=B16, stream=s) for _ in range(6) for s in streams]
    torch.cuda.synchronize()
    binding.check_device_error()
    for out, fin in got:
        assert torch.equal(out, want[0]) and torch.equal(fin, want[1])


def test_one_tensor_as_query_and_key():
    c = make([500], H=4, H_k=2, seed=5)
    c["q"] = c["k"].clone()
    want = run(c)
    out, fin = run({**c, "q": c["k"]})
    assert torch.equal(out, want[0]) and torch.equal(fin, want[1])


def test_nan_in_a_query_stays_with_its_token():
    c = make([200], H=2, seed=6)
    want, fin = run(c, out_dtype=B16)
    c["q"][70, 1, 3] = float("nan")
    out, again = run(c, out_dtype=B16)
    assert torch.isnan(out[70, 1]).all() and torch.equal(again, fin)
    out[70, 1] = want[70, 1]
    assert torch.equal(out, want)


@pytest.mark.parametrize("recurrent", [False, True])
def test_tokens_past_31_bits(recurrent):
    """The last sequence of a call whose v and out hold more than 2^31 elements, bit by bit."""
    H, d, last = 128, 128, 200
    T = 2**31 // (H * d) + 5000
    tail = make([last], H=H, H_k=2, seed=2)
    c = make([T], H=1, H_k=1, d_k=8, d_v=8, init=False, seed=2)  # (small: widened on the device)
    wide = dict(q=torch.zeros(T, 2, d, device="cuda", dtype=B16), k=torch.zeros(T, 2, d, device="cuda", dtype=B16),
                v=torch.zeros(T, H, d, device="cuda", dtype=B16), log_decay=c["log_decay"].expand(T, H).contiguous(),
                beta=c["beta"].expand(T, H).contiguous())
    wide["k"][:, :, 0] = 1
    wide["v"][:, :, 1] = 1
    for n, t in wide.items():
        t[-last:] = tail[n]
    cu = torch.tensor([0, T - last, T], dtype=torch.int32, device="cuda")
    init = torch.zeros(2, H, d, d, device="cuda")
    init[1] = tail["init_state"][0]
    out, fin = binding.delta_prefill(**wide, cu_seqlens=cu, init_state=init, out_dtype=B16, recurrent=recurrent, workspace=None)
    want, end = binding.delta_prefill(**tail, out_dtype=B16, recurrent=recurrent, workspace=None)
    binding.check_device_error()
    assert out.numel() > 2**31 and torch.equal(out[-last:], want) and torch.equal(fin[1], end[0])
    assert torch.isfinite(out[-last - 1]).all()


@pytest.mark.parametrize("recurrent", [False, True])
def test_states_past_31_bits(recurrent):
    H, d, N, each = 128, 128, 1100, 9
    tail = make([each, each], H=H, H_k=2, seed=4)
    state = torch.zeros(N, H, d, d, device="cuda")
    state[-2:] = tail["init_state"]
    wide = {n: torch.cat([torch.zeros((N - 2) * each, *tail[n].shape[1:], device="cuda", dtype=tail[n].dtype), tail[n]])
            for n in ("q", "k", "v", "log_decay", "beta")}
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda") * each
    out, fin = binding.delta_prefill(**wide, cu_seqlens=cu, init_state=state, final_state=state, recurrent=recurrent)
    want, end = binding.delta_prefill(**tail, recurrent=recurrent)
    assert fin.numel() > 2**31 and torch.equal(out[-2 * each:], want) and torch.equal(fin[-2:], end)
    assert not fin[:-2].any()
    one = {n: wide[n][::each].contiguous() for n in ("q", "k", "v", "log_decay", "beta")}
    small = end.clone()
    out = binding.delta_decode(*one.values(), state)
    want = binding.delta_decode(*(t[-2:].contiguous() for t in one.values()), small)
    binding.check_device_error()
    # Few states take narrower tiles, whose sums meet in another order: 130 roundings of 2^-24 of the column's
    # norm in each of S'^T k, S'^T q and (k . q) u, on either side.
    assert torch.allclose(out[-2:], want, rtol=0, atol=130 * 2.0**-24 * float(small.norm(dim=2).max()) * 6)
    assert torch.allclose(state[-2:], small, rtol=0, atol=130 * 2.0**-24 * float(small.norm(dim=2).max()) * 6)
    assert not state[:-2].any()


@pytest.mark.parametrize("d", [128, 127])
def test_rotated_rows_past_31_bits(d):
    H, last = 128, 60
    T = 2**31 // (H * d) + 1000
    x = torch.ones(T, H, d, device="cuda", dtype=B16)
    x[-last:] = torch.randn(last, H, d, device="cuda").to(B16)
    pos, f = torch.arange(T, device="cuda") * 1000003, torch.rand(d // 2, device="cuda")
    want, _ = binding.norm_rotate(x[-last:].clone(), None, pos[-last:].clone(), f)
    out, _ = binding.norm_rotate(x, None, pos, f, q_out=x)
    assert out is x and x.numel() > 2**31 and torch.equal(out[-last:], want)


def test_axes_as_an_array():
    """pair_axis in any form that holds integers: a list, a tuple, a tensor."""
    q = torch.randn(50, 3, 32, device="cuda")
    pos, f = torch.randint(0, 1000, (3, 50), device="cuda"), torch.rand(16, device="cuda")
    axes = [i % 3 for i in range(16)]
    want, _ = binding.norm_rotate(q, None, pos, f, pair_axis=axes)
    for form in (tuple(axes), torch.tensor(axes), torch.tensor(axes).numpy(), bytes(axes)):
        got, _ = binding.norm_rotate(q, None, pos, f, pair_axis=form)
        assert torch.equal(got, want)
    flat, _ = binding.norm_rotate(q, None, pos[0].contiguous(), f)
    assert not torch.equal(flat, want)
