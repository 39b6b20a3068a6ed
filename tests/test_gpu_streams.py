"""Calls with ``stream=``: what they allocate may not be memory that the current stream still uses."""

import pytest
import torch

from kimi_delta_attention_02_gb300 import binding, workloads
from linear_cases import make

pytestmark = pytest.mark.gpu


def _check_beside_pending_work(call):
    """``call(stream)`` returns its outputs. Blocks of every size that it allocates have just been freed
    on the current stream, while copies of them still wait there: a call on another stream must
    neither write them nor hand them out."""
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(None) if t is not None]
    torch.cuda.synchronize()
    sizes = []
    real = torch.empty

    def recording(shape, **kw):
        t = real(shape, **kw)
        sizes.append((t.shape, t.dtype))
        return t

    torch.empty = recording
    try:
        call(None)
    finally:
        torch.empty = real
    assert sizes
    torch.cuda.synchronize()
    junk = [torch.full(shape, 3, dtype=dtype, device="cuda") for shape, dtype in sizes]
    copies = [torch.zeros_like(t) for t in junk]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    for c, t in zip(copies, junk):
        c.copy_(t)
    del junk, t
    got = [t for t in call(side) if t is not None]
    side.synchronize()
    torch.cuda.synchronize()
    binding.check_device_error()
    assert all((c == 3).all() for c in copies)
    assert len(got) == len(want) and all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("recurrent", [False, True])
def test_linear_prefill(recurrent):
    c = make([3000], H=2, d_k=64, d_v=72, decay=0.01, seed=1)
    _check_beside_pending_work(lambda s: binding.linear_prefill(**c, stream=s, recurrent=recurrent))


def test_linear_decode():
    c = make([1] * 64, H=8, d_k=64, d_v=64, seed=1)
    states = iter([c["init_state"].clone() for _ in range(3)])
    _check_beside_pending_work(lambda s: [binding.linear_decode(c["q"], c["k"], c["v"], c["log_decay"], next(states),
                                                                stream=s)])


def test_block_norm():
    x, y = (torch.randn(300, 1000, device="cuda") for _ in range(2))
    _check_beside_pending_work(lambda s: binding.block_norm(x, y, post_norm=True, stream=s))


@pytest.mark.parametrize("form", ["prefill", "recurrent", "gated", "ex"])
def test_kda_prefill(form):
    T = 600 if form == "recurrent" else 20000
    c = workloads.make_prefill([T], H=2, device="cuda", seed=3, gated=True)
    head, tail = (c.q, c.k, c.v), (c.beta, c.cu_seqlens)
    assert form == "recurrent" or binding.workspace_size(T, 1, 2) > 0
    call = {"prefill": lambda s: binding.prefill(*head, c.log_alpha, *tail, c.init_state, stream=s),
            "recurrent": lambda s: binding.prefill(*head, c.log_alpha, *tail, c.init_state, stream=s, recurrent=True),
            "gated": lambda s: binding.prefill_gated(*head, c.z, c.A_log, *tail, c.init_state, stream=s),
            "ex": lambda s: binding.prefill_ex(*head, *tail, log_alpha=c.log_alpha, init_state=c.init_state, stream=s)}
    if c.log_alpha is None:
        c.log_alpha = -5 * torch.sigmoid(c.z.float())
    _check_beside_pending_work(call[form])


@pytest.mark.parametrize("form", ["decode", "gated", "ex"])
def test_kda_decode(form):
    c = workloads.make_decode_step(0, 64, 4, device="cuda", seed=3, gated=True)
    states = iter([workloads.make_decode_state(64, 4, device="cuda", seed=3) for _ in range(3)])
    la = -5 * torch.sigmoid(c.z.float())
    call = {"decode": lambda s: [binding.decode(c.q, c.k, c.v, la, c.beta, next(states), stream=s)],
            "gated": lambda s: [binding.decode_gated(c.q, c.k, c.v, c.z, c.A_log, c.beta, next(states), stream=s)],
            "ex": lambda s: [binding.decode_ex(c.q, c.k, c.v, c.beta, next(states), log_alpha=la, stream=s)]}
    _check_beside_pending_work(call[form])


def test_prologue():
    c = workloads.make_prologue([300, 40], H=3, device="cuda", seed=5)
    _check_beside_pending_work(lambda s: binding.prologue(c.q_raw, c.k_raw, c.v_raw, c.conv_weight, c.cu_seqlens,
                                                          c.conv_init, stream=s))
