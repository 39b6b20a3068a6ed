"""Calls with ``stream=``: what they allocate may not be memory that the current stream still uses."""

import pytest
import torch

from kimi_delta_attention_02_gb300 import binding
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
