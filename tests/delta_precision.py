"""How far the tensor-core kernel of the gated delta rule may be off in the 2-norm: ``check_pairs``, shared by its
tests.

Ten roundings of pairs on a chunk's way, 2^-18 / sqrt(3) each with random signs, and the read-out's come to 2e-5.
A bf16 output is the value nearest to one that is off by that, so entry by entry

    |out - exact| <= |bf16(exact) - exact| + 2 |that one - exact| ."""

import numpy as np
import torch

from delta_cases import bounds, check, f64, half_step

PAIRS = 2e-5


def off(got, want):
    return np.linalg.norm(f64(got) - want) / max(np.linalg.norm(want), 1e-30)


def check_pairs(c, out, fin, ref, tolerance=PAIRS):
    """Entry by entry within the bound for chunks of pairs, and in the 2-norm."""
    o, f = ref
    bo, bf, _ = bounds(c, pairs=True)
    check(fin, f, bf, "final")
    assert off(fin, f) < tolerance, off(fin, f)
    if out.dtype == torch.bfloat16:
        check(out, o, 2 * bo + half_step(o, out.dtype), "out")
        own = off(torch.from_numpy(o).to(torch.bfloat16), o)
        assert off(out, o) < own + 2 * tolerance, (off(out, o), own)
    else:
        check(out, o, bo, "out")
        assert off(out, o) < tolerance, off(out, o)
