"""Norms and rotation, and the same on the way into the 8-bit cache, at the edges of what they take, on
the GPU."""
import numpy as np
import pytest

import norm_rope_ref as ref
import test_norm_rope_gpu as base

pytestmark = pytest.mark.gpu
EPS = base.EPS


def test_plans_as_plain_tuples(fa):
    """A tuple of a plan's parts is looked at as a plan is."""
    import torch
    q, k, w, pos, axis = base.make(torch, 1, (9,), 4, 2, 64, "bf16", 64, axes=2)
    p = base.plan(fa, 64, axis, False)
    want = fa.norm_rope_forward(q, k, pos, p, norm=False)
    got = fa.norm_rope_forward(q, k, pos, tuple(p), norm=False)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for error, parts in [
        (ValueError, (p.turns, p.axes[:16], 2, False)), (ValueError, (p.turns, p.axes.cpu(), 2, False)),
        (ValueError, (p.turns[:20], p.axes[:20], 2, False)), (TypeError, (p.turns.int(), p.axes, 2, False)),
        (TypeError, (p.turns, p.axes.long(), 2, False)),
    ]:
        with pytest.raises(error):
            fa.norm_rope_forward(q, k, pos, parts, norm=False)
        with pytest.raises(error):
            fa.norm_rope_backward(q, k, q, k, pos, parts, norm=False)
