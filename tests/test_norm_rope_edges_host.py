"""Norms and rotation at the edges of what they take, on the host (no GPU needed)."""
import copy
import pickle

import pytest


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_tcgen05_gb300 import build as b
    b.build()
    import exact_io_aware_tcgen05_gb300 as fa
    fa.load()
    return fa


def _parts(torch, n=16, axes=None, num_axes=1):
    return [torch.zeros(n, dtype=torch.int64), axes, num_axes, False]


def test_plans_put_together_by_hand(lib):
    import torch
    axes = torch.zeros(16, dtype=torch.int32)
    for parts in (_parts(torch), _parts(torch, 64), _parts(torch, 16, axes, 3), _parts(torch, 16, axes, 1)):
        p = lib.RopePlan(parts)
        assert p.turns is parts[0] and p.axes is parts[1] and p.num_axes == parts[2] and p.interleaved is False
    made = lib.rope_plan([1.0, 2.0] * 8, axes=[0, 1] * 8, interleaved=True, device="cpu")
    for q in (copy.copy(made), copy.deepcopy(made), pickle.loads(pickle.dumps(made))):
        assert isinstance(q, lib.RopePlan) and torch.equal(q.turns, made.turns) and torch.equal(q.axes, made.axes)
        assert q.num_axes == 2 and q.interleaved


@pytest.mark.parametrize("error,change", [
    # what the kernels would read beyond its end, in another type or in another place
    (ValueError, lambda t, p: p[:3]),
    (TypeError, lambda t, p: [[0] * 16, *p[1:]]),
    (TypeError, lambda t, p: [p[0].int(), *p[1:]]),
    (TypeError, lambda t, p: [t.zeros(32, dtype=t.int64)[::2], *p[1:]]),
    (ValueError, lambda t, p: [p[0][:12], *p[1:]]),
    (ValueError, lambda t, p: [p[0].view(2, 8), *p[1:]]),
    (ValueError, lambda t, p: [t.zeros(72, dtype=t.int64), *p[1:]]),
    (ValueError, lambda t, p: [p[0][:0], *p[1:]]),
    (ValueError, lambda t, p: [p[0], None, 2, False]),
    (ValueError, lambda t, p: [p[0], t.zeros(8, dtype=t.int32), 2, False]),
    (ValueError, lambda t, p: [p[0], t.zeros(16, dtype=t.int32, device="meta"), 2, False]),
    (TypeError, lambda t, p: [p[0], t.zeros(16, dtype=t.int64), 2, False]),
    (TypeError, lambda t, p: [p[0], t.zeros(32, dtype=t.int32)[::2], 2, False]),
    (TypeError, lambda t, p: [p[0], [0] * 16, 2, False]),
    (ValueError, lambda t, p: [p[0], None, 0, False]),
    (ValueError, lambda t, p: [p[0], t.zeros(16, dtype=t.int32), 5, False]),
    (ValueError, lambda t, p: [p[0], t.zeros(16, dtype=t.int32), 2.0, False]),
])
def test_plans_that_do_not_hold_together_are_refused(lib, error, change):
    import torch
    with pytest.raises(error):
        lib.RopePlan(change(torch, _parts(torch)))
