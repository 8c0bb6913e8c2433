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


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
def test_single_tokens_of_one_block_at_once(fa, d, dtype):
    """Few tokens, each a run of its own, some blocks' by several warps at once, the blocks begun with scales
    that are no powers of two: those blocks' contents are undefined, and nothing else; the call ends."""
    import torch
    Hkv, page, pages = 3, 16, 40
    rng = np.random.default_rng(d)
    for step in range(20):
        ids = rng.permutation(pages)
        # four tokens each of one block in turn with another's, then single tokens of blocks of their own
        slots = [int(ids[2 * i + j]) * page + 1 + 2 * n for i in range(6) for n in range(4) for j in range(2)]
        alone = [int(b) * page + int(rng.integers(1, 16)) for b in ids[12:30]]
        slots += alone
        cache = fa.Kv8Cache(tuple(
            torch.from_numpy(x).cuda().view(t) for x, t in (
                (rng.integers(0, 256, (pages, Hkv, page, d)).astype(np.uint8), torch.float8_e4m3fn),
                (2.0 ** rng.uniform(-9, 1, (pages, Hkv, 1)).astype(np.float32), torch.float32)) * 2))
        q, k, w, pos, axis = base.make(torch, step, (len(slots),), 4, Hkv, d, dtype, d, norm=False)
        k *= 2.0 ** (step % 4)
        s = torch.tensor(slots, dtype=torch.int32, device="cuda")
        before = cache.k8.clone(), cache.k_scale.clone()
        p = base.plan(fa, d, axis, False)
        got = fa.kv8_append_norm_rope(cache, q, k, torch.randn_like(k), s, pos, p, norm=False)
        torch.cuda.synchronize()
        assert torch.equal(got, fa.norm_rope_forward(q, k, pos, p, norm=False)[0])
        y, bound = ref.forward(k, None, base.angle(pos, d, axis), False, False, EPS)
        open_ = torch.from_numpy(ids[:12].copy()).cuda()
        for x, old in zip((cache.k8.view(torch.uint8), cache.k_scale), (before[0].view(torch.uint8), before[1])):
            x[open_] = old[open_]
        sure = [x if t >= len(slots) - len(alone) else -1 for t, x in enumerate(slots)]
        base.check_keys(torch, before, (cache.k8, cache.k_scale), y, bound, sure)


@pytest.mark.parametrize("eps", [1e-6, 2.0 ** -100, 2.0 ** -126, 2.0 ** -128, 2.0 ** -149])
@pytest.mark.parametrize("T", [1, 3, 40, 6000])
def test_keys_of_zeros_and_the_least_eps(fa, T, eps):
    """Rows of zeros, whose inverse norm is eps ** -0.5, into blocks whose scale is the least there is, beside
    rows that are not zero."""
    import torch
    Hkv, d, page = 2, 128, 64
    q, k, w, pos, axis = base.make(torch, T, (T,), 4, Hkv, d, "bf16", d)
    k[:, 0] = 0.0
    q[T // 2:, 1] = 0.0
    pages = -(-T // page) + 1
    cache = fa.kv8_cache(pages, Hkv, d, page=page)
    before = cache.k8.clone(), cache.k_scale.clone()
    slots = list(range(T))
    kw = dict(q_weight=w[0], k_weight=w[1], eps=eps)
    p = base.plan(fa, d, axis, False)
    got = fa.kv8_append_norm_rope(cache, q, k, k, torch.tensor(slots, dtype=torch.int32, device="cuda"), pos, p, **kw)
    assert (cache.k8.view(torch.uint8)[:, 0] & 127 == 0).all()
    assert (got[T // 2:, 1] == 0).all() and torch.equal(got, fa.norm_rope_forward(q, k, pos, p, **kw)[0])
    y, bound = ref.forward(k, w[1], base.angle(pos, d, axis), False, True, eps)
    base.check_keys(torch, before, (cache.k8, cache.k_scale), y, bound, slots)


def test_keys_with_large_weights(fa):
    """x r w where x w goes beyond fp32."""
    import torch
    T, Hkv, d, page = 50, 2, 64, 16
    q, k, _, pos, axis = base.make(torch, 5, (T,), 4, Hkv, d, "bf16", 0)
    w = torch.full((d,), 2.0 ** 80, device="cuda")
    k = (k.float() * 2.0 ** 55).to(k.dtype)
    cache = fa.kv8_cache(4, Hkv, d, page=page)
    before = cache.k8.clone(), cache.k_scale.clone()
    slots = list(range(T))
    fa.kv8_append_norm_rope(cache, q, k, k, torch.tensor(slots, dtype=torch.int32, device="cuda"), k_weight=w, eps=EPS)
    y, bound = ref.forward(k, w, None, False, True, EPS)
    base.check_keys(torch, before, (cache.k8, cache.k_scale), y, bound, slots)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_as_long_as_fp32_holds(fa, d):
    """Rows whose squares sum to just below 2^128 are rows as others; from there on r is 0."""
    import torch
    T, Hkv, page = 40, 2, 64
    q, k, w, pos, axis = base.make(torch, 7, (T,), 3, Hkv, d, "bf16", d)
    sign = lambda x: torch.where(x < 0, -1.0, 1.0).to(x.dtype)
    most = 2.0 ** 60 if d == 128 else 1.4140625 * 2.0 ** 60     # d x^2 = 2^127 and just below it
    q[::2], k[::2] = sign(q[::2]) * most, sign(k[::2]) * most   # (the others: as they come)
    q[1, 1], k[1, 1] = sign(q[1, 1]) * 2.0 ** 61, sign(k[1, 1]) * 2.0 ** 61   # squares of 2^122 each: 2^128 at d = 64
    q[3, 0], k[3, 0, 5] = sign(q[3, 0]) * 2.0 ** 100, 2.0 ** 64
    dy = [torch.randn_like(q), torch.randn_like(k)]
    p, kw = base.plan(fa, d, axis, False), dict(q_weight=w[0], k_weight=w[1])
    a = base.angle(pos, d, axis)
    got, grads = fa.norm_rope_forward(q, k, pos, p, **kw), fa.norm_rope_backward(q, k, *dy, pos, p, **kw)
    cache = fa.kv8_cache(1, Hkv, d, page=page)
    before = cache.k8.clone(), cache.k_scale.clone()
    slots = list(range(T))
    s = torch.tensor(slots, dtype=torch.int32, device="cuda")
    assert torch.equal(fa.kv8_append_norm_rope(cache, q, k, k, s, pos, p, **kw), got[0])
    for i, x in enumerate((q, k)):
        long_ = x.double().square().sum(-1) >= 2.0 ** 128
        assert int(long_.sum()) == 2
        x = torch.where(long_[..., None], 0.0, x)               # (a row of zeros: outputs 0)
        want, bound = ref.forward(x, w[i], a, False, True, EPS)
        ref.check("y", got[i], want, bound, "bf16")
        if i:
            base.check_keys(torch, before, (cache.k8, cache.k_scale), want, bound, slots)
        assert (grads[i][long_] == 0).all()
        dx, dx_bound, dw, dw_bound = ref.backward(x, torch.where(long_[..., None], 0.0, dy[i]), w[i], a, False, True, EPS)
        ref.check("dx", grads[i], dx, dx_bound, "bf16")
        ref.check("dw", grads[2 + i], dw, dw_bound, None)


@pytest.mark.parametrize("side", [0, 1])
def test_one_sides_weight_alone(fa, side):
    """A norm with weights for queries or for keys only, its gradient too."""
    import torch
    q, k, w, pos, axis = base.make(torch, 8 + side, (333,), 6, 2, 128, "bf16", 64, wide=True)
    w[1 - side] = None
    dy = [torch.randn_like(q), torch.randn_like(k)]
    p, kw = base.plan(fa, 64, axis, False), dict(q_weight=w[0], k_weight=w[1])
    a = base.angle(pos, 64, axis)
    got, grads = fa.norm_rope_forward(q, k, pos, p, **kw), fa.norm_rope_backward(q, k, *dy, pos, p, **kw)
    for i, x in enumerate((q, k)):
        ref.check("y", got[i], *ref.forward(x, w[i], a, False, True, EPS), "bf16")
        dx, bound, dw, dw_bound = ref.backward(x, dy[i], w[i], a, False, True, EPS)
        ref.check("dx", grads[i], dx, bound, "bf16")
        if i == side:
            ref.check("dw", grads[2 + i], dw, dw_bound, None)
        else:
            assert grads[2 + i] is None


@pytest.mark.parametrize("name", ["test_norm_rope_edges_gpu.py", "test_kv8_gpu.py"])
def test_suites_under_the_bounds_checking_build(fa, name):
    """These tests, and those of the cache's writer without norms, with the library that checks the addresses it
    forms; the status word has to be clear after each."""
    import os
    import subprocess
    import sys
    if fa.fa_debug_checks_enabled():
        pytest.skip("this is the checking build")
    from exact_io_aware_tcgen05_gb300 import build as b
    env = dict(os.environ, FA_GB300_LIBRARY=b.build(debug=True), FA_GB300_CHECK_STATUS="1")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                        os.path.join("tests", name), "-k", "not bounds_checking"], cwd=root, env=env,
                       capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout[-4000:], r.stderr[-2000:])
