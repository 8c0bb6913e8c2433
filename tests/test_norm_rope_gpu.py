"""Norms and rotation of queries and keys, and their gradients, on the GPU."""

import random

import numpy as np
import pytest

import kv8_ref as kv8
import norm_rope_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(torch, seed, lead, Hq, Hkv, d, dtype, rot, axes=1, fused=False, wide=False, norm=True, far=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = ref.TYPES[dtype]
    heads = Hq + 2 * Hkv
    x = (torch.randn(*lead, heads, d, generator=g, device="cuda") * (1 + torch.arange(heads, device="cuda") % 3)[:, None]).to(dt)
    q, k = x[..., :Hq, :], x[..., Hq:Hq + Hkv, :]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(torch.float32 if wide else dt) if norm else None
         for _ in range(2)]
    pos = None
    if rot:
        shape = lead if axes == 1 else (axes, *lead)
        pos = torch.randint(0, 5000, shape, generator=g, device="cuda", dtype=torch.int32) + far
    rnd = random.Random(seed)
    axis = [rnd.randrange(axes) for _ in range(rot // 2)] if axes > 1 else None
    if axis:
        axis[0] = axes - 1
    return q, k, w, pos, axis


def angle(pos, rot, axis):
    if not rot:
        return None
    return ref.angles(pos.reshape(len(pos), -1) if axis else pos, ref.frequencies(rot), axis)


def plan(fa, rot, axis, interleaved):
    return fa.rope_plan(ref.frequencies(rot), axes=axis, interleaved=interleaved) if rot else None


CASES = [
    # lead, Hq, Hkv, d, dtype, rot, axes, interleaved, fused, wide, norm, far
    ((1,), 1, 1, 64, "bf16", 64, 1, False, False, False, True, 0),
    ((1,), 32, 8, 128, "bf16", 128, 1, False, True, False, True, 100000),
    ((3, 5), 4, 4, 128, "f16", 128, 1, True, False, True, True, 0),
    ((257,), 12, 4, 64, "f16", 32, 1, True, False, False, False, 0),
    ((1000,), 8, 1, 128, "bf16", 96, 3, False, True, True, True, 2 ** 27 - 6000),
    ((1000,), 7, 3, 64, "bf16", 16, 4, True, True, False, True, 77),
    ((2, 333), 16, 2, 64, "bf16", 0, 1, False, False, True, True, 0),
    ((2, 1025), 16, 16, 128, "f16", 64, 2, False, True, False, True, -4000),
    ((4099,), 32, 8, 128, "bf16", 128, 1, False, True, False, True, 0),
    ((4099,), 64, 8, 64, "f16", 48, 3, False, False, True, False, 0),
    ((20011,), 5, 5, 64, "bf16", 64, 1, False, True, False, True, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward(fa, case):
    import torch
    lead, Hq, Hkv, d, dtype, rot, axes, il, fused, wide, norm, far = CASES[case]
    q, k, w, pos, axis = make(torch, case, lead, Hq, Hkv, d, dtype, rot, axes, fused, wide, norm, far)
    got = fa.norm_rope_forward(q, k, pos, plan(fa, rot, axis, il), q_weight=w[0], k_weight=w[1], norm=norm, eps=EPS)
    a = angle(pos, rot, axis)
    for name, x, y, wt in (("q", q, got[0], w[0]), ("k", k, got[1], w[1])):
        assert y.shape == x.shape and y.is_contiguous() and y.dtype == x.dtype
        want, bound = ref.forward(x.reshape(-1, x.shape[-2], d), wt, a, il, norm, EPS)
        ref.check(name, y, want, bound, dtype)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_backward(fa, case):
    import torch
    lead, Hq, Hkv, d, dtype, rot, axes, il, fused, wide, norm, far = CASES[case]
    q, k, w, pos, axis = make(torch, case, lead, Hq, Hkv, d, dtype, rot, axes, fused, wide, norm, far)
    dy = [torch.randn_like(x.contiguous()) for x in (q, k)]
    kw = dict(q_weight=w[0], k_weight=w[1], norm=norm, eps=EPS)
    p = plan(fa, rot, axis, il)
    got = fa.norm_rope_backward(q, k, *dy, pos, p, **kw)
    a = angle(pos, rot, axis)
    for i, (name, x) in enumerate((("q", q), ("k", k))):
        want, bound, dw, dw_bound = ref.backward(x.reshape(-1, x.shape[-2], d), dy[i].reshape(-1, x.shape[-2], d), w[i], a, il, norm, EPS)
        ref.check("d" + name, got[i], want, bound, dtype)
        if norm:
            assert got[2 + i].dtype == torch.float32
            ref.check(f"d{name}_weight", got[2 + i], dw, dw_bound, None)
        else:
            assert got[2 + i] is None
    again = fa.norm_rope_backward(q, k, *dy, pos, p, **kw)
    for x, y in zip(got, again):
        assert (x is None and y is None) or torch.equal(x, y)


# ------------------------------------------------------------------- into the 8-bit cache

APPENDS = [
    # H, Hkv, d, page, dtype, rot, axes, interleaved, norm, wide, new tokens of each request at each step
    (4, 1, 64, 16, "bf16", 64, 1, False, True, False, [[1], [1], [1]]),
    (6, 3, 128, 32, "f16", 96, 2, False, True, True, [[5, 0, 40], [1, 1, 1], [30, 7, 2]]),
    (8, 2, 128, 128, "bf16", 128, 1, True, False, False, [[200], [1], [90]]),
    (32, 8, 128, 64, "bf16", 128, 3, False, True, False, [[1] * 20, [1] * 20, [17] * 20]),
    (2, 2, 64, 16, "f16", 32, 1, True, True, True, [[700, 3], [1, 20], [0, 17]]),
    (12, 4, 64, 128, "bf16", 0, 1, False, True, False, [[33, 16], [1, 1], [15, 160]]),
    (8, 8, 64, 64, "bf16", 48, 4, False, True, False, [[2500, 3000], [1, 900], [40, 1]]),
]


def check_keys(torch, before, after, y, bound, slots, new):
    """The keys' side of a cache after tokens y (64 bits, within `bound`) went to `slots`: scales, new codes,
    what blocks held before rounded again, and all else as it was."""
    codes0, scales0, codes1, scales1 = (x.clone() for x in (*before, *after))
    pages, H, page, d = codes0.shape
    want_codes, want_scales = codes0.view(torch.uint8).clone(), scales0.clone()
    val = torch.tensor(kv8.VALUES, device="cuda")
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        e = t + 1
        while e < len(slots) and slots[e] == slots[e - 1] + 1 and slots[e] % 16:
            e += 1
        pg, at = slots[t] // page, slots[t] % page
        blk, off = at // 16, at % 16
        new, far = y[t:e].transpose(0, 1), bound[t:e].transpose(0, 1)     # [H, n, d]
        fine = torch.isfinite(new)
        mag = torch.where(fine, new.abs(), 0.0)
        lo = torch.where(fine, (mag - far).clamp(min=0), 0.0).amax((1, 2))
        hi = torch.where(fine, mag + far, 0.0).amax((1, 2))
        s = scales1[pg, :, blk].double()
        for h in range(H):
            least, most = (kv8.scale_of_amax(float(v[h])) for v in (lo, hi))
            if off:
                least, most = (max(v, float(scales0[pg, h, blk])) for v in (least, most))
            assert least <= float(s[h]) <= most, (t, h, least, float(s[h]), most)
        # the new codes
        got = val[codes1.view(torch.uint8)[pg, :, at:at + e - t].long()]
        assert torch.equal(torch.isnan(got), ~fine)
        x = torch.where(fine, new, 0.0) / s[:, None, None]
        room = torch.where(fine, far, 0.0) / s[:, None, None]
        step = torch.maximum((x.abs() + room) * 2.0 ** -4, torch.full_like(x, 2.0 ** -10))
        err = (torch.where(fine, got, 0.0) - x).abs()
        assert (err <= step + room).all(), float((err / (step + room)).max())
        # the tokens before them
        if off:
            held = want_codes[pg, :, blk * 16:at].cpu().numpy()
            ratio = (scales0[pg, :, blk].double() / s).cpu().numpy()
            want = kv8.e4m3_codes(kv8.VALUES[held] * ratio[:, None, None])
            mine = codes1.view(torch.uint8)[pg, :, blk * 16:at].cpu().numpy()
            assert np.array_equal(kv8.VALUES[want], kv8.VALUES[mine], equal_nan=True)
        for x0, x1, place in ((want_codes, codes1.view(torch.uint8), slice(blk * 16, at + e - t)), (want_scales, scales1, blk)):
            x0[pg, :, place] = x1[pg, :, place]
        t = e
    assert torch.equal(want_codes, codes1.view(torch.uint8)) and torch.equal(want_scales, scales1)


@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(fa, case):
    import torch
    Hq, Hkv, d, page, dtype, rot, axes, il, norm, wide, steps = APPENDS[case]
    rng = np.random.default_rng(case)
    B = len(steps[0])
    total = np.sum(steps, axis=0)
    width = int(-(-total.max() // page))
    pages = B * width + 2
    table = rng.permutation(pages)[:B * width].reshape(B, width)
    byte = lambda: torch.from_numpy(rng.integers(0, 256, (pages, Hkv, page, d)).astype(np.uint8)).cuda().view(torch.float8_e4m3fn)
    scale = lambda: torch.from_numpy(rng.uniform(0, 8, (pages, Hkv, page // 16)).astype(np.float32)).cuda()
    cache = fa.Kv8Cache((byte(), scale(), byte(), scale()))
    twin = fa.Kv8Cache([x.clone() for x in cache])
    have = np.zeros(B, int)
    for step, n in enumerate(steps):
        slots = []
        for b in range(B):
            for i in range(n[b]):
                pos = have[b] + i
                slots.append(table[b, pos // page] * page + pos % page)
            if b % 2:
                slots.append(-1)      # a token with no place
        have += n
        q, k, w, pos, axis = make(torch, 10 * case + step, (len(slots),), Hq, Hkv, d, dtype, rot, axes, True, wide, norm)
        v = torch.randn(len(slots), Hkv, d, device="cuda").to(q.dtype)
        if norm:
            w[1] = (w[1] * 3.0 ** step).to(w[1].dtype)
        else:
            k = (k * 3.0 ** step).to(k.dtype)
        if step == 2 and not rot:
            k = k.clone()
            k[0, 0, 3], k[-1, -1, 7] = torch.nan, torch.inf
        s = torch.tensor(slots, dtype=torch.int32, device="cuda")
        p = plan(fa, rot, axis, il)
        kw = dict(q_weight=w[0], k_weight=w[1], norm=norm, eps=EPS)
        old = cache.k8.clone(), cache.k_scale.clone()
        got = fa.kv8_append_norm_rope(cache, q, k, v, s, pos, p, **kw)
        assert torch.equal(got, fa.norm_rope_forward(q, k, pos, p, **kw)[0])
        y, bound = ref.forward(k, w[1], angle(pos, rot, axis), il, norm, EPS)
        check_keys(torch, old, (cache.k8, cache.k_scale), y, bound, slots, n)
        fa.kv8_append(twin, v, v, s)
        assert torch.equal(cache.v8.view(torch.uint8), twin.v8.view(torch.uint8)) and torch.equal(cache.v_scale, twin.v_scale)
