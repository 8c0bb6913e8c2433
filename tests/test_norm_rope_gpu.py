"""Norms and rotation of queries and keys, their gradients, and the same on the way into the 8-bit
cache, on the GPU."""
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


def check_keys(torch, before, after, y, bound, slots):
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
        check_keys(torch, old, (cache.k8, cache.k_scale), y, bound, slots)
        fa.kv8_append(twin, v, v, s)
        assert torch.equal(cache.v8.view(torch.uint8), twin.v8.view(torch.uint8)) and torch.equal(cache.v_scale, twin.v_scale)


BEGUN = [
    # H, Hkv, d, page, dtype, tokens held, new tokens: blocks that another writer began, scales that are no
    # powers of two and larger or smaller than the new tokens want
    (2, 1, 64, 16, "bf16", [5, 15, 1], [1, 1, 1]),
    (8, 4, 128, 64, "f16", [3, 9, 70, 31], [20, 7, 300, 1]),
    (4, 8, 128, 32, "bf16", [13] * 40, [90] * 40),
]


@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("case", range(len(BEGUN)))
def test_append_to_blocks_that_others_began(fa, case, bad):
    import torch
    Hq, Hkv, d, page, dtype, held, new = BEGUN[case]
    rng = np.random.default_rng(50 + case)
    width = max(-(-(h + n) // page) for h, n in zip(held, new))
    pages = len(held) * width + 1
    table = rng.permutation(pages)[:len(held) * width].reshape(len(held), width)
    codes = [torch.from_numpy(rng.integers(0, 256, (pages, Hkv, page, d)).astype(np.uint8)).cuda().view(torch.float8_e4m3fn)
             for _ in range(2)]
    scales = [torch.from_numpy(2.0 ** rng.uniform(-9, 1, (pages, Hkv, page // 16)).astype(np.float32)).cuda() for _ in range(2)]
    cache = fa.Kv8Cache((codes[0], scales[0], codes[1], scales[1]))
    slots = [int(table[b, t // page]) * page + t % page for b in range(len(held)) for t in range(held[b], held[b] + new[b])]
    q, k, w, pos, axis = make(torch, case, (len(slots),), Hq, Hkv, d, dtype, d // 2, 1, False, False, True)
    v = torch.randn_like(k)
    if bad:
        k[:, 0, 3] = torch.inf        # all of a row becomes NaN or 0 by its norm
        k[::3, -1, 5] = torch.nan
    s = torch.tensor(slots, dtype=torch.int32, device="cuda")
    before = cache.k8.clone(), cache.k_scale.clone()
    kw = dict(q_weight=w[0], k_weight=w[1], eps=EPS)
    p = plan(fa, d // 2, axis, False)
    fa.kv8_append_norm_rope(cache, q, k, v, s, pos, p, **kw)
    y, bound = ref.forward(k, w[1], angle(pos, d // 2, axis), False, True, EPS)
    check_keys(torch, before, (cache.k8, cache.k_scale), y, bound.nan_to_num(0.0, 0.0), slots)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
def test_blocks_whose_tokens_come_in_several_runs(fa, d, dtype):
    """Two blocks' tokens in turn leave what these blocks hold undefined, and nothing else: the call
    ends, whatever the blocks' scales were, and the other blocks and the queries are as ever."""
    import torch
    Hkv, page, T = 3, 16, 5120          # 16 tokens in turn from two blocks, then 16 of one block, and so on
    rng = np.random.default_rng(d)
    pages = T // 32 * 3
    ids = rng.permutation(pages).reshape(-1, 3)
    slots = []
    for a, b, c in ids:
        slots += [int(x) * page + 1 + i for i in range(8) for x in (a, b)] + [int(c) * page + i for i in range(16)]
    for step in range(4):
        codes = [torch.from_numpy(rng.integers(0, 256, (pages, Hkv, page, d)).astype(np.uint8)).cuda().view(torch.float8_e4m3fn)
                 for _ in range(2)]
        scales = [torch.from_numpy(2.0 ** rng.uniform(-9, 1, (pages, Hkv, 1)).astype(np.float32)).cuda() for _ in range(2)]
        cache = fa.Kv8Cache((codes[0], scales[0], codes[1], scales[1]))
        q, k, w, pos, axis = make(torch, step, (T,), 4, Hkv, d, dtype, d, 1, False, False, False)
        k *= (2.0 ** -torch.arange(T, device="cuda").remainder(32).div(2, rounding_mode="floor"))[:, None, None] * 2.0 ** step
        s = torch.tensor(slots, dtype=torch.int32, device="cuda")
        before = cache.k8.clone(), cache.k_scale.clone()
        p = plan(fa, d, axis, False)
        got = fa.kv8_append_norm_rope(cache, q, k, torch.randn_like(k), s, pos, p, norm=False)
        torch.cuda.synchronize()
        assert torch.equal(got, fa.norm_rope_forward(q, k, pos, p, norm=False)[0])
        y, bound = ref.forward(k, None, angle(pos, d, axis), False, False, EPS)
        open_ = torch.from_numpy(ids[:, :2].copy()).cuda().flatten()
        for x, old in zip((cache.k8.view(torch.uint8), cache.k_scale), (before[0].view(torch.uint8), before[1])):
            x[open_] = old[open_]
        sure = [x if t % 32 >= 16 else -1 for t, x in enumerate(slots)]
        check_keys(torch, before, (cache.k8, cache.k_scale), y, bound, sure)


@pytest.mark.parametrize("norm,rot,il", [(False, 64, False), (False, 64, True), (False, 32, False), (True, 64, False), (False, 0, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinities_and_nan_stay_in_their_pairs(fa, norm, rot, il, dtype):
    import torch
    q, k, w, pos, axis = make(torch, 1, (6,), 3, 2, 64, dtype, rot, norm=norm)
    q[0, 0, 5], q[1, 1, 40], q[2, 2, 63], k[3, 0, 20], k[4, 1, 0] = torch.inf, torch.nan, -torch.inf, torch.inf, torch.nan
    got = fa.norm_rope_forward(q, k, pos, plan(fa, rot, axis, il), q_weight=w[0], k_weight=w[1], norm=norm)
    a = angle(pos, rot, axis)
    for x, y, wt in ((q, got[0], w[0]), (k, got[1], w[1])):
        want, bound = ref.forward(x, wt, a, il, norm, EPS)
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        inf = torch.isinf(want)
        assert torch.equal(torch.isinf(y), inf) and torch.equal(y[inf].double(), want[inf])
        fine = torch.isfinite(want)
        ref.check("fine", torch.where(fine, y, 0.0), torch.where(fine, want, 0.0), torch.where(fine, bound, 0.0), dtype)


def test_the_largest_and_smallest_numbers(fa):
    """fp16's largest numbers, zeros and rows far below eps."""
    import torch
    q, k, w, pos, axis = make(torch, 2, (5,), 2, 2, 128, "f16", 128)
    q[0] = 65504.0
    q[1] = 0.0
    q[2] = 2.0 ** -24
    k[3] *= 2.0 ** -12
    k[4, 0], k[4, 1] = -65504.0, 0.0
    got = fa.norm_rope_forward(q, k, pos, plan(fa, 128, axis, False), q_weight=w[0], k_weight=w[1])
    dy = [torch.randn_like(q), torch.randn_like(k)]
    grads = fa.norm_rope_backward(q, k, *dy, pos, plan(fa, 128, axis, False), q_weight=w[0], k_weight=w[1])
    a = angle(pos, 128, axis)
    for i, x in enumerate((q, k)):
        want, bound = ref.forward(x, w[i], a, False, True, EPS)
        ref.check("y", got[i], want, bound, "f16")
        want, bound, dw, dw_bound = ref.backward(x, dy[i], w[i], a, False, True, EPS)
        ref.check("dx", grads[i], want, bound, "f16")
        ref.check("dw", grads[2 + i], dw, dw_bound, None)


def test_positions_as_far_as_they_go(fa):
    import torch
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, -123456789, 10 ** 9]
    q, k, w, _, _ = make(torch, 3, (len(pos),), 2, 1, 128, "bf16", 128)
    freq = [1.0, 3.0, 0.7, 1e-9] + ref.frequencies(128)[4:]
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for il in (False, True):
        got = fa.norm_rope_forward(q, k, p, fa.rope_plan(freq, interleaved=il), norm=False)
        a = ref.exact_angles(pos, freq).cuda()
        for x, y in zip((q, k), got):
            # (a plan's frequency is the nearest 2^-64 of a turn: 2^-34 of a turn at 2^31)
            want, bound = ref.forward(x, None, a, il, False, EPS)
            ref.check("y", y, want, bound, "bf16")


def test_in_place_and_into_slices(fa):
    import torch
    T, Hq, Hkv, d = 700, 8, 2, 64
    _, _, w, pos, axis = make(torch, 4, (T,), Hq, Hkv, d, "bf16", 64)
    wide = torch.randn(T, Hq + 2 * Hkv, d, device="cuda").to(torch.bfloat16)
    q, k, v = wide[:, :Hq], wide[:, Hq:Hq + Hkv], wide[:, Hq + Hkv:]
    p, kw = plan(fa, 64, axis, False), dict(q_weight=w[0], k_weight=w[1])
    want = fa.norm_rope_forward(q, k, pos, p, **kw)
    dy = torch.randn_like(want[0]), torch.randn_like(want[1])
    grads = fa.norm_rope_backward(q, k, *dy, pos, p, **kw)
    # gradients into slices of the projection's, and in the place of dy
    into = torch.full_like(wide, 3.0)
    out = fa.norm_rope_backward(q, k, *dy, pos, p, out=(into[:, :Hq], into[:, Hq:Hq + Hkv]), **kw)
    assert out[0].data_ptr() == into.data_ptr() and torch.equal(into[:, :Hq], grads[0])
    assert torch.equal(into[:, Hq:Hq + Hkv], grads[1]) and (into[:, Hq + Hkv:] == 3).all()
    dz = [x.clone() for x in dy]
    out = fa.norm_rope_backward(q, k, *dz, pos, p, out=dz, **kw)
    assert all(torch.equal(a, b) for a, b in zip(dz, grads)) and torch.equal(out[2], grads[2])
    # the forward in its own place
    rest = v.clone()
    fa.norm_rope_forward(q, k, pos, p, out=(q, k), **kw)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, rest)


def test_offsets_beyond_32_bits(fa):
    import torch
    far = 2 ** 30
    big = torch.empty(2 * far + 1024, dtype=torch.bfloat16, device="cuda")
    q, k = big.as_strided((3, 4, 64), (far, 64, 1)), big.as_strided((3, 2, 64), (far, 64, 1), 512)
    a, b, w, pos, axis = make(torch, 5, (3,), 4, 2, 64, "bf16", 64)
    q.copy_(a)
    k.copy_(b)
    p, kw = plan(fa, 64, axis, False), dict(q_weight=w[0], k_weight=w[1])
    want = fa.norm_rope_forward(a, b, pos, p, **kw)
    got = fa.norm_rope_forward(q, k, pos, p, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    grads = fa.norm_rope_backward(a, b, *want, pos, p, **kw)
    out = fa.norm_rope_backward(q, k, *want, pos, p, out=(q, k), **kw)     # (in the place of q and k: row by row)
    assert all(torch.equal(x, y) for x, y in zip(out, grads))
    caches = [fa.kv8_cache(3, 2, 64, page=16) for _ in range(2)]
    q.copy_(a)
    k.copy_(b)
    s = torch.tensor([3, 4, 40], dtype=torch.int32, device="cuda")
    outs = [fa.kv8_append_norm_rope(c, x, y, y, s, pos, p, **kw) for c, x, y in zip(caches, (a, q), (b, k))]
    assert torch.equal(*outs)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(*caches))
    del big, q, k
    torch.cuda.empty_cache()


def test_no_tokens(fa):
    import torch
    q, k = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    p = plan(fa, 64, None, False)
    a, b = fa.norm_rope_forward(q, k, pos, p, q_weight=w, k_weight=w)
    assert a.shape == q.shape and b.shape == k.shape
    got = fa.norm_rope_backward(q, k, a, b, pos, p, q_weight=w, k_weight=w)
    assert (got[2] == 0).all() and (got[3] == 0).all()
    cache = fa.kv8_cache(2, 2, 64, page=16)
    assert fa.kv8_append_norm_rope(cache, q, k, k, pos, pos, p).shape == q.shape


def test_refusals(fa):
    import torch
    q, k, w, pos, _ = make(torch, 6, (5,), 4, 2, 64, "bf16", 64)
    p, p3 = plan(fa, 64, None, False), fa.rope_plan([1.0] * 32, axes=[0, 1, 2, 0] * 8)
    kw = dict(q_weight=w[0], k_weight=w[1])
    fwd = fa.norm_rope_forward
    for error, call in [
        (ValueError, lambda: fwd(q, k, None, p)), (ValueError, lambda: fwd(q, k, pos)),
        (TypeError, lambda: fwd(q, k, pos.long(), p)), (ValueError, lambda: fwd(q, k, pos[:4], p)),
        (ValueError, lambda: fwd(q, k, pos, p3)), (ValueError, lambda: fwd(q, k, torch.stack([pos] * 2), p3)),
        (TypeError, lambda: fwd(q, k, torch.stack([pos] * 5, 1).T[:3], p3)),
        (ValueError, lambda: fwd(q[:4], k, pos, p)), (ValueError, lambda: fwd(q, k[..., :32], pos, p)),
        (ValueError, lambda: fwd(q[..., :32], k[..., :32], pos, p)), (ValueError, lambda: fwd(q[0], k[0], pos, p)),
        (ValueError, lambda: fwd(q, k, pos.cpu(), p)), (ValueError, lambda: fwd(q, k.cpu(), pos, p)),
        (ValueError, lambda: fwd(q, k, pos, fa.rope_plan([1.0] * 32, device="cpu"))),
        (ValueError, lambda: fwd(q, k, pos, p, q_weight=w[0][:32])), (ValueError, lambda: fwd(q, k, pos, p, q_weight=w[0].cpu())),
        (TypeError, lambda: fwd(q, k, pos, p, q_weight=w[0].half())),
        (TypeError, lambda: fwd(q, k, pos, p, q_weight=w[0], k_weight=w[1].float())),
        (ValueError, lambda: fwd(q, k, pos, p, norm=False, **kw)), (fa.FAError, lambda: fwd(q, k, pos, p, eps=0.0)),
        (ValueError, lambda: fwd(q[:1].expand(5, 4, 64), k, pos, p)), (ValueError, lambda: fwd(q, k.transpose(0, 1), pos, p)),
        (ValueError, lambda: fwd(q, k, pos, p, out=(q, k[:, :1]))), (TypeError, lambda: fwd(q, k, pos, p, out=(q, k.float()))),
        (ValueError, lambda: fwd(q, k, pos, p, out=(q[:1].expand(5, 4, 64), k))),
        (ValueError, lambda: fa.norm_rope_backward(q, k, q, q, pos, p)),
        (ValueError, lambda: fa.norm_rope_backward(q, k, q[:4], k, pos, p)),
        (fa.FAError, lambda: fa.norm_rope_backward(q, k, q, k, pos, p, workspace=torch.empty(64, device="cuda"), **kw)),
        (ValueError, lambda: fa.norm_rope_backward(q, k, q, k, pos, p, workspace=torch.empty(1 << 20), **kw)),
    ]:
        with pytest.raises(error):
            call()
    cache = fa.kv8_cache(2, 2, 64, page=16)
    s = torch.arange(5, dtype=torch.int32, device="cuda")
    app = fa.kv8_append_norm_rope
    for error, call in [
        (ValueError, lambda: app(cache, q, q, q, s, pos, p)), (ValueError, lambda: app(cache, q, k, k[:, :1], s, pos, p)),
        (ValueError, lambda: app(cache, q, k, k[:4], s, pos, p)), (ValueError, lambda: app(cache, q, k, k, s[:4], pos, p)),
        (TypeError, lambda: app(cache, q, k, k, s.long(), pos, p)), (TypeError, lambda: app(cache, q, k, k.half(), s, pos, p)),
        (ValueError, lambda: app(cache, q[None], k[None], k[None], s, pos[None], p)),
        (ValueError, lambda: app(cache, q, k, k, s, pos, p, out=q[:, :2])),
    ]:
        with pytest.raises(error):
            call()
    fa.fa_device_status()


def test_streams_and_graphs(fa):
    """Calls on streams of their own at once, and captured ones replayed on new inputs."""
    import torch
    sets = [make(torch, 30 + i, (3000 + i,), 8, 2, 128, "bf16", 128) for i in range(2)]
    p = plan(fa, 128, None, False)

    def both(q, k, w, pos, stream=None):
        kw = dict(q_weight=w[0], k_weight=w[1], stream=stream)
        y = fa.norm_rope_forward(q, k, pos, p, **kw)
        return (*y, *fa.norm_rope_backward(q, k, *y, pos, p, **kw))

    want = [both(*s[:4]) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(10):
        for i, s in enumerate(sets):
            got[i] = both(*s[:4], stream=streams[i])
    torch.cuda.synchronize()
    for g, x in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, x))
    q, k, w, pos, _ = sets[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(q, k, w, pos)
    for seed in (50, 51):
        a, b, _, c, _ = make(torch, seed, (3000,), 8, 2, 128, "bf16", 128)
        q.copy_(a)
        k.copy_(b)
        pos.copy_(c)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(out, both(a, b, w, c)))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
def test_a_training_step(fa, dtype, d):
    """Projection's output -> norm and rotation -> attention -> back to the projection's gradient, against
    autograd in 64 bits."""
    import torch
    B, N, Hq, Hkv = 2, 300, 4, 2
    dt = ref.TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g, device="cuda").to(dt)
    w = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")) for _ in range(2)]
    do = torch.randn(B, N, Hq, d, generator=g, device="cuda").to(dt)
    pos = torch.arange(N, dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    p = plan(fa, d, None, False)
    q, k, v = x[..., :Hq, :], x[..., Hq:Hq + Hkv, :], x[..., Hq + Hkv:, :].contiguous()
    kw = dict(q_weight=w[0], k_weight=w[1])
    qr, kr = fa.norm_rope_forward(q, k, pos, p, **kw)
    o, lse = fa.attention_forward(qr, kr, v, causal=True)
    dqr, dkr, dv = fa.attention_backward(qr, kr, v, o, lse, do, causal=True)
    dx = torch.empty_like(x)
    _, _, dqw, dkw = fa.norm_rope_backward(q, k, dqr, dkr, pos, p, out=(dx[..., :Hq, :], dx[..., Hq:Hq + Hkv, :]), **kw)
    dx[..., Hq + Hkv:, :] = dv
    fa.fa_device_status()

    xd, wd = x.double().requires_grad_(), [t.double().requires_grad_() for t in w]
    a = ref.angles(pos.view(-1), ref.frequencies(d))

    def side(t, wt):
        t = t.reshape(B * N, -1, d)
        n = t / torch.sqrt(t.square().mean(-1, keepdim=True) + EPS) * wt
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
        u, z = n[..., :d // 2], n[..., d // 2:]
        return torch.cat([u * c - z * s, z * c + u * s], -1).view(B, N, -1, d).transpose(1, 2)

    qd, kd = side(xd[..., :Hq, :], wd[0]), side(xd[..., Hq:Hq + Hkv, :], wd[1])
    vd = xd[..., Hq + Hkv:, :].transpose(1, 2)
    kd, vd = (t.repeat_interleave(Hq // Hkv, 1) for t in (kd, vd))
    s = (qd @ kd.transpose(2, 3)) * d ** -0.5
    s = s.masked_fill(torch.ones(N, N, device="cuda").triu(1).bool(), -torch.inf)
    od = (torch.softmax(s, -1) @ vd).transpose(1, 2)
    od.backward(do.double())
    # as for the attention's own gradients: probabilities, scores' gradients and outputs are rounded to 16 bits
    rel = lambda u, z: float((u.double() - z.detach()).norm() / z.detach().norm())
    assert rel(o, od) < 2e-2
    for name, u, z in (("dx", dx, xd.grad), ("dq_weight", dqw, wd[0].grad), ("dk_weight", dkw, wd[1].grad)):
        assert rel(u, z) < 2e-2, name


@pytest.mark.parametrize("d,dtype,page", [(128, "bf16", 64), (64, "f16", 16)])
def test_serving_steps_replayed_from_a_graph(fa, d, dtype, page):
    """plan, append and attention behind shared prefixes as one captured step, replayed while the requests
    grow, end and begin: each step's cache and outputs as by calls one by one, and the outputs as by the
    formula over that cache."""
    import torch
    import kv8_ref64
    import test_kv8_prefix_gpu as prefix
    Hq, Hkv, B, T, width, pages = 8, 2, 5, 12, 6, 60
    g = torch.Generator(device="cuda").manual_seed(d)
    dt = ref.TYPES[dtype]
    dev = dict(device="cuda")
    w = [(1 + 0.2 * torch.randn(d, generator=g, **dev)).to(dt) for _ in range(2)]
    p = plan(fa, d, None, False)
    kw = dict(q_weight=w[0], k_weight=w[1])
    # two prefixes on pages 0 .. of their own
    P = [3 * page - 5, page + 1]
    prefix_table = torch.tensor([[0, 1, 2], [3, 4, 0]], dtype=torch.int32, **dev)
    prefix_lens = torch.tensor(P, dtype=torch.int32, **dev)

    def start():
        cache = fa.kv8_cache(pages, Hkv, d, page=page)
        for row, n in zip(prefix_table, P):
            at = torch.arange(n, **dev)
            slots = (row[at // page] * page + at % page).int()
            gg = torch.Generator(device="cuda").manual_seed(n)
            x = torch.randn(n, 3 * Hkv, d, generator=gg, **dev).to(dt)
            fa.kv8_append_norm_rope(cache, x[:, :Hkv], x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:], slots, at.int(), p, **kw)
        ring = torch.cat([torch.arange(5, pages, dtype=torch.int32, **dev), torch.full((5,), -1, dtype=torch.int32, **dev)])
        return dict(cache=cache, lens=torch.zeros(B, dtype=torch.int32, **dev), table=torch.full((B, width), -1, dtype=torch.int32, **dev),
                    ring=ring, state=torch.tensor([0, pages - 5, 0], dtype=torch.int32, **dev))

    group = torch.tensor([0, 0, 0, 1, 1], **dev)   # requests 0 .. 2 behind the first prefix

    def step(st, x, grow):
        lens, cu, slots, state = fa.kv8_plan(st["lens"], grow, st["table"], st["ring"], st["state"], page=page, tokens=T)
        # a token's position: its prefix, its request's length before, its place among the new ones
        t = torch.arange(T, **dev)
        b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
        pos = (prefix_lens[group[b]] + lens[b] - (cu[b + 1] - cu[b]) + t - cu[b]).int()
        q = fa.kv8_append_norm_rope(st["cache"], x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots, pos, p, **kw)
        bounds = torch.stack([cu[0], cu[3], cu[5]])
        o, lse = fa.attention_forward_kv8_prefix(q, st["cache"], prefix_table, prefix_lens, bounds, st["table"], lens,
                                                 cu_seqlens=cu, max_seqlen=T)
        st["lens"].copy_(lens)
        st["state"].copy_(state)
        return q, o, lse, cu

    x, grow = torch.zeros(T, Hq + 2 * Hkv, d, dtype=dt, **dev), torch.zeros(B, dtype=torch.int32, **dev)
    plain, held = start(), start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(start(), x, grow)     # (warm-up, on a cache of its own)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(held, x, grow)
    for grows in ([3, 1, 4, 0, 2], [1, 1, 1, 1, 1], [-1, 2, 0, 5, 1], [7, 0, 1, -1, 1], [1, 1, 1, 1, 1]):
        x.copy_(torch.randn(x.shape, generator=g, **dev))
        grow.copy_(torch.tensor(grows, dtype=torch.int32))
        graph.replay()
        q, o, lse, cu = step(plain, x, grow)
        n = int(cu[-1])
        assert torch.equal(q, captured[0]) and torch.equal(o[:n], captured[1][:n]) and torch.equal(lse[:, :n], captured[2][:, :n])
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(plain["cache"], held["cache"]))
        c = dict(q=q[:n], cache=tuple(plain["cache"]), table=plain["table"], lens=plain["lens"], cu=cu, dtype=dtype,
                 prefix_table=prefix_table, prefix_lens=prefix_lens, prefix_cu=torch.stack([cu[0], cu[3], cu[5]]))
        kv8_ref64.close(c, o[:n], lse[:, :n], prefix.attend(c))
    fa.fa_device_status()


@pytest.mark.parametrize("name", ["test_norm_rope_gpu.py", "test_kv8_prefix_gpu.py"])
def test_suites_under_the_bounds_checking_build(fa, name):
    """These tests again with the library that checks its indices; the status word has to be clear after
    each."""
    import os
    import subprocess
    import sys
    if fa.fa_debug_checks_enabled():
        pytest.skip("this is the checking build")
    from exact_io_aware_tcgen05_gb300 import build as b
    env = dict(os.environ, FA_GB300_LIBRARY=b.build(debug=True), FA_GB300_CHECK_STATUS="1")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                        os.path.join("tests", name)], cwd=root, env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout[-4000:], r.stderr[-2000:])
