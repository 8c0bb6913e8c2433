"""The 8-bit paged cache on the GPU where a call can go wrong: rows that see nothing between long
requests, and others that come up in a server's batches."""
import numpy as np
import pytest

import kv8_ref as ref
import kv8_ref64 as r64

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- items without keys

# Long requests with requests that see nothing between them, one and several in a row, so many
# that every CTA has items of both kinds: (tokens, new tokens) of one stretch, repeated.
SEATS = {
    "one": [(4096, 1), (0, 1), (3000, 1)],
    "six": [(2048, 1)] + [(0, 1)] * 6 + [(129, 1)],
    "ends": [(0, 1)] * 5 + [(5000, 1)] + [(0, 1)] * 2,
    "short": [(1, 1), (0, 1), (128, 1), (0, 1), (0, 1)],
}


@pytest.mark.parametrize("Hkv", [1, 8])
@pytest.mark.parametrize("group", [1, 8, 16, 24])
@pytest.mark.parametrize("kind", list(SEATS))
def test_idle_seats_between_long_requests(fa, kind, group, Hkv):
    """Single tokens (up to 8 and up to 16 rows, and items of 128)."""
    times = 40 if Hkv == 1 else 10
    stretch = SEATS[kind] * times
    lens, new = [x[0] for x in stretch], [x[1] for x in stretch]
    c = r64.make(3, lens, new, group * Hkv, Hkv, 64 if group == 8 else 128, 64, "f16" if group == 1 else "bf16")
    r64.close(c, *r64.run(fa, c), r64.attend(c))


@pytest.mark.parametrize("Hkv", [1, 8])
@pytest.mark.parametrize("group,new", [(2, 4), (4, 4), (8, 20), (1, 300)])
def test_refused_prompts_between_long_requests(fa, group, new, Hkv):
    """Requests with more new tokens than keys: their first blocks of rows see nothing."""
    stretch = [(2500, new), (0, new), (3, new), (new // 2, new), (700, new), (0, new), (0, new), (0, new),
               (0, new), (0, new), (1500, 1)] * (8 if Hkv == 1 else 3)
    c = r64.make(4, [x[0] for x in stretch], [x[1] for x in stretch], group * Hkv, Hkv, 128, 32, "bf16")
    r64.close(c, *r64.run(fa, c), r64.attend(c))
    r64.close(c, *r64.run(fa, c, window=100), r64.attend(c, window=100))


def test_nothing_but_idle_seats(fa):
    for n, group in ((1, 8), (2, 8), (40, 8)):
        c = r64.make(5, [0] * 50, [n] * 50, group * 2, 2, 128, 64, "bf16")
        o, lse = r64.run(fa, c)
        assert (o == 0).all() and (lse == -float("inf")).all()


def test_a_refused_prompt_in_a_step(fa):
    """A prompt that kv8_plan refuses keeps its place in cu_seqlens; the others' rows are right."""
    import torch
    H, Hq, d, page, pages = 2, 8, 128, 64, 160
    cache = fa.kv8_cache(pages, H, d, page=page)
    grow = [3000, 500, 2500, 1, 400]
    T = sum(grow)
    table = torch.zeros(5, 60, dtype=torch.int32, device="cuda")
    ring = torch.arange(pages, dtype=torch.int32, device="cuda")
    state = torch.tensor([0, 100, 0], dtype=torch.int32, device="cuda")   # 100 free pages: 47 + 8 + 40 + 1
    lens = torch.zeros(5, dtype=torch.int32, device="cuda")
    x = torch.randn(T, Hq + 2 * H, d, device="cuda").bfloat16()
    ln, cu, slots, st = fa.kv8_plan(lens, torch.tensor(grow, dtype=torch.int32, device="cuda"), table, ring, state,
                                    page=page, tokens=T)
    assert ln.tolist() == [3000, 500, 2500, 1, 0] and st.tolist()[2] == 1
    fa.kv8_append(cache, x[:, Hq:Hq + H], x[:, Hq + H:], slots)
    c = dict(q=x[:, :Hq].contiguous(), cache=tuple(cache), table=table, lens=ln, cu=cu, new=grow, dtype="bf16")
    r64.close(c, *r64.run(fa, c), r64.attend(c))


# ------------------------------------------------------------------------- windows

@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 50, 2 ** 30, 140, 1])
@pytest.mark.parametrize("group,new", [(1, 9), (2, 8), (4, 200)])
def test_any_window_with_more_tokens_than_keys(fa, group, new, window):
    """Positions below 0 and windows as long as an int, in items of up to 8, 16 and 128 rows."""
    c = r64.make(6, [5, 300, 0, new // 2], [new, 1, new, new], group * 2, 2, 128, 16, "bf16")
    r64.close(c, *r64.run(fa, c, window=window), r64.attend(c, window=window))


# ------------------------------------------------------- queries that are not finite

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,group,new", [(128, 1, 6), (64, 2, 7), (128, 4, 6), (64, 1, 150)])
def test_queries_that_are_not_finite_and_rows_that_see_nothing(fa, d, group, new, dtype):
    """An infinity or NaN in a query makes its row NaN where the row sees a key, and no other row; a
    row that sees none has O = 0 and LSE = -inf, whatever its query holds."""
    import torch
    # positions from -3 on; pages that the cache does not have in the second and third
    c = r64.make(7, [new - 3, 200, 64 + new], [new, new, new], group * 2, 2, d, 16, dtype)
    c["table"][1, :] = -1
    c["table"][2, 4:] = 2 ** 30
    clean = r64.run(fa, c)
    want = r64.attend(c)
    r64.close(c, *clean, want)
    bad = torch.zeros(c["q"].shape[:2], dtype=torch.bool, device="cuda")
    for b in range(3):
        for i, (h, x) in zip((0, 2, 3, new - 1), ((0, "nan"), (1, "inf"), (group * 2 - 1, "-inf"), (0, "inf"))):
            c["q"][b * new + i, h, 5 * i % d] = float(x)
            bad[b * new + i, h] = True
    o, lse = r64.run(fa, c)
    sees = (want[1] > -float("inf")).T                     # [T, Hq]
    assert bool((sees & bad).any()) and bool((~sees & bad).any())
    assert torch.isnan(o[sees & bad]).all() and torch.isnan(lse.T[sees & bad]).all()
    assert (o[~sees] == 0).all() and (lse.T[~sees] == -float("inf")).all()
    fine = ~(sees & bad)
    assert torch.equal(o[fine], clean[0][fine]) and torch.equal(lse.T[fine], clean[1].T[fine])


def test_a_step_without_tokens(fa):
    """Plan, append and attend of a packed batch that holds no token."""
    import torch
    cache = fa.kv8_cache(8, 2, 128, page=16)
    was = [t.view(torch.uint8).clone() for t in cache]
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, table = torch.tensor([20, 0, 7], **i32), torch.tensor([[1, 2], [0, 0], [3, 0]], **i32)
    ln, cu, slots, st = fa.kv8_plan(lens, torch.zeros(3, **i32), table, torch.arange(8, **i32),
                                    torch.tensor([4, 4, 0], **i32), page=16, tokens=0)
    assert ln.tolist() == [20, 0, 7] and cu.tolist() == [0] * 4 and slots.numel() == 0 and st.tolist() == [4, 4, 0]
    x = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    fa.kv8_append(cache, x[:, 4:6], x[:, 6:], slots)
    for n in (1, 2 ** 30):
        o, lse = fa.attention_forward_kv8(x[:, :4], cache, table, ln, cu_seqlens=cu, max_seqlen=n)
        assert o.shape == (0, 4, 128) and lse.shape == (4, 0)
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(was, cache))
    fa.fa_device_status()


# --------------------------------------------------------------- scales in the writer

def _blocks(rng, dtype, n, d):
    """n blocks that hold some tokens at scales that are no powers of two, and tokens for the places
    behind them: codes [n, 1, 16, d], scales [n], offsets and values [n][new, d].  Many values lie so
    near the middle between two codes that a rounding on the way there decides otherwise."""
    import torch
    mid = (ref.VALUES[8:126] + ref.VALUES[9:127]) / 2           # ties of normal codes
    codes = rng.integers(0, 256, (n, 1, 16, d)).astype(np.uint8)
    scales, offs, new = np.empty(n), rng.integers(1, 16, n), []
    for i in range(n):
        x = torch.from_numpy(rng.normal(0, 1, (16 - offs[i], d))).to(r64.TYPES[dtype]).double().numpy()
        if i % 2:
            # the block keeps its scale: some value over it is a tie, but for 32 bits
            m = rng.choice(mid)
            s = np.float32(x.flat[0] / m if x.flat[0] else 1.0)
            s = abs(s) if abs(s) * 448 >= np.abs(x).max() else np.float32(abs(x.flat[0]) / mid[rng.integers(0, 9)])
            while s * 448 < np.abs(x).max():
                s = np.float32(s * 2)
        else:
            # the scale grows: some code held is a tie at the new one, but for 32 bits
            grown = ref.scale_of_amax(np.abs(x).max())
            c = rng.integers(16, 126)
            s = np.float32(rng.choice(mid[mid < ref.VALUES[c]]) * grown / ref.VALUES[c])
            codes[i, 0, :, ::3] = c
        scales[i] = s
        new.append(x)
    return codes, scales, offs, new


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_to_blocks_of_any_scale(fa, d, dtype):
    """Blocks that another writer began: e4m3(x / scale) and e4m3(code old / new), rounded once."""
    import torch
    rng = np.random.default_rng(d)
    n = 400
    codes, scales, offs, new = _blocks(rng, dtype, n, d)
    scales = scales.reshape(n, 1, 1)
    slots = np.concatenate([16 * i + np.arange(o, 16) for i, o in enumerate(offs)]).astype(np.int32)
    x = np.concatenate(new)[:, None]
    # rounding twice gives other codes
    keeps = np.arange(n) % 2 == 1
    with np.errstate(over="ignore"):
        twice = np.concatenate([(np.float32(v) * (np.float32(1) / np.float32(s))).astype(np.float64).ravel()
                                for v, s, k in zip(new, scales.ravel(), keeps) if k])
    once = np.concatenate([(v / s).ravel() for v, s, k in zip(new, scales.ravel(), keeps) if k])
    assert (ref.e4m3_codes(np.clip(twice, -448, 448)) != ref.e4m3_codes(once)).sum() > 10
    cache = []
    for _ in range(2):
        cache += [torch.from_numpy(codes.copy()).cuda().view(torch.float8_e4m3fn),
                  torch.from_numpy(scales.astype(np.float32)).cuda()]
    k = torch.from_numpy(x).to(r64.TYPES[dtype]).cuda()
    fa.kv8_append(fa.Kv8Cache(cache), k, k, torch.from_numpy(slots).cuda())
    ref.append(codes, scales, x, slots)
    for c, s in (cache[:2], cache[2:]):
        assert np.array_equal(s.double().cpu().numpy(), scales)
        got = c.view(torch.uint8).cpu().numpy()
        assert np.array_equal(ref.VALUES[got], ref.VALUES[codes], equal_nan=True), int((got != codes).sum())


def test_append_of_infinities_to_a_block_of_any_scale(fa):
    import torch
    cache = fa.kv8_cache(1, 1, 64, page=16)
    for s in (cache.k_scale, cache.v_scale):
        s.fill_(0.3)
    x = torch.zeros(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 1], x[1, 0, 2], x[2, 0, 3], x[2, 0, 4], x[2, 0, 5] = 3.0, float("inf"), float("-inf"), float("nan"), -0.3
    fa.kv8_append(cache, x, x, torch.arange(5, 8, dtype=torch.int32, device="cuda"))
    got = cache.k8.float()[0, 0, 5:8]
    assert torch.equal(cache.k_scale.flatten(), torch.full((1,), 0.3, device="cuda"))
    assert torch.isnan(got).nonzero().tolist() == [[1, 2], [2, 3], [2, 4]]
    assert got[0, 1] == 10 and got[2, 5] == -1 and torch.nan_to_num(got).abs().sum() == 11
    assert torch.equal(cache.k8.view(torch.uint8), cache.v8.view(torch.uint8))


# --------------------------------------------------------------------- hidden values

import test_kv8_gpu as base   # noqa: E402  (its cases, with a comparison that a NaN fails)


@pytest.mark.parametrize("case", base.CASES, ids=[str(i) for i in range(len(base.CASES))])
def test_no_nan_of_a_free_place_comes_out(fa, case):
    lens, new, Hq, Hkv, d, page, dtype, causal, window = case
    c = r64.make(8, lens, new, Hq, Hkv, d, page, dtype, spread=1.0)
    r64.close(c, *r64.run(fa, c, causal=causal, window=window), r64.attend(c, causal=causal, window=window))


NAN_CASES = [
    # (lens, new, Hq, Hkv, d, page, dtype, causal, window): up to 8, 16 and 128 rows, whole and split items
    ([300, 77], [4, 2], 4, 2, 128, 64, "bf16", True, 0),
    ([300, 77], [4, 2], 4, 2, 64, 16, "f16", True, 0),
    ([4000], [4], 4, 2, 128, 128, "bf16", True, 0),
    ([300, 77], [7, 3], 2, 2, 128, 32, "f16", True, 40),
    ([300, 200], [6, 8], 2, 2, 64, 32, "bf16", True, 3),
    ([300, 77], [4, 4], 8, 2, 128, 64, "bf16", True, 0),
    ([9000], [2], 16, 2, 64, 64, "f16", True, 0),
    ([300, 600], [5, 15], 2, 2, 128, 16, "bf16", True, 130),
    ([300, 77], [4, 2], 4, 2, 128, 64, "bf16", False, 0),
    ([300, 77], [20, 77], 4, 2, 128, 64, "f16", True, 0),
    ([300, 77], [20, 77], 4, 2, 64, 32, "f16", True, 40),
    ([3000, 700], [140, 40], 4, 2, 64, 64, "f16", True, 0),
    ([3000, 700], [140, 40], 4, 2, 128, 128, "bf16", True, 200),
    ([300, 77], [50, 77], 4, 2, 128, 16, "f16", False, 0),
]


@pytest.mark.parametrize("case", NAN_CASES, ids=[str(i) for i in range(len(NAN_CASES))])
def test_nan_reaches_the_rows_that_see_it(fa, case):
    """NaN codes among the values of some tokens: those channels of the rows that see them, of that
    head's queries, and nothing else; among the keys: those rows."""
    import torch
    lens, new, Hq, Hkv, d, page, dtype, causal, window = case
    c = r64.make(9, lens, new, Hq, Hkv, d, page, dtype, spread=1.0)
    kw = dict(causal=causal, window=window)
    clean = r64.run(fa, c, **kw)
    r64.close(c, *clean, r64.attend(c, **kw))
    spots = []                                             # (request, token, key/value head, channel)
    for b, (n, m) in enumerate(zip(lens, new)):
        first = n - m
        for i, j in enumerate({n - 1, n - 2, max(first, 0), max(first - window + 2, 0), n // 2, 0}):
            spots.append((b, j, i % Hkv, (37 * i + 5) % d))
    cu = c["cu"].tolist()

    def sees(b, j):
        pos = torch.arange(lens[b] - new[b], lens[b], device="cuda")
        see = torch.full_like(pos, j < lens[b], dtype=torch.bool)
        if causal:
            see = see & (j <= pos)
        if window:
            see = see & (pos - j < window)
        return see

    G = Hq // Hkv
    for side in (2, 0):                                    # values, then keys
        cache = list(c["cache"])
        cache[side] = codes = cache[side].view(torch.uint8).clone()
        want = torch.zeros(c["q"].shape, dtype=torch.bool, device="cuda")
        for b, j, h, ch in spots:
            codes[int(c["table"][b, j // page]), h, j % page, ch] = 127 if j % 2 else 255
            for g in range(h * G, h * G + G):
                want[cu[b]:cu[b + 1], g, ch if side else slice(None)] |= sees(b, j) if side else sees(b, j)[:, None]
        cache[side] = codes.view(torch.float8_e4m3fn)
        o, lse = r64.run(fa, c | dict(cache=tuple(cache)), **kw)
        assert torch.equal(torch.isnan(o), want)
        assert torch.equal(o[~want], clean[0][~want])
        if side:
            assert torch.equal(lse, clean[1])
        else:
            assert torch.equal(torch.isnan(lse), want[..., 0].T)
            assert torch.equal(lse[~want[..., 0].T], clean[1][~want[..., 0].T])


# ------------------------------------------------------- ranges that the header states

ROWS = [(2, 4), (8, 2), (4, 20)]        # (heads a group, new tokens): up to 8, 16 and 128 rows


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group,new", ROWS)
def test_queries_with_one_large_element(fa, group, new, dtype):
    """Elements of q far below the row's largest, and keys that are small where that one is: an
    element is held to 2^-17 of the largest."""
    import torch
    for large in (2.0 ** 10, 2.0 ** 13):
        c = r64.make(10, [700, 90], [new, new], group * 2, 2, 128, 64, dtype)
        c["q"][..., 7] = torch.where(torch.rand(c["q"].shape[:2], device="cuda") < 0.7, large, 1.0).to(c["q"].dtype)
        k8 = c["cache"][0].view(torch.uint8)
        k8[..., 7] = torch.where(k8[..., 7] & 127 == 127, k8[..., 7], 0)
        r64.close(c, *r64.run(fa, c), r64.attend(c))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("n", [200, 8192])
@pytest.mark.parametrize("first", [True, False])
def test_value_scales_far_apart(fa, first, n, group, new, dtype):
    """Blocks of values 2^99 / tokens apart, scores that are about the same: every key counts in the
    sum of the probabilities, wherever the large ones are (the first half of the blocks, every other
    one, and the last)."""
    import torch
    far = 99 - (n - 1).bit_length()
    for low in (-64, -80, 0):
        high = low + far
        if high > 120 or dtype == "f16" and high > 4:
            high = 4 if dtype == "f16" else 120
            low = high - far
            if low < -80:
                low = -80
        c = r64.make(11, [n], [new], group, 1, 64, 16, dtype)
        vs = c["cache"][3]
        blocks = c["table"][0, :-(-n // 16)].long()
        half = torch.zeros(len(blocks), dtype=torch.bool)
        if first:
            half[:len(half) // 2] = True
        else:
            half[1::2] = True
        half[-1] = not first
        vs[blocks, 0, 0] = torch.where(half.cuda(), 2.0 ** high, 2.0 ** low)
        if low == -64 and first:                           # blocks of zeros, as kv8_append writes them
            c["cache"][2].view(torch.uint8)[blocks[~half]] = 0
        c["q"] *= 0.25
        r64.close(c, *r64.run(fa, c), r64.attend(c))


@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("exponent", [-80, -64, 0, 100])
def test_value_scales_at_their_bounds(fa, exponent, group, new):
    c = r64.make(12, [3000, 40], [new, new], group * 2, 2, 128, 32, "bf16")
    c["cache"][3].mul_(2.0 ** 7 * 2.0 ** exponent)
    r64.close(c, *r64.run(fa, c), r64.attend(c))


# ------------------------------------------------------------------------ timeouts

@pytest.mark.parametrize("group,new", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_waits_that_run_out_over_many_short_items(fa, dtype, group, new):
    """Waits that give up, at once or later, in CTAs of some hundred items of a tile or two, requests
    without keys among them: the kernels end, and the next call is right."""
    import torch
    lens = [100, 200, 0, 30, 129, 0, 0, 64] * 500
    c = r64.make(13, lens, [min(new, max(n, 1)) for n in lens], group * 8, 8, 64, 16, dtype)
    want = r64.run(fa, c)
    args = c["q"], fa.Kv8Cache(c["cache"]), c["table"], c["lens"]
    for limit in (1, 300, 2000, 5000):
        fa.fa_set_wait_limit_cycles(limit)
        try:
            fa.attention_forward_kv8(*args, cu_seqlens=c["cu"], max_seqlen=new)
            status = fa.fa_device_status(check=False)
        finally:
            fa.fa_set_wait_limit_cycles(0)
        assert status in (fa.FA_OK, fa.FA_ERR_TIMEOUT) and (limit > 1 or status == fa.FA_ERR_TIMEOUT)
    got = r64.run(fa, c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
