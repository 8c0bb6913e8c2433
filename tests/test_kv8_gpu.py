"""The 8-bit paged cache on the GPU: block tables and slots, the writer, attention over it."""
import numpy as np
import pytest

import kv8_ref as ref

pytestmark = pytest.mark.gpu

# probabilities are rounded to 9 bits (bf16) or 11 (fp16) after a rounding to fp16's 11
P_ROUND = {"bf16": 2.0 ** -9 + 2.0 ** -11, "f16": 2.0 ** -11 + 2.0 ** -12}
OUT_ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def tdtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def f64(t):
    return t.double().cpu().numpy()


def to_cache(fa, codes, scales, vcodes, vscales):
    import torch
    return fa.Kv8Cache((dev(codes).view(torch.float8_e4m3fn), dev(scales.astype(np.float32)),
                        dev(vcodes).view(torch.float8_e4m3fn), dev(vscales.astype(np.float32))))


# ------------------------------------------------------------------------------- plan

@pytest.mark.parametrize("B,page,most,grow,ended,free,extra", [
    (1, 16, 0, 1, 0, 1.0, 0), (1, 128, 1000, 300, 0, 1.0, 7), (5, 64, 200, 1, 2, 1.0, 0),
    (64, 64, 4096, 1, 5, 1.0, 3), (300, 16, 700, 90, 40, 1.0, 500), (300, 32, 700, 90, 40, 0.5, 0),
    (40, 16, 300, 50, 10, 0.0, 0), (1500, 16, 100, 40, 300, 0.7, -100), (8192, 16, 40, 3, 1000, 0.9, 9),
])
def test_plan(fa, B, page, most, grow, ended, free, extra):
    rng = np.random.default_rng(B * page + grow)
    lens = rng.integers(0, most + 1, B)
    g = rng.integers(0, grow + 1, B)
    g[0] = grow
    g[rng.permutation(B)[:ended]] = -1
    width = (most + grow) // page + 1
    have, after = -(-lens // page), -(-(lens + np.maximum(g, 0)) // page)
    if B > 3:
        lens[1] = min(width * page, lens[1] + page * width)   # a full row: refused where it grows
        have[1], after[1] = -(-lens[1] // page), width
    left = int((after - have).sum() * free)
    pages = int(have.sum()) + left + 3
    ids = rng.permutation(pages)
    table = np.full((B, width), -9, np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    head = int(rng.integers(0, pages))
    ring = np.full(pages, -5, np.int32)
    for i in range(left):
        ring[(head + i) % pages] = ids[at + i]
    T = max(int(np.maximum(g, 0).sum()) + extra, 0)
    state = np.array([head, left, 77], np.int32)
    d = [dev(x.astype(np.int32)) for x in (lens, g, table, ring, state)]
    want = ref.plan(lens, g, table, ring, state, page, T)
    for _ in range(2):   # running it again on the same inputs gives the same outputs
        got = fa.kv8_plan(*d, page=page, tokens=T)
        for name, x, y in zip(("lens", "cu", "slots", "state"), got, want):
            assert np.array_equal(x.cpu().numpy(), y), name
        assert np.array_equal(d[2].cpu().numpy(), table)
        assert np.array_equal(d[3].cpu().numpy(), ring)


def test_plan_takes_broken_state(fa):
    """Lengths, counts and page ids outside their ranges are clamped or get no slot."""
    import torch
    lens = dev(np.array([-5, 1000, 20], np.int32))
    table = dev(np.array([[3, 9], [0, 1], [2, 99]], np.int32))
    ring = dev(np.array([50, -3, 1, 2], np.int32))
    state = dev(np.array([-2, 100, 0], np.int32))
    lens_out, cu, slots, st = fa.kv8_plan(lens, dev(np.array([1, 1, 1], np.int32)), table, ring, state,
                                          page=16, tokens=3)
    torch.cuda.synchronize()
    # request 0 (no tokens) takes ring[(-2) mod 4] = 1; 1 is full; 2's last page is none
    assert lens_out.tolist() == [1, 32, 21] and slots.tolist() == [16, -1, -1]
    assert cu.tolist() == [0, 1, 2, 3] and st.tolist() == [3, 3, 1]


# ----------------------------------------------------------------------------- append

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,page,steps", [(1, 16, [[1], [1], [1]]), (3, 32, [[5, 0, 40], [1, 1, 1], [30, 7, 2]]),
                                          (2, 128, [[200], [1], [90]]), (8, 64, [[1] * 20, [1] * 20, [17] * 20])])
def test_append_steps(fa, d, dtype, H, page, steps):
    """Several calls one after the other: every token held has the codes and scales of the plain form."""
    import torch
    rng = np.random.default_rng(d + H)
    B = len(steps[0])
    total = np.sum(steps, axis=0)
    width = int(-(-total.max() // page))
    pages = B * width + 2
    table = rng.permutation(pages)[:B * width].reshape(B, width)
    codes = rng.integers(0, 256, (2, pages, H, page, d)).astype(np.uint8)
    scales = rng.uniform(0, 8, (2, pages, H, page // 16)).astype(np.float32)
    cache = to_cache(fa, codes[0], scales[0], codes[1], scales[1])
    scales = scales.astype(np.float64)
    have = np.zeros(B, int)
    for step, n in enumerate(steps):
        slots, cuts = [], []
        for b in range(B):
            for i in range(n[b]):
                pos = have[b] + i
                slots.append(table[b, pos // page] * page + pos % page)
            if b % 2:
                slots.append(-1)      # a token with no place
        have += n
        slots = np.array(slots, np.int32)
        # magnitudes that rise from step to step, zeros, infinities and NaN among them; k and v
        # are slices of one wider tensor
        wide = rng.normal(0, 3.0 ** step, (len(slots), 3 * H, d))
        wide[rng.random(wide.shape) < 0.02] = 0
        if step == 2:
            wide[0, :, 3], wide[0, :, 5], wide[-1, :, 7] = np.inf, np.nan, -np.inf
        wide[:, 2 * H:] = 1e30
        x = dev(wide, tdtype(dtype))
        fa.kv8_append(cache, x[:, :H], x[:, H:2 * H], dev(slots))
        y = f64(x)
        for side in range(2):
            ref.append(codes[side], scales[side], y[:, side * H:side * H + H], slots)
    for side, (c, s) in enumerate(((cache.k8, cache.k_scale), (cache.v8, cache.v_scale))):
        # (a NaN has two codes)
        assert np.array_equal(ref.VALUES[c.view(torch.uint8).cpu().numpy()], ref.VALUES[codes[side]],
                              equal_nan=True)
        assert np.array_equal(f64(s), scales[side])


@pytest.mark.parametrize("dtype,values", [
    ("bf16", [0.0, 1e-30, 448.0, 449.0, 3.3e38, 2.0 ** -120, 1.75, 1.7578125, -896.0, 2.0 ** -64]),
    ("f16", [0.0, 6e-8, 448.0, 448.25, 65504.0, 6.1e-5, 1.75, 1.7509765625, -896.0, 2.0 ** -14]),
])
def test_append_scales_at_their_edges(fa, dtype, values):
    """amax just at and above 448 2^k, the smallest and largest numbers of the type."""
    cache = fa.kv8_cache(len(values), 1, 64, page=16)
    x = np.zeros((len(values), 1, 64))
    x[:, 0, 9] = values
    x[:, 0, 10:] = np.array(values)[:, None] * np.linspace(-1, 1, 54)
    k = dev(x, tdtype(dtype))
    slots = np.arange(len(values), dtype=np.int32) * 16
    fa.kv8_append(cache, k, k, dev(slots))
    codes, scales = np.zeros((len(values), 1, 16, 64), np.uint8), np.ones((len(values), 1, 1))
    ref.append(codes, scales, f64(k), slots)
    import torch
    assert np.array_equal(f64(cache.k_scale), scales) and np.array_equal(f64(cache.v_scale), scales)
    assert np.array_equal(cache.k8.view(torch.uint8).cpu().numpy(), codes)


# ----------------------------------------------------------------------------- attend

def make(rng, B, lens, new, Hq, Hkv, d, page, dtype, spread=0.0, q_scale=1.0):
    """A cache with `lens` tokens (in pages of no order, anything in the places no request holds:
    NaN codes, NaN scales), queries of the last `new` tokens."""
    width = max(-(-int(max(lens)) // page), 1) + 1
    pages = sum(-(-int(n) // page) for n in lens) + 3
    order = rng.permutation(pages)
    table = rng.integers(-2 ** 31, 2 ** 31 - 1, (B, width)).astype(np.int32)
    codes = rng.integers(0, 256, (2, pages, Hkv, page, d)).astype(np.uint8)
    scales = np.full((2, pages, Hkv, page // 16), np.nan)
    at = 0
    for b in range(B):
        for j in range(-(-int(lens[b]) // page)):
            pg = table[b, j] = order[at]
            at += 1
            held = min(page, int(lens[b]) - j * page)
            x = rng.normal(0, 1, (2, Hkv, held, d))
            codes[:, pg, :, :held] = ref.e4m3_codes(np.clip(x * 120, -448, 448))
            nb = -(-held // 16)
            scales[:, pg, :, :nb] = 2.0 ** np.round(rng.normal(0, spread, (2, Hkv, nb))) / 128
    T = int(sum(new))
    import torch
    q = torch.from_numpy(rng.normal(0, q_scale, (T, Hq, d))).to(tdtype(dtype))
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(q=q, codes=codes, scales=scales, table=table, lens=np.array(lens, np.int32), cu=cu, new=new)


def check(fa, c, d, dtype, causal=True, window=0, scale=None, dense=False):
    scale = d ** -0.5 if scale is None else scale
    cache = to_cache(fa, c["codes"][0], c["scales"][0], c["codes"][1], c["scales"][1])
    q = c["q"].cuda()
    Hq = q.shape[1]
    if dense:
        B, n = len(c["lens"]), c["new"][0]
        o, lse = fa.attention_forward_kv8(q.view(B, n, Hq, d), cache, dev(c["table"]), dev(c["lens"]),
                                          causal=causal, window=window, scale=scale)
        o, lse = o.view(B * n, Hq, d), lse.transpose(0, 1).reshape(Hq, B * n)
    else:
        o, lse = fa.attention_forward_kv8(q, cache, dev(c["table"]), dev(c["lens"]), causal=causal,
                                          window=window, scale=scale, cu_seqlens=dev(c["cu"]),
                                          max_seqlen=max(c["new"]))
    fa.fa_device_status()
    wo, wl, bo, bl = ref.attend(f64(c["q"]), c["codes"][0], c["scales"][0], c["codes"][1], c["scales"][1],
                                c["table"], c["lens"], c["cu"], scale, causal, window, P_ROUND[dtype],
                                OUT_ROUND[dtype])
    o, lse = f64(o), f64(lse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(wl))
    fine = np.isfinite(wl)
    assert (np.abs(lse - wl)[fine] <= bl[fine]).all(), float((np.abs(lse - wl)[fine] / bl[fine]).max())
    # below the least normal output a rounding is off by half the least step
    tiny = 2.0 ** -25 if dtype == "f16" else 2.0 ** -134
    bad = np.abs(o - wo) > bo + tiny
    assert not bad.any(), (int(bad.sum()), float((np.abs(o - wo) / (bo + tiny)).max()))
    return o, lse


CASES = [
    # (lens, new, Hq, Hkv, d, page, dtype, causal, window)
    ([1], [1], 1, 1, 128, 16, "bf16", True, 0),
    ([1], [1], 8, 1, 64, 128, "f16", True, 0),
    ([127, 128, 129, 1, 0, 255], [1] * 6, 8, 2, 128, 64, "bf16", True, 0),
    ([127, 128, 129, 1, 0, 255], [1] * 6, 8, 2, 64, 16, "bf16", True, 0),
    ([1000, 17, 300], [1] * 3, 4, 4, 128, 16, "f16", True, 0),
    ([700, 333, 5], [1] * 3, 32, 2, 128, 32, "bf16", True, 0),          # 16 heads a group
    ([700, 333, 5], [1] * 3, 40, 2, 64, 32, "f16", True, 0),           # 20 heads a group
    ([513], [1], 71, 1, 128, 128, "bf16", True, 0),                    # 71 heads a group
    ([513, 20], [1] * 2, 6, 2, 128, 64, "bf16", False, 0),
    ([4000, 2], [1] * 2, 8, 1, 128, 64, "bf16", True, 0),
    ([900, 100, 1], [1] * 3, 4, 2, 128, 64, "bf16", True, 100),        # sliding windows
    ([900, 129, 260], [1] * 3, 4, 2, 64, 16, "f16", True, 1),
    ([300, 40, 9, 130], [5, 1, 9, 2], 8, 2, 128, 64, "bf16", True, 0),   # drafts
    ([300, 40, 9, 130], [5, 0, 9, 2], 8, 2, 64, 16, "f16", True, 33),
    ([300, 40, 3, 0], [5, 1, 9, 2], 4, 4, 128, 64, "bf16", True, 0),     # rows that see nothing
    ([300, 40, 3, 0], [5, 1, 9, 2], 4, 4, 64, 32, "bf16", False, 0),
    ([257], [257], 2, 1, 128, 64, "bf16", True, 0),                     # a whole prompt
    ([260, 70], [130, 70], 6, 2, 64, 32, "f16", True, 0),
    ([400, 70], [200, 33], 3, 1, 128, 128, "bf16", True, 50),
    ([300], [150], 16, 2, 128, 16, "bf16", True, 0),
    ([140, 150], [129, 140], 4, 2, 128, 64, "f16", False, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention(fa, case):
    lens, new, Hq, Hkv, d, page, dtype, causal, window = case
    rng = np.random.default_rng(len(lens) * 1000 + d + Hq)
    c = make(rng, len(lens), lens, new, Hq, Hkv, d, page, dtype)
    check(fa, c, d, dtype, causal, window)


@pytest.mark.parametrize("B,most", [(257, 1), (700, 1), (700, 9), (300, 40)])
def test_attention_of_many_requests(fa, B, most):
    """More requests than a CTA has threads, long runs of requests without tokens among them."""
    rng = np.random.default_rng(B + most)
    lens = rng.integers(0, 150, B)
    lens[40:200] = 0
    lens[B - 1] = 900
    new = np.minimum(rng.integers(0, most + 1, B), lens)
    new[B - 1] = most
    c = make(rng, B, lens.tolist(), new.tolist(), 4, 2, 64, 16, "bf16")
    check(fa, c, 64, "bf16")


@pytest.mark.parametrize("window", [0, 100])
def test_more_new_tokens_than_announced(fa, window):
    """The rows of max_seqlen tokens of each request are right whatever the others hold."""
    rng = np.random.default_rng(16)
    c = make(rng, 3, [600, 450, 300], [1, 9, 1], 4, 2, 128, 64, "bf16")
    want = fa_out(fa, c, window=window)
    got = fa_out(fa, c, window=window, max_seqlen=1)
    fa.fa_device_status()
    for t in (0, 1, 10):
        # probabilities rounded to 9 and to 11 bits (2^-9 together at most), each output to bf16;
        # values are 448 / 128 at most
        assert (got[0][t].float() - want[0][t].float()).abs().max() <= 3 * 2.0 ** -8 * 3.5


def test_calls_and_graphs_at_once(fa):
    """Calls on two streams, each with its own workspace, and graphs of them that replay together."""
    import torch
    rng = np.random.default_rng(17)
    want, args = [], []
    for new, lens in ((1, [4000, 3000, 100] * 5), (50, [900, 2000] * 3)):
        c = make(rng, len(lens), lens, [new] * len(lens), 8, 2, 128, 64, "bf16")
        want.append(fa_out(fa, c))
        cache = to_cache(fa, c["codes"][0], c["scales"][0], c["codes"][1], c["scales"][1])
        args.append((c["q"].cuda(), cache, dev(c["table"]), dev(c["lens"]),
                     dict(cu_seqlens=dev(c["cu"]), max_seqlen=new)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    graphs, outs = [], []
    for s, (q, cache, table, lens, kw) in zip(streams, args):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(fa.attention_forward_kv8(q, cache, table, lens, **kw))
        graphs.append(g)
    for _ in range(20):
        got = [fa.attention_forward_kv8(q, cache, table, lens, stream=s, **kw)
               for s, (q, cache, table, lens, kw) in zip(streams, args)]
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, a, b in zip(want, got, outs):
            assert all(torch.equal(x, y) for x, y in zip(w, a)) and all(torch.equal(x, y) for x, y in zip(w, b))
    fa.fa_device_status()


def test_suite_under_the_bounds_checking_build(fa):
    """This file's tests again with the library that checks its indices; the status word has to be
    clear after each."""
    import os
    import subprocess
    import sys
    if fa.fa_debug_checks_enabled():
        pytest.skip("this is the checking build")
    from exact_io_aware_tcgen05_gb300 import build as b
    env = dict(os.environ, FA_GB300_LIBRARY=b.build(debug=True), FA_GB300_CHECK_STATUS="1")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                        os.path.join("tests", "test_kv8_gpu.py")], cwd=root, env=env, capture_output=True,
                       text=True, timeout=1200)
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout[-4000:], r.stderr[-2000:])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 3, 70])
def test_attention_dense(fa, n, dtype):
    rng = np.random.default_rng(n)
    c = make(rng, 3, [200, 71, 333], [n] * 3, 8, 2, 128, 64, dtype)
    check(fa, c, 128, dtype, dense=True)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
def test_attention_with_scales_far_apart(fa, d, dtype):
    """Blocks whose scales differ by many powers of two, sharp and flat rows."""
    rng = np.random.default_rng(5)
    c = make(rng, 2, [700, 90], [1, 4], 8, 2, d, 64, dtype, spread=4.0)
    check(fa, c, d, dtype)
    c = make(rng, 2, [700, 90], [1, 4], 8, 2, d, 64, dtype, q_scale=20.0)
    check(fa, c, d, dtype)


def test_attention_keeps_a_long_flat_tail(fa):
    """One key far above thousands of others whose weights, each 2^-13 or less of its, sum up to
    as much: none is lost."""
    rng = np.random.default_rng(6)
    n, d = 9000, 128
    c = make(rng, 1, [n], [1], 2, 1, d, 128, "bf16")
    ids = c["table"][0, :-(-n // 128)]
    codes = c["codes"][0]
    codes[ids, 0, :, 0] = ref.e4m3_codes(np.array(32.0))
    codes[ids[3], 0, 40, 0] = ref.e4m3_codes(np.array(448.0))
    codes[ids[:, None], 0, :, 1:] = 0
    c["scales"][0][ids] = 1 / 32.0
    c["q"][:] = 0
    c["q"][..., 0] = 0.75
    check(fa, c, d, "bf16", scale=1.0)


def test_hidden_values_stay_hidden(fa):
    """NaN codes in places that some rows see and others do not: only those rows' channels."""
    import torch
    rng = np.random.default_rng(7)
    for d, page, window in ((128, 64, 0), (64, 16, 0), (128, 32, 40)):
        c = make(rng, 2, [300, 77], [20, 77], 4, 2, d, page, "bf16")
        cu = c["cu"]
        at = lambda b, j: (c["table"][b, j // page], slice(None), j % page)   # noqa: E731
        for b, j, ch in ((0, 290, 3), (1, 50, 9), (1, 70, d - 1)):
            c["codes"][1][at(b, j)][:, ch] = 127
        clean = {**c, "codes": c["codes"].copy()}
        for b, j, ch in ((0, 290, 3), (1, 50, 9), (1, 70, d - 1)):
            clean["codes"][1][at(b, j)][:, ch] = 0
        cache = to_cache(fa, c["codes"][0], c["scales"][0], c["codes"][1], c["scales"][1])
        o, lse = fa.attention_forward_kv8(c["q"].cuda(), cache, dev(c["table"]), dev(c["lens"]),
                                          window=window, cu_seqlens=dev(cu), max_seqlen=77)
        fa.fa_device_status()
        want = np.zeros(o.shape, bool)
        for b, j, ch in ((0, 290, 3), (1, 50, 9), (1, 70, d - 1)):
            for i in range(c["new"][b]):
                pos = c["lens"][b] - c["new"][b] + i
                if j <= pos and (not window or pos - j < window):
                    want[cu[b] + i, :, ch] = True
        got = f64(o)
        assert np.array_equal(np.isnan(got), want)
        oc, lc = check(fa, clean, d, "bf16", window=window)
        assert np.array_equal(got[~want], oc[~want]) and np.array_equal(f64(lse), lc)
        # a key of NaN: the rows that see it, all their channels
        c = clean
        c["codes"][0][at(1, 60)][:, 5] = 255
        cache = to_cache(fa, c["codes"][0], c["scales"][0], c["codes"][1], c["scales"][1])
        o, lse = fa.attention_forward_kv8(c["q"].cuda(), cache, dev(c["table"]), dev(c["lens"]),
                                          window=window, cu_seqlens=dev(cu), max_seqlen=77)
        sees = np.zeros(o.shape[0], bool)
        for i in range(77):
            sees[cu[1] + i] = 60 <= i and (not window or i - 60 < window)
        assert np.array_equal(np.isnan(f64(o)), np.broadcast_to(sees[:, None, None], o.shape))
        assert np.array_equal(np.isnan(f64(lse)), np.broadcast_to(sees, lse.shape))


def test_queries_that_are_not_finite(fa):
    """An infinity or NaN in a query makes that row NaN and no other."""
    rng = np.random.default_rng(8)
    c = make(rng, 2, [200, 50], [1, 5], 8, 2, 128, 64, "bf16")
    clean = f64(fa_out(fa, c)[0])
    c["q"][0, 3, 7] = float("nan")
    c["q"][4, 1, 0] = float("inf")
    o = f64(fa_out(fa, c)[0])
    bad = np.zeros(o.shape, bool)
    bad[0, 3] = bad[4, 1] = True
    assert np.isnan(o[bad]).all() and np.array_equal(o[~bad], clean[~bad])


def fa_out(fa, c, **kw):
    cache = to_cache(fa, c["codes"][0], c["scales"][0], c["codes"][1], c["scales"][1])
    args = dict(cu_seqlens=dev(c["cu"]), max_seqlen=max(c["new"])) | kw
    return fa.attention_forward_kv8(c["q"].cuda(), cache, dev(c["table"]), dev(c["lens"]), **args)


def test_bad_pages_are_hidden(fa):
    rng = np.random.default_rng(9)
    c = make(rng, 3, [300, 80, 64], [1, 3, 1], 4, 2, 128, 32, "bf16")
    c["table"][0, 2], c["table"][0, 9] = -1, 2 ** 31 - 1
    c["table"][1, 1], c["table"][2, :2] = c["codes"].shape[1], -7
    check(fa, c, 128, "bf16")


def test_lengths_outside_their_range(fa):
    """Lengths are clamped to what a table row can hold."""
    rng = np.random.default_rng(10)
    c = make(rng, 2, [128, 64], [1, 1], 4, 2, 64, 64, "bf16")
    c["table"] = np.ascontiguousarray(c["table"][:, :2])
    c["table"][1, 1] = c["table"][0, 1]
    c["codes"][:, c["table"][0]] = 56
    c["scales"][:] = 1.0
    c["lens"][:] = (2 ** 31 - 1, -4)
    check(fa, c, 64, "bf16")


def test_rows_behind_the_last_request_are_left(fa):
    import torch
    rng = np.random.default_rng(11)
    c = make(rng, 2, [90, 30], [4, 2], 4, 2, 128, 64, "bf16")
    T = 6 + 50
    q = torch.randn(T, 4, 128, device="cuda").bfloat16()
    q[:6] = c["q"].cuda()
    out = torch.full((T, 4, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((4, T), 9.0, device="cuda")
    cache = to_cache(fa, c["codes"][0], c["scales"][0], c["codes"][1], c["scales"][1])
    ws = torch.empty(fa.fa_fwd_kv8_workspace_size(2, 4, 2, 4, 128, T), dtype=torch.uint8, device="cuda")
    r = fa.attention_forward_kv8(q, cache, dev(c["table"]), dev(c["lens"]), cu_seqlens=dev(c["cu"]),
                                 max_seqlen=4, out=out, lse=lse, workspace=ws)
    assert r[0] is out and r[1] is lse
    o, l = fa_out(fa, c)
    assert torch.equal(out[:6], o) and torch.equal(lse[:, :6], l)
    assert (out[6:] == 7).all() and (lse[:, 6:] == 9).all()


def test_slices_and_streams(fa):
    """q, k and v as slices of one projection's output, on a stream of the caller's."""
    import torch
    rng = np.random.default_rng(12)
    for new, dense in (([3, 2, 6], False), ([2, 2, 2], True)):
        c = make(rng, 3, [90, 30, 260], new, 4, 2, 128, 64, "bf16")
        want = fa_out(fa, c)
        T = sum(new)
        wide = torch.randn(T, 8, 128, device="cuda").bfloat16()
        wide[:, :4] = c["q"].cuda()
        q = wide[:, :4]
        kw = dict(cu_seqlens=dev(c["cu"]), max_seqlen=max(new))
        if dense:
            q, kw = wide.view(3, 2, 8, 128)[:, :, :4], {}
        cache = to_cache(fa, c["codes"][0], c["scales"][0], c["codes"][1], c["scales"][1])
        table, lens = dev(c["table"]), dev(c["lens"])
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for s in (side, side.cuda_stream):
            o, lse = fa.attention_forward_kv8(q, cache, table, lens, stream=s, **kw)
            side.synchronize()
            assert torch.equal(o.reshape(T, 4, 128), want[0])


def test_far_offsets(fa):
    """Pages whose codes lie beyond 2^32 bytes."""
    import torch
    H, page, d = 8, 128, 128
    pages = (1 << 32) // (H * page * d) + 40
    cache = fa.kv8_cache(pages, H, d, page=page)
    n = 300
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, device="cuda")
    slots = (table[0, pos // page] * page + pos % page).int()
    x = torch.randn(2, n, H, d, device="cuda").bfloat16()
    fa.kv8_append(cache, x[0], x[1], slots)
    small = fa.Kv8Cache([t[pages - 3:].clone() for t in cache])
    q = torch.randn(1, 1, 16, d, device="cuda").bfloat16()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    o, lse = fa.attention_forward_kv8(q, cache, table, lens)
    o2, lse2 = fa.attention_forward_kv8(q, small, table - (pages - 3), lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    k = (small.k8.float() * small.k_scale.repeat_interleave(16, 2)[..., None])[[2, 0, 1]]
    k = k.transpose(1, 2).reshape(-1, H, d)[:n]
    assert ((k - x[0].float()).abs() <= x[0].float().abs() * 2.0 ** -4 + 2.0 ** -9).all()


# ----------------------------------------------------------------------------- together

@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
def test_serving_steps_replayed_from_a_graph(fa, d, dtype):
    """Plan, append and attend, captured once and replayed as the requests grow, end and come
    anew; two graphs with workspaces of their own; every step against the plain forms."""
    import torch
    rng = np.random.default_rng(13)
    B, Hq, H, page, pages, width = 5, 8, 2, 16, 24, 8
    cache = fa.kv8_cache(pages, H, d, page=page)
    codes = np.zeros((2, pages, H, page, d), np.uint8)
    scales = np.ones((2, pages, H, page // 16))
    table, ring = np.zeros((B, width), np.int32), rng.permutation(pages).astype(np.int32)
    lens, state = np.zeros(B, np.int32), np.array([0, pages, 0], np.int32)
    dv = dict(lens=dev(lens), grow=dev(lens), table=dev(table), ring=dev(ring), state=dev(state))
    T = 24
    qkv = torch.zeros(T, Hq + 2 * H, d, device="cuda", dtype=tdtype(dtype))

    def step():
        ln, cu, slots, st = fa.kv8_plan(dv["lens"], dv["grow"], dv["table"], dv["ring"], dv["state"],
                                        page=page, tokens=T)
        fa.kv8_append(cache, qkv[:, Hq:Hq + H], qkv[:, Hq + H:], slots)
        o, lse = fa.attention_forward_kv8(qkv[:, :Hq], cache, dv["table"], ln, cu_seqlens=cu, max_seqlen=T)
        dv["lens"].copy_(ln)
        dv["state"].copy_(st)
        return ln, slots, st, o, lse

    keep = [dv[n].clone() for n in dv] + [t.clone() for t in cache]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for t, was in zip([dv[n] for n in dv] + list(cache), keep):
        t.copy_(was) if t.dtype != torch.float8_e4m3fn else t.view(torch.uint8).copy_(was.view(torch.uint8))
    refused = 0
    for i in range(14):
        grow = rng.integers(0, 2 if i % 3 else 8, B)
        if i % 4 == 3:
            grow[rng.integers(0, B)] = -1
        dv["grow"].copy_(dev(grow.astype(np.int32)))
        x = torch.from_numpy(rng.normal(0, 1 + i % 3, qkv.shape)).to(qkv.dtype)
        qkv.copy_(x)
        g, (ln, slots, st, o, lse) = graphs[i % 2]
        g.replay()
        fa.fa_device_status()
        lens, cu, want_slots, state = ref.plan(lens, grow, table, ring, state, page, T)
        assert np.array_equal(ln.cpu().numpy(), lens) and np.array_equal(st.cpu().numpy(), state)
        assert np.array_equal(slots.cpu().numpy(), want_slots)
        refused += int(state[2])
        x = f64(x)
        for sd in range(2):
            ref.append(codes[sd], scales[sd], x[:, Hq + sd * H:Hq + sd * H + H], want_slots)
        n = int(cu[-1])
        wo, wl, bo, bl = ref.attend(x[:n, :Hq], codes[0], scales[0], codes[1], scales[1], table, lens, cu,
                                    d ** -0.5, True, 0, P_ROUND[dtype], OUT_ROUND[dtype])
        assert (np.abs(f64(o)[:n] - wo) <= bo + 2.0 ** -25).all()
        assert (np.abs(f64(lse)[:, :n] - wl)[np.isfinite(wl)] <= bl[np.isfinite(wl)]).all()


def test_same_inputs_same_bits(fa):
    import torch
    rng = np.random.default_rng(14)
    c = make(rng, 3, [2000, 700, 64], [1, 3, 64], 8, 2, 128, 64, "bf16")
    a, b = fa_out(fa, c), fa_out(fa, c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_over_a_cache_against_the_16_bit_forward(fa):
    """A prompt written to the cache and attended to, next to attention_forward on the values
    that the cache holds (exact in bf16: a code has 4 significant bits)."""
    import torch
    B, N, Hq, H, d, page = 2, 200, 8, 2, 128, 64
    x = torch.randn(B * N, Hq + 2 * H, d, device="cuda").bfloat16()
    ring = torch.arange(8, dtype=torch.int32, device="cuda")
    table = torch.zeros(B, 4, dtype=torch.int32, device="cuda")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    state = torch.tensor([0, 8, 0], dtype=torch.int32, device="cuda")
    lens, cu, slots, state = fa.kv8_plan(zero, zero + N, table, ring, state, page=page, tokens=B * N)
    cache = fa.kv8_cache(8, H, d, page=page)
    fa.kv8_append(cache, x[:, Hq:Hq + H], x[:, Hq + H:], slots)
    o, lse = fa.attention_forward_kv8(x[:, :Hq], cache, table, lens, cu_seqlens=cu, max_seqlen=N)

    def held(codes, scales):
        y = codes.float() * scales.repeat_interleave(16, 2)[..., None]
        y = y[table.long()].transpose(2, 3).reshape(B, 4 * page, H, d)[:, :N]
        return y.bfloat16().contiguous()

    q = x[:, :Hq].reshape(B, N, Hq, d).contiguous()
    v = held(cache.v8, cache.v_scale)
    o2, lse2 = fa.attention_forward(q, held(cache.k8, cache.k_scale), v, causal=True)
    assert (lse - lse2.transpose(0, 1).reshape(Hq, -1)).abs().max() < 1e-4
    # each rounds its probabilities (half a step of bf16 at most) and its output (likewise)
    far = (o.float() - o2.reshape(B * N, Hq, d).float()).abs()
    assert far.max() <= 4 * 2.0 ** -8 * v.float().abs().max()


@pytest.mark.parametrize("n,d", [(1, 128), (1, 64), (40, 128), (40, 64)])
def test_wait_budget_expiry_reports_timeout_then_recovers(fa, n, d):
    """Waits that give up end the kernels, whatever the other warps were at."""
    rng = np.random.default_rng(15)
    lens = [3000, 700, 90, 200] * 6
    c = make(rng, len(lens), lens, [min(n, x) for x in lens], 8, 2, d, 64, "bf16")
    want = fa_out(fa, c)
    fa.fa_device_status()
    fa.fa_set_wait_limit_cycles(1)
    try:
        fa_out(fa, c)
        assert fa.fa_device_status(check=False) == fa.FA_ERR_TIMEOUT
    finally:
        fa.fa_set_wait_limit_cycles(0)
    assert fa.fa_device_status(check=False) == fa.FA_OK
    got = fa_out(fa, c)
    fa.fa_device_status()
    assert (got[0] == want[0]).all() and (got[1] == want[1]).all()
