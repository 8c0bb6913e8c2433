"""Attention over shared prefixes in the 8-bit cache on the GPU."""
import math

import pytest

import kv8_ref64 as ref

pytestmark = pytest.mark.gpu


def make(seed, groups, Hq, Hkv, d, page, dtype, spread=0.0, behind=0):
    """`groups`: (tokens of the prefix or None for requests outside all groups, [(own tokens, new ones), ...]);
    requests outside groups come first or last."""
    import torch
    requests = [r for _, rs in groups for r in rs]
    prefixes = [(n, rs) for n, rs in groups if n is not None]
    lens, new = [r[0] for r in requests], [r[1] for r in requests]
    c = ref.make(seed, lens + [n for n, _ in prefixes], new + [0] * len(prefixes), Hq, Hkv, d, page, dtype, spread)
    B, dev = len(requests), "cuda"
    first = sum(r[1] for r in groups[0][1]) if groups[0][0] is None else 0
    cu = [first]
    for _, rs in prefixes:
        cu.append(cu[-1] + sum(r[1] for r in rs))
    c |= dict(prefix_table=c["table"][B:].contiguous(), prefix_lens=c["lens"][B:].contiguous(),
              prefix_cu=torch.tensor(cu, dtype=torch.int32, device=dev), table=c["table"][:B].contiguous(),
              lens=c["lens"][:B].contiguous(), cu=c["cu"][:B + 1].contiguous(), new=new)
    if behind:
        c["q"] = torch.cat([c["q"], torch.randn(behind, Hq, d, device=dev).to(c["q"].dtype)])
    return c


def attend(c, scale=None):
    """O, LSE and bounds as in kv8_ref64.attend, for sequences of a prefix and a request's own tokens.  The
    join adds a rounding of each part's LSE (2^-24 of it, which changes its weight by as much) and a few of
    32 bits."""
    import torch
    q, (k8, ks, v8, vs), dtype = c["q"].double(), c["cache"], c["dtype"]
    T, Hq, d = q.shape
    pages, H, page = k8.shape[:3]
    scale = d ** -0.5 if scale is None else scale
    o, bo = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((Hq, T), -math.inf, dtype=torch.float64, device=q.device)
    bl = torch.zeros_like(lse)
    cu, lens, pcu, plens = (c[n].tolist() for n in ("cu", "lens", "prefix_cu", "prefix_lens"))

    def keys(table, total, codes, scales):
        total = min(max(total, 0), table.numel() * page)
        ids = table[:-(-total // page)].long()
        known = (ids >= 0) & (ids < pages)
        x, s = ref._side(codes, scales, torch.where(known, ids, 0), total)
        known = known.repeat_interleave(page)[:total]
        return x, s, known

    for b, total in enumerate(lens):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        g = [p for p in range(len(plens)) if pcu[p] <= cu[b] < pcu[p + 1]]
        parts = [(c["prefix_table"][g[0]], plens[g[0]])] if g else []
        parts.append((c["table"][b], total))
        k = torch.cat([keys(t, m, k8, ks)[0] for t, m in parts], 1)
        v, vscale, known = zip(*[keys(t, m, v8, vs) for t, m in parts])
        v, vscale, known = torch.cat(v, 1), torch.cat(vscale, 1), torch.cat(known)
        total = k.shape[1]
        if total == 0:
            continue
        pos = torch.arange(total - n, total, device=q.device)[:, None]
        see = (torch.arange(total, device=q.device) <= pos) & known
        any_row = see.any(0)
        v = torch.where(any_row[:, None], v, 0.0)
        vscale = torch.where(any_row, vscale, 0.0)
        rows = slice(cu[b], cu[b + 1])
        for h in range(Hq):
            i = h // (Hq // H)
            x = q[rows, h]
            s = (scale * (x @ k[i].T)).masked_fill(~see, -math.inf)
            size = scale * (x.abs() @ k[i].abs().T) + 2.0 ** 1.25 * scale * x.abs().amax(1, keepdim=True) * k[i].abs().sum(1)
            size = size.masked_fill(~see, 0.0).amax(1)
            z = torch.logsumexp(s, 1)
            zz = torch.where(z > -math.inf, z, 0.0)
            p = torch.exp(s - zz[:, None])
            lse[h, rows] = z
            o[rows, h] = p @ v[i]
            # (a part's LSE may be below the joint one; where its rounding is larger it counts for as much less)
            e = 2.0 ** -19 * size + 2.0 ** -19 + 2.0 ** -22 * zz.abs()
            bl[h, rows] = 2 * e
            lost = 2.0 ** -28 * (p * vscale[i]).amax(1) * 448 * see.sum(1)
            far = (ref.P_ROUND[dtype] + 2 * e)[:, None] * (p @ v[i].abs()) + lost[:, None]
            bo[rows, h] = far + ref.OUT_ROUND[dtype] * (o[rows, h].abs() + far)
    return o, lse, bo, bl


def run(fa, c, **kw):
    args = dict(cu_seqlens=c["cu"], max_seqlen=max(c["new"])) | kw
    out = fa.attention_forward_kv8_prefix(c["q"], fa.Kv8Cache(c["cache"]), c["prefix_table"], c["prefix_lens"],
                                          c["prefix_cu"], c["table"], c["lens"], **args)
    fa.fa_device_status()
    return out


CASES = [
    # groups, Hq, Hkv, d, page, dtype
    ([(1, [(1, 1)])], 1, 1, 64, 16, "bf16"),
    ([(1000, [(7, 1), (300, 1)])], 8, 8, 128, 64, "bf16"),
    ([(129, [(5, 5), (1, 1), (40, 3)])], 8, 2, 64, 16, "f16"),
    ([(0, [(20, 1), (300, 2)]), (2000, [(1, 1)] * 9), (33, [(0, 0), (64, 64)])], 12, 4, 128, 32, "bf16"),
    ([(None, [(50, 2), (9, 1)]), (700, [(17, 1), (18, 2)]), (64, [(130, 1)])], 16, 2, 64, 64, "f16"),
    ([(777, [(90, 30), (700, 1)]), (None, [(128, 128), (3, 0), (1, 1)])], 4, 4, 128, 128, "f16"),
    ([(5000, [(100 + 3 * i, 1) for i in range(64)])], 32, 8, 128, 64, "bf16"),
    ([(3000, [(200, 200), (1, 1), (77, 50)]), (4097, [(300, 128)] * 3)], 16, 4, 64, 16, "bf16"),
    ([(400, [(0, 0)]), (300, [(2, 2)]), (200, [(0, 0), (1, 1)])], 5, 1, 128, 16, "bf16"),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_formula(fa, case):
    c = make(case, *CASES[case], spread=case % 3)
    ref.close(c, *run(fa, c), attend(c))


@pytest.mark.parametrize("n,dtype", [(1, "bf16"), (3, "f16"), (70, "bf16")])
def test_dense(fa, n, dtype):
    B = 5
    c = make(n, [(500, [(n + 11 * i, n) for i in range(2)]), (90, [(n + i, n) for i in range(3)])], 8, 2, 64, 32, dtype)
    want = attend(c)
    q = c["q"]
    c["q"] = q.view(B, n, 8, 64)
    o, lse = run(fa, c, cu_seqlens=None, max_seqlen=None)
    assert o.shape == (B, n, 8, 64) and lse.shape == (B, 8, n)
    ref.close(c, o.view(B * n, 8, 64), lse.transpose(0, 1).reshape(8, B * n), want)


def test_scale_and_far_scales(fa):
    c = make(3, [(600, [(100, 4), (50, 1)])], 8, 2, 128, 64, "bf16", spread=6.0)
    ref.close(c, *run(fa, c, scale=0.3), attend(c, scale=0.3))


def test_nothing_to_see(fa):
    """Empty prefixes and requests without tokens: O = 0 and LSE = -inf."""
    import torch
    c = make(5, [(0, [(0, 0), (4, 4)]), (40, [(3, 3)])], 8, 2, 64, 16, "bf16")
    c["lens"][1] = 0       # its 4 new tokens got no place
    c["prefix_lens"][1] = -7
    o, lse = run(fa, c)
    assert (o[:4] == 0).all() and (lse[:, :4] == -math.inf).all()
    ref.close(c, o, lse, attend(c))
    assert torch.isfinite(lse[:, 4:]).all()


def test_rows_behind_the_last_request_are_left(fa):
    import torch
    c = make(6, [(300, [(10, 2), (70, 1)])], 8, 2, 128, 64, "f16", behind=3)
    want = attend(c)
    out = torch.full_like(c["q"], 7.0)
    lse = torch.full((8, len(c["q"])), 9.0, device="cuda")
    run(fa, c, out=out, lse=lse)
    assert (out[3:] == 7).all() and (lse[:, 3:] == 9).all()
    c["q"] = c["q"][:3]
    ref.close(c, out[:3], lse[:, :3], [x[:3] if x.shape[0] == 6 else x[:, :3] for x in want])


def test_bad_pages_and_lengths(fa):
    """Pages that the cache does not have hide their tokens; lengths beyond the table are cut."""
    c = make(7, [(500, [(200, 3), (40, 1)])], 8, 2, 64, 16, "bf16")
    c["prefix_table"][0, 3], c["prefix_table"][0, 30], c["table"][0, 1] = -1, 2 ** 31 - 1, -5
    ref.close(c, *run(fa, c), attend(c))
    c["prefix_table"] = c["prefix_table"][:, :31].contiguous()   # 496 of the 500
    c["prefix_lens"][0] = 2 ** 31 - 1
    ref.close(c, *run(fa, c), attend(c))


def test_nan_stays_with_those_who_see_it(fa):
    import torch
    c = make(8, [(64, [(40, 2)]), (64, [(50, 2)])], 4, 2, 64, 16, "bf16")
    want = attend(c)
    v8 = c["cache"][2].view(torch.uint8)
    v8[c["prefix_table"][0, 1].long(), 1, 5, 9] = 127                 # seen by the first group alone
    v8[c["table"][1, 3].long(), 0, 1, 3] = 127                        # by the second request's second token
    o, lse = run(fa, c)
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[0:2, 2:4, 9] = True
    bad[3, 0:2, 3] = True
    assert torch.equal(torch.isnan(o), bad)
    ref.close(c, torch.where(bad, want[0].to(o.dtype), o), lse, want)
    assert torch.isfinite(lse).all()


def test_as_without_sharing(fa):
    """Against attention over tables that name the prefix's pages for every request."""
    import torch
    page, P = 64, 640
    c = make(9, [(P, [(30 + 7 * i, 1 + i % 3) for i in range(12)])], 16, 4, 128, page, "f16")
    table = torch.cat([c["prefix_table"][:, :P // page].expand(12, -1), c["table"]], 1).contiguous()
    o, lse = run(fa, c)
    o2, lse2 = fa.attention_forward_kv8(c["q"], fa.Kv8Cache(c["cache"]), table, c["lens"] + P, cu_seqlens=c["cu"],
                                        max_seqlen=max(c["new"]))
    want, _, bo, _ = attend(c)
    assert ((o.double() - o2.double()).abs() <= 2 * bo).all()
    assert (lse - lse2).abs().max() < 1e-4


def test_streams_graphs_and_two_calls_at_once(fa):
    import torch
    cs = [make(20 + i, [(900 + i, [(60, 2), (300, 1), (5, 1)])], 8, 2, 128, 64, "bf16") for i in range(2)]
    want = [run(fa, c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(20):
        for i, c in enumerate(cs):
            got[i] = fa.attention_forward_kv8_prefix(
                c["q"], fa.Kv8Cache(c["cache"]), c["prefix_table"], c["prefix_lens"], c["prefix_cu"], c["table"],
                c["lens"], cu_seqlens=c["cu"], max_seqlen=2, stream=streams[i])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [fa.attention_forward_kv8_prefix(
            c["q"], fa.Kv8Cache(c["cache"]), c["prefix_table"], c["prefix_lens"], c["prefix_cu"], c["table"], c["lens"],
            cu_seqlens=c["cu"], max_seqlen=2) for c in cs]
    for _ in range(3):
        for o, lse in outs:
            o.zero_()
            lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(outs, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    fa.fa_device_status()
