"""Attention over the 8-bit cache in 64 bits, by torch operations on whole requests (kv8_ref.py has
the same a row at a time), for batches of many keys: random caches, the formula, bounds on the
kernels' errors, and a comparison that a NaN fails."""
from __future__ import annotations

import math

import torch

BLOCK = 16

# a probability's rounding: to 9 bits (bf16, up to 16 rows) or 11, after one to fp16's 11
P_ROUND = {"bf16": 2.0 ** -9 + 2.0 ** -11, "f16": 2.0 ** -11 + 2.0 ** -12}
OUT_ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def make(seed, lens, new, Hq, Hkv, d, page, dtype, spread=0.0, device="cuda"):
    """A cache with `lens` tokens (pages in no order; any byte, NaN among them, and NaN scales in the
    places that no request holds) and queries of each request's last `new` tokens."""
    g = torch.Generator(device=device).manual_seed(seed)
    kw = dict(generator=g, device=device)
    B = len(lens)
    width = max(-(-max(lens) // page), 1) + 1
    per = [-(-n // page) for n in lens]
    pages = sum(per) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, width), generator=torch.Generator().manual_seed(seed + 1),
                          dtype=torch.int64).int()
    held = torch.zeros(pages, dtype=torch.int64)
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = order[at:at + k]
        held[order[at:at + k].long()] = (lens[b] - page * torch.arange(k)).clamp(max=page)
        at += k
    held = held.to(device)
    codes, scales = [], []
    for _ in range(2):
        x = torch.randn(pages, Hkv, page, d, **kw).mul_(120).clamp_(-448, 448).to(torch.float8_e4m3fn)
        junk = torch.randint(0, 256, x.shape, dtype=torch.uint8, **kw)
        free = torch.arange(page, device=device) >= held[:, None]
        codes.append(torch.where(free[:, None, :, None], junk, x.view(torch.uint8)).view(torch.float8_e4m3fn))
        s = torch.exp2(torch.round(torch.randn(pages, Hkv, page // BLOCK, **kw) * spread)) / 128
        none = BLOCK * torch.arange(page // BLOCK, device=device) >= held[:, None]
        scales.append(s.masked_fill(none[:, None], math.nan))
    q = torch.randn(sum(new), Hq, d, **kw).to(TYPES[dtype])
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
    return dict(q=q, cache=(codes[0], scales[0], codes[1], scales[1]), table=table.to(device),
                lens=torch.tensor(lens, dtype=torch.int32, device=device), cu=cu.to(device), new=list(new),
                dtype=dtype)


def _side(codes, scales, ids, n):
    """Tokens 0 .. n - 1 on pages `ids`, [Hkv, n, d], and their scales, [Hkv, n]."""
    H, page, d = codes.shape[1:]
    s = scales[ids].double().repeat_interleave(BLOCK, 2).transpose(0, 1).reshape(H, -1)[:, :n]
    x = codes.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double().transpose(0, 1).reshape(H, -1, d)[:, :n]
    return x * s[..., None], s


def attend(c, scale=None, causal=True, window=0):
    """O [T, Hq, d], LSE [Hq, T] and bounds on their errors.

    A score is a sum of d products (2 or 3 pieces of q each) in 32 bits, off by at most 2^-19 scale
    sum|q||k|; a piece is rounded to e4m3's least step at the latest, which leaves an element of q
    within 2^-10 where the row's largest is 224 or more, that is within 2^-17.8 of that one.  An
    exponential and what scales it are off by 2^-20 relative.  All change each probability by the
    factor 1 + e, and O by at most 2 e sum P|v| (numerator and sum).  Weights (the probability times
    V's scale) below 2^-28 of the row's largest may be lost."""
    q, (k8, ks, v8, vs), dtype = c["q"].double(), c["cache"], c["dtype"]
    T, Hq, d = q.shape
    pages, H, page = k8.shape[:3]
    G = Hq // H
    scale = d ** -0.5 if scale is None else scale
    dev = q.device
    o, bo = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((Hq, T), -math.inf, dtype=torch.float64, device=dev)
    bl = torch.zeros_like(lse)
    cu, lens = c["cu"].tolist(), c["lens"].tolist()
    for b, total in enumerate(lens):
        n, total = cu[b + 1] - cu[b], min(max(total, 0), c["table"].shape[1] * page)
        if n == 0 or total == 0:
            continue
        ids = c["table"][b, :-(-total // page)].long()
        known = ((ids >= 0) & (ids < pages)).repeat_interleave(page)[:total]
        ids = torch.where((ids >= 0) & (ids < pages), ids, 0)
        k, _ = _side(k8, ks, ids, total)
        v, vscale = _side(v8, vs, ids, total)
        pos = torch.arange(total - n, total, device=dev)[:, None]
        j = torch.arange(total, device=dev)
        see = known[None, :].expand(n, total)
        if causal:
            see = see & (j <= pos)
        if window:
            see = see & (j > pos - window)
        hidden = ~see[None]                                            # [1, n, total]
        any_row = see.any(0)
        v = torch.where(any_row[:, None], v, 0.0)
        vscale = torch.where(any_row, vscale, 0.0)
        for h in range(Hq):
            g = h // G
            x = q[cu[b]:cu[b + 1], h]                                  # [n, d]
            s = (scale * (x @ k[g].T)).masked_fill(hidden[0], -math.inf)
            size = scale * (x.abs() @ k[g].abs().T)
            size = size + 2.0 ** 1.25 * scale * x.abs().amax(1, keepdim=True) * k[g].abs().sum(1)
            size = size.masked_fill(hidden[0], 0.0).amax(1)
            z = torch.logsumexp(s, 1)
            p = torch.exp(s - torch.where(z > -math.inf, z, 0.0)[:, None])
            rows = slice(cu[b], cu[b + 1])
            lse[h, rows] = z
            o[rows, h] = p @ v[g]
            e = 2.0 ** -19 * size + 2.0 ** -20
            bl[h, rows] = 2 * e + 2.0 ** -22 * torch.where(z > -math.inf, z, 0.0).abs()
            lost = 2.0 ** -28 * (p * vscale[g]).amax(1) * 448 * see.sum(1)
            far = (P_ROUND[dtype] + 2 * e)[:, None] * (p @ v[g].abs()) + lost[:, None]
            bo[rows, h] = far + OUT_ROUND[dtype] * (o[rows, h].abs() + far)
    return o, lse, bo, bl


def close(c, o, lse, want):
    """Whether O and LSE lie within the bounds; a NaN does not."""
    wo, wl, bo, bl = want
    o, lse = o.double(), lse.double()
    seen = wl > -math.inf
    assert torch.equal(lse == -math.inf, ~seen)
    err = torch.where(seen, (lse - wl).abs(), 0.0)
    assert (err <= bl).all(), float((err / bl.clamp(min=1e-30)).max())
    # below the least normal output a rounding is off by half the least step
    tiny = 2.0 ** -25 if c["dtype"] == "f16" else 2.0 ** -134
    err = (o - wo).abs()
    assert (err <= bo + tiny).all(), (int((~(err <= bo + tiny)).sum()), float((err / (bo + tiny)).max()))


def run(fa, c, **kw):
    args = dict(cu_seqlens=c["cu"], max_seqlen=max(c["new"])) | kw
    out = fa.attention_forward_kv8(c["q"], fa.Kv8Cache(c["cache"]), c["table"], c["lens"], **args)
    fa.fa_device_status()
    return out
