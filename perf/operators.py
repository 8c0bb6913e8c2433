"""The serving operators over the 8-bit paged key/value cache, as they are measured: their
cases, their plain forms in elementary torch operations, and the calls a user makes.

Three operators make one serving step:

  plan    kv8_plan               pages for the requests' new tokens, their slots
  append  kv8_append             the new tokens' keys and values into the cache, in 8 bits
  attend  attention_forward_kv8  the new tokens' attention over the cache

The cache holds e4m3 codes, [pages, Hkv, page, d], and a float32 scale for each block of 16
tokens and head, [pages, Hkv, page / 16]; a value is its code times its block's scale.
"""
import math
import random

import torch

own = False

BLOCK = 16          # tokens of one scale block
LEAST = -64         # least exponent of a scale
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------- the cases

def _plan(name, B, context, page, grow, ended, seats=0):
    return dict(name=name, op="plan", B=B, context=context, page=page, grow=grow, ended=ended,
                seats=seats)


def _append(name, B, context, grow, Hkv, d, page, dtype):
    return dict(name=name, op="append", B=B, context=context, grow=grow, Hkv=Hkv, d=d, page=page,
                dtype=dtype)


def _attend(name, B, context, n, Hq, Hkv, d, page, dtype, window=0, ragged=True, fresh=False):
    return dict(name=name, op="attend", B=B, context=context, n=n, Hq=Hq, Hkv=Hkv, d=d, page=page,
                dtype=dtype, window=window, ragged=ragged, fresh=fresh)


def listed():
    return [
        # a decoding step's bookkeeping: a token for each of 64 requests, some requests over
        _plan("plan_step_b64", 64, 8192, 64, 1, 3),
        # a server's busy moment: 384 requests, prompts' chunks among them, a padded token batch
        _plan("plan_chunks_b384_page16", 384, 16384, 16, 257, 40, 1000),
        # a decoding step's new keys and values, one layer
        _append("append_step_b64_h8_d128", 64, 8192, 1, 8, 128, 64, "bf16"),
        # short prompts behind contexts that end inside a block, fp16
        _append("append_chunks_b37_h8_d64_f16", 37, 2048, 301, 8, 64, 16, "f16"),
        # long prompts taken in whole
        _append("append_prompts_b8_h8_d128", 8, 0, 8192, 8, 128, 64, "bf16"),
        # one request's next token: what a single user waits for
        _attend("decode_b1_1000_h32kv8_d128", 1, 1000, 1, 32, 8, 128, 64, "bf16", ragged=False),
        # a server's decoding step, requests of many lengths
        _attend("decode_b64_8192_h32kv8_d128", 64, 8192, 1, 32, 8, 128, 64, "bf16"),
        # the same with small heads, small pages and fp16, many requests
        _attend("decode_b128_2048_h32kv8_d64_f16", 128, 2048, 1, 32, 8, 64, 16, "f16"),
        # few requests over long documents, a key/value head for each query head
        _attend("decode_b2_131072_h16kv16_d128", 2, 131072, 1, 16, 16, 128, 128, "bf16", ragged=False),
        # a sliding window's decoding step, drafts of up to 5 tokens to be checked at once
        _attend("drafts_b24_16384_w4096_h32kv8_d128", 24, 16384, 5, 32, 8, 128, 64, "bf16", 4096),
        # a chunk of a long prompt over what came before it
        _attend("chunk_b1_2048_of_16384_h32kv8_d128", 1, 16384, 2048, 32, 8, 128, 64, "bf16",
                ragged=False),
        # whole prompts of many lengths, nothing before them
        _attend("prompts_b16_2048_h32kv8_d64", 16, 2048, 2048, 32, 8, 64, 64, "bf16", fresh=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    d = rng.choice([64, 128])
    if op == "plan":
        B = _log(rng, 1, 512)
        c = _plan("", B, _log(rng, page, 16384), page, _log(rng, 1, max(2, 65536 // B)),
                  rng.randint(0, B // 4), rng.choice([0, 0, rng.randint(1, 512)]))
    elif op == "append":
        B, Hkv = _log(rng, 1, 256), rng.choice([1, 2, 8, 16])
        c = _append("", B, _log(rng, 1, 4096), _log(rng, 1, max(2, 65536 * 8 // Hkv // B)), Hkv, d,
                    page, dtype)
        while B * c["grow"] * Hkv * d > 8 * 8192 * 8 * 128:
            c["grow"] = c["grow"] // 2 + 1
    else:
        Hq, Hkv = rng.choice([(32, 8), (16, 16), (8, 8), (16, 1), (32, 4), (64, 8), (12, 4)])
        B = _log(rng, 1, 128)
        n = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 1024)])
        context = max(n, _log(rng, 1, 65536))
        # no more than the largest listed cases read and multiply
        while B * context * Hkv * d > 2 * 131072 * 16 * 128 or B * n * context * Hq * d > 2048 * 16384 * 32 * 128:
            if B > 1:
                B = (B + 1) // 2
            else:
                n, context = (n + 1) // 2, (context + 1) // 2
        c = _attend("", B, context, n, Hq, Hkv, d, page, dtype,
                    rng.choice([0, 0, 0, _log(rng, 1, 4096)]), rng.random() < 0.7,
                    n > 8 and rng.random() < 0.3)
    del c["name"]
    return c


def _ragged(rng, B, most, least=1):
    """B whole numbers up to `most`, spread over their logarithm, the largest one `most`."""
    least = max(1, min(least, most))
    out = [_log(rng, least, most) for _ in range(B)]
    out[rng.randrange(B)] = most
    return out


def _lengths(case):
    """(tokens before, tokens new) of each request: they go by the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B = case["B"]
    if case["op"] == "plan":
        before = _ragged(rng, B, case["context"], case["context"] // 64)
        new = _ragged(rng, B, case["grow"])
        for b in rng.sample(range(B), case["ended"]):
            new[b] = -1
        return before, new
    if case["op"] == "append":
        before = [0] * B if not case["context"] else [rng.randint(0, case["context"]) for _ in range(B)]
        return before, [case["grow"]] * B if not case["context"] else _ragged(rng, B, case["grow"])
    n = _ragged(rng, B, case["n"], case["n"] // 16) if case["ragged"] else [case["n"]] * B
    if case["fresh"]:
        return [0] * B, n
    total = _ragged(rng, B, case["context"], case["context"] // 16) if case["ragged"] else [case["context"]] * B
    return [max(t - x, 0) for t, x in zip(total, n)], n


# ------------------------------------------------------------------------- the inputs

def _table(rng, lens, width, page, pages):
    """Pages of `lens` tokens each, in no order, and what pages are left."""
    order = list(range(pages))
    rng.shuffle(order)
    rows, at = [], 0
    for n in lens:
        k = -(-n // page)
        rows.append(order[at:at + k] + [-1] * (width - k))
        at += k
    return rows, order[at:]


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _exponent(amax):
    """The least k >= LEAST with amax <= 448 * 2^k."""
    m, e = torch.frexp(amax)
    return torch.clamp(torch.where(m <= 0.875, e - 9, e - 8), min=LEAST)


def _pow2(k):
    return torch.ldexp(torch.ones_like(k, dtype=torch.float32), k)


def _filled(gen, case, pages, lens, rows):
    """One side of a cache with normal values in the tokens the requests hold, a few channels
    larger, and what recycled pages hold (any byte) everywhere else."""
    Hkv, d, page = case["Hkv"], case["d"], case["page"]
    gain = torch.ones(Hkv, 1, 1, d, device="cuda")
    gain[:, 0, 0, torch.randint(0, d, (3,), generator=gen, device="cuda")] = 5.0
    x = torch.randn(pages, Hkv, page // BLOCK, BLOCK, d, generator=gen, device="cuda") * gain
    k = _exponent(x.abs().amax((3, 4)))
    codes = (x * _pow2(-k)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = codes.view(pages, Hkv, page, d)
    held = torch.zeros(pages + 1, dtype=torch.int32)
    for n, row in zip(lens, rows):
        for j in range(-(-n // page)):
            held[row[j]] = min(page, n - j * page)
    free = torch.arange(page, device="cuda") >= held[:pages].cuda()[:, None]
    junk = torch.randint(0, 256, (pages, 1, page, 1), generator=gen, device="cuda").to(torch.uint8)
    codes = torch.where(free[:, None, :, None], junk, codes)
    return codes.view(torch.float8_e4m3fn).contiguous(), _pow2(k)


def prepare(case, seed):
    before, new = _lengths(case)
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    page, B = case["page"], case["B"]
    st = dict(case=dict(case), page=page)
    after = [x + max(g, 0) for x, g in zip(before, new)]
    width = max(-(-x // page) for x in after) + 1
    need = sum(-(-x // page) for x in after)
    pages = need + need // 8 + 2
    if case["op"] == "plan":
        rows, left = _table(rng, before, width, page, pages)
        head = rng.randrange(pages)
        ring = [-1] * pages
        for i, x in enumerate(left):
            ring[(head + i) % pages] = x
        st |= dict(lens=_int(before), grow=_int(new), table=_int(rows), ring=_int(ring),
                   state=_int([head, len(left), 0]),
                   tokens=sum(max(g, 0) for g in new) + case["seats"])
        return st
    rows, _ = _table(rng, after, width, page, pages)
    dt = TYPES[case["dtype"]]
    st["table"] = _int(rows)
    if case["op"] == "append":
        st["k8"], st["ks"] = _filled(gen, case, pages, before, rows)
        st["v8"], st["vs"] = _filled(gen, case, pages, before, rows)
        slots = [row[t // page] * page + t % page
                 for row, x, g in zip(rows, before, new) for t in range(x, x + g)]
        st["slots"] = _int(slots)
        shape = (len(slots), case["Hkv"], case["d"])
        for name in ("k", "v"):
            st[name] = (torch.randn(shape, generator=gen, device="cuda") * 1.5).to(dt)
        return st
    st["k8"], st["ks"] = _filled(gen, case, pages, after, rows)
    st["v8"], st["vs"] = _filled(gen, case, pages, after, rows)
    st["lens"] = _int(after)
    st["n"] = max(new)
    st["dense"] = min(new) == max(new)
    starts = [0]
    for g in new:
        starts.append(starts[-1] + g)
    st["cu"] = _int(starts)
    shape = (B, new[0]) if st["dense"] else (starts[-1],)
    q = torch.randn(*shape, case["Hq"], case["d"], generator=gen, device="cuda")
    st["q"] = q.to(dt)
    return st


# ------------------------------------------------------------------------- the plain forms

def _run_plan(st):
    lens, grow, page = st["lens"].long(), st["grow"].long(), st["page"]
    table, ring = st["table"].clone(), st["ring"].clone()
    B, width, cap, T = lens.numel(), table.shape[1], ring.numel(), st["tokens"]
    head, count = st["state"][0].long(), st["state"][1].long()
    add = grow.clamp(min=0)
    end = add.cumsum(0)
    have = (lens + page - 1) // page
    fits = (grow >= 0) & (lens + add <= width * page) & (end <= T)
    need = torch.where(fits, (lens + add + page - 1) // page - have, 0)
    last = need.cumsum(0)
    served = fits & ((need == 0) | (last <= count))
    first = last - need
    # the slot of each token, and the pages that its request gets
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(end, t, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    pos = lens[b] + t - (end[b] - add[b])
    blk = (pos // page).clamp(max=width - 1)
    fresh = blk - have[b]
    taken = ring[(head + first[b] + fresh.clamp(min=0)) % cap]
    at = torch.where(fresh >= 0, taken, table[b, blk]).long()
    good = real & served[b]
    slots = torch.where(good, at * page + pos % page, -1).int()
    write = torch.where(good & (fresh >= 0), b * width + blk, B * width)
    flat = torch.cat([table.reshape(-1), table.new_zeros(1)])
    flat[write] = at.int()
    table = flat[:-1].view(B, width)
    # the pages of requests that ended, behind the ring's last
    gone = torch.where(grow < 0, have, 0)
    back = gone.cumsum(0) - gone
    j = torch.arange(width, device="cuda")
    put = torch.where(j < gone[:, None], (head + count + back[:, None] + j) % cap, cap)
    ring = torch.cat([ring, ring.new_zeros(1)])
    ring[put.reshape(-1)] = st["table"].reshape(-1)
    used = torch.where(served, need, 0).sum()
    after = torch.where(grow < 0, 0, torch.where(served, lens + add, lens)).int()
    state = torch.stack([(head + used) % cap, count - used + gone.sum(), ((grow >= 0) & ~served).sum()])
    cu = torch.cat([end.new_zeros(1), end])
    return dict(lens=after, cu=cu.int(), slots=slots, table=table, ring=ring[:-1], state=state.int())


def _append_side(codes, scales, x, slots):
    """The tokens `x` into one side of the cache."""
    pages, Hkv, page, d = codes.shape
    x = x.float()
    blocks, which = torch.unique(slots.long() // BLOCK, return_inverse=True)
    n = blocks.numel()
    offset = torch.full((n,), BLOCK, device="cuda", dtype=torch.long)
    offset = offset.scatter_reduce(0, which, slots.long() % BLOCK, "amin")
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(2)
    amax = torch.zeros(n, Hkv, device="cuda").scatter_reduce(0, which[:, None].expand(-1, Hkv), amax, "amax")
    need = _pow2(_exponent(amax))
    pg, sub = blocks // (page // BLOCK), blocks % (page // BLOCK)
    old = scales[pg, :, sub]
    new = torch.where(offset[:, None] > 0, torch.maximum(old, need), need)
    scales[pg, :, sub] = new
    # the tokens that the blocks held already, at the new scales
    view = codes.view(torch.uint8).view(pages, Hkv, page // BLOCK, BLOCK, d)
    held = view[pg, :, sub].view(torch.float8_e4m3fn).float()
    held = (held * (old / new)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = torch.arange(BLOCK, device="cuda") < offset[:, None]
    held = torch.where(keep[:, None, :, None], held, view[pg, :, sub])
    # a number that is not finite is stored as NaN
    x = x / new[which][..., None]
    held[which, :, slots.long() % BLOCK] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    view[pg, :, sub] = held
    return codes, scales


def _run_append(st):
    k8, ks = _append_side(st["k8"], st["ks"], st["k"], st["slots"])
    v8, vs = _append_side(st["v8"], st["vs"], st["v"], st["slots"])
    return dict(k8=k8, k_scale=ks, v8=v8, v_scale=vs)


def _values(codes, scales, table):
    """What the requests' pages stand for, [B, Hkv, tokens, d]; `table` without missing pages."""
    x = codes.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
    x = x * scales[table].repeat_interleave(BLOCK, 3)[..., None]
    B, W, H, P, d = x.shape
    return x.transpose(1, 2).reshape(B, H, W * P, d)


def _run_attend(st):
    case, q, lens = st["case"], st["q"], st["lens"].long()
    B, n, Hq, Hkv, d = case["B"], st["n"], case["Hq"], case["Hkv"], case["d"]
    G = Hq // Hkv
    table = st["table"].long().clamp(min=0)
    k = _values(st["k8"], st["ks"], table)
    v = _values(st["v8"], st["vs"], table)
    cu = st["cu"].long()
    mine = cu[1:] - cu[:-1]
    i = torch.arange(n, device="cuda")
    row = torch.minimum(cu[:-1, None] + i, cu[1:, None] - 1)
    qf = q.reshape(-1, Hq, d).float()[row].view(B, n, Hkv, G, d)
    qf = qf.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    pos = lens[:, None] - mine[:, None] + i
    j = torch.arange(k.shape[2], device="cuda")
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])
    if case["window"]:
        seen &= j > pos[..., None] - case["window"]
    live = (j < lens[:, None])[:, None, :, None]
    s = torch.matmul(qf, torch.where(live, k, 0.0).transpose(2, 3)).view(B, Hkv, G, n, -1)
    s = torch.where(seen[:, None, None], s * d ** -0.5, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    p = p / torch.where(total > 0, total, 1.0)
    o = torch.matmul(p.view(B, Hkv, G * n, -1), torch.where(live, v, 0.0))
    o = o.view(B, Hq, n, d).transpose(1, 2)
    lse = lse.view(B, Hq, n)
    if st["dense"]:
        return dict(o=o.to(q.dtype), lse=lse)
    real = (i < mine[:, None]).view(-1)
    return dict(o=o.reshape(B * n, Hq, d)[real].to(q.dtype),
                lse=lse.transpose(0, 1).reshape(Hq, B * n)[:, real])


def run(st):
    op = st["case"]["op"]
    if own:
        import exact_io_aware_tcgen05_gb300 as fa
        if op == "plan":
            lens, cu, slots, state = fa.kv8_plan(st["lens"], st["grow"], st["table"], st["ring"],
                                                 st["state"], page=st["page"], tokens=st["tokens"])
            return dict(lens=lens, cu=cu, slots=slots, table=st["table"], ring=st["ring"], state=state)
        cache = fa.Kv8Cache((st["k8"], st["ks"], st["v8"], st["vs"]))
        if op == "append":
            fa.kv8_append(cache, st["k"], st["v"], st["slots"])
            return dict(k8=st["k8"], k_scale=st["ks"], v8=st["v8"], v_scale=st["vs"])
        cu, n = (None, None) if st["dense"] else (st["cu"], st["n"])
        o, lse = fa.attention_forward_kv8(st["q"], cache, st["table"], st["lens"], causal=True,
                                          window=st["case"]["window"], cu_seqlens=cu, max_seqlen=n)
        return dict(o=o, lse=lse)
    return {"plan": _run_plan, "append": _run_append, "attend": _run_attend}[op](st)


# ------------------------------------------------------------------------- the work

def _visible(before, n, window):
    """Keys that a request's new tokens see: pairs, and the keys that any of them sees."""
    total = before + n
    if not window:
        return n * before + n * (n + 1) // 2, total
    pairs = sum(min(before + i + 1, window) for i in range(n))
    return pairs, min(total, window + n - 1)


def work(case):
    before, new = _lengths(case)
    page = case["page"]
    if case["op"] == "plan":
        tokens = sum(max(g, 0) for g in new) + case["seats"]
        moved = sum(-(-x // page) if g < 0 else -(-(x + g) // page) - -(-x // page)
                    for x, g in zip(before, new))
        return {"bytes": 4 * (4 * case["B"] + tokens + 2 * moved + 7), "flops": 0}
    if case["op"] == "append":
        tokens = sum(new)
        blocks = sum(-(-(x + g) // BLOCK) - x // BLOCK for x, g in zip(before, new))
        values = 2 * tokens * case["Hkv"] * case["d"]
        return {"bytes": 3 * values + 2 * 4 * blocks * case["Hkv"] + 4 * tokens, "flops": 2 * values}
    pairs = keys = 0
    for x, g in zip(before, new):
        p, k = _visible(x, g, case["window"])
        pairs, keys = pairs + p, keys + k
    rows = sum(new) * case["Hq"]
    cached = 2 * keys * case["Hkv"] * case["d"]
    return {"bytes": cached + 2 * 4 * (keys // BLOCK) * case["Hkv"] + 4 * rows * case["d"] + 4 * rows
            + 4 * (keys // page), "flops": 4 * case["d"] * pairs * case["Hq"]}


# ------------------------------------------------------------------------- in 64 bits

def _exact_plan(st):
    lens, grow = st["lens"].tolist(), st["grow"].tolist()
    table, ring = st["table"].tolist(), st["ring"].tolist()
    old = [list(r) for r in table]
    head, count, _ = st["state"].tolist()
    page, T, cap, width = st["page"], st["tokens"], len(ring), len(table[0])
    after, cu, slots, wanted, used, put, missed = [], [0], [-1] * T, 0, 0, 0, 0
    for b, (x, g) in enumerate(zip(lens, grow)):
        have = -(-x // page)
        if g < 0:
            for j in range(have):
                ring[(head + count + put) % cap] = old[b][j]
                put += 1
            after.append(0)
            cu.append(cu[-1])
            continue
        ok = x + g <= width * page and cu[-1] + g <= T
        need = -(-(x + g) // page) - have if ok else 0
        wanted += need
        ok = ok and (need == 0 or wanted <= count)
        if ok:
            for j in range(need):
                table[b][have + j] = ring[(head + wanted - need + j) % cap]
            for t in range(g):
                slots[cu[-1] + t] = table[b][(x + t) // page] * page + (x + t) % page
            used += need
        missed += not ok
        after.append(x + g if ok else x)
        cu.append(cu[-1] + g)
    return dict(lens=_int(after), cu=_int(cu), slots=_int(slots), table=_int(table), ring=_int(ring),
                state=_int([(head + used) % cap, count - used + put, missed]))


def _to_code(x):
    """The e4m3 value nearest to x, ties to even; |x| <= 448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e - 1, min=-6) - 3)
    return torch.round(x / step) * step


def _exact_append(codes, scales, x, slots):
    pages, Hkv, page, d = codes.shape
    codes, scales, x = codes.double().cpu(), scales.double().cpu(), x.double().cpu()
    at = slots.tolist()
    t = 0
    while t < len(at):
        # the tokens of one block
        e = t + 1
        while e < len(at) and at[e] // BLOCK == at[t] // BLOCK:
            e += 1
        pg, off = at[t] // page, at[t] % page
        blk, off = off // BLOCK, off % BLOCK
        amax = x[t:e].abs().amax((0, 2))
        k = torch.clamp(torch.ceil(torch.log2(amax / 448)), min=LEAST)
        k = torch.where(amax > 448 * 2.0 ** k, k + 1, k)
        new = 2.0 ** k
        if off:
            old = scales[pg, :, blk]
            new = torch.maximum(old, new)
            rows = slice(blk * BLOCK, blk * BLOCK + off)
            codes[pg, :, rows] = _to_code(codes[pg, :, rows] * (old / new)[:, None, None])
        scales[pg, :, blk] = new
        first = blk * BLOCK + off
        codes[pg, :, first:first + e - t] = _to_code(x[t:e] / new[:, None]).transpose(0, 1)
        t = e
    return codes.cuda(), scales.cuda()


def _exact_attend(st):
    case, lens, cu = st["case"], st["lens"].tolist(), st["cu"].tolist()
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    q = st["q"].reshape(-1, Hq, d).double()
    o = torch.zeros_like(q)
    lse = torch.full((Hq, q.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    for b, total in enumerate(lens):
        n = cu[b + 1] - cu[b]
        ids = st["table"][b, :-(-total // page)].long()

        def side(codes, scales):
            x = codes.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double().view(len(ids), Hkv, page // BLOCK, BLOCK, d)
            x = x * scales[ids].double()[..., None, None]
            return x.view(len(ids), Hkv, page, d).transpose(0, 1).reshape(Hkv, -1, d)[:, :total]

        k, v = side(st["k8"], st["ks"]), side(st["v8"], st["vs"])
        pos = torch.arange(total - n, total, device="cuda")[:, None]
        j = torch.arange(total, device="cuda")
        hide = (j > pos) | ((j <= pos - case["window"]) if case["window"] else (j < 0))
        for h in range(Hq):
            g = h // (Hq // Hkv)
            s = (q[cu[b]:cu[b + 1], h] @ k[g].T) / math.sqrt(d)
            s = s.masked_fill(hide, -math.inf)
            z = torch.logsumexp(s, 1)
            lse[h, cu[b]:cu[b + 1]] = z
            o[cu[b]:cu[b + 1], h] = torch.exp(s - torch.where(z > -math.inf, z, 0.0)[:, None]) @ v[g]
    if st["dense"]:
        B, n = case["B"], st["n"]
        return dict(o=o.view(B, n, Hq, d), lse=lse.view(Hq, B, n).transpose(0, 1))
    return dict(o=o, lse=lse)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(st)
    if case["op"] == "append":
        k8, ks = _exact_append(st["k8"], st["ks"], st["k"], st["slots"])
        v8, vs = _exact_append(st["v8"], st["vs"], st["v"], st["slots"])
        return dict(k8=k8, k_scale=ks, v8=v8, v_scale=vs)
    return _exact_attend(st)
