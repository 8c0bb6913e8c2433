"""What stands around attention, as it is measured: the preparation of queries and keys (a norm
for each head, then the rotation by position), its gradient, the same on the way into the 8-bit
paged cache, and attention of a batch whose requests share a prefix in that cache.  Cases, plain
forms in elementary torch operations, and the calls a user makes.

  forward   norm_rope_forward             queries and keys of a projection, ready for attention
  backward  norm_rope_backward            the gradients of that, the norms' weights among them
  append    kv8_append_norm_rope          a serving step: queries ready, keys and values in the cache
  prefix    attention_forward_kv8_prefix  attention over shared prefixes and the requests' own tokens

A head's row x of d channels becomes n = x / sqrt(mean(x^2) + eps) * weight, and its first `rot`
channels are rotated in pairs by position * frequency; with several axes (time, height, width) each
frequency takes its own axis' position.  The cache holds e4m3 codes, [pages, Hkv, page, d], and a
float32 scale for each block of 16 tokens and head, [pages, Hkv, page / 16].
"""
import math
import random

import torch

own = False

BLOCK = 16          # tokens of one scale block
LEAST = -64         # least exponent of a scale
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------- the cases

def _rope(op, name, B, n, Hq, Hkv, d, dtype, rot, axes=1, interleaved=False, norm=True, wide=False,
          fused=False, far=0):
    """`wide`: the weights are float32; `fused`: q and k are slices of one projection's output."""
    return dict(name=name, op=op, B=B, n=n, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, rot=rot, axes=axes,
                interleaved=interleaved, norm=norm, wide=wide, fused=fused, far=far)


def _append(name, B, context, grow, Hq, Hkv, d, page, dtype, rot, axes=1, interleaved=False, norm=True):
    return dict(name=name, op="append", B=B, context=context, grow=grow, Hq=Hq, Hkv=Hkv, d=d, page=page,
                dtype=dtype, rot=rot, axes=axes, interleaved=interleaved, norm=norm, far=0)


def _prefix(name, B, groups, shared, context, n, Hq, Hkv, d, page, dtype, ragged=True):
    return dict(name=name, op="prefix", B=B, groups=groups, shared=shared, context=context, n=n, Hq=Hq,
                Hkv=Hkv, d=d, page=page, dtype=dtype, ragged=ragged)


def listed():
    return [
        # one request's next token: what a single user waits for
        _rope("forward", "forward_b1_1_h32kv8_d128", 1, 1, 32, 8, 128, "bf16", 128, fused=True, far=4096),
        # a training step's sequences in earnest, a key/value head for each query head
        _rope("forward", "forward_b2_8192_h16_d128", 2, 8192, 16, 16, 128, "bf16", 128),
        # an odd number of tokens, part of the channels rotated in neighbouring pairs, no norm, fp16
        _rope("forward", "forward_b1_5003_h12kv4_d64_f16", 1, 5003, 12, 4, 64, "f16", 32, interleaved=True,
              norm=False),
        # images and video: positions in time, height and width, straight from the fused projection
        _rope("forward", "forward_b1_32768_h32kv8_d128_axes3", 1, 32768, 32, 8, 128, "bf16", 128, axes=3,
              fused=True, wide=True, far=100000),
        # a short sequence's step
        _rope("backward", "backward_b1_300_h4kv2_d128", 1, 300, 4, 2, 128, "bf16", 128),
        # the gradients of the training step above
        _rope("backward", "backward_b2_8192_h16_d128", 2, 8192, 16, 16, 128, "bf16", 128, fused=True),
        # packed sequences with small heads, fp16, float32 weights
        _rope("backward", "backward_b1_32771_h32kv8_d64_f16_axes3", 1, 32771, 32, 8, 64, "f16", 64, axes=3,
              wide=True),
        # a decoding step: a token for each of 64 requests
        _append("append_step_b64_h32kv8_d128", 64, 8192, 1, 32, 8, 128, 64, "bf16", 128),
        # short prompts behind contexts that end inside a block, small heads and pages, fp16
        _append("append_chunks_b37_h32kv8_d64_f16", 37, 2048, 301, 32, 8, 64, 16, "f16", 32, axes=2,
                interleaved=True),
        # long prompts taken in whole
        _append("append_prompts_b8_h32kv8_d128", 8, 0, 8192, 32, 8, 128, 64, "bf16", 128),
        # a decoding step of 64 requests behind one system prompt
        _prefix("prefix_step_b64_8192_h32kv8_d128", 64, 1, 8192, 512, 1, 32, 8, 128, 64, "bf16"),
        # questions of up to 200 tokens about three documents, fp16
        _prefix("prefix_questions_b24_16384_h16kv4_d64_f16", 24, 3, 16384, 200, 200, 16, 4, 64, 16, "f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "backward", "append", "prefix"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    d = rng.choice([64, 128])
    Hq, Hkv = rng.choice([(32, 8), (16, 16), (16, 2), (64, 8), (12, 4), (8, 1)])
    page = rng.choice([16, 32, 64, 128])
    rot = rng.choice([d, d, d, d // 2, d // 4, 3 * d // 4])
    axes = rng.choice([1, 1, 2, 3, 4])
    interleaved, norm = rng.random() < 0.3, rng.random() < 0.8
    if op in ("forward", "backward"):
        # no more tokens than the largest listed case's values allow
        most = 32768 * 40 * 128 // ((Hq + Hkv) * d)
        tokens = _log(rng, 1, min(most, 65536))
        B = _log(rng, 1, min(tokens, 64))
        c = _rope(op, "", B, max(tokens // B, 1), Hq, Hkv, d, dtype, rng.choice([rot, rot, rot, 0]) if norm else rot,
                  axes, interleaved, norm, rng.random() < 0.5, d == 128 and rng.random() < 0.5,
                  rng.choice([0, 0, _log(rng, 1, 1000000)]))
    elif op == "append":
        B = _log(rng, 1, 256)
        c = _append("", B, _log(rng, 1, 4096), _log(rng, 1, max(2, 65536 // B)), Hq, Hkv, d, page, dtype, rot,
                    axes, interleaved, norm)
        while B * c["grow"] * (Hq + 2 * Hkv) * d > 8 * 8192 * 48 * 128:
            c["grow"] = c["grow"] // 2 + 1
    else:
        B = _log(rng, 2, 96)
        n = rng.choice([1, 1, rng.randint(2, 6), _log(rng, 7, 256)])
        shared = _log(rng, 1, 32768)
        while B * n * Hq * shared * d > 24 * 200 * 16 * 16384 * 64:
            if n > 1:
                n = (n + 1) // 2
            else:
                shared = shared // 2 + 1
        c = _prefix("", B, rng.randint(1, min(B, 4)), shared, max(n, _log(rng, 1, 2048)), n, Hq, Hkv, d, page,
                    dtype, rng.random() < 0.7)
    del c["name"]
    return c


def _ragged(rng, B, most, least=1):
    """B whole numbers up to `most`, spread over their logarithm, the largest one `most`."""
    least = max(1, min(least, most))
    out = [_log(rng, least, most) for _ in range(B)]
    out[rng.randrange(B)] = most
    return out


def _case_rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """(tokens before, tokens new) of each request: they go by the case alone."""
    rng = _case_rng(case)
    B = case["B"]
    if case["op"] == "append":
        before = [0] * B if not case["context"] else [rng.randint(0, case["context"]) for _ in range(B)]
        return before, [case["grow"]] * B if not case["context"] else _ragged(rng, B, case["grow"])
    n = _ragged(rng, B, case["n"], case["n"] // 16) if case["ragged"] else [case["n"]] * B
    total = _ragged(rng, B, case["context"], case["context"] // 16) if case["ragged"] else [case["context"]] * B
    return [max(t - x, 0) for t, x in zip(total, n)], n


def _groups(case):
    """(tokens of each shared prefix, requests of each group)."""
    rng = _case_rng(case)
    rng.random()
    P, B = case["groups"], case["B"]
    shared = _ragged(rng, P, case["shared"], case["shared"] // 8)
    cuts = sorted(rng.sample(range(1, B), P - 1))
    return shared, [b - a for a, b in zip([0] + cuts, cuts + [B])]


# ------------------------------------------------------------------------- the inputs

def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _exponent(amax):
    """The least k >= LEAST with amax <= 448 * 2^k."""
    m, e = torch.frexp(amax)
    return torch.clamp(torch.where(m <= 0.875, e - 9, e - 8), min=LEAST)


def _pow2(k):
    return torch.ldexp(torch.ones_like(k, dtype=torch.float32), k)


def _filled(gen, case, pages, held):
    """One side of a cache with normal values in the places that are held, a few channels larger, and
    what recycled pages hold (any byte) everywhere else."""
    Hkv, d, page = case["Hkv"], case["d"], case["page"]
    gain = torch.ones(Hkv, 1, 1, d, device="cuda")
    gain[:, 0, 0, torch.randint(0, d, (3,), generator=gen, device="cuda")] = 5.0
    x = torch.randn(pages, Hkv, page // BLOCK, BLOCK, d, generator=gen, device="cuda") * gain
    k = _exponent(x.abs().amax((3, 4)))
    codes = (x * _pow2(-k)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = codes.view(pages, Hkv, page, d)
    free = torch.arange(page, device="cuda") >= held[:, None]
    junk = torch.randint(0, 256, (pages, 1, page, 1), generator=gen, device="cuda").to(torch.uint8)
    codes = torch.where(free[:, None, :, None], junk, codes)
    return codes.view(torch.float8_e4m3fn).contiguous(), _pow2(k)


def _table(order, lens, page):
    """Block tables for `lens` tokens each, from the page numbers `order` (used up)."""
    width = max(max(-(-x // page) for x in lens), 1)
    return [[order.pop() for _ in range(-(-x // page))] + [-1] * (width - -(-x // page)) for x in lens]


def _held(pages, page, *tables):
    held = torch.zeros(pages, dtype=torch.int32)
    for lens, rows in tables:
        for n, row in zip(lens, rows):
            for j in range(-(-n // page)):
                held[row[j]] = min(page, n - j * page)
    return held.cuda()


def _rotation(case, st):
    """Frequencies and the axis of each; the framework's plan, which a program makes once."""
    half = case["rot"] // 2
    if not half:
        st |= dict(freq=None, rope=None)
        return
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    # the axes' frequencies one block behind the other, the first axis' the shortest
    cuts = [half * (i + 1) // (case["axes"] + 1) for i in range(1, case["axes"])]
    axis = [sum(i >= c for c in cuts) for i in range(half)]
    st |= dict(freq=f, axis=torch.tensor(axis, device="cuda"), rope=None)
    if own:
        import exact_io_aware_tcgen05_gb300 as fa
        st["rope"] = fa.rope_plan(f, axes=axis if case["axes"] > 1 else None, interleaved=case["interleaved"])


def _weights(gen, case, st):
    dt = torch.float32 if case.get("wide") else TYPES[case["dtype"]]
    for name in ("q_weight", "k_weight"):
        w = 1.45 * (1 + 0.1 * torch.randn(case["d"], generator=gen, device="cuda"))
        st[name] = w.to(dt) if case["norm"] else None


def _positions(case, along):
    """Positions on the case's axes for places `along` (int64) of the sequences: a picture is 64 wide
    and high."""
    axes = [along // 4096, along // 64 % 64, along % 64, along] if case["axes"] > 1 else [along]
    pos = torch.stack([p + case["far"] for p in axes[:case["axes"]]]).int()
    return pos[0] if case["axes"] == 1 else pos


def _projected(gen, case, lead, gain):
    """q, k and v, as three tensors or as slices of one."""
    Hq, Hkv, d, dt = case["Hq"], case["Hkv"], case["d"], TYPES[case["dtype"]]
    heads = Hq + 2 * Hkv
    x = torch.randn(*lead, heads, d, generator=gen, device="cuda") * gain
    x = x.to(dt)
    parts = x[..., :Hq, :], x[..., Hq:Hq + Hkv, :], x[..., Hq + Hkv:, :]
    return parts if case.get("fused", True) else tuple(p.contiguous() for p in parts)


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=dict(case))
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] in ("forward", "backward"):
        B, n = case["B"], case["n"]
        lead = (B, n) if B > 1 else (n,)
        gain = 1.0 + 0.5 * torch.randn(Hq + 2 * Hkv, 1, generator=gen, device="cuda").abs()
        st["q"], st["k"], _ = _projected(gen, case, lead, gain)
        _rotation(case, st)
        _weights(gen, case, st)
        along = torch.arange(n, device="cuda") + rng.randrange(4)
        st["positions"] = _positions(case, along.expand(lead)) if case["rot"] else None
        if case["op"] == "backward":
            dt = TYPES[case["dtype"]]
            st["dq"] = torch.randn(*lead, Hq, d, generator=gen, device="cuda").to(dt)
            st["dk"] = torch.randn(*lead, Hkv, d, generator=gen, device="cuda").to(dt)
            if case["fused"]:   # the projection's gradient, of which these two become slices
                st["grad"] = torch.zeros(*lead, Hq + 2 * Hkv, d, device="cuda", dtype=dt)
        return st
    before, new = _lengths(case)
    page = case["page"]
    after = [x + g for x, g in zip(before, new)]
    shared, members = _groups(case) if case["op"] == "prefix" else ([], [])
    need = sum(-(-x // page) for x in after + shared)
    pages = need + need // 8 + 2
    order = list(range(pages))
    rng.shuffle(order)
    rows = _table(order, after, page)
    if case["op"] == "append":
        held = _held(pages, page, (before, rows))
        st["k8"], st["ks"] = _filled(gen, case, pages, held)
        st["v8"], st["vs"] = _filled(gen, case, pages, held)
        places = [(row[t // page] * page + t % page, t)
                  for row, x, g in zip(rows, before, new) for t in range(x, x + g)]
        st["slots"] = _int([s for s, _ in places])
        st["q"], st["k"], st["v"] = _projected(gen, case, (len(places),), 1.5)
        _rotation(case, st)
        _weights(gen, case, st)
        st["positions"] = _positions(case, torch.tensor([t for _, t in places], device="cuda"))
        return st
    prefix_rows = _table(order, shared, page)
    held = _held(pages, page, (after, rows), (shared, prefix_rows))
    st["k8"], st["ks"] = _filled(gen, case, pages, held)
    st["v8"], st["vs"] = _filled(gen, case, pages, held)
    starts = [0]
    for g in new:
        starts.append(starts[-1] + g)
    bounds, at = [0], 0
    for m in members:
        at += m
        bounds.append(starts[at])
    st |= dict(table=_int(rows), lens=_int(after), n=max(new), dense=min(new) == max(new), cu=_int(starts),
               prefix_table=_int(prefix_rows), prefix_lens=_int(shared), prefix_cu=_int(bounds))
    shape = (case["B"], new[0]) if st["dense"] else (starts[-1],)
    st["q"] = torch.randn(*shape, Hq, d, generator=gen, device="cuda").to(TYPES[case["dtype"]])
    return st


# ------------------------------------------------------------------------- the plain forms

def _angles(st):
    """cos and sin, [tokens..., 1, rot / 2]: the angles in 64 bits, since positions may be far."""
    pos = st["positions"].double()
    pos = pos[..., None].expand(*pos.shape, st["freq"].numel()) if st["case"]["axes"] == 1 else \
        pos[st["axis"]].movedim(0, -1)
    a = (pos * st["freq"]).unsqueeze(-2)
    return torch.cos(a).float(), torch.sin(a).float()


def _turned(x, cs, interleaved, back=False):
    """The first channels of x rotated."""
    if cs is None:
        return x
    cos, sin = cs
    half = cos.shape[-1]
    sin = -sin if back else sin
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _ready(x, weight, cs, case):
    """x normed and rotated, in 32 bits."""
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    return _turned(x, cs, case["interleaved"])


def _run_forward(st):
    case, dt = st["case"], st["q"].dtype
    cs = _angles(st) if st["freq"] is not None else None
    return dict(q=_ready(st["q"], st["q_weight"], cs, case).to(dt), k=_ready(st["k"], st["k_weight"], cs, case).to(dt))


def _back(x, dy, weight, cs, case):
    dn = _turned(dy.float(), cs, case["interleaved"], back=True)
    if not case["norm"]:
        return dn, None
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    g = dn * weight.float()
    dx = r * (g - x * (r * r * (g * x).mean(-1, keepdim=True)))
    return dx, (dn * (x * r)).double().flatten(0, -2).sum(0).float()


def _run_backward(st):
    case, dt = st["case"], st["q"].dtype
    cs = _angles(st) if st["freq"] is not None else None
    dq, dqw = _back(st["q"], st["dq"], st["q_weight"], cs, case)
    dk, dkw = _back(st["k"], st["dk"], st["k_weight"], cs, case)
    out = dict(dq=dq.to(dt), dk=dk.to(dt))
    return out | dict(dq_weight=dqw, dk_weight=dkw) if case["norm"] else out


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
    x = x / new[which][..., None]
    held[which, :, slots.long() % BLOCK] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    view[pg, :, sub] = held
    return codes, scales


def _run_append(st):
    case = st["case"]
    cs = _angles(st)
    q = _ready(st["q"], st["q_weight"], cs, case).to(st["q"].dtype)
    k8, ks = _append_side(st["k8"], st["ks"], _ready(st["k"], st["k_weight"], cs, case), st["slots"])
    v8, vs = _append_side(st["v8"], st["vs"], st["v"], st["slots"])
    return dict(q=q, k8=k8, k_scale=ks, v8=v8, v_scale=vs)


def _values(codes, scales, table):
    """What pages stand for, [B, Hkv, tokens, d]; `table` without missing pages."""
    x = codes.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
    x = x * scales[table].repeat_interleave(BLOCK, 3)[..., None]
    B, W, H, P, d = x.shape
    return x.transpose(1, 2).reshape(B, H, W * P, d)


def _seen(q, k, v, seen, scale):
    """Maximum, sum and weighted values of each row, over the keys that it sees."""
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(s - top)
    return torch.where(seen.any(-1, keepdim=True), top, -math.inf), p.sum(-1, keepdim=True), torch.matmul(p, v)


def _run_prefix(st):
    case, q, lens = st["case"], st["q"], st["lens"].long()
    B, n, Hq, Hkv, d = case["B"], st["n"], case["Hq"], case["Hkv"], case["d"]
    G, scale = Hq // Hkv, case["d"] ** -0.5
    flat = q.reshape(-1, Hq, d).float()
    T = flat.shape[0]
    cache = st["k8"], st["ks"], st["v8"], st["vs"]
    # the shared keys: every group's rows against its prefix, once (the groups lie one behind the
    # other, and how long they are a program knows)
    shared, members = _groups(case)
    _, new = _lengths(case)
    top0 = torch.full((T, Hq, 1), -math.inf, device="cuda")
    sum0 = torch.zeros(T, Hq, 1, device="cuda")
    o0 = torch.zeros(T, Hq, d, device="cuda")
    at = first = 0
    for g, (length, m) in enumerate(zip(shared, members)):
        rows = slice(at, at + sum(new[first:first + m]))
        at, first = rows.stop, first + m
        ids = st["prefix_table"][g, :-(-length // case["page"])].long()[None]
        k = _values(cache[0], cache[1], ids)[0, :, :length]
        v = _values(cache[2], cache[3], ids)[0, :, :length]
        x = flat[rows].view(-1, Hkv, G, d).permute(1, 0, 2, 3).reshape(Hkv, -1, d)
        every = torch.ones(1, 1, length, dtype=torch.bool, device="cuda")
        for to, y in zip((top0, sum0, o0), _seen(x, k, v, every, scale)):
            to[rows] = y.expand(Hkv, x.shape[1], y.shape[-1]).reshape(Hkv, -1, G, y.shape[-1]).transpose(0, 1).reshape(-1, Hq, y.shape[-1])
    # the requests' own keys
    table = st["table"].long().clamp(min=0)
    k, v = _values(cache[0], cache[1], table), _values(cache[2], cache[3], table)
    cu = st["cu"].long()
    mine = cu[1:] - cu[:-1]
    i = torch.arange(n, device="cuda")
    row = torch.minimum(cu[:-1, None] + i, cu[1:, None] - 1)
    x = flat[row].view(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4)
    pos = lens[:, None] - mine[:, None] + i
    j = torch.arange(k.shape[2], device="cuda")
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])
    live = (j < lens[:, None])[:, None, :, None]
    own_parts = _seen(x, torch.where(live, k, 0.0)[:, :, None], torch.where(live, v, 0.0)[:, :, None],
                      seen[:, None, None], scale)
    real = (i < mine[:, None]).reshape(-1)
    top1, sum1, o1 = (y.permute(0, 3, 1, 2, 4).reshape(B * n, Hq, -1)[real] for y in own_parts)
    # joined
    top = torch.maximum(top0, top1)
    ref = torch.where(top > -math.inf, top, 0.0)
    f0, f1 = torch.exp(top0 - ref), torch.exp(top1 - ref)
    total = f0 * sum0 + f1 * sum1
    o = (f0 * o0 + f1 * o1) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + ref)[..., 0].transpose(0, 1)
    if st["dense"]:
        return dict(o=o.view(B, n, Hq, d).to(q.dtype), lse=lse.reshape(Hq, B, n).transpose(0, 1).contiguous())
    return dict(o=o.to(q.dtype), lse=lse.contiguous())


def run(st):
    op = st["case"]["op"]
    if own:
        import exact_io_aware_tcgen05_gb300 as fa
        if op == "prefix":
            cache = fa.Kv8Cache((st["k8"], st["ks"], st["v8"], st["vs"]))
            cu, n = (None, None) if st["dense"] else (st["cu"], st["n"])
            o, lse = fa.attention_forward_kv8_prefix(
                st["q"], cache, st["prefix_table"], st["prefix_lens"], st["prefix_cu"], st["table"], st["lens"],
                cu_seqlens=cu, max_seqlen=n)
            return dict(o=o, lse=lse)
        kw = dict(q_weight=st["q_weight"], k_weight=st["k_weight"], norm=st["case"]["norm"], eps=EPS)
        if op == "append":
            cache = fa.Kv8Cache((st["k8"], st["ks"], st["v8"], st["vs"]))
            q = fa.kv8_append_norm_rope(cache, st["q"], st["k"], st["v"], st["slots"], st["positions"], st["rope"], **kw)
            return dict(q=q, k8=st["k8"], k_scale=st["ks"], v8=st["v8"], v_scale=st["vs"])
        if op == "forward":
            q, k = fa.norm_rope_forward(st["q"], st["k"], st["positions"], st["rope"], **kw)
            return dict(q=q, k=k)
        Hq, Hkv = st["case"]["Hq"], st["case"]["Hkv"]
        into = (st["grad"][..., :Hq, :], st["grad"][..., Hq:Hq + Hkv, :]) if "grad" in st else None
        dq, dk, dqw, dkw = fa.norm_rope_backward(st["q"], st["k"], st["dq"], st["dk"], st["positions"], st["rope"],
                                                 out=into, **kw)
        out = dict(dq=dq, dk=dk)
        return out | dict(dq_weight=dqw, dk_weight=dkw) if st["case"]["norm"] else out
    return {"forward": _run_forward, "backward": _run_backward, "append": _run_append, "prefix": _run_prefix}[op](st)


# ------------------------------------------------------------------------- the work

def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] in ("forward", "backward"):
        tokens = case["B"] * case["n"]
        values = tokens * (Hq + Hkv) * d
        passes = 2 if case["op"] == "forward" else 3 if case["norm"] else 2
        each = (4 if case["norm"] else 0) + (3 if case["rot"] else 0)
        weights = 2 * d * (4 if case["wide"] else 2) if case["norm"] else 0
        if case["op"] == "backward":
            each = 2 * each + 3
            weights += 8 * d if case["norm"] else 0
        return {"bytes": 2 * passes * values + weights + (4 * case["axes"] * tokens if case["rot"] else 0),
                "flops": each * values}
    before, new = _lengths(case)
    tokens = sum(new)
    if case["op"] == "append":
        blocks = sum(-(-(x + g) // BLOCK) - x // BLOCK for x, g in zip(before, new))
        values = 2 * tokens * Hkv * d
        return {"bytes": 4 * tokens * Hq * d + 3 * values + 8 * blocks * Hkv + 4 * tokens * (1 + case["axes"]),
                "flops": 7 * tokens * (Hq + Hkv) * d + 2 * values}
    shared, members = _groups(case)
    pairs, first = 0, 0
    for length, m in zip(shared, members):
        pairs += length * sum(new[first:first + m])
        first += m
    pairs += sum(g * x + g * (g + 1) // 2 for x, g in zip(before, new))
    keys = sum(shared) + sum(before) + tokens
    rows = tokens * Hq
    return {"bytes": 2 * keys * Hkv * d + 8 * (keys // BLOCK) * Hkv + 4 * rows * d + 4 * rows
            + 4 * (keys // case["page"]), "flops": 4 * d * pairs * Hq}


# ------------------------------------------------------------------------- in 64 bits

def _exact_rotated(st, x, sign=1.0):
    """Complex products, one for each pair."""
    case, half = st["case"], st["case"]["rot"] // 2
    if not half:
        return x
    pos = st["positions"].double()
    pos = pos[None] if case["axes"] == 1 else pos
    turn = torch.stack([pos[int(a)] * f for a, f in zip(st["axis"].tolist(), st["freq"].tolist())], -1)
    z = torch.polar(torch.ones_like(turn), sign * turn)[..., None, :]
    y = x.clone()
    first = slice(0, 2 * half, 2) if case["interleaved"] else slice(0, half)
    second = slice(1, 2 * half, 2) if case["interleaved"] else slice(half, 2 * half)
    w = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _exact_ready(st, x, weight):
    x = x.double()
    if st["case"]["norm"]:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    return _exact_rotated(st, x)


def _exact_back(st, x, dy, weight):
    g = _exact_rotated(st, dy.double(), -1.0)
    if not st["case"]["norm"]:
        return g, None
    x, d = x.double(), x.shape[-1]
    size = torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS)
    unit = x / size
    dw = (g * unit).reshape(-1, d).sum(0)
    g = g * weight.double()
    return (g - unit * (g * unit).sum(-1, keepdim=True) / d) / size, dw


def _to_code(x):
    """The e4m3 value nearest to x, ties to even; |x| <= 448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e - 1, min=-6) - 3)
    return torch.round(x / step) * step


def _exact_append(codes, scales, x, slots):
    """Each block's 16 places at once: old tokens, new tokens, or neither."""
    pages, Hkv, page, d = codes.shape
    codes = codes.double().view(pages, Hkv, page // BLOCK, BLOCK, d).transpose(1, 2).reshape(-1, Hkv, BLOCK, d)
    scales = scales.double().transpose(1, 2).reshape(-1, Hkv).clone()
    at = slots.long()
    ids = torch.unique(at // BLOCK)
    token = torch.full((codes.shape[0] * BLOCK,), -1, device="cuda", dtype=torch.long)
    token[at] = torch.arange(at.numel(), device="cuda")
    token = token.view(-1, BLOCK)[ids]                        # [blocks, 16]
    for some in torch.arange(ids.numel(), device="cuda").split(4096):
        b, t = ids[some], token[some]
        here = (t >= 0)[:, None, :, None]
        y = torch.where(here, x[t.clamp(min=0)].double().transpose(1, 2), 0.0)   # [blocks, Hkv, 16, d]
        amax = y.abs().amax((2, 3))
        k = torch.clamp(torch.ceil(torch.log2(amax / 448)), min=LEAST)
        k = torch.where(amax > 448 * 2.0 ** k, k + 1, k)
        k = torch.where(amax <= 448 * 2.0 ** (k - 1), k - 1, k).clamp(min=LEAST)
        new, old = 2.0 ** k, scales[b]
        begun = (t[:, 0] < 0)[:, None]
        new = torch.where(begun, torch.maximum(old, new), new)
        ahead = (t >= 0).long().argmax(1)[:, None] > torch.arange(BLOCK, device="cuda")
        was = codes[b]
        again = torch.where(ahead[:, None, :, None], _to_code(was * (old / new)[..., None, None]), was)
        codes[b] = torch.where(here, _to_code(y / new[..., None, None]), again)
        scales[b] = new
    codes = codes.view(pages, page // BLOCK, Hkv, BLOCK, d).transpose(1, 2).reshape(pages, Hkv, page, d)
    return codes, scales.view(pages, page // BLOCK, Hkv).transpose(1, 2).contiguous()


def _exact_prefix(st):
    case, lens, cu = st["case"], st["lens"].tolist(), st["cu"].tolist()
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    q = st["q"].reshape(-1, Hq, d).double()
    o = torch.zeros_like(q)
    lse = torch.full((Hq, q.shape[0]), -math.inf, dtype=torch.float64, device="cuda")

    def side(codes, scales, ids, total):
        x = codes.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double().view(len(ids), Hkv, page // BLOCK, BLOCK, d)
        x = x * scales[ids].double()[..., None, None]
        return x.view(len(ids), Hkv, page, d).transpose(0, 1).reshape(Hkv, -1, d)[:, :total]

    bounds = st["prefix_cu"].tolist()
    for b, total in enumerate(lens):
        n = cu[b + 1] - cu[b]
        g = max(i for i in range(len(bounds) - 1) if bounds[i] <= cu[b])
        length = int(st["prefix_lens"][g])
        before = st["prefix_table"][g, :-(-length // page)].long()
        ids = st["table"][b, :-(-total // page)].long()
        k = torch.cat([side(st["k8"], st["ks"], before, length), side(st["k8"], st["ks"], ids, total)], 1)
        v = torch.cat([side(st["v8"], st["vs"], before, length), side(st["v8"], st["vs"], ids, total)], 1)
        pos = torch.arange(length + total - n, length + total, device="cuda")[:, None]
        hide = torch.arange(length + total, device="cuda") > pos
        rows = slice(cu[b], cu[b + 1])
        for h in range(Hq):
            s = (q[rows, h] @ k[h // (Hq // Hkv)].T) / math.sqrt(d)
            s = s.masked_fill(hide, -math.inf)
            z = torch.logsumexp(s, 1)
            lse[h, rows] = z
            o[rows, h] = torch.exp(s - z[:, None]) @ v[h // (Hq // Hkv)]
    if st["dense"]:
        B, n = case["B"], st["n"]
        return dict(o=o.view(B, n, Hq, d), lse=lse.view(Hq, B, n).transpose(0, 1).contiguous())
    return dict(o=o, lse=lse)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prefix":
        return _exact_prefix(st)
    if case["op"] == "backward":
        dq, dqw = _exact_back(st, st["q"], st["dq"], st["q_weight"])
        dk, dkw = _exact_back(st, st["k"], st["dk"], st["k_weight"])
        out = dict(dq=dq, dk=dk)
        return out | dict(dq_weight=dqw, dk_weight=dkw) if case["norm"] else out
    q, k = _exact_ready(st, st["q"], st["q_weight"]), _exact_ready(st, st["k"], st["k_weight"])
    if case["op"] == "forward":
        return dict(q=q, k=k)
    k8, ks = _exact_append(st["k8"], st["ks"], k, st["slots"])
    v8, vs = _exact_append(st["v8"], st["vs"], st["v"], st["slots"])
    return dict(q=q, k8=k8, k_scale=ks, v8=v8, v_scale=vs)
