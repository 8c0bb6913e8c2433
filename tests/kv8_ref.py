"""Plain float64 / integer forms of the 8-bit cache's operators (fa_kv8_* of include/fa.h),
on numpy arrays."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16


def e4m3_values():
    """The value of each code, 0 .. 255."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m / 8, -6) if e == 0 else math.ldexp(1 + m / 8, e - 7)
        out[c] = math.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return out


VALUES = e4m3_values()


def e4m3_codes(x):
    """The codes nearest to x (|x| <= 448 or not finite), ties to the even code."""
    mag = VALUES[:127]
    a = np.abs(x)
    fine = np.isfinite(x)
    a = np.where(fine, a, 0.0)
    hi = np.clip(np.searchsorted(mag, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = mag[hi] - a, a - mag[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = code + np.where(np.signbit(x), 128, 0)
    return np.where(fine, code, 127).astype(np.uint8)


def plan(lens, grow, table, ring, state, page, T):
    """(lens, cu, slots, state), table and ring updated in place."""
    before = table.copy()
    B, width = table.shape
    cap = len(ring)
    head, count = int(state[0]), int(state[1])
    out, cu, slots = [], [0], np.full(T, -1, np.int32)
    wanted = used = put = refused = 0
    for b in range(B):
        have = -(-int(lens[b]) // page)
        g = int(grow[b])
        cu.append(cu[-1] + max(g, 0))
        if g < 0:
            for j in range(have):
                ring[(head + count + put) % cap] = before[b, j]
                put += 1
            out.append(0)
            continue
        total = int(lens[b]) + g
        fits = total <= width * page and cu[-1] <= T
        need = -(-total // page) - have if fits else 0
        wanted += need
        if not fits or (need and wanted > count):
            refused += 1
            out.append(int(lens[b]))
            continue
        for j in range(need):
            table[b, have + j] = ring[(head + wanted - need + j) % cap]
        used += need
        for i in range(g):
            pos = int(lens[b]) + i
            slots[cu[b] + i] = table[b, pos // page] * page + pos % page
        out.append(total)
    return (np.array(out, np.int32), np.array(cu, np.int32), slots,
            np.array([(head + used) % cap, count - used + put, refused], np.int32))


def scale_of_amax(amax):
    """2^k for the least k >= -64 with amax <= 448 2^k."""
    k = -64
    while amax > 448 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def append(codes, scales, x, slots):
    """Tokens x [T, Hkv, d] (float64) into one side of the cache, in place."""
    pages, H, page, d = codes.shape
    t = 0
    while t < len(slots):
        if not 0 <= slots[t] < pages * page:
            t += 1
            continue
        e = t + 1
        while e < len(slots) and slots[e] == slots[e - 1] + 1 and slots[e] % BLOCK:
            e += 1
        pg, at = int(slots[t]) // page, int(slots[t]) % page
        blk, off = at // BLOCK, at % BLOCK
        for h in range(H):
            new = x[t:e, h]
            fine = np.isfinite(new)
            s = scale_of_amax(np.max(np.where(fine, np.abs(new), 0.0)))
            if off:
                old = float(scales[pg, h, blk])
                s = max(s, old)
                held = slice(blk * BLOCK, at)
                codes[pg, h, held] = e4m3_codes(VALUES[codes[pg, h, held]] * (old / s))
            scales[pg, h, blk] = s
            codes[pg, h, at:at + e - t] = e4m3_codes(new / s)
        t = e


def attend(q, codes, scales, vcodes, vscales, table, lens, cu, scale, causal=True, window=0,
           p_round=0.0, out_round=0.0):
    """O [T, Hq, d], LSE [Hq, T] and bounds on their errors for kernels that hold sums in 32
    bits, round each probability by a relative p_round at most and O by out_round.

    A score is a sum of d products (2 or 3 pieces of q each) in 32 bits: off by at most
    2^-19 scale sum|q||k|; an exponential and what scales it by 2^-20 relative.  Both change
    each probability by the factor 1 + e, and O by at most 2 e sum P|v| (numerator and sum)."""
    T, Hq, d = q.shape
    pages, H, page, _ = codes.shape
    G = Hq // H
    o, lse = np.zeros((T, Hq, d)), np.full((Hq, T), -math.inf)
    bo, bl = np.zeros((T, Hq, d)), np.zeros((Hq, T))
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        total = min(max(int(lens[b]), 0), table.shape[1] * page)
        if n == 0 or total == 0:
            continue
        j = np.arange(total)
        ids = table[b, j // page]
        known = (ids >= 0) & (ids < pages)
        ids = np.where(known, ids, 0)
        for g in range(H):
            ks, vs = scales[ids, g, j % page // BLOCK], vscales[ids, g, j % page // BLOCK]
            k = VALUES[codes[ids, g, j % page]] * ks.astype(np.float64)[:, None]
            v = VALUES[vcodes[ids, g, j % page]] * vs.astype(np.float64)[:, None]
            for i in range(n):
                pos = total - n + i
                see = known & ((j <= pos) if causal else True)
                if window:
                    see = see & (j > pos - window)
                if not see.any():
                    continue
                t = int(cu[b]) + i
                for h in range(g * G, g * G + G):
                    s = scale * (k[see] @ q[t, h])
                    size = scale * (np.abs(k[see]) @ np.abs(q[t, h]))
                    m = s.max()
                    p = np.exp(s - m)
                    z = p.sum()
                    lse[h, t] = m + math.log(z)
                    p /= z
                    o[t, h] = p @ v[see]
                    e = 2.0 ** -19 * size.max() + 2.0 ** -20
                    bl[h, t] = 2 * e + 2.0 ** -22 * abs(lse[h, t])
                    # what underflows: a weight below 2^-28 of the largest (P times V's scale)
                    lost = 2.0 ** -28 * (p * vs[see]).max() * 448 * see.sum()
                    mass = p @ np.abs(v[see])
                    bo[t, h] = (p_round + 2 * e) * mass + lost
                    bo[t, h] = bo[t, h] + out_round * (np.abs(o[t, h]) + bo[t, h])
    return o, lse, bo, bl
