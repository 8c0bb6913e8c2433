// fa_kv8_work.cuh -- what the kernels of attention over the paged 8-bit cache share: the
// even split of the work over the CTAs, the producer that brings a part's pages and scales
// in, and the cutting of numbers into 8-bit pieces.
#pragma once

#include "fa_kernels.h"
#include "fa_ptx.cuh"
#include "fa_seq.cuh"

#include <climits>
#include <type_traits>

namespace fa {

namespace kv8 {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kKeys = 128;          // keys of a tile
// Weights are kept times 2^12.  A column's reference M moves when a key exceeds it by more
// than 2^3 (its weight then is above 2^15, near fp16's largest number, 65504), so that it
// mostly does not: the maxima over the lanes and the accumulators' rescaling are rare.
constexpr float kShift = 12.f;
constexpr float kGrow = 3.f;
constexpr float kNone = -1e30f;     // in place of a column's reference that has none yet
constexpr int kWindow = 64;         // requests whose lengths a CTA keeps in shared memory
constexpr int kThreads = 256;

constexpr int kCtaSmem = 233472 / 2 - 1024;   // two CTAs per SM
constexpr int kMaxSlots = 12;
constexpr int kParts = 4;         // parts the producer may be ahead
constexpr int kScaleSlots = 16;   // tiles whose scales are kept: more than the ring is long

// ------------------------------------------------------------- work distribution
//
// An item is a block of C rows of one request and key/value head, a row being a (new token,
// head of the group) pair.  An item has the key tiles that its rows see, counted in units of
// a tile, and kItemCost more units stand for its fixed cost.  All items lie one behind the
// other and CTA c takes an equal, contiguous share of the units, whatever items begin and
// end in it; its part of an item that it shares with other CTAs goes to the workspace.
//
// With a causal mask a request's later blocks see more keys.  Its blocks are taken in
// pairs, the first with the last and so on, which all see about as many keys together, so
// that every pair has the same units (a few of them empty) and no sums over blocks are
// needed to find a CTA's place.

struct Request {
    int start, n;   // new tokens
    int len;        // tokens in the cache, the new ones among them
};

// (As seq_bounds of fa_seq.cuh.  These kernels begin while the ones before them, which write
// lengths, bounds, table, cache and queries, may be running, so they read nothing through the
// read-only path, which is for data that nobody writes while a kernel lives.)
__device__ __forceinline__ Request load_request(const Kv8FwdParams& p, int b) {
    Request r;
    if (p.seq.cu_seqlens) {
        r.start = min(max(p.seq.cu_seqlens[b], 0), p.seq.total_tokens);
        r.n = min(max(p.seq.cu_seqlens[b + 1], r.start), p.seq.total_tokens) - r.start;
    } else {
        r.start = b * p.seq.N;
        r.n = p.seq.N;
    }
    const long long room = static_cast<long long>(p.width) << p.page_log2;
    r.len = static_cast<int>(min(max(static_cast<long long>(p.lens[b]), 0LL), room));
    return r;
}

template <int C>
constexpr int kItemCost = C <= 16 ? 1 : 4;

// The first key that a token at position `pos` sees, max(pos - window + 1, 0) with a window.
// (A request with more new tokens than keys has positions below 0, and a window may be as
// large as an int: their difference need not be one.)
__device__ __forceinline__ int first_key(int window, int pos) {
    return window > 0 ? max(pos, window - 1) - (window - 1) : 0;
}

// The items of a request for one key/value head: `blocks` blocks of C rows in `pairs`
// pairs of `cost` units each.
struct Items {
    int blocks, pairs, cost;
};

// A request's rows are one block where items are narrow (kv8_columns chose them so), and its
// units fit 32 bits (fa_fwd_kv8 sees to it).
template <int C>
constexpr bool kOneBlock = C <= 16;
template <int C>
using Units = std::conditional_t<kOneBlock<C>, int, long long>;

// (Out of line, like the division: the kernels' many roles make much code, and what does not
// fit the SM's instruction cache has to be fetched again and again.)
template <int C>
static __device__ __noinline__ Items items_of_blocks(const Kv8FwdParams& p, int n, int len) {
    Items it;
    const int G = p.seq.group;
    it.blocks = (n * G + C - 1) / C;
    it.pairs = (it.blocks + 1) / 2;
    int most = (len + kKeys - 1) / kKeys;   // tiles of a block
    if (p.seq.window > 0) {
        // a block's rows see window + (its tokens - 1) consecutive keys at most
        const long long span = static_cast<long long>(p.seq.window) + (C - 1) / G + 1;
        most = static_cast<int>(min(static_cast<long long>(most), (span + kKeys - 2) / kKeys + 1));
    }
    if (it.blocks <= 1) {
        it.cost = most + kItemCost<C>;
        return it;
    }
    int both = 2 * most;
    if (p.seq.causal) {
        // blocks i and blocks - 1 - i end at positions that add up to this or less
        const long long ends = 2LL * (len - n) + (it.blocks + 1) * static_cast<long long>(C) / G;
        both = static_cast<int>(min(static_cast<long long>(both), max(ends / kKeys + 2, static_cast<long long>(most))));
    }
    it.cost = both + 2 * kItemCost<C>;
    return it;
}

template <int C>
__device__ __forceinline__ Items items_of(const Kv8FwdParams& p, int n, int len) {
    if constexpr (!kOneBlock<C>) {
        return items_of_blocks<C>(p, n, len);
    } else {
        Items it;
        it.blocks = it.pairs = n > 0 ? 1 : 0;
        int tiles = (len + kKeys - 1) / kKeys;
        if (p.seq.window > 0) {
            const long long span = static_cast<long long>(p.seq.window) + p.seq.N;
            tiles = static_cast<int>(min(static_cast<long long>(tiles), (span + kKeys - 2) / kKeys + 1));
        }
        it.cost = tiles + kItemCost<C>;
        return it;
    }
}

static __device__ __noinline__ long long divide_long(long long a, long long b) { return a / b; }

__device__ __forceinline__ int divide(int a, int b) {
    return static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}
// 64-bit division that mostly is a 32-bit one.
__device__ __forceinline__ long long divide(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return divide_long(a, b);
}

// CTA c of the first G takes units [c total / G, (c + 1) total / G) of `total`; G is the
// number of CTAs, or of units where there are fewer, so that no share among them is empty.
template <class U>
__device__ __forceinline__ int sharers(U total, int ctas) {
    return static_cast<int>(min(total, static_cast<U>(ctas)));
}
template <class U>
__device__ __forceinline__ U share_begin(U total, int c, int G) {   // (G < 2^10)
    const U q = static_cast<U>(divide(total, static_cast<U>(G)));
    return q * c + static_cast<U>(static_cast<uint32_t>((total - q * G) * c) / static_cast<uint32_t>(G));
}
__device__ __forceinline__ int share_of(long long total, long long unit, int G) {
    return static_cast<int>(divide((unit + 1) * G - 1, total));
}

// One CTA's part of an item.
struct Part {
    Request req;
    int b, h, row0;     // request, key/value head, first row
    int tile0, tiles;   // the part's key tiles (absolute); 0: an item whose rows see nothing
    bool whole;         // all of the item's tiles
    bool begins;        // the item's first tile is the part's
    long long unit0;    // the item's first unit
    int item_tiles;
    int lo_key, hi_key; // the keys that any row of the item sees: [lo_key, hi_key]
    int all_lo, all_hi; // the keys that every row sees
};

// Where a CTA's share begins, found by all its threads.
struct Share {
    long long begin, end, total;
    int b0, h, pair, off;   // the request, head, pair of blocks and unit of that pair it begins at
};

// A walk over a CTA's parts (the producer's; it hands them to the other roles).
template <int C>
struct Walk {
    const Kv8FwdParams& p;
    const int3* window;      // (start, n, len) of requests b0 .. b0 + kWindow - 1, in shared memory
    int b0, b, h, pair, off; // request, head, pair of blocks, units of that pair behind us
    long long left, unit;    // units left, the next one's number
    Request req;
    Items it;

    __device__ Walk(const Kv8FwdParams& p_, const Share& s, const int3* w)
        : p(p_), window(w), b0(s.b0), b(s.b0), h(s.h), pair(s.pair), off(s.off),
          left(s.end - s.begin), unit(s.begin) {
        load();
    }
    __device__ void load() {
        if (b >= p.seq.B || left == 0) return;
        if (b - b0 < kWindow) {
            const int3 w = window[b - b0];
            req.start = w.x;
            req.n = w.y;
            req.len = w.z;
        } else {
            req = load_request(p, b);
        }
        it = items_of<C>(p, req.n, req.len);
    }
    // The keys that the rows of block `blk` see.
    __device__ __forceinline__ void see(int blk, Part& part) const {
        part.row0 = blk * C;
        int first = req.len - req.n, last = first;   // positions of its first and last token
        if constexpr (kOneBlock<C>) {
            last += min(req.n, C) - 1;
        } else {
            const int G = p.seq.group;
            first += part.row0 / G;
            last += min((part.row0 + C - 1) / G, req.n - 1);
        }
        part.hi_key = p.seq.causal ? last : req.len - 1;
        part.all_hi = p.seq.causal ? first : req.len - 1;
        part.lo_key = first_key(p.seq.window, first);
        part.all_lo = first_key(p.seq.window, last);
        part.tile0 = part.lo_key / kKeys;
        part.item_tiles = part.hi_key >= part.lo_key ? part.hi_key / kKeys - part.tile0 + 1 : 0;
        // (more new tokens than the call announced: no more keys than there are units for)
        if (kOneBlock<C>) part.item_tiles = min(part.item_tiles, it.cost - kItemCost<C>);
    }
    __device__ __forceinline__ bool next(Part& part) {
#pragma unroll 1
        while (left > 0 && b < p.seq.B) {
            if (off >= it.cost) {
                off = 0;
                ++pair;
            }
            if (pair >= it.pairs) {
                pair = 0;
                if (it.pairs == 0 || ++h == p.seq.Hkv) {
                    h = 0;
                    ++b;
                    load();
                }
                continue;
            }
            int before = 0;   // units of the pair before this item's
            see(pair, part);
            if (!kOneBlock<C> && off >= part.item_tiles + kItemCost<C> && it.blocks - 1 - pair != pair) {
                before = part.item_tiles + kItemCost<C>;
                see(it.blocks - 1 - pair, part);
            }
            const int at = off - before;
            const bool none = at >= part.item_tiles + kItemCost<C>;   // the pair's empty units
            const int end = none ? it.cost - before : part.item_tiles + kItemCost<C>;
            const int take = static_cast<int>(min(left, static_cast<long long>(end - at)));
            part.unit0 = unit - at;
            off += take;
            left -= take;
            unit += take;
            if (none) continue;
            const int t1 = min(at + take, part.item_tiles);
            part.req = req;
            part.b = b;
            part.h = h;
            part.tile0 += at;
            part.tiles = max(t1 - at, 0);
            part.begins = at == 0;
            part.whole = part.begins && t1 == part.item_tiles;
            if (part.tiles > 0 || part.whole) return true;
        }
        return false;
    }
};

// The 16-byte unit u of row r in a tile of rows of D bytes, swizzled over D bytes.
template <int D>
__device__ __forceinline__ int unit_offset(int r, int u) {
    return r * D + ((u ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Exponent of the power of two that brings a row's largest magnitude into (224, 448].
__device__ __forceinline__ int row_exponent(uint32_t amax_bits) {
    const int e = static_cast<int>(amax_bits >> 23) - 127;
    return max(e - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0), -100);
}

__device__ __forceinline__ float pow2f(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

// Eight consecutive elements of a row of queries (D / 8 neighbouring lanes have the row, all
// of them take part), cut into KQ e4m3 pieces for `dst` (pieces `piece` bytes apart): the row
// times the power of two that brings its largest element into (224, 448], as fp16 numbers
// (exact: 8 or 11 bits), each piece the rounding of what the ones before it leave.  Returns
// the row's scale.  An infinity or NaN makes all the row's pieces NaN, and with them its
// products (its scale stays a number: masked products must stay -inf whatever they are
// multiplied by, so that a row that sees nothing comes out as one).
template <int D, int E, int KQ>
__device__ __forceinline__ float cut_queries(uint4 w, uint8_t* dst, int piece) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t top = 0;   // magnitudes, as the integers of two 16-bit numbers
#pragma unroll
    for (int j = 0; j < 4; ++j) top = __vmaxu2(top, u[j] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t amax = __float_as_uint(unpack2<E>(top).x);
    const bool fine = amax < 0x7f800000u;
    const int k = fine ? row_exponent(amax) : 0;
    const float inv = pow2f(-k);
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = unpack2<E>(u[j]);
        h[j] = fine ? pack2<kElemF16>(f.x * inv, f.y * inv) : 0x7fff7fffu;
    }
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
        uint32_t c[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            asm("{\n\t.reg .b16 lo, hi;\n\t"
                "cvt.rn.satfinite.e4m3x2.f16x2 lo, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 hi, %2;\n\t"
                "mov.b32 %0, {lo, hi};\n\t}"
                : "=r"(c[j]) : "r"(h[2 * j]), "r"(h[2 * j + 1]));
        *reinterpret_cast<uint2*>(dst + q * piece) = make_uint2(c[0], c[1]);
        if (q + 1 < KQ) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t lo, hi;
                asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                    "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                    : "=r"(lo), "=r"(hi) : "r"(c[j]));
                h[2 * j] = sub_f16x2(h[2 * j], lo);
                h[2 * j + 1] = sub_f16x2(h[2 * j + 1], hi);
            }
        }
    }
    return pow2f(k);
}

// Bytes of a word that are e4m3 NaN (0x7f or 0xff), as 0x80 in each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// a / b for 0 <= a < 2^16, with inv = ceil(2^32 / b): the product is within 2^-16 of a / b
// from above.  (b = 1: inv would be 2^32.)
__device__ __forceinline__ int small_div(int a, int b, uint32_t inv) {
    if (b == 1) return a;
    return a < 65536 ? static_cast<int>(__umulhi(static_cast<uint32_t>(a), inv)) : a / b;
}

// Inclusive sums over the block of one value per thread, and the block's total.
template <class U>
__device__ __forceinline__ U block_units(U v, long long* warp_sums, U* total) {
    U* sums = reinterpret_cast<U*>(warp_sums);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const U u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    U before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const U x = sums[w];
        if (w < warp) before += x;
        all += x;
    }
    *total = all;
    return v + before;
}

// Finds this CTA's share: sums of the requests' units, by all threads.
template <int C, class Smem>
__device__ __forceinline__ void find_share(const Kv8FwdParams& p, Smem& sm) {
    const int cta = blockIdx.x, B = p.seq.B;
    using U = Units<C>;
    U begin = 0, before = 0, total = 0;
    Request r{0, 0, 0};
    auto units = [&](int b) -> U {
        if (b >= B) return 0;
        r = load_request(p, b);
        const Items it = items_of<C>(p, r.n, r.len);
        return static_cast<U>(it.pairs) * p.seq.Hkv * it.cost;
    };
    // request b's units end at `end`, `mine` of them: does the share begin there?
    auto look = [&](int b, U mine, U end) {
        if (begin >= end - mine && begin < end) {
            const Items it = items_of<C>(p, r.n, r.len);
            const U at = begin - (end - mine), item = static_cast<U>(divide(at, static_cast<U>(it.cost)));
            const int h = kOneBlock<C> ? static_cast<int>(item) : static_cast<int>(divide(item, static_cast<U>(it.pairs)));
            sm.share.b0 = b;
            sm.share.off = static_cast<int>(at - item * it.cost);
            sm.share.h = h;
            sm.share.pair = static_cast<int>(item - static_cast<U>(h) * it.pairs);
        }
    };
    const U first = units(threadIdx.x);
    U sum = first;
#pragma unroll 1
    for (int b = threadIdx.x + kThreads; b < B; b += kThreads) sum += units(b);
    const U upto = block_units(sum, sm.warp_sums, &total);
    const int G = sharers(total, gridDim.x);
    begin = cta < G ? share_begin(total, cta, G) : total;
    if (threadIdx.x == 0) {
        sm.share.begin = begin;
        sm.share.end = cta < G ? share_begin(total, cta + 1, G) : total;
        sm.share.total = total;
    }
    if (B <= kThreads) {
        look(threadIdx.x, first, upto);
        __syncthreads();
        const int at = static_cast<int>(threadIdx.x) - sm.share.b0;
        if (at >= 0 && at < kWindow) sm.window[at] = make_int3(r.start, r.n, r.len);
    } else {
#pragma unroll 1
        for (int b0 = 0; b0 < B; b0 += kThreads) {
            const int b = b0 + threadIdx.x;
            const U mine = units(b);
            U all;
            const U end = before + block_units(mine, sm.warp_sums, &all);
            look(b, mine, end);
            before += all;
        }
        __syncthreads();
        const int b = sm.share.b0 + threadIdx.x;
        if (threadIdx.x < kWindow && sm.share.begin < total) {
            r = Request{0, 0, 0};
            if (b < B) r = load_request(p, b);
            sm.window[threadIdx.x] = make_int3(r.start, r.n, r.len);
        }
    }
}

// The part of a wait that is not over at once, out of line: the kernels' roles wait in many
// places.  The hardware suspends the thread for up to 0.5 us at a time, so that waiting warps
// take no issue slots from the others; gives up as mbar_wait does.  (More registers here, for a
// time worked out from the limit, cost the 128-row kernel 1 to 5 % in its callers.)
static __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort, long long limit,
                                            int* status) {
    const long long t0 = clock64();
    while (true) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity), "r"(500u)
            : "memory");
        if (done) return *abort == 0;   // (produce: a place given back for an abort is not free)
        if (*abort) return false;
        if (clock64() - t0 > limit) {
            *abort = 1;
            atomicExch(status, kDevTimeout);
            return false;
        }
    }
}

template <class Smem>
__device__ __forceinline__ bool wait_for(const Kv8FwdParams& p, Smem& sm, uint64_t* bar, int phase) {
    return mbar_try_wait(smem_addr(bar), phase & 1) ||
           wait_on(smem_addr(bar), phase & 1, &sm.abort, p.timeout_cycles, p.status);
}

// A wait that ignores the abort flag, out of line: for what still comes after an abort.  It
// comes at the latest when every other wait has given up, so this one waits for longer than
// any of those may.  (A limit out of the parameters costs 3 to 5 % of the 128-row kernel's
// time, by the registers that the call then takes: hence a constant, above a bound that the
// host keeps.)
constexpr long long kKv8DrainCycles = 2 * kKv8MaxWaitCycles + 2 * kDrainCycles;
static __device__ __noinline__ void drain_on(uint32_t bar, uint32_t parity) {
    mbar_wait_drain(bar, parity, kKv8DrainCycles);
}

// Part number np, in registers; false behind the last.  After an abort too every role goes
// through all the parts (their named barriers pair up), so these waits ignore it.
template <class Smem>
__device__ __forceinline__ bool take_part(Smem& sm, int np, Part& part) {
    drain_on(smem_addr(&sm.part_full[np % kParts]), (np / kParts) & 1);
    part = sm.parts[np % kParts];
    return part.tiles >= 0;
}

// O = 0 and LSE = -inf for an item that sees no keys: `rows` rows from row0 on, by a warp.
template <int D>
static __device__ __noinline__ void rows_without_keys(const Kv8FwdParams& p, int b, int h, int start, int row0,
                                                      int rows) {
    const int lane = threadIdx.x & 31, G = p.seq.group;
#pragma unroll 1
    for (int r = row0; r < row0 + rows; ++r) {
        const int tok = r / G, head = h * G + r % G;
        const long long token = start + tok;
        if (!fa_index_ok(token, p.seq.total_tokens, p.status)) continue;
        uint16_t* out = static_cast<uint16_t*>(p.o) + (token * p.seq.Hq + head) * D;
        if (lane < D / 8) *reinterpret_cast<uint4*>(out + 8 * lane) = make_uint4(0, 0, 0, 0);
        if (lane == 0) p.lse[row_stat_index(p.seq, b, head, start, tok)] = kNegInf;
    }
}

// The producer warp: walks the CTA's share, hands its parts out, and for each part's tiles
// copies K and V in units of U keys (K's units, then V's) through the ring of slots (pages by
// TMA, rows of d bytes swizzled over d bytes), and with the first of them the tile's 16
// scales (K's, then V's; -1 for V's where a block's tokens are hidden: behind the last key
// that is seen, or on a page that the cache does not have).
//
// An item whose rows see nothing (an idle seat, a refused prompt) it writes itself and does not
// hand out.  The issuer looks one tile ahead, into the next part, before it issues this part's
// last product, so a part that it waits for there must not depend on that product.  A part with
// tiles does not: its place among the parts and its queries' place were given back by parts
// before this one.  Without tiles any number of parts could follow, and would.
//
// One warp's instructions for a tile take about as long as a narrow tile does, so what its
// copies have in common is worked out once and the table is read while the part is handed
// over.  (A lane has a copy; the lanes' copies are issued one by one, some 80 cycles each, 16 a
// tile with pages of 16 tokens.  A second producer warp, for V, made that case slower, 42.7 ->
// 50.3 us for 128 requests of up to 2048 tokens at d = 64: the kernel's roles share the
// instruction cache, and more code in flight costs more than the wait.)
template <int D, int C, int U, int kSlots, class Smem>
__device__ __forceinline__ void produce(const Kv8FwdParams& p, Smem& sm, uint8_t* sKV) {
    constexpr int kUnits = kKeys / U;          // of a side
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    const int page = 1 << p.page_log2, per_tile = kKeys >> p.page_log2;
    const int box_log2 = min(p.page_log2, U == 128 ? 7 : 6);
    const int key = lane << box_log2;          // this lane's copy: keys from here on (none from 128 on)
    const int unit_boxes = U >> box_log2;
    const int blocks_log2 = p.page_log2 - 4;   // scale blocks of a page
    const int side_blk = lane & 7;             // lanes 0..7: K's scales, 8..15: V's
    int c = 0;                                 // tiles
    int slot = 0, use = 0;                     // the next unit's slot, how often it was used
    bool ok = true, joined = false;
    Part part;
    Walk<C> walk(p, sm.share, sm.window);      // (a CTA without a share has no parts)
#pragma unroll 1
    for (int np = 0;;) {
        const bool more = walk.next(part);
        if (more && part.tiles == 0) {
            rows_without_keys<D>(p, part.b, part.h, part.req.start, part.row0,
                                 min(C, part.req.n * p.seq.group - part.row0));
            continue;
        }
        if (!more) part.tiles = -1;
        const int* row = p.table + static_cast<long long>(part.b) * p.width;
        const int lim = min(part.hi_key + 1, part.req.len);   // tokens from here on are not needed
        const int last_page = min((lim + page - 1) >> p.page_log2, p.width);
        // the table's entries, 32 at a time, the next ones on their way
        int base = part.tile0 * per_tile;
        auto entry = [&](int i) { return i < last_page ? row[i] : -1; };
        int cur = more ? entry(base + lane) : -1;
        int nxt = more ? entry(base + 32 + lane) : -1;
        if (np >= kParts)
            drain_on(smem_addr(&sm.part_empty[np % kParts]), (np / kParts - 1) & 1);
        if (lane == 0) {
            sm.parts[np % kParts] = part;
            mbar_arrive(smem_addr(&sm.part_full[np % kParts]));
            if (more && part.begins && !part.whole) {
                Kv8Join j;
                j.last = share_of(sm.share.total, part.unit0 + part.item_tiles - 1,
                                  sharers(sm.share.total, gridDim.x));
                j.b = part.b;
                j.h = part.h;
                j.start = part.req.start;
                j.n = part.req.n;
                j.row0 = part.row0;
                p.joins[blockIdx.x] = j;
                joined = true;
            }
        }
        __syncwarp();
        if (!more) break;
        ++np;
#pragma unroll 1
        for (int i = 0; i < part.tiles && ok; ++i, ++c) {
            const int tile = part.tile0 + i;
            if (tile * per_tile >= base + 32) {
                base += 32;
                cur = nxt;
                nxt = entry(base + 32 + lane);
            }
            const int first = tile * per_tile - base;
            const int id = __shfl_sync(0xffffffffu, cur, (first + (key >> p.page_log2)) & 31);
            const bool load = key < kKeys && id >= 0 && id < p.num_pages && tile * kKeys + key < lim;
            const uint32_t loads = __ballot_sync(0xffffffffu, load);
            const int page_row = id * p.seq.Hkv + part.h;
            const int sid = __shfl_sync(0xffffffffu, cur, (first + (side_blk >> blocks_log2)) & 31);
#pragma unroll 1
            for (int unit = 0; unit < 2 * kUnits; ++unit) {
                if (use > 0) {
                    // After an abort the issuer gives places back whatever became of their copies,
                    // and nothing may be copied to one that has a copy on its way.  (Both loads are on
                    // their way together; the abort comes long before a place given back for it.)
                    const int abort = *const_cast<volatile int*>(&sm.abort);
                    const uint32_t bar = smem_addr(&sm.kv_empty[slot]);
                    const int phase = (use - 1) & 1;
                    ok = mbar_try_wait(bar, phase) ? abort == 0
                                                   : wait_on(bar, phase, &sm.abort, p.timeout_cycles, p.status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                const uint32_t full = smem_addr(&sm.kv_full[slot]);
                if (lane == 0) {
                    const uint32_t n = __popc(loads >> (unit % kUnits * unit_boxes) & ((1u << unit_boxes) - 1u));
                    mbar_arrive_expect_tx(full, (n << box_log2) * D);
                }
                __syncwarp();
                if (load && (kUnits == 1 || key / U == unit % kUnits))
                    tma_load_3d(smem_addr(sKV + (slot * U + key % U) * D), unit < kUnits ? &p.tm_k : &p.tm_v, full,
                                0, key & (page - 1), page_row);
                if (++slot == kSlots) {
                    slot = 0;
                    ++use;
                }
                if (unit == 0) {
                    // the scales (their slot's last tile is long done)
                    const uint32_t sbar = smem_addr(&sm.scales_full[c % kScaleSlots]);
                    bool plain = true;
                    if (lane < 16) {
                        float* to = &sm.scales[c % kScaleSlots][lane];
                        if (sid >= 0 && sid < p.num_pages && tile * kKeys + side_blk * kKv8Block < lim) {
                            const long long at =
                                ((static_cast<long long>(sid) * p.seq.Hkv + part.h) << blocks_log2) +
                                (side_blk & ((1 << blocks_log2) - 1));
                            cp_async4(smem_addr(to), (lane < 8 ? p.k_scale : p.v_scale) + at);
                            plain = false;
                        } else {
                            *to = lane < 8 ? 0.f : -1.f;   // hidden
                        }
                    }
                    if (plain) mbar_arrive(sbar);
                    else cp_async_arrive(sbar);
                }
            }
        }
    }
    if (lane == 0 && !joined) p.joins[blockIdx.x].last = 0;
    // every copy lands before the CTA exits, whatever became of the other roles
#pragma unroll 1
    for (int i = 0; i < kSlots; ++i) {
        const int last = i < slot ? use : use - 1;
        if (last >= 0) drain_on(smem_addr(&sm.kv_full[i]), last & 1);
    }
    // (a tile has its scales from its first unit on)
    const int tiles = (use * kSlots + slot + 2 * kUnits - 1) / (2 * kUnits);
#pragma unroll 1
    for (int i = max(0, tiles - kScaleSlots); i < tiles; ++i)
        drain_on(smem_addr(&sm.scales_full[i % kScaleSlots]), (i / kScaleSlots) & 1);
}

// A launch that may begin while the kernel before it on the stream is ending (it waits for
// that one's results itself).
template <class Params>
cudaError_t launch_dependent(void (*kern)(Params), dim3 grid, int threads, int smem, cudaStream_t stream,
                             const Params& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace kv8
}  // namespace fa
