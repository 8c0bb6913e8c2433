// fa_kv8_cache.cu -- the paged 8-bit cache's bookkeeping (block tables, slots, free
// pages) and its writer.  The formats and rules are those of fa_kv8_plan and
// fa_kv8_append in include/fa.h.
#include "fa_kv8_work.cuh"
#include "fa_norm_rope.cuh"

#include <algorithm>
#include <climits>

namespace fa {
namespace {

// ------------------------------------------------------------------------- plan

// Inclusive sums over the block of one value per thread, and the block's total.
// `warp_sums` holds one value per warp (32 at most).
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    auto scan = [&](long long x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += u;
        }
        return x;
    };
    v = scan(v);
    __syncthreads();   // the last scan's sums have been read
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    // every warp scans the warps' sums for itself
    const long long sums = scan(lane < warps ? warp_sums[lane] : 0);
    *total = __shfl_sync(0xffffffffu, sums, 31);
    return v + (warp > 0 ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0);
}

// What every CTA knows of each request after the scans.
struct PlanRequest {
    int end;      // its tokens end here in the packed batch
    int len;      // tokens it holds
    int first;    // pages taken from the ring before its own; -1: it gets none (refused or ended)
    int back;     // pages given back before its own; -1: it has not ended
};

// Every CTA does the sums over all requests itself, from memory that no CTA writes (B
// is at most 8192, the loads come from L2), so one launch does the whole plan and no CTA
// waits for another; then the threads of the grid share the tokens out among themselves
// (a binary search of the requests' ends in shared memory), and the warps the ended
// requests.  The table entries and ring places that are read (old blocks, free pages)
// are never among those that are written (new blocks, behind the free pages).  Bound by
// latency (a few KB in all): 4.5 us for 64 requests of a token, 5.1 us for 384 of up to 257, and
// 10.4 us where 40 of those end, the longest with 993 pages: a request's pages are given back by
// one warp, 32 at a time, each load behind the store before it.
__global__ void __launch_bounds__(1024) kv8_plan_kernel(const Kv8PlanParams p) {
    extern __shared__ PlanRequest req[];   // [B]
    __shared__ long long warp_sums[32];
    __shared__ int used;     // pages taken from the ring: the served requests with the largest sum
    if (threadIdx.x == 0) used = 0;
    grid_launch_dependents();
    grid_dependency_wait();
    const int page = 1 << p.page_log2;
    const int cap = p.num_pages;
    int head = p.state[0] % cap;
    if (head < 0) head += cap;
    const int count = min(max(p.state[1], 0), cap);
    const long long room = static_cast<long long>(p.width) << p.page_log2;

    long long tokens = 0, wanted = 0, gone = 0, refused = 0;
    for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        const bool in = b < p.B;
        const int g = in ? p.grow[b] : 0;
        const long long len = in ? min(max(static_cast<long long>(p.lens[b]), 0LL), room) : 0;
        const long long add = max(g, 0);
        long long sum;
        const long long end = tokens + block_scan(add, warp_sums, &sum);
        tokens += sum;
        const long long have = (len + page - 1) >> p.page_log2;
        const bool fits = in && g >= 0 && len + add <= room && end <= p.T;
        const long long need = fits ? ((len + add + page - 1) >> p.page_log2) - have : 0;
        const long long last = wanted + block_scan(need, warp_sums, &sum);
        wanted += sum;
        const bool served = fits && (need == 0 || last <= count);
        const long long freed = in && g < 0 ? have : 0;
        const long long back = gone + block_scan(freed, warp_sums, &sum) - freed;
        gone += sum;
        if (served && need > 0) atomicMax(&used, static_cast<int>(last));
        refused += __syncthreads_count(in && g >= 0 && !served);
        if (in) {
            PlanRequest r;
            r.end = static_cast<int>(min(end, static_cast<long long>(INT_MAX)));
            r.len = static_cast<int>(len);
            r.first = served ? static_cast<int>(last - need) : -1;
            r.back = g < 0 ? static_cast<int>(min(back, static_cast<long long>(INT_MAX))) : -1;
            req[b] = r;
            if (blockIdx.x == 0) {
                p.lens_out[b] = static_cast<int>(g < 0 ? 0 : served ? len + add : len);
                p.cu_out[b + 1] = r.end;
            }
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.cu_out[0] = 0;
        p.state_out[0] = static_cast<int>((head + used) % cap);
        p.state_out[1] = static_cast<int>(min(count - used + gone, static_cast<long long>(cap)));
        p.state_out[2] = static_cast<int>(refused);
    }
    __syncthreads();

    const int threads = gridDim.x * blockDim.x;
    for (long long t = blockIdx.x * blockDim.x + threadIdx.x; t < p.T; t += threads) {
        int lo = 0, hi = p.B;   // the first request whose end is behind t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (req[mid].end > t) hi = mid;
            else lo = mid + 1;
        }
        int slot = -1;
        if (lo < p.B) {
            const PlanRequest r = req[lo];
            if (r.first >= 0) {
                const int pos = r.len + static_cast<int>(t) - (lo ? req[lo - 1].end : 0);
                const int blk = pos >> p.page_log2;
                const int k = blk - ((r.len + page - 1) >> p.page_log2);
                int* entry = p.table + static_cast<long long>(lo) * p.width + blk;
                int id;
                if (k >= 0) {
                    id = p.ring[(static_cast<long long>(head) + r.first + k) % cap];
                    if ((pos & (page - 1)) == 0) *entry = id;
                } else {
                    id = *entry;
                }
                if (id >= 0 && id < cap) slot = (id << p.page_log2) + (pos & (page - 1));
            }
        }
        p.slots[t] = slot;
    }
    const int lane = threadIdx.x & 31;
    for (int b = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; b < p.B; b += threads >> 5) {
        const PlanRequest r = req[b];
        if (r.back < 0) continue;
        const int have = (r.len + page - 1) >> p.page_log2;
        for (int k = lane; k < have; k += 32) {
            // (a ring that claims more free pages than there can be is not overrun)
            const long long at = static_cast<long long>(count) + r.back + k;
            if (at < cap) p.ring[(head + at) % cap] = p.table[static_cast<long long>(b) * p.width + k];
        }
    }
}

// ----------------------------------------------------------------------- append

// Exponent of the least power of two, 2^-64 at least, with amax <= 448 * 2^k: with
// amax = m 2^e, 1 <= m < 2, and 448 = 1.75 * 2^8, k = e - 8 where m <= 1.75 and e - 7
// beyond.
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
    const int e = static_cast<int>(amax_bits >> 23) - 127;
    return max(e - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0), -64);
}

__device__ __forceinline__ float pow2f(int k) { return __uint_as_float((k + 127) << 23); }

// Four e4m3 codes widened to fp32 (exact; NaN stays NaN).
__device__ __forceinline__ void unpack4_e4m3(uint32_t w, float (&f)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    const float2 x = unpack2<kElemF16>(lo), y = unpack2<kElemF16>(hi);
    f[0] = x.x;
    f[1] = x.y;
    f[2] = y.x;
    f[3] = y.y;
}

// a * b and a / b in fp32, rounded to odd: toward zero, and the last bit set where that was not
// exact.  A value so rounded rounds on to e4m3's 4 bits as the exact one does (the 20 bits
// between hold whether it lies above, below or on a tie).  An exact one stays as it is.
__device__ __forceinline__ float to_odd(float x, bool exact) {
    return exact ? x : __uint_as_float(__float_as_uint(x) | 1u);
}
__device__ __forceinline__ float mul_odd(float a, float b) {
    const float x = __fmul_rz(a, b);
    return to_odd(x, __fmaf_rn(a, b, -x) == 0.f);
}
__device__ __forceinline__ float div_odd(float a, float b) {
    const float x = __fdiv_rz(a, b);
    return to_odd(x, __fmaf_rn(-x, b, a) == 0.f);
}

// Whether the addresses formed lie in their tensors (checking build): 8 codes, or a scale, of one side of the
// cache (keys 0, values 1), and 8 channels of a new token, as it is written without norm and rotation.
template <int D>
__device__ __forceinline__ bool codes_ok(const Kv8AppendParams& p, int side, const void* at) {
    return fa_row_ok(p.codes[side], at, 8, static_cast<long long>(p.num_slots) * p.Hkv, D, D, p.status);
}
__device__ __forceinline__ bool scale_ok(const Kv8AppendParams& p, int side, const float* at) {
    return fa_index_ok(at - p.scales[side], static_cast<long long>(p.num_slots) / kKv8Block * p.Hkv, p.status);
}
template <int D>
__device__ __forceinline__ bool values_ok(const Kv8AppendParams& p, int side, const void* at) {
    return fa_row_ok(p.x[side], at, 16, p.T, 2LL * D * p.Hkv, 2 * p.stride, p.status);
}

// The codes of n new tokens of a block whose scale is not a power of two, by a warp: a block that
// another writer began (this one's scales are powers of two).  `x` and `row` are the lane's 8
// values of the first token.
template <int D, int E>
__device__ __noinline__ void append_by_division(const Kv8AppendParams& p, int side, const uint16_t* x, uint8_t* row, int n,
                                                float scale) {
    const long long stride = p.stride;
    for (int r = (threadIdx.x & 31) / (D / 8); r < n; r += 32 / (D / 8)) {
        if (!values_ok<D>(p, side, x + r * stride) || !codes_ok<D>(p, side, row + static_cast<long long>(r) * D)) continue;
        const uint4 w = *reinterpret_cast<const uint4*>(x + r * stride);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 g = unpack2<E>(u[j]);
            f[2 * j] = div_odd(g.x, scale) + g.x * 0.f;   // (inf * 0 is NaN: infinities become NaN codes)
            f[2 * j + 1] = div_odd(g.y, scale) + g.y * 0.f;
        }
        *reinterpret_cast<uint2*>(row + static_cast<long long>(r) * D) = make_uint2(pack4_e4m3(f[0], f[1], f[2], f[3]), pack4_e4m3(f[4], f[5], f[6], f[7]));
    }
}

// The next run of consecutive slots of one block among a batch's tokens, from token t on.
struct BlockRun {
    int slot, off, n;   // its first slot, that one's place in the block, its tokens
    bool skip;          // no place in the cache, or a block that an earlier warp began
};
__device__ __forceinline__ BlockRun next_run(const Kv8AppendParams& p, int t, long long c0) {
    const int lane = threadIdx.x & 31;
    BlockRun r;
    r.slot = fa_index_ok(t, p.T, p.status) ? p.slots[t] : -1;
    r.off = r.slot & (kKv8Block - 1);
    const bool real = r.slot >= 0 && r.slot < p.num_slots;
    const int mine = lane < kKv8Block && t + lane < p.T ? p.slots[t + lane] : -1;
    const uint32_t follows = __ballot_sync(
        0xffffffffu, real && r.off + lane < kKv8Block && mine == r.slot + lane);
    r.n = real ? __ffs(~follows) - 1 : 1;   // lane 16 never follows
    r.skip = !real || (r.off > 0 && t == c0 && t > 0 && p.slots[t - 1] == r.slot - 1);
    return r;
}

// The `off` tokens that a block held, rounded again to a larger scale, by a warp; `row` is the
// lane's 8 codes of the block's first token, `ratio` the old scale by the new one (exact, the new
// scale being a power of two, or too small for any code).
template <int D>
__device__ __forceinline__ void round_again(const Kv8AppendParams& p, int side, uint8_t* row, int off, float ratio) {
    for (int r = (threadIdx.x & 31) / (D / 8); r < off; r += 32 / (D / 8)) {
        uint2* at = reinterpret_cast<uint2*>(row + static_cast<long long>(r) * D);
        if (!codes_ok<D>(p, side, at)) continue;
        uint2 c = *at;
        float f[4];
        unpack4_e4m3(c.x, f);
        c.x = pack4_e4m3(mul_odd(f[0], ratio), mul_odd(f[1], ratio), mul_odd(f[2], ratio), mul_odd(f[3], ratio));
        unpack4_e4m3(c.y, f);
        c.y = pack4_e4m3(mul_odd(f[0], ratio), mul_odd(f[1], ratio), mul_odd(f[2], ratio), mul_odd(f[3], ratio));
        *at = c;
    }
}

// One warp takes the blocks of 16 slots whose first new token is among its `chunk`
// tokens, for one head of K or V, one block after the other: D / 8 lanes hold one token
// (8 values, a 16-byte load), so the warp holds the block's new tokens at once and reads
// each value once.  Nothing is shared between warps: a block belongs to one warp.
// Bound by memory traffic (3 bytes a value): the loads of a block's tokens are all in
// flight together, neighbouring warps take neighbouring heads of the same tokens, and
// eight codes leave a lane in one store.  Measured: 8 prompts of 8192 tokens (Hkv 8, d = 128,
// bf16) 66.8 us, 6.0 TB/s, 89 % of the measured copy rate (74 us with every value looked at for
// an infinity on its own: then the ALUs were as busy as the memory); 64 single tokens 3.2 us, a
// launch and the loads that wait for one another (slot, then values and scale).
template <int D, int E>
__device__ __forceinline__ void append_chunk(const Kv8AppendParams& p, int side, int h, long long c0) {
    constexpr int kLanes = D / 8;          // lanes of one token
    constexpr int kRows = 32 / kLanes;     // tokens the warp loads at a time
    constexpr int kSteps = kKv8Block / kRows;
    const int lane = threadIdx.x & 31;
    if (c0 >= p.T) return;
    const int c1 = static_cast<int>(min(c0 + p.chunk, static_cast<long long>(p.T)));
    const uint16_t* x = static_cast<const uint16_t*>(p.x[side]) + static_cast<long long>(h) * D +
                        (lane % kLanes) * 8;
    int t = static_cast<int>(c0);
    while (t < c1) {
        // the run of consecutive slots from t on, to the end of its block
        const BlockRun run = next_run(p, t, c0);
        const int slot = run.slot, off = run.off, n = run.n;
        if (run.skip) {
            t += n;
            continue;
        }
        uint4 w[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = i * kRows + lane / kLanes;
            w[i] = r < n && values_ok<D>(p, side, x + (t + r) * p.stride) ? *reinterpret_cast<const uint4*>(x + (t + r) * p.stride)
                                                                        : make_uint4(0, 0, 0, 0);
        }
        // amax of the finite values, as integers (the order of magnitudes): of pairs of 16-bit
        // ones, or one by one where there is an infinity or NaN to leave out
        uint32_t pairs = 0;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) pairs = __vmaxu2(pairs, u[j] & 0x7fff7fffu);
        }
        const uint32_t largest = __reduce_max_sync(0xffffffffu, max(pairs & 0xffffu, pairs >> 16));
        const bool finite = largest < (E == kElemBf16 ? 0x7f80u : 0x7c00u);
        uint32_t top = __float_as_uint(unpack2<E>(largest).x);
        if (!finite) {
            top = 0;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = unpack2<E>(u[j]);
                    const uint32_t a = __float_as_uint(f.x) & 0x7fffffffu, b = __float_as_uint(f.y) & 0x7fffffffu;
                    top = max(top, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
                }
            }
            top = __reduce_max_sync(0xffffffffu, top);
        }
        const int need = scale_exponent(top);
        const int page = slot >> p.page_log2;
        const int in_page = slot & ((1 << p.page_log2) - 1);
        const long long row0 = (static_cast<long long>(page) * p.Hkv + h) << p.page_log2;
        float* scale_at = p.scales[side] + (row0 + in_page) / kKv8Block;
        uint8_t* row = p.codes[side] + (row0 + in_page) * D + (lane % kLanes) * 8;
        float scale = pow2f(need);
        const bool known = scale_ok(p, side, scale_at);
        if (off > 0 && known) {
            const float old = *scale_at;
            scale = fmaxf(old, scale);
            if (scale > old) round_again<D>(p, side, row - static_cast<long long>(off) * D, off, old / scale);
        }
        if ((__float_as_uint(scale) & 0x7fffffu) != 0) {
            append_by_division<D, E>(p, side, x + t * p.stride, row, n, scale);
        } else {
            const float inv = 1.f / scale;   // exact for a power of two
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int r = i * kRows + lane / kLanes;
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                float f[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 g = unpack2<E>(u[j]);
                    f[2 * j] = g.x * inv;
                    f[2 * j + 1] = g.y * inv;
                    if (!finite) {   // inf * 0 is NaN: infinities become NaN codes
                        f[2 * j] += g.x * 0.f;
                        f[2 * j + 1] += g.y * 0.f;
                    }
                }
                if (r < n && codes_ok<D>(p, side, row + static_cast<long long>(r) * D))
                    *reinterpret_cast<uint2*>(row + static_cast<long long>(r) * D) =
                        make_uint2(pack4_e4m3(f[0], f[1], f[2], f[3]), pack4_e4m3(f[4], f[5], f[6], f[7]));
            }
        }
        __syncwarp();   // every lane has read the old scale
        if (lane == 0 && known) *scale_at = scale;
        t += n;
    }
}

template <int D, int E>
__global__ void __launch_bounds__(256) kv8_append_kernel(const Kv8AppendParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    const long long item = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    append_chunk<D, E>(p, static_cast<int>(item / p.Hkv % 2), static_cast<int>(item % p.Hkv),
                       item / p.Hkv / 2 * p.chunk);
}

// The lane's part of a key, normed and rotated.  (The norm's factor could be put off to the product with the
// block's 1 / scale, rotation keeping factors, which made the prompts below 0.5 % faster; but that product
// is infinite for a row of zeros with a small eps, and x w may be where x r w is not.)
template <int D, int E, bool IL>
__device__ __forceinline__ void key_row(const NormRopeParams& q, const RowLane<D, IL>& at, const float* cosines,
                                        const float* sines, uint4 a, uint4 b, const float (&w)[16], float (&v)[16]) {
    widen<E>(a, b, v);
    if (q.norm) scale_row(v, inverse_norm<D>(v, q.eps), w);
    Rotation rot;
    rotation_from<D, IL>(cosines, sines, at, rot);
    rotate<D, IL, false>(at, rot, v);
}

// append_chunk for keys that are normed and rotated on their way, from which 32-bit numbers the
// block's scale and codes come, so that a key is rounded once.  With PAIR two warps have a block, the
// first and the last 8 of its new tokens, and both walk the chunk's runs (one warp's 64 numbers a lane
// did not fit its registers beside the rest: 322 us in place of 301 for 8 prompts of 8192 tokens, Hq 32,
// Hkv 8, d = 128); `tops` is theirs, for two runs in turn.  Without, runs have 512 / D tokens at most,
// what a warp loads at a time.
// `cosines` and `sines`: rows of D / 2 for the tokens from c0 on; w: the lane's weights.
//
// Returns the first token that is not done: c1, or, without RARE, where a run needs RARE: there are
// infinities or NaN among its keys, or the block's scale is not a power of two (another writer began
// it).
template <int D, int E, bool IL, bool PAIR, bool RARE>
__device__ __forceinline__ int append_rotated(const Kv8AppendParams& p, const NormRopeParams& q, const RowLane<D, IL>& at,
                                              const float (&w)[16], int h, long long c0, int t, int c1,
                                              const float* cosines, const float* sines, uint2 (*tops)[2], int& turn) {
    constexpr int kLanes = D / 16;               // lanes of one token
    constexpr int kRows = 32 / kLanes;           // tokens the warp loads at a time
    constexpr int kMine = kKv8Block / 2, kSteps = PAIR ? kMine / kRows : 1;
    const int lane = threadIdx.x & 31, pair = threadIdx.x / 64, second = PAIR ? threadIdx.x / 32 & 1 : 0;
    const int mine = second * kMine + lane / kLanes;   // the lane's first token in a run
    // The larger of both warps' numbers, and the first one's first lane's `old`: where a block comes in
    // several runs, another warp (of the pair or of any CTA) may write its scale while this one reads it,
    // and all lanes of a pair must go the same way (the buffers take turns: a warp that writes one again
    // has met the other since that one read it).  A single warp's lanes vote, below; handing its `old` round
    // here made the pairs' code slower as it was then laid out (310 us in place of 298 for the prompts below).
    auto both = [&](uint32_t top, float& old) {
        top = __reduce_max_sync(0xffffffffu, top);
        if (!PAIR) return top;
        uint2* x = tops[turn & 1];
        ++turn;
        if (lane == 0) x[second] = make_uint2(top, __float_as_uint(old));
        named_bar_sync(1 + pair, 64);
        old = __uint_as_float(x[0].y);
        return max(x[0].x, x[1].x);
    };
    while (t < c1) {
        const BlockRun run = next_run(p, t, c0);
        if (run.skip) {
            t += run.n;
            continue;
        }
        const int off = run.off, n = run.n;
        const uint16_t* x = static_cast<const uint16_t*>(q.x[1]) + (t + mine) * q.x_stride[1] + static_cast<long long>(h) * D;
        auto ok = [&](const uint16_t* from) {   // (q.heads[1] is 0 where the queries have a kernel of their own)
            return fa_row_ok(q.x[1], from, 16, p.T, 2LL * D * p.Hkv, 2 * q.x_stride[1], p.status);
        };
        uint4 in[kSteps][2];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            in[i][0] = in[i][1] = make_uint4(0, 0, 0, 0);
            if (i * kRows + mine < n && ok(x + 8 * at.unit[0]) && ok(x + 8 * at.unit[1])) {
                in[i][0] = *reinterpret_cast<const uint4*>(x + 8 * at.unit[0]);
                in[i][1] = *reinterpret_cast<const uint4*>(x + 8 * at.unit[1]);
            }
            x += kRows * q.x_stride[1];
        }
        const int page = run.slot >> p.page_log2;
        const int in_page = run.slot & ((1 << p.page_log2) - 1);
        const long long row0 = (static_cast<long long>(page) * p.Hkv + h) << p.page_log2;
        float* scale_at = p.scales[0] + (row0 + in_page) / kKv8Block;
        uint8_t* row = p.codes[0] + (row0 + in_page) * D;
        const bool known = scale_ok(p, 0, scale_at);
        float old = off > 0 && known ? *scale_at : 0.f;
        float v[kSteps][16];
        float most = 0.f;   // the largest magnitude (NaN does not count)
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int place = static_cast<int>(t - c0) + min(i * kRows + mine, n - 1);
            key_row<D, E, IL>(q, at, cosines + place * (D / 2), sines + place * (D / 2), in[i][0], in[i][1], w, v[i]);
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 16; j += 2) m = fmax3(m, fabsf(v[i][j]), fabsf(v[i][j + 1]));
            if (i * kRows + mine < n) most = fmaxf(most, m);
        }
        uint32_t top = both(__float_as_uint(most), old);
        if (RARE && top >= 0x7f800000u) {
            top = 0;
            for (int i = 0; i < kSteps; ++i)
                for (int j = 0; j < 16; ++j) {
                    const uint32_t a = __float_as_uint(v[i][j]) & 0x7fffffffu;
                    if (i * kRows + mine < n && a < 0x7f800000u) top = max(top, a);
                }
            top = both(top, old);
        }
        const float scale = fmaxf(pow2f(scale_exponent(top)), old);
        const bool rare = top >= 0x7f800000u || (__float_as_uint(scale) & 0x7fffffu) != 0;
        if (!RARE && (PAIR ? rare : __any_sync(0xffffffffu, rare))) return t;
        if (second == 0) {   // (both warps have read the old scale)
            if (off > 0 && scale > old)
                round_again<D>(p, 0, row - static_cast<long long>(off) * D + lane % (D / 8) * 8, off, old / scale);
            if (lane == 0 && known) *scale_at = scale;
        }
        const float unscale = 1.f / scale;   // exact for a power of two
        uint8_t* to = row + mine * D;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                // (inf * 0 is NaN: infinities become NaN codes)
                if (RARE) v[i][j] = div_odd(v[i][j], scale) + v[i][j] * 0.f;
                else v[i][j] *= unscale;
            }
            if (i * kRows + mine < n) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (codes_ok<D>(p, 0, to + i * kRows * D + 8 * at.unit[j]))
                        *reinterpret_cast<uint2*>(to + i * kRows * D + 8 * at.unit[j]) =
                            make_uint2(pack4_e4m3(v[i][8 * j], v[i][8 * j + 1], v[i][8 * j + 2], v[i][8 * j + 3]),
                                       pack4_e4m3(v[i][8 * j + 4], v[i][8 * j + 5], v[i][8 * j + 6], v[i][8 * j + 7]));
            }
        }
        t += n;
    }
    return c1;
}

template <int D, int E, bool IL, bool PAIR>
__device__ __noinline__ int append_rotated_rare(const Kv8AppendParams& p, const NormRopeParams& q, int h, long long c0,
                                                int t, int c1, const float* cosines, const float* sines,
                                                uint2 (*tops)[2], int turn) {
    const RowLane<D, IL> at(threadIdx.x % (D / 16), q.rope.rot);
    float w[16];
    if (q.norm) load_weights<D, E, IL>(q.w[1], q.wide, at, w);
    append_rotated<D, E, IL, PAIR, true>(p, q, at, w, h, c0, t, c1, cosines, sines, tops, turn);
    return turn;
}

// Items (a head and one of the CTA's chunks of tokens) by pairs of warps, or by single ones.
template <int D, int E, bool IL, bool PAIR>
__device__ __forceinline__ void append_keys(const Kv8AppendParams& p, const NormRopeParams& q, long long c0, int tokens,
                                            const float (*cosines)[D / 2], const float (*sines)[D / 2],
                                            uint2 (*tops)[2][2]) {
    constexpr int kTeams = kNormThreads / (PAIR ? 64 : 32);
    const int team = threadIdx.x / (PAIR ? 64 : 32);
    const RowLane<D, IL> at(threadIdx.x % (D / 16), q.rope.rot);
    float w[16];
    if (q.norm) load_weights<D, E, IL>(q.w[1], q.wide, at, w);
    int turn = 0;
    for (int i = team; i < p.Hkv * p.chunks; i += kTeams) {
        const int first = i / p.Hkv * p.chunk, h = i % p.Hkv;
        const int t0 = static_cast<int>(c0) + first, t1 = static_cast<int>(c0) + min(first + p.chunk, tokens);
        uint2 (*mine)[2] = tops[PAIR ? team : 0];
        const int t = append_rotated<D, E, IL, PAIR, false>(p, q, at, w, h, t0, t0, t1, cosines[first], sines[first], mine, turn);
        if (t < t1) turn = append_rotated_rare<D, E, IL, PAIR>(p, q, h, t0, t, t1, cosines[first], sines[first], mine, turn);
    }
}

// What a CTA of kv8_append_norm_rope_kernel does (blockIdx.y), for some tokens: their blocks of keys
// (two warps for a head and `chunk` tokens) or of values (a warp), or their queries, a group of D / 16 lanes for a
// token and some of the heads.  For keys and queries the CTA first has the tokens' cosines and sines
// in shared memory.  (A block that begins among them may go on behind them: up to 15 tokens more,
// whose angles are there too.)
//
// In long batches the queries have norm_rope_kernel, which keeps more warps on an SM (queries here, all
// kinds of CTAs side by side: 315 us and more for the prompts below).  Measured (one GB300, bf16, Hq 32,
// Hkv 8, d = 128): 8 prompts of 8192 tokens 298 us, 73 % of the measured copy rate: the queries 168 us, 94 %,
// then keys and values 132 us, where the keys wait for their loads and for the other warp of a block (issue
// slots 46 % used, DRAM 36 %; four warps to a block, with 24 warps an SM: 300); 64 single tokens 3.8 us, a
// launch and the slots, positions and rows that wait for one another.  At d = 128 this kernel's 128 registers
// do not hold everything: 100 bytes a thread are spilled (44 with neighbouring pairs).
constexpr int kAppendValues = 0, kAppendKeys = 1, kAppendQueries = 2;

template <int D, int E, bool IL>
__global__ void __launch_bounds__(kNormThreads, 2) kv8_append_norm_rope_kernel(
    const __grid_constant__ Kv8AppendParams p, const __grid_constant__ NormRopeParams q) {
    constexpr int kTokens = 3 * kKv8Block - 1, kWarps = kNormThreads / 32;
    __shared__ alignas(16) float cosines[kTokens][D / 2], sines[kTokens][D / 2];
    __shared__ uint2 tops[kWarps / 2][2][2];
    grid_launch_dependents();
    grid_dependency_wait();
    const int role = blockIdx.y, warp = threadIdx.x / 32;
    const long long c0 = static_cast<long long>(blockIdx.x) * p.chunk * p.chunks;   // the CTA's first token
    const int tokens = static_cast<int>(min(static_cast<long long>(p.chunk) * p.chunks, p.T - c0));
    if (role == kAppendValues) {
        for (int i = warp; i < p.Hkv * p.chunks; i += kWarps)
            append_chunk<D, E>(p, 1, i % p.Hkv, c0 + i / p.Hkv * p.chunk);
        return;
    }
    const int half = q.rope.rot / 2, lane = threadIdx.x % 32;
    if (half > 0) {
        int all = tokens, last = 0;
        if (role == kAppendKeys) {
            last = fa_index_ok(c0 + tokens - 1, p.T, p.status) ? p.slots[c0 + tokens - 1] : -1;
            all = min(tokens + kKv8Block - 1 - (last & (kKv8Block - 1)), static_cast<int>(min(p.T - c0, 64LL)));
        }
        for (int row = warp; row < all && fa_index_ok(row, kTokens, p.status); row += kWarps) {
            if (row >= tokens && p.slots[c0 + row] != last + row - tokens + 1) continue;
#pragma unroll
            for (int f = lane; f < D / 2; f += 32)
                if (f < half) {
                    const int place = place_of<D, IL>(f);
                    cos_sin(q.rope, f, c0 + row, cosines[row][place], sines[row][place]);
                }
        }
    }
    __syncthreads();
    if (role == kAppendKeys) {
        // (a decoding step's single tokens need no pairs of warps)
        if (tokens == 1 && next_run(p, static_cast<int>(c0), c0).n <= 512 / D)
            append_keys<D, E, IL, false>(p, q, c0, tokens, cosines, sines, tops);
        else
            append_keys<D, E, IL, true>(p, q, c0, tokens, cosines, sines, tops);
        return;
    }
    constexpr int L = D / 16, kGroups = kNormThreads / L;
    const int group = threadIdx.x / L, per = kGroups / (p.chunk * p.chunks);   // groups for a token
    const int row = group % (p.chunk * p.chunks), first = group / (p.chunk * p.chunks);
    const bool real = row < tokens && first < per;
    const long long token = c0 + (real ? row : 0);
    const RowLane<D, IL> at(threadIdx.x % L, q.rope.rot);
    const uint16_t* x = static_cast<const uint16_t*>(q.x[0]) + token * q.x_stride[0];
    uint16_t* y = static_cast<uint16_t*>(q.y[0]) + token * q.y_stride[0];
    Rotation rot;
    float w[16];
    rotation_from<D, IL>(cosines[token - c0], sines[token - c0], at, rot);
    if (q.norm) load_weights<D, E, IL>(q.w[0], q.wide, at, w);
#pragma unroll 1
    for (int h0 = 0; h0 < q.heads[0]; h0 += 2 * per) {
        uint4 in[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = h0 + u * per + first;
                const uint16_t* from = x + h * D + 8 * at.unit[j];
                in[u][j] = real && h < q.heads[0] && channels_ok<D>(q, 0, q.x[0], from, q.x_stride[0])
                               ? *reinterpret_cast<const uint4*>(from)
                               : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int h = h0 + u * per + first;
            float v[16];
            widen<E>(in[u][0], in[u][1], v);
            if (q.norm) scale_row(v, inverse_norm<D>(v, q.eps), w);
            rotate<D, IL, false>(at, rot, v);
            if (real && h < q.heads[0]) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (channels_ok<D>(q, 0, q.y[0], y + h * D + 8 * at.unit[j], q.y_stride[0]))
                        *reinterpret_cast<uint4*>(y + h * D + 8 * at.unit[j]) = narrow<E>(v + 8 * j);
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv8_plan(const Kv8PlanParams& p, int sms, cudaStream_t stream) {
    // a token per thread up to one CTA per SM; small plans take a small CTA, whose sums
    // have fewer warps to add up
    const int threads = p.B <= 256 && p.T <= 256 ? 256 : 1024;
    const int grid = std::min(std::max((p.T + threads - 1) / threads, 1), sms);
    const int smem = p.B * static_cast<int>(sizeof(PlanRequest));
    if (smem > 48 * 1024 - 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            kv8_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    return kv8::launch_dependent(kv8_plan_kernel, grid, threads, smem, stream, p);
}

cudaError_t launch_kv8_append(const Kv8AppendParams& p, int d, cudaStream_t stream) {
    constexpr int kThreads = 256;
    const long long chunks = (static_cast<long long>(p.T) + p.chunk - 1) / p.chunk;
    const long long warps = chunks * p.Hkv * 2;
    const long long grid = (warps * 32 + kThreads - 1) / kThreads;
    if (grid > INT_MAX) return cudaErrorInvalidValue;
    auto kern = d == 128 ? (p.elem == kElemBf16Code ? kv8_append_kernel<128, kElemBf16> : kv8_append_kernel<128, kElemF16>)
                         : (p.elem == kElemBf16Code ? kv8_append_kernel<64, kElemBf16> : kv8_append_kernel<64, kElemF16>);
    return kv8::launch_dependent(kern, static_cast<int>(grid), kThreads, 0, stream, p);
}

cudaError_t launch_kv8_append_norm_rope(const Kv8AppendParams& a, const NormRopeParams& n, int d, cudaStream_t stream) {
    const long long tokens = static_cast<long long>(a.chunk) * a.chunks;
    const dim3 grid(static_cast<unsigned>((a.T + tokens - 1) / tokens), n.ctas[0] > 0 ? 2 : 3);
    const bool f16 = a.elem == kElemF16Code, il = n.rope.interleaved != 0;
    auto kern = d == 128 ? (f16 ? (il ? kv8_append_norm_rope_kernel<128, kElemF16, true> : kv8_append_norm_rope_kernel<128, kElemF16, false>)
                                : (il ? kv8_append_norm_rope_kernel<128, kElemBf16, true> : kv8_append_norm_rope_kernel<128, kElemBf16, false>))
                         : (f16 ? (il ? kv8_append_norm_rope_kernel<64, kElemF16, true> : kv8_append_norm_rope_kernel<64, kElemF16, false>)
                                : (il ? kv8_append_norm_rope_kernel<64, kElemBf16, true> : kv8_append_norm_rope_kernel<64, kElemBf16, false>));
    cudaError_t e = kv8::launch_dependent(kern, grid, kNormThreads, 0, stream, a, n);
    if (e == cudaSuccess && n.ctas[0] > 0) e = launch_norm_rope(n, d, stream);
    return e;
}

}  // namespace fa
