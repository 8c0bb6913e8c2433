// fa_kv8_cache.cu -- the paged 8-bit cache's bookkeeping (block tables, slots, free
// pages) and its writer.  The formats and rules are those of fa_kv8_plan and
// fa_kv8_append in include/fa.h.
#include "fa_kv8_work.cuh"

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

// The codes of n new tokens of a block whose scale is not a power of two, by a warp: a block that
// another writer began (this one's scales are powers of two).  `x` and `row` are the lane's 8
// values of the first token.
template <int D, int E>
__device__ __noinline__ void append_by_division(const uint16_t* x, long long stride, uint8_t* row, int n, float scale) {
    for (int r = (threadIdx.x & 31) / (D / 8); r < n; r += 32 / (D / 8)) {
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
__global__ void __launch_bounds__(256) kv8_append_kernel(const Kv8AppendParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    constexpr int kLanes = D / 8;          // lanes of one token
    constexpr int kRows = 32 / kLanes;     // tokens the warp loads at a time
    constexpr int kSteps = kKv8Block / kRows;
    const int lane = threadIdx.x & 31;
    const long long item = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int h = static_cast<int>(item % p.Hkv);
    const int side = static_cast<int>(item / p.Hkv % 2);
    const long long c0 = item / p.Hkv / 2 * p.chunk;
    if (c0 >= p.T) return;
    const int c1 = static_cast<int>(min(c0 + p.chunk, static_cast<long long>(p.T)));
    const uint16_t* x = static_cast<const uint16_t*>(p.x[side]) + static_cast<long long>(h) * D +
                        (lane % kLanes) * 8;
    int t = static_cast<int>(c0);
    while (t < c1) {
        // the run of consecutive slots from t on, to the end of its block
        const int slot = p.slots[t];
        const int off = slot & (kKv8Block - 1);
        const bool real = slot >= 0 && slot < p.num_slots;
        const int mine = lane < kKv8Block && t + lane < p.T ? p.slots[t + lane] : -1;
        const uint32_t follows = __ballot_sync(
            0xffffffffu, real && off + lane < kKv8Block && mine == slot + lane);
        const int n = real ? __ffs(~follows) - 1 : 1;   // lane 16 never follows
        if (!real || (off > 0 && t == c0 && t > 0 && p.slots[t - 1] == slot - 1)) {
            t += n;    // no place in the cache, or a block that an earlier warp began
            continue;
        }
        uint4 w[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = i * kRows + lane / kLanes;
            w[i] = r < n ? *reinterpret_cast<const uint4*>(x + (t + r) * p.stride) : make_uint4(0, 0, 0, 0);
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
        if (off > 0) {
            const float old = *scale_at;
            scale = fmaxf(old, scale);
            if (scale > old) {
                // the tokens that the block held, rounded again to the larger scale
                const float ratio = old / scale;   // (exact, the new scale being a power of two, or too small for any code)
                for (int r = lane / kLanes; r < off; r += kRows) {
                    uint2* at = reinterpret_cast<uint2*>(row + static_cast<long long>(r - off) * D);
                    uint2 c = *at;
                    float f[4];
                    unpack4_e4m3(c.x, f);
                    c.x = pack4_e4m3(mul_odd(f[0], ratio), mul_odd(f[1], ratio), mul_odd(f[2], ratio), mul_odd(f[3], ratio));
                    unpack4_e4m3(c.y, f);
                    c.y = pack4_e4m3(mul_odd(f[0], ratio), mul_odd(f[1], ratio), mul_odd(f[2], ratio), mul_odd(f[3], ratio));
                    *at = c;
                }
            }
        }
        if ((__float_as_uint(scale) & 0x7fffffu) != 0) {
            append_by_division<D, E>(x + t * p.stride, p.stride, row, n, scale);
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
                if (r < n)
                    *reinterpret_cast<uint2*>(row + static_cast<long long>(r) * D) =
                        make_uint2(pack4_e4m3(f[0], f[1], f[2], f[3]), pack4_e4m3(f[4], f[5], f[6], f[7]));
            }
        }
        __syncwarp();   // every lane has read the old scale
        if (lane == 0) *scale_at = scale;
        t += n;
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

}  // namespace fa
