// fa_norm_rope.cu -- norms of queries and keys for each head with the rotation by position in
// the same pass, and its gradient.  The formulas are those of fa_norm_rope and fa_norm_rope_bwd
// in include/fa.h, the layout in registers that of fa_norm_rope.cuh.
//
// Both are bound by memory: the forward reads and writes each value once (4 bytes), the backward
// reads two and writes one (6 bytes).  What it takes to come near: enough rows on their way (an SM
// needs some 50 KB), few instructions a row (some 180 for the 4 or 8 rows of a warp, half of them the
// arithmetic), and angles worked out once for many heads.
//
// Measured (one GB300, bf16, in a graph, the shares of the measured copy rate): forward 32768 tokens, Hq 32,
// Hkv 8, d = 128, three axes, slices of a projection 107.6 us, 92 % (a plain copy of such rows runs at 97 %);
// 16384 tokens of 16 and 16 heads 47.8 us, 83 %, where the last CTAs leave SMs idle; one token 2.6 us, a
// launch and the loads that wait for one another.  A warp on four heads of one token, its angles
// shared, waited longer at every token's start (121 to 131 us); passes of rows through rings in shared
// memory, by bulk or by asynchronous copies, took 118 to 126 us, bound by their instructions.
#include "fa_kv8_work.cuh"
#include "fa_norm_rope.cuh"

#include <algorithm>

namespace fa {
namespace {

// A unit of work is one token's run of heads of one side (q or k), for a group of D / 16 lanes; the
// groups of a warp have neighbouring tokens.
struct Unit {
    long long token;
    int head;
    __device__ __forceinline__ Unit(const NormRopeParams& p, int side, long long unit) {
        const long long part = kv8::divide(unit, static_cast<long long>(p.T));
        token = unit - part * p.T;
        head = static_cast<int>(part) * p.run[side];
    }
};

// This lane's two 16-byte units of the rows of a unit of work, kStep bytes from row to row.
template <int D, bool IL>
struct LaneRows {
    static constexpr int kStep = D * 2;
    char* unit[2];
    __device__ __forceinline__ LaneRows(const void* x, long long stride, const Unit& u, const RowLane<D, IL>& at) {
        char* first = static_cast<char*>(const_cast<void*>(x)) + 2 * (u.token * stride + u.head * D);
        unit[0] = first + 16 * at.unit[0];
        unit[1] = first + 16 * at.unit[1];
    }
    __device__ __forceinline__ bool ok(const NormRopeParams& p, int side, const void* x, long long stride, int row) const {
        return channels_ok<D>(p, side, x, unit[0] + row * kStep, stride) && channels_ok<D>(p, side, x, unit[1] + row * kStep, stride);
    }
    __device__ __forceinline__ void load(int row, uint4 (&v)[2]) const {
        v[0] = *reinterpret_cast<const uint4*>(unit[0] + row * kStep);
        v[1] = *reinterpret_cast<const uint4*>(unit[1] + row * kStep);
    }
    template <int E>
    __device__ __forceinline__ void store(int row, const float (&v)[16]) const {
        *reinterpret_cast<uint4*>(unit[0] + row * kStep) = narrow<E>(v);
        *reinterpret_cast<uint4*>(unit[1] + row * kStep) = narrow<E>(v + 8);
    }
    __device__ __forceinline__ void advance(int rows) {
        unit[0] += rows * kStep;
        unit[1] += rows * kStep;
    }
};

template <int D, int E, bool IL>
__global__ void __launch_bounds__(kNormThreads, 3) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int kAhead = 2, kLanes = RowLane<D, IL>::kLanes, kGroups = kNormThreads / kLanes;
    grid_launch_dependents();
    grid_dependency_wait();
    const int side = static_cast<int>(blockIdx.x) >= p.ctas[0] ? 1 : 0, run = p.run[side];
    const long long units = static_cast<long long>(p.T) * (p.heads[side] / run);
    const long long unit = static_cast<long long>(blockIdx.x - (side ? p.ctas[0] : 0)) * kGroups + threadIdx.x / kLanes;
    const bool real = unit < units;   // (the others take part in the sums)
    const Unit un(p, side, real ? unit : units - 1);
    const RowLane<D, IL> at(threadIdx.x % kLanes, p.rope.rot);
    LaneRows<D, IL> from(p.x[side], p.x_stride[side], un, at), to(p.y[side], p.y_stride[side], un, at);
    Rotation rot;
    float w[16];
    if (p.norm) load_weights<D, E, IL>(p.w[side], p.wide, at, w);
    // a batch of rows whose loads are on their way together; whole: all of them are there
    auto batch = [&](bool fresh, auto whole, int left) {
        uint4 in[kAhead][2];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if ((whole || u < left) && from.ok(p, side, p.x[side], p.x_stride[side], u)) from.load(u, in[u]);
        if (fresh) lane_rotation<D, IL>(p.rope, at, un.token, rot);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (!whole && u >= left) break;
            float v[16];
            widen<E>(in[u][0], in[u][1], v);
            if (p.norm) scale_row(v, inverse_norm<D>(v, p.eps), w);
            rotate<D, IL, false>(at, rot, v);
            if (real && to.ok(p, side, p.y[side], p.y_stride[side], u)) to.template store<E>(u, v);
        }
        from.advance(kAhead);
        to.advance(kAhead);
    };
    int left = run;
#pragma unroll 1
    for (; left >= kAhead; left -= kAhead) batch(left == run, std::true_type{}, left);
    if (left > 0) batch(left == run, std::false_type{}, left);
}

// A row's dn (in g) to dx, and its part of dw:
//   xh = x r,  g = dn w,  dx = r (g - xh mean(g xh)),  dw += dn xh.
template <int D>
__device__ __forceinline__ void norm_back(float (&g)[16], float (&x)[16], float r, const float (&w)[16], float (&dw)[16]) {
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] *= r;
        dw[i] = fmaf(g[i], x[i], dw[i]);
        g[i] *= w[i];
        q[i & 1] = fmaf(g[i], x[i], q[i & 1]);
    }
    const float mean = row_sum<D>(q[0] + q[1]) * (-1.f / D);
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = r * fmaf(x[i], mean, g[i]);
}

// A CTA keeps to one side and goes through many units; it adds its rows' parts of dw up in
// registers, then over its groups of lanes in shared memory, and norm_rope_weights_kernel adds the
// CTAs' sums up in their order, so the result has one order of additions for given sizes.
//
// The rows come by asynchronous copies, kBwdAhead - 1 rows ahead and over the ends of units, into places
// in shared memory that each thread reads back itself: no thread waits for another, and what is on its
// way takes none of the registers, which dw, the weights and the angles fill.  With the rows loaded into
// registers, two at a time, 16384 tokens of 16 and 16 heads (d = 128) took 79.6 us in place of 69.8
// (5.8 TB/s, 85 % of the measured copy rate); more rows ahead, or rows in 2 KB pieces by bulk copies
// (72.5), were no faster.
constexpr int kBwdAhead = 3;

template <int D, int E, bool IL>
__global__ void __launch_bounds__(kNormThreads, 2) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int kAhead = kBwdAhead, kLanes = RowLane<D, IL>::kLanes, kGroups = kNormThreads / kLanes;
    extern __shared__ uint4 places[];   // [kAhead][4][threads]; at the end [kGroups][D] floats
    grid_launch_dependents();
    grid_dependency_wait();
    const int side = static_cast<int>(blockIdx.x) >= p.ctas[0] ? 1 : 0, run = p.run[side];
    const long long units = static_cast<long long>(p.T) * (p.heads[side] / run);
    const RowLane<D, IL> at(threadIdx.x % kLanes, p.rope.rot);
    float w[16], dw[16];
    if (p.norm) load_weights<D, E, IL>(p.w[side], p.wide, at, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[i] = 0.f;
    const long long start = static_cast<long long>(blockIdx.x - (side ? p.ctas[0] : 0)) * kGroups;
    const long long step = static_cast<long long>(p.ctas[side]) * kGroups;
    long long next = start;   // the unit that copies are in, its row
    int row = 0, put = 0;
    const uint16_t *cx = nullptr, *cdy = nullptr;
    auto seek = [&] {
        const long long mine = next + threadIdx.x / kLanes;
        cx = cdy = nullptr;
        if (mine >= units) return;
        const Unit un(p, side, mine);
        cdy = static_cast<const uint16_t*>(p.dy[side]) + un.token * p.dy_stride[side] + un.head * D;
        cx = static_cast<const uint16_t*>(p.x[side]) + un.token * p.x_stride[side] + un.head * D;
    };
    auto copy = [&] {
        if (next < units) {
            if (cdy) {
                uint4* to = places + put * 4 * kNormThreads + threadIdx.x;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (channels_ok<D>(p, side, p.dy[side], cdy + 8 * at.unit[j], p.dy_stride[side]))
                        cp_async16(smem_addr(to + j * kNormThreads), cdy + 8 * at.unit[j]);
                    if (p.norm && channels_ok<D>(p, side, p.x[side], cx + 8 * at.unit[j], p.x_stride[side]))
                        cp_async16(smem_addr(to + (2 + j) * kNormThreads), cx + 8 * at.unit[j]);
                }
                cdy += D;
                cx += D;
            }
            if (++row == run) {
                row = 0;
                next += step;
                seek();
            }
        }
        put = put + 1 == kAhead ? 0 : put + 1;
        cp_async_commit();
    };
    seek();
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) copy();
    int take = 0;
#pragma unroll 1
    for (long long first = start; first < units; first += step) {
        const bool real = first + threadIdx.x / kLanes < units;   // (the others take part in the sums)
        const Unit un(p, side, real ? first + threadIdx.x / kLanes : units - 1);
        uint16_t* y = static_cast<uint16_t*>(p.y[side]) + un.token * p.y_stride[side] + un.head * D;
        Rotation rot;
        lane_rotation<D, IL>(p.rope, at, un.token, rot);
#pragma unroll 1
        for (int h = 0; h < run; ++h) {
            cp_async_wait<kAhead - 2>();
            const uint4* from = places + take * 4 * kNormThreads + threadIdx.x;
            take = take + 1 == kAhead ? 0 : take + 1;
            float g[16], v[16];
            widen<E>(from[0], from[kNormThreads], g);
            if (p.norm) widen<E>(from[2 * kNormThreads], from[3 * kNormThreads], v);
            copy();
            if (!real) {   // (no row adds nothing to dw)
#pragma unroll
                for (int i = 0; i < 16; ++i) g[i] = v[i] = 0.f;
            }
            rotate<D, IL, true>(at, rot, g);
            if (p.norm) norm_back<D>(g, v, inverse_norm<D>(v, p.eps), w, dw);
            if (real) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (channels_ok<D>(p, side, p.y[side], y + 8 * at.unit[j], p.y_stride[side]))
                        *reinterpret_cast<uint4*>(y + 8 * at.unit[j]) = narrow<E>(g + 8 * j);
            }
            y += D;
        }
    }
    if (!p.partial) return;
    __syncthreads();
    float (*sums)[D] = reinterpret_cast<float (*)[D]>(places);
#pragma unroll
    for (int i = 0; i < 16; ++i) sums[threadIdx.x / kLanes][8 * at.unit[i / 8] + i % 8] = dw[i];
    __syncthreads();
    if (threadIdx.x < D) {
        float v = 0.f;
#pragma unroll 8
        for (int i = 0; i < kGroups; ++i) v += sums[i][threadIdx.x];
        const long long sum = static_cast<long long>(blockIdx.x) * D + threadIdx.x;
        if (fa_index_ok(sum, (static_cast<long long>(p.ctas[0]) + p.ctas[1]) * D, p.status)) p.partial[sum] = v;
    }
}

// The weights' gradients from the CTAs' sums: a CTA takes 32 channels of one side.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_weights_kernel(const __grid_constant__ NormRopeParams p) {
    __shared__ double sums[32][33];
    grid_launch_dependents();
    grid_dependency_wait();
    const int side = blockIdx.x / (D / 32), ch = blockIdx.x % (D / 32) * 32 + threadIdx.x % 32;
    const int row = threadIdx.x / 32;
    if (!p.dw[side]) return;
    double v = 0.0;
#pragma unroll 8
    for (int i = row; i < p.ctas[side]; i += 32) {
        const long long sum = static_cast<long long>(i + (side ? p.ctas[0] : 0)) * D + ch;
        if (fa_index_ok(sum, (static_cast<long long>(p.ctas[0]) + p.ctas[1]) * D, p.status)) v += p.partial[sum];
    }
    sums[row][threadIdx.x % 32] = v;
    __syncthreads();
    if (row == 0) {
        v = 0.0;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += sums[i][threadIdx.x];
        p.dw[side][ch] = static_cast<float>(v);
    }
}

template <int D, int E>
cudaError_t launch(const NormRopeParams& p, cudaStream_t stream) {
    return kv8::launch_dependent(p.rope.interleaved ? norm_rope_kernel<D, E, true> : norm_rope_kernel<D, E, false>,
                                 p.ctas[0] + p.ctas[1], kNormThreads, 0, stream, p);
}

template <int D, int E>
cudaError_t launch_bwd(const NormRopeParams& p, cudaStream_t stream) {
    auto kern = p.rope.interleaved ? norm_rope_bwd_kernel<D, E, true> : norm_rope_bwd_kernel<D, E, false>;
    constexpr int smem = kBwdAhead * 4 * 16 * kNormThreads;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = kv8::launch_dependent(kern, p.ctas[0] + p.ctas[1], kNormThreads, smem, stream, p);
    if (e != cudaSuccess || !p.partial) return e;
    return kv8::launch_dependent(norm_rope_weights_kernel<D>, 2 * (D / 32), 1024, 0, stream, p);
}

// The heads of a unit: the largest divisor of `heads` (128 at most, by when angles cost nothing) that
// leaves `want` units or more, 1 where even single heads do not.
int heads_of_unit(long long T, int heads, long long want) {
    int best = 1;
    for (int r = 2; r <= std::min(heads, 128); ++r)
        if (heads % r == 0 && T * (heads / r) >= want) best = r;
    return best;
}

}  // namespace

// Units of one token and a run of heads.  A unit's start (its angles) costs about as much as four
// heads, so few units are wanted, but enough for every SM: four CTAs' worth for each.  Where that
// leaves runs of more than 8 heads, twice as many even out the last CTAs: 16384 tokens of 16 and 16
// heads took 47.2 us with runs of 8 and 49.5 with 16; 5003 of 12 and 4 (d = 64) 4.3 us with runs of 2 and
// 5.9 with 1.
int norm_rope_plan(NormRopeParams& p, int d, int sms, bool backward) {
    const int groups = kNormThreads / (d / 16);   // of a CTA
    const long long want = static_cast<long long>(sms) * 4 * groups;
    long long ctas[2];
    for (int side = 0; side < 2; ++side) {
        p.run[side] = 1;
        ctas[side] = 0;
        if (p.heads[side] == 0) continue;
        const long long mine = want * p.heads[side] / (p.heads[0] + p.heads[1]);
        p.run[side] = heads_of_unit(p.T, p.heads[side], mine);
        if (p.run[side] > 8) p.run[side] = std::max(heads_of_unit(p.T, p.heads[side], 2 * mine), std::min(p.run[side], 8));
        while (p.heads[side] % p.run[side] != 0) --p.run[side];
        ctas[side] = (static_cast<long long>(p.T) * (p.heads[side] / p.run[side]) + groups - 1) / groups;
    }
    // the backward's CTAs, as many as are resident, go through several units each, so that few sums
    // are left to add up
    const long long most = 2LL * sms;
    if (backward && ctas[0] + ctas[1] > most) {
        ctas[0] = std::max(1LL, std::min(most - 1, most * p.heads[0] / (p.heads[0] + p.heads[1])));
        ctas[1] = most - ctas[0];
    }
    if (ctas[0] + ctas[1] > INT_MAX) return 0;
    p.ctas[0] = static_cast<int>(ctas[0]);
    p.ctas[1] = static_cast<int>(ctas[1]);
    return p.ctas[0] + p.ctas[1];
}

cudaError_t launch_norm_rope(const NormRopeParams& p, int d, cudaStream_t stream) {
    const bool f16 = p.elem == kElemF16Code;
    if (d == 128) return f16 ? launch<128, kElemF16>(p, stream) : launch<128, kElemBf16>(p, stream);
    return f16 ? launch<64, kElemF16>(p, stream) : launch<64, kElemBf16>(p, stream);
}

cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, int d, cudaStream_t stream) {
    const bool f16 = p.elem == kElemF16Code;
    if (d == 128) return f16 ? launch_bwd<128, kElemF16>(p, stream) : launch_bwd<128, kElemBf16>(p, stream);
    return f16 ? launch_bwd<64, kElemF16>(p, stream) : launch_bwd<64, kElemBf16>(p, stream);
}

}  // namespace fa
