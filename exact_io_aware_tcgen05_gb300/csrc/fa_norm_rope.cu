// fa_norm_rope.cu -- norms of queries and keys for each head with the rotation by position in
// the same pass, and its gradient.  The formulas are those of fa_norm_rope and fa_norm_rope_bwd
// in include/fa.h, the layout in registers that of fa_norm_rope.cuh.
//
// Both are bound by memory: the forward reads and writes each value once (4 bytes), the backward
// reads two and writes one (6 bytes).  A unit of work is one token's run of heads of one side (q
// or k) for D / 16 lanes, which work out the token's cosines and sines once and keep two (the
// backward) or four rows on their way.
#include "fa_kv8_work.cuh"
#include "fa_norm_rope.cuh"

#include <algorithm>

namespace fa {
namespace {

template <int D, int E, bool IL>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int side = static_cast<int>(blockIdx.x) >= p.ctas[0] ? 1 : 0;
    norm_rope_rows<D, E, IL>(p, side, blockIdx.x - (side ? p.ctas[0] : 0));
}

// dn = dy turned back; with r the row's inverse norm, xh = x r and g = dn w:
//   dx = r (g - xh mean(g xh)),  dw = sum over tokens and heads of dn xh.
// A CTA keeps to one side and adds its rows' dn xh up in registers, then over its groups in
// shared memory; norm_rope_weights_kernel adds the CTAs' sums up in their order, so the result
// has one order of additions for a given shape and device.
template <int D, int E, bool IL>
__global__ void __launch_bounds__(kNormThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int L = D / 16, kGroups = kNormThreads / L, kAhead = 2;
    __shared__ float sums[kGroups][D];
    grid_launch_dependents();
    grid_dependency_wait();
    const int side = static_cast<int>(blockIdx.x) >= p.ctas[0] ? 1 : 0, run = p.run[side];
    const int cta = blockIdx.x - (side ? p.ctas[0] : 0), in_warp = threadIdx.x / L % (32 / L);
    const RowLane<D, IL> at(threadIdx.x % L, p.rope.rot);
    const long long units = static_cast<long long>(p.T) * (p.heads[side] / run);
    float w[16], dw[16];
    if (p.norm) load_weights<D, E, IL>(p.w[side], p.wide, at, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[i] = 0.f;
    // (every lane of a warp goes through as many units: the sums shuffle)
#pragma unroll 1
    for (long long first = static_cast<long long>(cta) * kGroups + threadIdx.x / 32 * (32 / L); first < units;
         first += static_cast<long long>(p.ctas[side]) * kGroups) {
        const long long mine = first + in_warp;
        const bool real = mine < units;
        const long long unit = real ? mine : units - 1;
        const long long part = unit / p.T, token = unit - part * p.T;
        const uint16_t* x = static_cast<const uint16_t*>(p.x[side]) + token * p.x_stride[side] + part * run * D;
        const uint16_t* dy = static_cast<const uint16_t*>(p.dy[side]) + token * p.dy_stride[side] + part * run * D;
        uint16_t* y = static_cast<uint16_t*>(p.y[side]) + token * p.y_stride[side] + part * run * D;
        float c[8], s[8];
        rotation_of<D, IL>(p.rope, at, token, c, s);
#pragma unroll 1
        for (int h0 = 0; h0 < run; h0 += kAhead) {
            uint4 gin[kAhead][2], in[kAhead][2];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const bool row = real && h0 + u < run;
                    const int o = (h0 + u) * D + 8 * at.unit[j];
                    gin[u][j] = row ? *reinterpret_cast<const uint4*>(dy + o) : make_uint4(0, 0, 0, 0);
                    in[u][j] = row && p.norm ? *reinterpret_cast<const uint4*>(x + o) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                float g[16];
                widen<E>(gin[u][0], gin[u][1], g);
                rotate<D, IL, true>(at, c, s, g);
                if (p.norm) {
                    float xh[16];
                    widen<E>(in[u][0], in[u][1], xh);
                    const float r = inverse_norm<D>(xh, p.eps);
                    float q[2] = {0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        xh[i] *= r;
                        dw[i] = fmaf(g[i], xh[i], dw[i]);
                        g[i] *= w[i];
                        q[i & 1] = fmaf(g[i], xh[i], q[i & 1]);
                    }
                    const float mean = row_sum<D>(q[0] + q[1]) * (1.f / D);
#pragma unroll
                    for (int i = 0; i < 16; ++i) g[i] = r * fmaf(-xh[i], mean, g[i]);
                }
                uint4 out[2];
                narrow<E>(g, out[0], out[1]);
                if (real && h0 + u < run && fa_index_ok(token, p.T, p.status)) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        *reinterpret_cast<uint4*>(y + (h0 + u) * D + 8 * at.unit[j]) = out[j];
                }
            }
        }
    }
    if (!p.partial) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) sums[threadIdx.x / L][8 * at.unit[i / 8] + i % 8] = dw[i];
    __syncthreads();
    if (threadIdx.x < D) {
        float v = 0.f;
#pragma unroll 8
        for (int i = 0; i < kGroups; ++i) v += sums[i][threadIdx.x];
        p.partial[static_cast<long long>(blockIdx.x) * D + threadIdx.x] = v;
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
    for (int i = row; i < p.ctas[side]; i += 32)
        v += p.partial[static_cast<long long>(i + (side ? p.ctas[0] : 0)) * D + ch];
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
cudaError_t launch(NormRopeParams& p, cudaStream_t stream) {
    const bool il = p.rope.interleaved != 0;
    return kv8::launch_dependent(il ? norm_rope_kernel<D, E, true> : norm_rope_kernel<D, E, false>,
                                 p.ctas[0] + p.ctas[1], kNormThreads, 0, stream, p);
}

template <int D, int E>
cudaError_t launch_bwd(NormRopeParams& p, cudaStream_t stream) {
    const bool il = p.rope.interleaved != 0;
    const cudaError_t e = kv8::launch_dependent(il ? norm_rope_bwd_kernel<D, E, true> : norm_rope_bwd_kernel<D, E, false>,
                                                p.ctas[0] + p.ctas[1], kNormThreads, 0, stream, p);
    if (e != cudaSuccess || !p.partial) return e;
    return kv8::launch_dependent(norm_rope_weights_kernel<D>, 2 * (D / 32), 1024, 0, stream, p);
}

// The heads of a unit: the largest divisor of `heads` that leaves `want` units or more (1 where
// even single heads do not).
int heads_of_unit(long long T, int heads, long long want) {
    int best = 1;
    for (int r = 2; r <= heads; ++r)
        if (heads % r == 0 && T * (heads / r) >= want) best = r;
    return best;
}

}  // namespace

// Units of one token and a run of heads; enough of them for every SM, and runs no longer than
// that allows, so that a token's angles serve many heads.
int norm_rope_plan(NormRopeParams& p, int d, int sms, bool backward) {
    const int groups = kNormThreads / (d / 16);   // of a CTA
    const long long want = static_cast<long long>(sms) * 8 * groups;
    long long ctas[2], all = 0;
    for (int side = 0; side < 2; ++side) {
        p.run[side] = heads_of_unit(p.T, p.heads[side], want * p.heads[side] / (p.heads[0] + p.heads[1]));
        ctas[side] = (static_cast<long long>(p.T) * (p.heads[side] / p.run[side]) + groups - 1) / groups;
        all += ctas[side];
    }
    // the backward's CTAs go through several units each, so that few sums are left to add up
    const long long most = 4LL * sms;
    if (backward && all > most) {
        ctas[0] = std::max(1LL, std::min(most - 1, most * p.heads[0] / (p.heads[0] + p.heads[1])));
        ctas[1] = most - ctas[0];
    }
    if (ctas[0] + ctas[1] > INT_MAX) return 0;
    p.ctas[0] = static_cast<int>(ctas[0]);
    p.ctas[1] = static_cast<int>(ctas[1]);
    return p.ctas[0] + p.ctas[1];
}

cudaError_t launch_norm_rope(NormRopeParams& p, int d, cudaStream_t stream) {
    const bool f16 = p.elem == kElemF16Code;
    if (d == 128) return f16 ? launch<128, kElemF16>(p, stream) : launch<128, kElemBf16>(p, stream);
    return f16 ? launch<64, kElemF16>(p, stream) : launch<64, kElemBf16>(p, stream);
}

cudaError_t launch_norm_rope_bwd(NormRopeParams& p, int d, cudaStream_t stream) {
    const bool f16 = p.elem == kElemF16Code;
    if (d == 128) return f16 ? launch_bwd<128, kElemF16>(p, stream) : launch_bwd<128, kElemBf16>(p, stream);
    return f16 ? launch_bwd<64, kElemF16>(p, stream) : launch_bwd<64, kElemBf16>(p, stream);
}

}  // namespace fa
