// fa_norm_rope.cuh -- a head's row in registers, its norm and its rotation by position: what
// the kernels that prepare queries and keys share (fa_norm_rope.cu, fa_kv8_cache.cu).
//
// D / 16 lanes hold a row of D channels, two 16-byte units (8 channels each) a lane, chosen so
// that both channels of every rotated pair lie in one lane: pairs (f, f + rot / 2) put units u
// and u + rot / 16 together, neighbouring pairs lie in a unit anyway.  Nothing but the sum of
// squares crosses lanes, and a lane's 8 cosines and sines serve all heads of its token.
//
// An angle is position * frequency.  A frequency is kept as a fraction of a turn in units of
// 2^-64, so that the low 64 bits of the product are the angle without its whole turns, exactly
// (frequency's own rounding: position * 2^-65 turns); its upper half goes to sincospif.  That is
// three integer products an angle, where 64-bit floating point would be the slow unit here and a
// table of cosines a second stream from memory.
#pragma once

#include "fa_kernels.h"
#include "fa_ptx.cuh"

namespace fa {

template <int D, bool IL>   // IL: neighbouring pairs (2 f, 2 f + 1)
struct RowLane {
    static constexpr int kLanes = D / 16;
    int unit[2];     // the lane's units
    bool turned[2];  // whether they are rotated
    int freq[2];     // IL: the first of each unit's 4 frequencies; else [0]: the first of 8

    __device__ __forceinline__ RowLane(int lane, int rot) {
        if constexpr (IL) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                unit[j] = lane + j * kLanes;
                turned[j] = 8 * unit[j] < rot;
                freq[j] = 4 * unit[j];
            }
        } else {
            const int r = rot / 16;
            unit[0] = lane < r ? lane : 2 * r + 2 * (lane - r);
            unit[1] = lane < r ? lane + r : unit[0] + 1;
            turned[0] = turned[1] = lane < r;
            freq[0] = freq[1] = 8 * lane;
        }
    }
};

// Cosine and sine of the lane's pairs for one token: pair i is (x[i], x[8 + i]), or with IL
// (x[2 i], x[2 i + 1]) of the lane's 16 channels.  Not set for units that are not rotated.
template <int D, bool IL>
__device__ __forceinline__ void rotation_of(const RopeParams& r, const RowLane<D, IL>& at, long long token,
                                            float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (!at.turned[j]) continue;
#pragma unroll
        for (int i = 4 * j; i < 4 * j + 4; ++i) {
            const int f = IL ? at.freq[j] + i - 4 * j : at.freq[0] + i;
            int axis = r.axes ? r.axes[f] : 0;
            if (static_cast<unsigned>(axis) >= static_cast<unsigned>(r.num_axes)) axis = 0;
            const long long pos = r.positions[axis * r.axis_stride + token];
            const unsigned long long turn = static_cast<unsigned long long>(pos) * r.turns[f];
            // the upper 32 bits as half turns, -1 <= x < 1
            const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;
            sincospif(x, &s[i], &c[i]);
        }
    }
}

// The lane's 16 channels turned by its angles (back: by their negatives).
template <int D, bool IL, bool BACK>
__device__ __forceinline__ void rotate(const RowLane<D, IL>& at, const float (&c)[8], const float (&s)[8],
                                       float (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (!at.turned[j]) continue;
#pragma unroll
        for (int i = 4 * j; i < 4 * j + 4; ++i) {
            float& a = x[IL ? 2 * i : i];
            float& b = x[IL ? 2 * i + 1 : 8 + i];
            const float sn = BACK ? -s[i] : s[i];
            const float y = a * c[i] - b * sn;
            b = b * c[i] + a * sn;
            a = y;
        }
    }
}

template <int E>
__device__ __forceinline__ void widen(uint4 a, uint4 b, float (&x)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = unpack2<E>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <int E>
__device__ __forceinline__ void narrow(const float (&x)[16], uint4& a, uint4& b) {
    a = make_uint4(pack2<E>(x[0], x[1]), pack2<E>(x[2], x[3]), pack2<E>(x[4], x[5]), pack2<E>(x[6], x[7]));
    b = make_uint4(pack2<E>(x[8], x[9]), pack2<E>(x[10], x[11]), pack2<E>(x[12], x[13]), pack2<E>(x[14], x[15]));
}

// Sum over the D / 16 lanes of a row, in all of them.
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1 / sqrt(mean of squares + eps)
template <int D>
__device__ __forceinline__ float inverse_norm(const float (&x)[16], float eps) {
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i & 1] = fmaf(x[i], x[i], q[i & 1]);
    return rsqrtf(fmaf(row_sum<D>(q[0] + q[1]), 1.f / D, eps));
}

// The lane's 16 weights of one side (1 without weights).
template <int D, int E, bool IL>
__device__ __forceinline__ void load_weights(const void* w, bool wide, const RowLane<D, IL>& at, float (&v)[16]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 1.f;
    } else if (wide) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + 8 * at.unit[i / 2] + 4 * (i & 1));
            v[4 * i] = f.x;
            v[4 * i + 1] = f.y;
            v[4 * i + 2] = f.z;
            v[4 * i + 3] = f.w;
        }
    } else {
        const uint4* u = static_cast<const uint4*>(w);
        widen<E>(u[at.unit[0]], u[at.unit[1]], v);
    }
}

constexpr int kNormThreads = 256;

// The forward for one CTA, number `cta` of a side's: a group of D / 16 lanes has one token's run
// of heads, kAhead rows of it on their way at a time.
template <int D, int E, bool IL>
__device__ __forceinline__ void norm_rope_rows(const NormRopeParams& p, int side, int cta) {
    constexpr int L = D / 16, kAhead = 4;
    const int run = p.run[side];
    const RowLane<D, IL> at(threadIdx.x % L, p.rope.rot);
    const long long units = static_cast<long long>(p.T) * (p.heads[side] / run);
    const long long mine = static_cast<long long>(cta) * (kNormThreads / L) + threadIdx.x / L;
    const bool real = mine < units;   // (the others take part in the sums)
    const long long unit = real ? mine : units - 1;
    const long long part = unit / p.T, token = unit - part * p.T;
    const uint16_t* x = static_cast<const uint16_t*>(p.x[side]) + token * p.x_stride[side] + part * run * D;
    uint16_t* y = static_cast<uint16_t*>(p.y[side]) + token * p.y_stride[side] + part * run * D;
    float c[8], s[8], w[16];
    rotation_of<D, IL>(p.rope, at, token, c, s);
    if (p.norm) load_weights<D, E, IL>(p.w[side], p.wide, at, w);
#pragma unroll 1
    for (int h0 = 0; h0 < run; h0 += kAhead) {
        uint4 in[kAhead][2];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                in[u][j] = h0 + u < run ? *reinterpret_cast<const uint4*>(x + (h0 + u) * D + 8 * at.unit[j])
                                        : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            float v[16];
            widen<E>(in[u][0], in[u][1], v);
            if (p.norm) {
                const float r = inverse_norm<D>(v, p.eps);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = v[i] * r * w[i];
            }
            rotate<D, IL, false>(at, c, s, v);
            uint4 out[2];
            narrow<E>(v, out[0], out[1]);
            if (real && h0 + u < run && fa_index_ok(token, p.T, p.status)) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<uint4*>(y + (h0 + u) * D + 8 * at.unit[j]) = out[j];
            }
        }
    }
}

}  // namespace fa
