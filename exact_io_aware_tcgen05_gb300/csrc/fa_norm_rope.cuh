// fa_norm_rope.cuh -- a head's row in registers, its norm and its rotation by position: what
// the kernels that prepare queries and keys share (fa_norm_rope.cu, fa_kv8_cache.cu).
//
// D / 16 lanes hold a row of D channels, two 16-byte units (8 channels each) a lane, chosen so
// that both channels of every rotated pair lie in one lane: pairs (f, f + rot / 2) put units u
// and u + rot / 16 together, neighbouring pairs lie in a unit anyway.  Nothing but the sum of
// squares crosses lanes, and a lane's 8 cosines and sines serve all heads of its token.  (The
// instructions that take two fp32 numbers saved as much arithmetic as they cost in moves: pairs
// must lie in neighbouring registers.)
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

constexpr int kNormThreads = 256;

template <int D, bool IL>   // IL: neighbouring pairs (2 f, 2 f + 1)
struct RowLane {
    static constexpr int kLanes = D / 16;
    int unit[2];     // the lane's units
    bool turned[2];  // whether they are rotated
    int freq[2];     // the first of four frequencies: pairs 0 .. 3 and 4 .. 7 of the lane

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
            freq[0] = 8 * lane;
            freq[1] = 8 * lane + 4;
        }
    }
};

__device__ __forceinline__ int axis_of(const RopeParams& r, int f) {
    const int axis = r.axes ? r.axes[f] : 0;
    return static_cast<unsigned>(axis) < static_cast<unsigned>(r.num_axes) ? axis : 0;
}

// Cosine and sine of frequency f's angle for one token.  The nearest quarter turn is taken off as an
// integer first: what is left, an eighth of a turn at most, is an fp32 number to 2^-28 of a turn, where
// a whole turn would be one to 2^-26.
__device__ __forceinline__ void cos_sin(const RopeParams& r, int f, long long token, float& c, float& s) {
    if (!fa_index_ok(f, r.rot / 2, r.status) || !fa_index_ok(token, r.axis_stride, r.status)) {
        c = s = 0.f;
        return;
    }
    const long long pos = r.positions[axis_of(r, f) * r.axis_stride + token];
    const uint32_t turn = static_cast<uint32_t>((static_cast<unsigned long long>(pos) * r.turns[f]) >> 32);
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    float x, y;
    sincospif(static_cast<float>(static_cast<int>(turn - (quarter << 30))) * 0x1p-31f, &y, &x);   // (half turns)
    const uint32_t a = __float_as_uint(quarter & 1 ? y : x), b = __float_as_uint(quarter & 1 ? x : y);
    c = __uint_as_float(a ^ ((quarter + 1) & 2) << 30);
    s = __uint_as_float(b ^ (quarter & 2) << 30);
}

// A lane's cosines and sines: pair i is the lane's channels (i, 8 + i), or with IL (2 i, 2 i + 1).
// (Not set for units that are not rotated.)
struct Rotation {
    alignas(16) float c[8], s[8];
};

// For one token, worked out by the lane itself.
template <int D, bool IL>
__device__ __forceinline__ void lane_rotation(const RopeParams& p, const RowLane<D, IL>& at, long long token, Rotation& r) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (!at.turned[j]) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) cos_sin(p, at.freq[j] + i, token, r.c[4 * j + i], r.s[4 * j + i]);
    }
}

// From rows of cosines and of sines in shared memory, where frequency f is at place_of(f): the lanes of
// a row read neighbouring 16 bytes.
template <int D, bool IL>
__device__ __forceinline__ int place_of(int f) {
    return IL ? f : (f & 4 ? D / 4 : 0) + f / 8 * 4 + f % 4;
}
template <int D, bool IL>
__device__ __forceinline__ void rotation_from(const float* cos_row, const float* sin_row, const RowLane<D, IL>& at,
                                              Rotation& r) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (!at.turned[j]) continue;
        const int place = place_of<D, IL>(at.freq[j]);
        *reinterpret_cast<float4*>(&r.c[4 * j]) = *reinterpret_cast<const float4*>(cos_row + place);
        *reinterpret_cast<float4*>(&r.s[4 * j]) = *reinterpret_cast<const float4*>(sin_row + place);
    }
}

// The lane's 16 channels turned by its angles (back: by their negatives).
template <int D, bool IL, bool BACK>
__device__ __forceinline__ void rotate(const RowLane<D, IL>& at, const Rotation& r, float (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (!at.turned[j]) continue;
#pragma unroll
        for (int i = 4 * j; i < 4 * j + 4; ++i) {
            float& a = x[IL ? 2 * i : i];
            float& b = x[IL ? 2 * i + 1 : 8 + i];
            const float s = BACK ? -r.s[i] : r.s[i], y = fmaf(a, r.c[i], -(b * s));
            b = fmaf(b, r.c[i], a * s);
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
__device__ __forceinline__ uint4 narrow(const float* x) {
    return make_uint4(pack2<E>(x[0], x[1]), pack2<E>(x[2], x[3]), pack2<E>(x[4], x[5]), pack2<E>(x[6], x[7]));
}

// Whether 8 channels at `at` lie in a token's heads of one side of the tensor at `base` (checking build).
template <int D>
__device__ __forceinline__ bool channels_ok(const NormRopeParams& p, int side, const void* base, const void* at, long long stride) {
    return fa_row_ok(base, at, 16, p.T, 2LL * D * p.heads[side], 2 * stride, p.status);
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
    float q[2] = {x[0] * x[0], x[1] * x[1]};
#pragma unroll
    for (int i = 2; i < 16; ++i) q[i & 1] = fmaf(x[i], x[i], q[i & 1]);
    const float a = fmaf(row_sum<D>(q[0] + q[1]), 1.f / D, eps), r = rsqrtf(a);
    // a step of Newton's: rsqrtf is good to two ulps (infinite squares: r = 0)
    return r > 0.f ? fmaf(0.5f * r, fmaf(-a * r, r, 1.f), r) : r;
}

// x = x r w, in that order.
__device__ __forceinline__ void scale_row(float (&x)[16], float r, const float (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
}

// The lane's 16 weights of one side (1 without weights).
template <int D, int E, bool IL>
__device__ __forceinline__ void load_weights(const void* w, bool wide, const RowLane<D, IL>& at, float (&v)[16]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 1.f;
    } else if (wide) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(&v[4 * i]) =
                *reinterpret_cast<const float4*>(static_cast<const float*>(w) + 8 * at.unit[i / 2] + 4 * (i & 1));
    } else {
        const uint4* u = static_cast<const uint4*>(w);
        widen<E>(u[at.unit[0]], u[at.unit[1]], v);
    }
}

}  // namespace fa
