// fa_kv8_fwd.cu -- attention of new tokens over the paged 8-bit cache (fa_fwd_kv8 in
// include/fa.h).
#include "fa_kernels.h"
#include "fa_ptx.cuh"
#include "fa_seq.cuh"

#include <climits>

namespace fa {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float e4m3_value(uint32_t code) {
    uint32_t h;
    asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(code));
    return unpack2<kElemF16>(h).x;
}

// One warp per (new token, query head): lanes take keys for the scores, channels for the
// sum over the values; the running maximum and sum of the online softmax are the warp's.
template <int D, int E>
__global__ void __launch_bounds__(128) fa_fwd_kv8_kernel(const Kv8FwdParams p) {
    __shared__ float sq[4][D];
    const SeqInfo& s = p.seq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * 4 + warp;
    const int h = static_cast<int>(item % s.Hq);
    const long long t = item / s.Hq;
    if (t >= s.total_tokens) return;
    int b, first, n;
    if (s.cu_seqlens) {
        int lo = 0, hi = s.B;   // the first request that ends behind t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s.cu_seqlens[mid + 1] > t) hi = mid;
            else lo = mid + 1;
        }
        if (lo == s.B) return;
        b = lo;
        first = s.cu_seqlens[b];
        n = s.cu_seqlens[b + 1] - first;
    } else {
        b = static_cast<int>(t / s.N);
        first = b * s.N;
        n = s.N;
    }
    const int page = 1 << p.page_log2;
    const int len = static_cast<int>(min(max(static_cast<long long>(p.lens[b]), 0LL),
                                         static_cast<long long>(p.width) << p.page_log2));
    const int pos = len - n + static_cast<int>(t - first);
    const int hi = s.causal ? pos : len - 1;
    const int lo = s.causal && s.window > 0 ? max(pos - s.window + 1, 0) : 0;
    const int g = h / s.group;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + t * p.q_stride + h * D;
    for (int c = lane; c < D; c += 32)
        sq[warp][c] = E == kElemBf16 ? __uint_as_float(static_cast<uint32_t>(q[c]) << 16)
                                     : unpack2<kElemF16>(q[c]).x;
    __syncwarp();
    float m = kNegInf, l = 0.f, o[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] = 0.f;
    for (int j0 = lo / 32 * 32; j0 <= hi; j0 += 32) {
        const int j = j0 + lane;
        long long row = -1;
        if (j >= lo && j <= hi) {
            const int id = p.table[static_cast<long long>(b) * p.width + (j >> p.page_log2)];
            if (id >= 0 && id < p.num_pages)
                row = ((static_cast<long long>(id) * s.Hkv + g) << p.page_log2) + (j & (page - 1));
        }
        float x = kNegInf, vs = 0.f;
        if (row >= 0) {
            const uint8_t* k = p.k8 + row * D;
            float dot = 0.f;
            for (int c = 0; c < D; ++c) dot += sq[warp][c] * e4m3_value(k[c]);
            x = dot * p.k_scale[row / kKv8Block] * p.scale_log2;
            vs = p.v_scale[row / kKv8Block];
        }
        float top = m;
#pragma unroll
        for (int w = 0; w < 32; ++w) top = fmaxf(top, __shfl_sync(0xffffffffu, x, w));
        const float ref = top == kNegInf ? 0.f : top;
        const float w = exp2f(x - ref);
        const float f = exp2f(m - ref);
        m = top;
        l *= f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[c] *= f;
        for (int u = 0; u < 32; ++u) {
            const long long r = __shfl_sync(0xffffffffu, row, u);
            const float wu = __shfl_sync(0xffffffffu, w, u), su = __shfl_sync(0xffffffffu, vs, u);
            if (r < 0) continue;
            l += wu;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[c] += wu * su * e4m3_value(p.v8[r * D + lane + 32 * c]);
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;   // (NaN divides on)
    uint16_t* out = static_cast<uint16_t*>(p.o) + (t * s.Hq + h) * D;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
        out[lane + 32 * c] = static_cast<uint16_t>(pack2<E>(o[c] * inv, 0.f));
    if (lane == 0) {
        const long long at = s.cu_seqlens ? static_cast<long long>(h) * s.total_tokens + t
                                          : (static_cast<long long>(b) * s.Hq + h) * s.N + (t - first);
        p.lse[at] = l != 0.f ? (m + log2f(l)) * kLn2 : kNegInf;
    }
}

}  // namespace

cudaError_t launch_fwd_kv8(const Kv8FwdParams& p, int d, cudaStream_t stream) {
    const long long grid = (static_cast<long long>(p.seq.total_tokens) * p.seq.Hq + 3) / 4;
    if (grid > INT_MAX) return cudaErrorInvalidValue;
    const unsigned g = static_cast<unsigned>(grid);
    if (d == 128 && p.elem == kElemBf16Code) fa_fwd_kv8_kernel<128, kElemBf16><<<g, 128, 0, stream>>>(p);
    else if (d == 128) fa_fwd_kv8_kernel<128, kElemF16><<<g, 128, 0, stream>>>(p);
    else if (p.elem == kElemBf16Code) fa_fwd_kv8_kernel<64, kElemBf16><<<g, 128, 0, stream>>>(p);
    else fa_fwd_kv8_kernel<64, kElemF16><<<g, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fa
