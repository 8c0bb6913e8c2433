// fa_kv8_rows.cu -- attention of many new tokens (chunks of prompts, whole prompts, drafts)
// over the paged 8-bit cache (fa_fwd_kv8 in include/fa.h) on sm_103a: items of 128 rows.
//
// With 128 rows the products fill the tensor cores' tiles the usual way round, rows on the
// 128 TMEM lanes, keys on the columns:
//   S [128 x 128 keys] = Q K^T     Q's pieces from shared memory, K as stored, K-major
//   O [128 x d]       += P V       P's pieces from TMEM, V as stored, read MN-major
// (kind::f8f6f4).  The number formats, the pieces and V's scale in the exponent are those
// of fa_kv8_fwd.cu; a key's scales are the same for the 16 columns of its block, and a
// softmax thread has a row, so no maximum crosses lanes.
//
// Bound by the tensor cores and the exponentials together: a 128 x 128 tile at d = 128
// takes 2 x 4 + 3 x 4 MMAs of 128 x 128 x 32 for bf16 (Q in 2 pieces, P in 3), 1280 cycles
// at the 8-bit rate, and 16384 exponentials, 1024 cycles at 16 a cycle.  A CTA's steps depend
// on one another (P takes the place of S in TMEM); the second CTA of the SM fills the gaps,
// each using the tensor cores while the other is in its softmax.
//
// One CTA (256 threads, two per SM, half the TMEM each: S and P 128 columns, O d):
//   warp 0       producer (fa_kv8_work.cuh)
//   warp 1       tcgen05 issuer; owns the TMEM allocation
//   warp 2       the tiles' scales, made ready for the exponents
//   warps 4..7   a row per thread: the row's queries scaled and cut into pieces, softmax,
//                the output.  They take the registers that the others give up.
#include "fa_kv8_work.cuh"

namespace fa {
namespace {

using namespace kv8;

constexpr int kRows = 128;

template <int D, int E>
struct RowsCfg {
    static constexpr int kQ = E == kElemBf16 ? 2 : 3;    // pieces of q
    static constexpr int kP = E == kElemBf16 ? 3 : 4;    // pieces of P
    static constexpr int kSlotBytes = kKeys * D;
    static constexpr int kQPiece = kRows * D;
    static constexpr int kQBytes = kQ * kQPiece;
    static constexpr int kSwizzle = D == 128 ? 2 : 4;
    static constexpr int kGroup = 8 * D;
};

struct RowsSmem {   // behind the tiles
    static constexpr bool kOutOfLine = false;
    float scales[kScaleSlots][16];   // of a tile: K's 8 blocks, V's 8 (V < 0: hidden)
    // the same, ready: K's scale and log2 of V's; 1 / V's (-1: hidden); whether any is hidden
    float2 ready[kScaleSlots][8];
    float inv_vs[kScaleSlots][8];
    int absent[kScaleSlots];
    int3 window[kWindow];
    Share share;
    Part parts[kParts];
    long long warp_sums[kThreads / 32];
    uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots], scales_full[kScaleSlots];
    uint64_t ready_full[kScaleSlots];
    uint64_t part_full[kParts], part_empty[kParts];
    uint64_t q_full, s_full, o_full, all_done;
    uint32_t tmem;
    int abort;
    int poison;                      // NaN found among values that only some rows see
};

template <int D, int E>
constexpr int rows_slots() {
    using K = RowsCfg<D, E>;
    const int n = (kCtaSmem - 1024 - K::kQBytes - static_cast<int>(sizeof(RowsSmem))) / K::kSlotBytes;
    return n < 8 ? n : 8;
}

template <int D, int E>
constexpr int rows_smem_bytes() {
    using K = RowsCfg<D, E>;
    return 1024 + rows_slots<D, E>() * K::kSlotBytes + K::kQBytes + static_cast<int>(sizeof(RowsSmem));
}

// Registers: 256 threads at 128; the first warpgroup gives up what the softmax warps take.
constexpr int kRegsCtl = 72;
constexpr int kRegsSoftmax = 184;
static_assert(128 * kRegsCtl + 128 * kRegsSoftmax <= kThreads * 128, "register split");

constexpr int kBarP = 1;     // weights written; the softmax warps and the issuer
constexpr int kBarRows = 2;  // the softmax warps among themselves

// The channels (a bit each) in which a row sees a NaN code among the part's values that
// not every row sees.  Rare: the codes are read again.
template <int D>
__device__ __forceinline__ void row_nan(const Kv8FwdParams& p, const Part& part, int lo, int hi, uint32_t (&mask)[D / 32]) {
    const int first = part.tile0 * kKeys, past = first + part.tiles * kKeys;
    for (int j = max(first, lo); j < min(past, hi + 1); ++j) {
        if (j >= part.all_lo && j <= part.all_hi) {
            j = part.all_hi;   // seen by all: the product has it
            continue;
        }
        const int id = __ldg(p.table + static_cast<long long>(part.b) * p.width + (j >> p.page_log2));
        if (id < 0 || id >= p.num_pages) continue;
        const long long r = ((static_cast<long long>(id) * p.seq.Hkv + part.h) << p.page_log2) +
                            (j & ((1 << p.page_log2) - 1));
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
#pragma unroll 1
            for (int c = 0; c < 32; ++c)
                if ((__ldg(p.v8 + r * D + 32 * w + c) & 0x7f) == 0x7f) mask[w] |= 1u << c;
    }
}

template <int D, int E>
__global__ void __launch_bounds__(kThreads, 2) fa_fwd_kv8_rows_kernel(const __grid_constant__ Kv8FwdParams p) {
    using K = RowsCfg<D, E>;
    constexpr int kSlots = rows_slots<D, E>();
    static_assert(kSlots >= 3 && kSlots / 2 + 2 < kScaleSlots, "ring of key/value tiles");
    constexpr uint32_t kIdescS = idesc_f32acc(kRows, kKeys, false, false, kElemFp8);
    // P's pieces are e5m2 (operand format code 1), V e4m3, MN-major
    constexpr uint32_t kIdescO = idesc_f32acc(kRows, D, false, true, kElemFp8) | (1u << 7);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sKV = smem;                               // [slots]
    uint8_t* sQ = smem + kSlots * K::kSlotBytes;       // [pieces][rows][D]
    RowsSmem& sm = *reinterpret_cast<RowsSmem*>(sQ + K::kQBytes);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    grid_launch_dependents();

    if (threadIdx.x == 0) {
        sm.abort = 0;
        sm.poison = 0;
#pragma unroll 1
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_addr(&sm.kv_full[i]), 1);
            mbar_init(smem_addr(&sm.kv_empty[i]), 1);
        }
#pragma unroll 1
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(smem_addr(&sm.scales_full[i]), 32);
            mbar_init(smem_addr(&sm.ready_full[i]), 1);
        }
        for (int i = 0; i < kParts; ++i) {
            mbar_init(smem_addr(&sm.part_full[i]), 1);
            mbar_init(smem_addr(&sm.part_empty[i]), 6);   // the issuer, the scales' warp, 4 softmax warps
        }
        mbar_init(smem_addr(&sm.q_full), 128);
        mbar_init(smem_addr(&sm.s_full), 1);
        mbar_init(smem_addr(&sm.o_full), 1);
        mbar_init(smem_addr(&sm.all_done), 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&sm.tmem), 256);
        tmem_relinquish();
    }
    // what the kernels before this one wrote is there from here on
    grid_dependency_wait();
    find_share<kRows>(p, sm);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;   // S and P: 128 columns, then O

    auto wait = [&](uint64_t* bar, int phase) { return wait_for(p, sm, bar, phase); };
    Part part;

    if (warp == 0) {
        regs_lower<kRegsCtl>();
        produce<D, kRows, kSlots>(p, sm, sKV);
    } else if (warp == 1) {
        // --------------------------------------------------------------- issuer
        // After an abort it goes on issuing on stale data, so that every barrier's phases
        // still complete.
        regs_lower<kRegsCtl>();
        const uint64_t k0 = sdesc<K::kSwizzle>(smem_addr(sKV), 16, K::kGroup);
        const uint64_t v0 = sdesc<K::kSwizzle>(smem_addr(sKV), K::kGroup, K::kGroup);
        const uint64_t q0 = sdesc<K::kSwizzle>(smem_addr(sQ), 16, K::kGroup);
        int T = 0, nq = 0;   // tiles, parts with tiles
        auto issue_s = [&](int tile) {   // lane 0
            const int st = (2 * tile) % kSlots;
            wait(&sm.kv_full[st], (2 * tile) / kSlots);
            tc_fence_after();
            const uint64_t kd = k0 + static_cast<uint64_t>((st * K::kSlotBytes) >> 4);
#pragma unroll
            for (int q = 0; q < K::kQ; ++q)
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                    mma_ss_f8(tmem, q0 + ((q * K::kQPiece) >> 4) + 2 * kk, kd + 2 * kk, kIdescS,
                              (q > 0 || kk > 0) ? 1u : 0u);
            mma_commit(smem_addr(&sm.s_full));
            mma_commit(smem_addr(&sm.kv_empty[st]));
        };
#pragma unroll 1
        for (int np = 0; take_part(sm, np, part); ++np) {
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_addr(&sm.part_empty[np % kParts]));
                if (part.tiles > 0) {
                    wait(&sm.q_full, nq);
                    issue_s(T);
                }
            }
            if (part.tiles > 0) ++nq;
            __syncwarp();
#pragma unroll 1
            for (int i = 0; i < part.tiles; ++i, ++T) {
                named_bar_sync(kBarP, 160);
                if (lane == 0) {
                    const int st = (2 * T + 1) % kSlots;
                    wait(&sm.kv_full[st], (2 * T + 1) / kSlots);
                    tc_fence_after();
                    const uint64_t vd = v0 + static_cast<uint64_t>((st * K::kSlotBytes) >> 4);
#pragma unroll
                    for (int q = 0; q < K::kP; ++q)
#pragma unroll
                        for (int kk = 0; kk < kKeys / 32; ++kk)
                            mma_ts_f8(tmem + 128, tmem + 32 * q + 8 * kk, vd + ((kk * 32 * D) >> 4), kIdescO,
                                      (i > 0 || q > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(smem_addr(&sm.kv_empty[st]));
                    // S of the next tile overwrites P behind this product
                    if (i + 1 < part.tiles) issue_s(T + 1);
                    else mma_commit(smem_addr(&sm.o_full));
                }
                __syncwarp();
            }
        }
        if (lane == 0) {
            mma_commit(smem_addr(&sm.all_done));
            mbar_wait_drain(smem_addr(&sm.all_done), 0, kDrainCycles);
        }
        __syncwarp();
    } else if (warp == 2) {
        // --------------------------------------------------------------- scales
        regs_lower<kRegsCtl>();
        int T = 0;
#pragma unroll 1
        for (int np = 0; take_part(sm, np, part); ++np) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[np % kParts]));
#pragma unroll 1
            for (int i = 0; i < part.tiles; ++i, ++T) {
                const int sc = T % kScaleSlots;
                wait(&sm.scales_full[sc], T / kScaleSlots);
                const int b = lane & 7;
                const float ks = sm.scales[sc][b], vs = sm.scales[sc][8 + b];
                const bool gone = vs < 0.f;
                const uint32_t vb = __float_as_uint(vs);
                float lvs = static_cast<float>(static_cast<int>(vb >> 23) - 127);
                float inv = __uint_as_float((254u << 23) - vb);
                if ((vb & 0x7fffffu) != 0 || vb < 0x00800000u || vb > 0x7e000000u) {
                    // not a power of two, or one without a normal inverse
                    lvs = log2f(vs);
                    inv = 1.f / vs;
                }
                const bool any = __any_sync(0xffffffffu, gone);
                if (lane < 8) {
                    sm.ready[sc][b] = gone ? make_float2(0.f, 0.f) : make_float2(ks, lvs);
                    sm.inv_vs[sc][b] = gone ? -1.f : inv;
                }
                if (lane == 0) sm.absent[sc] = any ? 1 : 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sm.ready_full[sc]));
            }
        }
    } else if (warp == 3) {
        regs_lower<kRegsCtl>();   // idle; its warpgroup gives registers away
    } else {
        // -------------------------------------------------------------- softmax
        regs_raise<kRegsSoftmax>();
        const int quad = warp - 4, row = quad * 32 + lane;   // TMEM lane; in V's tiles, the key
        const uint32_t tS = tmem + (static_cast<uint32_t>(quad * 32) << 16), tO = tS + 128;
        const int G = p.seq.group;
        int T = 0, no = 0;   // tiles, parts with tiles
        bool ok = true;
#pragma unroll 1
        for (int np = 0; take_part(sm, np, part); ++np) {
            const int r = part.row0 + row;
            const bool real = r < part.req.n * G;
            const int tok = r / G, head = part.h * G + (r - tok * G);
            const long long token = part.req.start + tok;
            const int pos_row = part.req.len - part.req.n + tok;
            // keys [lo, hi] are this row's
            const int hi = !real ? -1 : p.seq.causal ? pos_row : part.req.len - 1;
            const int lo = p.seq.window > 0 ? max(pos_row - p.seq.window + 1, 0) : 0;
            float rowc = 0.f;   // the row's scale, and the exponent's
            if (part.tiles > 0) {
                // the row's queries (the last part's products with the last ones are complete)
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                                  token * p.q_stride + head * D);
                uint4 w[D / 8];
#pragma unroll
                for (int u = 0; u < D / 8; ++u) w[u] = real ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
                uint32_t top = 0;
#pragma unroll
                for (int u = 0; u < D / 8; ++u) {
                    const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = unpack2<E>(x[j]);
                        top = max(top, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
                    }
                }
                // an infinity or NaN makes the row NaN, through its scale
                const bool fine = top < 0x7f800000u;
                const int k = fine ? row_exponent(top) : 0;
                const float inv = fine ? pow2f(-k) : 0.f;
                rowc = (fine ? pow2f(k) : __uint_as_float(0x7fc00000u)) * p.scale_log2;
#pragma unroll
                for (int u = 0; u < D / 16; ++u) {   // 16 elements, 16 bytes of each piece
                    float x[16];
                    const uint32_t y[8] = {w[2 * u].x, w[2 * u].y, w[2 * u].z, w[2 * u].w,
                                           w[2 * u + 1].x, w[2 * u + 1].y, w[2 * u + 1].z, w[2 * u + 1].w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 f = unpack2<E>(y[j]);
                        x[2 * j] = fine ? f.x * inv : 0.f;
                        x[2 * j + 1] = fine ? f.y * inv : 0.f;
                    }
#pragma unroll
                    for (int q = 0; q < K::kQ; ++q) {
                        uint32_t codes[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            codes[j] = pack4_e4m3(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
                            float f[4];
                            e4m3_floats(codes[j], f);
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[4 * j + i] -= f[i];
                        }
                        *reinterpret_cast<uint4*>(sQ + q * K::kQPiece + unit_offset<D>(row, u)) =
                            make_uint4(codes[0], codes[1], codes[2], codes[3]);
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(smem_addr(&sm.q_full));
            }
            float l = 0.f, ref = kNone;   // the exponents' offset: M - kShift
#pragma unroll 1
            for (int i = 0; i < part.tiles; ++i, ++T) {
                const int sc = T % kScaleSlots;
                if (ok)
                    ok = __all_sync(0xffffffffu, wait(&sm.ready_full[sc], T / kScaleSlots) && wait(&sm.s_full, T));
                if (ok) {
                    tc_fence_after();
                    float s[kKeys];
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c)
                        tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[c * 32]));
                    tmem_ld_wait();
                    reg_fence(*reinterpret_cast<uint32_t(*)[kKeys]>(&s[0]));
                    const int kb = (part.tile0 + i) * kKeys;
                    // exponents t - M + kShift in place of the products (M = 0 of a row that has
                    // no reference yet)
                    const bool none = ref == kNone;
                    const float base = none ? 0.f : ref;
#pragma unroll
                    for (int b = 0; b < 8; ++b) {
                        const float2 kv = sm.ready[sc][b];
                        const float kc = kv.x * rowc, off = kv.y - base;
                        const uint64_t c2 = f2_pack(kc, kc), o2 = f2_pack(off, off);
#pragma unroll
                        for (int c = 16 * b; c < 16 * b + 16; c += 2) {
                            const float2 e = f2_unpack(f2_fma(f2_pack(s[c], s[c + 1]), c2, o2));
                            s[c] = e.x;
                            s[c + 1] = e.y;
                        }
                    }
                    if (sm.absent[sc] || kb < part.all_lo || kb + kKeys - 1 > part.all_hi) {
                        const int clo = lo - kb, chi = min(hi, part.req.len - 1) - kb;
#pragma unroll
                        for (int b = 0; b < 8; ++b) {
                            const bool gone = sm.inv_vs[sc][b] < 0.f;
#pragma unroll
                            for (int c = 16 * b; c < 16 * b + 16; ++c)
                                if (c < clo || c > chi || gone) s[c] = kNegInf;
                        }
                        // 0 * NaN is NaN: no row's product may meet a NaN that it does not
                        // see.  (The values have to be there to be looked at.)  This thread
                        // looks after key kb + row.
                        const int vi = 2 * T + 1, pos = kb + row;
                        ok = __all_sync(0xffffffffu, wait(&sm.kv_full[vi % kSlots], vi / kSlots));
                        uint4* vrow = reinterpret_cast<uint4*>(sKV + (vi % kSlots) * K::kSlotBytes + row * D);
                        const bool hidden = sm.inv_vs[sc][row / 16] < 0.f || pos < part.lo_key ||
                                            pos > part.hi_key || pos >= part.req.len;
                        if (hidden) {
#pragma unroll
                            for (int u = 0; u < D / 16; ++u) vrow[u] = make_uint4(0, 0, 0, 0);
                        } else if (pos < part.all_lo || pos > part.all_hi) {
#pragma unroll 1
                            for (int u = 0; u < D / 16; ++u) {
                                uint4 w = vrow[u];
                                const uint32_t a = nan_bytes(w.x), b = nan_bytes(w.y), e = nan_bytes(w.z),
                                               f = nan_bytes(w.w);
                                if (a | b | e | f) {
                                    // those channels become NaN at the part's end, for the rows that see them
                                    w.x &= ~(a | (a - (a >> 7)));
                                    w.y &= ~(b | (b - (b >> 7)));
                                    w.z &= ~(e | (e - (e >> 7)));
                                    w.w &= ~(f | (f - (f >> 7)));
                                    vrow[u] = w;
                                    sm.poison = 1;
                                }
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    float top4[4];
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) top4[i4] = fmax3(s[3 * i4], s[3 * i4 + 1], s[3 * i4 + 2]);
#pragma unroll
                    for (int c = 12; c < kKeys - 4; c += 8)
#pragma unroll
                        for (int i4 = 0; i4 < 4; ++i4) top4[i4] = fmax3(top4[i4], s[c + 2 * i4], s[c + 2 * i4 + 1]);
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) top4[i4] = fmaxf(top4[i4], s[kKeys - 4 + i4]);
                    const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                    const bool moves = none ? top > kNegInf : top > kShift + kGrow;
                    if (__any_sync(0xffffffffu, moves)) {
                        // the row's reference moves up to its largest key
                        const float by = moves ? kShift - top : 0.f;
#pragma unroll
                        for (int c = 0; c < kKeys; ++c) s[c] += by;
                        const float f = none ? 1.f : ex2_approx(by);
                        l *= f;
                        if (moves) ref = base - by;
                        if (i > 0) {
                            // (the last tile's product was complete before this tile's S)
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t x[16];
                                tmem_ld16(tO + c, x);
                                tmem_ld_wait();
                                reg_fence(x);
#pragma unroll
                                for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f);
                                tmem_st16(tO + c, x);
                            }
                        }
                    }
                    // weights, their sum, and their pieces (32 keys are 8 columns of a piece)
#pragma unroll
                    for (int c0 = 0; c0 < kKeys; c0 += 32) {
                        uint32_t h[16];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            uint64_t sum2 = 0;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int c = c0 + 16 * b + 2 * j;
                                const float w0 = ex2_approx(s[c]), w1 = ex2_approx(s[c + 1]);
                                sum2 = j == 0 ? f2_pack(w0, w1) : f2_add(sum2, f2_pack(w0, w1));
                                h[8 * b + j] = pack2<kElemF16>(w0, w1);
                            }
                            const float2 sum = f2_unpack(sum2);
                            l = fmaf(sum.x + sum.y, sm.inv_vs[sc][c0 / 16 + b], l);
                        }
#pragma unroll
                        for (int q = 0; q < K::kP; ++q) {
                            uint32_t words[8];
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (K::kP == 3 && q == 2) h[j] += 0x00800080u;
#pragma unroll
                            for (int j = 0; j < 8; ++j) words[j] = __byte_perm(h[2 * j], h[2 * j + 1], 0x7531);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (q + 1 < K::kP) h[j] = sub_f16x2(h[j], h[j] & 0xff00ff00u);
                            tmem_st8(tS + 32 * q + c0 / 4, words);
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before();
                }
                named_bar_signal(kBarP, 160, ok);
            }
            // ------------------------------------------------ the part's end
            if (part.tiles > 0) {
                if (ok) ok = __all_sync(0xffffffffu, wait(&sm.o_full, no));
                ++no;
            }
            tc_fence_after();
            bool poison = false;
            if (part.tiles > 0 && (part.tile0 * kKeys < part.all_lo ||
                                   (part.tile0 + part.tiles) * kKeys - 1 > part.all_hi)) {
                // (parts with no such edge set no poison)
                named_bar_sync(kBarRows, 128);
                poison = sm.poison != 0;
                named_bar_sync(kBarRows, 128);
                if (row == 0) sm.poison = 0;
            }
            if (ok) {
                uint32_t nan[D / 32] = {};
                if (poison && real) row_nan<D>(p, part, lo, hi, nan);
                const bool whole = part.whole;
                const float mul = !whole ? 1.f : l != 0.f ? 1.f / l : 0.f;   // (NaN divides on)
                const long long slot = (2LL * blockIdx.x + (part.begins ? 1 : 0)) * kRows + row;
                const bool in = real && fa_index_ok(token, p.seq.total_tokens, p.status);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t x[32];
                    if (part.tiles > 0) {
                        tmem_ld32(tO + c * 32, x);
                        tmem_ld_wait();
                        reg_fence(x);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = 0;
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        x[j] = __float_as_uint(__uint_as_float(x[j]) * mul);
                        if ((nan[c] >> j) & 1u) x[j] = 0x7fc00000u;
                    }
                    if (in && whole) {
                        uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) +
                                                              (token * p.seq.Hq + head) * D + c * 32);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint32_t y[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                y[j] = pack2<E>(__uint_as_float(x[8 * u + 2 * j]), __uint_as_float(x[8 * u + 2 * j + 1]));
                            out[u] = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    } else if (in) {
                        uint4* out = reinterpret_cast<uint4*>(p.part_o + slot * D + c * 32);
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            out[u] = make_uint4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
                    }
                }
                const float m = ref == kNone ? 0.f : ref + kShift;
                if (in && whole)
                    p.lse[row_stat_index(p.seq, part.b, head, part.req.start, tok)] =
                        l != 0.f ? (m - kShift + log2f(l)) * kLn2 : kNegInf;
                else if (in)
                    p.part_stat[slot] = make_float2(ref == kNone ? kNegInf : m, l);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[np % kParts]));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 256);
}

template <int D, int E>
cudaError_t launch_rows(const Kv8FwdParams& p, cudaStream_t stream) {
    constexpr int smem = rows_smem_bytes<D, E>();
    static_assert(smem <= kCtaSmem, "shared memory per CTA");
    auto kern = fa_fwd_kv8_rows_kernel<D, E>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, p.ctas, kThreads, smem, stream, p);
}

}  // namespace

cudaError_t launch_fwd_kv8_rows(const Kv8FwdParams& p, int d, cudaStream_t stream) {
    if (d == 128)
        return p.elem == kElemBf16Code ? launch_rows<128, kElemBf16>(p, stream)
                                       : launch_rows<128, kElemF16>(p, stream);
    return p.elem == kElemBf16Code ? launch_rows<64, kElemBf16>(p, stream) : launch_rows<64, kElemF16>(p, stream);
}

}  // namespace fa
