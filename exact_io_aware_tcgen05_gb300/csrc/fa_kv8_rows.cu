// fa_kv8_rows.cu -- attention of many new tokens (chunks of prompts, whole prompts, drafts)
// over the paged 8-bit cache (fa_fwd_kv8 in include/fa.h) on sm_103a: items of 128 rows.
//
// With 128 rows the products fill the tensor cores' tiles the usual way round, rows on the
// 128 TMEM lanes, keys on the columns:
//   S [128 x 128 keys] = Q K^T     Q's pieces from shared memory, K as stored, K-major
//   O [128 x d]       += P V       P (fp16) from TMEM, V as fp16, read MN-major
// The first is kind::f8f6f4 with Q in pieces (fa_kv8_fwd.cu has the number formats) and K
// untouched.  For the second, each value's code is widened to fp16 (exact) once for all 128
// rows, by two warps, which costs far less than cutting 128 x 128 weights into 8-bit pieces,
// and one fp16 product takes two thirds of the time of three 8-bit ones.  The weights are
// rounded to fp16's 11 bits.  V's scale is in the exponent as in fa_kv8_fwd.cu; a key's scales
// are the same for the 16 columns of its block, and a softmax thread has a row, so no
// maximum crosses lanes.
//
// What it cannot do without: a 128 x 128 tile at d = 128 takes 1024 cycles of MMAs for bf16
// (2 x 4 of 128 x 128 x 32 8-bit, 8 of 128 x 128 x 16; MMAs of 64 columns ran no faster than
// those of 128) and 16384 exponentials, 512 cycles at 32 a cycle; at d = 64 the MMAs take 512
// too.  The softmax takes a tile in two halves of 64 keys, so that the first half's product runs
// during the second's softmax; P takes the place of the scores in TMEM.  Between a tile's
// second half and the next tile's scores the SM's other CTA has the units to itself.
//
// Measured (one GB300, bf16, Hq 32, Hkv 8): 2048 new tokens over 16384 keys at d = 128 463 us,
// 1110 TFLOP/s, 59 % of the measured bf16 rate; 16 whole prompts of up to 2048 at d = 64 229 us,
// twice what its exponentials and MMAs take.  Bound by the chain of a tile in its CTA (scores,
// two halves of softmax of some 1000 cycles each, product), two CTAs deep: the tensor pipe is
// active 48 % (d = 128) and the issue slots half used, so neither unit is the limit.  A softmax in
// a loop of 16 or 32 columns (short code, less at once in registers) ran 8 to 17 % slower, an
// earlier load of the queries, or one copy of the values and a longer ring, no faster: what
// takes a register more in the softmax costs up to a fifth.
//
// One CTA (256 threads, two per SM, half the TMEM each: S and P 128 columns, O d):
//   warp 0       producer (fa_kv8_work.cuh)
//   warp 1       tcgen05 issuer; owns the TMEM allocation
//   warps 2, 3   the tiles' values to fp16
//   warps 4..7   softmax and output, a row per thread
//   warps 2..7   an item's queries, scaled and cut into pieces
#include "fa_kv8_work.cuh"

namespace fa {
namespace {

using namespace kv8;

constexpr int kRows = 128;
// The weights are fp16 numbers here, times 2^9: a row's reference moves when a key exceeds it
// by more than 2^6 (fp16's largest number is near 2^16), which hardly happens once a row has
// seen some keys, and weights down to 2^-23 of it keep all 11 bits.
constexpr float kRowsShift = 9.f;
constexpr float kRowsGrow = 6.f;

constexpr int kHalf = 64;   // keys of a half tile

template <int D, int E>
struct RowsCfg {
    static constexpr int kQ = E == kElemBf16 ? 2 : 3;    // pieces of q
    static constexpr int kSlotBytes = kHalf * D;
    static constexpr int kQPiece = kRows * D;
    static constexpr int kQBytes = kQ * kQPiece;
    static constexpr int kV16Bytes = kHalf * D * 2;      // [d / 64][keys][64], swizzled over 128 bytes
    static constexpr int kV16Chunk = kHalf * 128;
    // the halves' values, each in its place, unless the queries leave no room for both
    static constexpr int kV16Bufs = kQBytes > 32768 ? 1 : 2;
    static constexpr int kSwizzle = D == 128 ? 2 : 4;
    static constexpr int kGroup = 8 * D;
};

struct RowsSmem {   // behind the tiles
    float scales[kScaleSlots][16];   // of a tile: K's 8 blocks, V's 8 (V < 0: hidden)
    // the same, ready for the exponents: K's scale, log2 of V's, 1 / V's (-1: hidden)
    float4 ready[kScaleSlots][8];
    int absent[kScaleSlots];         // whether a block is hidden
    float q_scale[kRows];
    int q_next;                      // claims of rows to cut (cut_rows)
    int3 window[kWindow];
    Share share;
    Part parts[kParts];
    long long warp_sums[kThreads / 32];
    uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots], scales_full[kScaleSlots];
    uint64_t ready_full[kScaleSlots];
    uint64_t part_full[kParts], part_empty[kParts];
    uint64_t q_full, q_empty, s_full, o_half[2], all_done;
    uint32_t tmem;
    int abort;
    int poison[2];                   // [part parity] NaN found among values that only some rows see
};

template <int D, int E>
constexpr int rows_fixed_bytes() {
    using K = RowsCfg<D, E>;
    return 1024 + K::kQBytes + K::kV16Bufs * K::kV16Bytes + static_cast<int>(sizeof(RowsSmem));
}

template <int D, int E>
constexpr int rows_slots() {
    const int n = (kCtaSmem - rows_fixed_bytes<D, E>()) / RowsCfg<D, E>::kSlotBytes;
    return (n < kMaxSlots ? n : kMaxSlots) / 2 * 2;   // (even: a tile's K units lie side by side)
}

template <int D, int E>
constexpr int rows_smem_bytes() {
    return rows_fixed_bytes<D, E>() + rows_slots<D, E>() * RowsCfg<D, E>::kSlotBytes;
}

// + half: weights and values there; softmax warps, values' warps, issuer.  Only the issuer waits
// there (and a warp without rows).  The others come again once the issuer has been there, or they
// would be counted twice: they wait for what it issued behind it, the softmax for a tile's scores,
// the values' warps for the products of a half, after an abort too (it goes on issuing).
constexpr int kBarP = 1;
constexpr int kBarRows = 3;  // the softmax warps among themselves
constexpr int kBarConv = 4;  // warps 2 and 3 among themselves

// A wait, by a warp, for what the issuer commits in any case.
__device__ __forceinline__ void wait_for_issuer(uint64_t* bar, int phase) {
    if (!mbar_try_wait(smem_addr(bar), phase & 1)) drain_on(smem_addr(bar), phase & 1);
    __syncwarp();
}

// Four e4m3 codes to fp16 (exact; NaN stays NaN).
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

// A part's queries into their pieces, by the warps that have nothing else to do: each claims
// a warp's load of rows at a time, the next one's load on its way while it cuts the last one,
// until there are none left.  `next` counts the claims of all parts, for each part kClaims
// and one more (too many) for each of the 6 warps.
template <int D, int E>
__device__ __noinline__ void cut_rows(const Kv8FwdParams& p, int& next, float* q_scale, uint8_t* sQ, int start,
                                      int n, int h, int row0) {
    using K = RowsCfg<D, E>;
    constexpr int kLanes = D / 8;          // threads of a row
    constexpr int kPass = 32 / kLanes;     // rows of a warp's load
    constexpr int kClaims = kRows / kPass;
    const int lane = threadIdx.x & 31, sub = lane % kLanes, G = p.seq.group, rows = n * G;
    const int tok0 = row0 / G, rem0 = row0 - tok0 * G;
    uint4 w = make_uint4(0, 0, 0, 0);
    int r = -1;
#pragma unroll 1
    while (true) {
        int c = lane == 0 ? atomicAdd(&next, 1) : 0;
        c = __shfl_sync(0xffffffffu, c, 0) % (kClaims + 6);
        const int r2 = c * kPass + lane / kLanes;
        uint4 w2 = make_uint4(0, 0, 0, 0);
        if (c < kClaims && row0 + r2 < rows) {
            const int more = small_div(rem0 + r2, G, p.group_inv);
            const int head = h * G + rem0 + r2 - more * G;
            const long long token = start + tok0 + more;
            w2 = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + token * p.q_stride +
                                                 head * D + sub * 8);
        }
        if (r >= 0) {
            const float scale = cut_queries<D, E, K::kQ>(
                w, sQ + unit_offset<D>(r, sub >> 1) + (sub & 1) * 8, K::kQPiece);
            if (sub == 0) q_scale[r] = scale;
        }
        if (c >= kClaims) return;
        w = w2;
        r = r2;
    }
}

// NaN for the channels in which a row sees a NaN code among the part's values that not every
// row sees.  Rare: the codes are read again.
template <int D>
__device__ __noinline__ void spoil_row(const Kv8FwdParams& p, const Part& part, int lo, int hi, uint16_t* out,
                                       float* partial) {
    const int first = part.tile0 * kKeys, past = first + part.tiles * kKeys;
    for (int j = max(first, lo); j < min(past, hi + 1); ++j) {
        if (j >= part.all_lo && j <= part.all_hi) {
            j = part.all_hi;   // seen by all: the product has it
            continue;
        }
        const int id = p.table[static_cast<long long>(part.b) * p.width + (j >> p.page_log2)];
        if (id < 0 || id >= p.num_pages) continue;
        const long long r = ((static_cast<long long>(id) * p.seq.Hkv + part.h) << p.page_log2) +
                            (j & ((1 << p.page_log2) - 1));
#pragma unroll 1
        for (int c = 0; c < D; ++c) {
            if ((p.v8[r * D + c] & 0x7f) != 0x7f) continue;
            if (out) out[c] = 0x7fff;   // a NaN of either type
            else partial[c] = __uint_as_float(0x7fc00000u);
        }
    }
}

template <int D, int E>
__global__ void __launch_bounds__(kThreads, 2) fa_fwd_kv8_rows_kernel(const __grid_constant__ Kv8FwdParams p) {
    using K = RowsCfg<D, E>;
    constexpr int kSlots = rows_slots<D, E>();
    static_assert(kSlots >= 4 && kSlots / 4 + 2 < kScaleSlots, "ring of key/value tiles");
    constexpr uint32_t kIdescS = idesc_f32acc(kRows, kKeys, false, false, kElemFp8);
    constexpr uint32_t kIdescO = idesc_f32acc(kRows, D, false, true, kElemF16);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sKV = smem;                               // [slots]
    uint8_t* sQ = smem + kSlots * K::kSlotBytes;       // [pieces][rows][D]
    uint8_t* sV = sQ + K::kQBytes;                     // [kV16Bufs]
    RowsSmem& sm = *reinterpret_cast<RowsSmem*>(sV + K::kV16Bufs * K::kV16Bytes);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    grid_launch_dependents();

    if (threadIdx.x == 0) {
        sm.abort = 0;
        sm.poison[0] = sm.poison[1] = 0;
        sm.q_next = 0;
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
            mbar_init(smem_addr(&sm.part_empty[i]), 7);   // every warp but the producer
        }
        mbar_init(smem_addr(&sm.q_full), 192);            // warps 2 .. 7
        mbar_init(smem_addr(&sm.q_empty), 5);             // the last S of the part, 4 softmax warps
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sm.o_half[i]), 1);
        }
        mbar_init(smem_addr(&sm.s_full), 1);
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
    const uint32_t tmem = sm.tmem;   // S and P of a tile's halves, 64 columns each, then O

    auto wait = [&](uint64_t* bar, int phase) { return wait_for(p, sm, bar, phase); };
    Part part;

    if (warp == 0) {
        produce<D, kRows, kHalf, kSlots>(p, sm, sKV);
    } else if (warp == 1) {
        // --------------------------------------------------------------- issuer
        // Walks the tiles of all parts one behind the other; S of a tile's half is issued
        // behind the last tile's product of that half, whose P it overwrites.  After an
        // abort it goes on issuing on stale data, so that every barrier's phases still
        // complete.
        const uint64_t k0 = sdesc<K::kSwizzle>(smem_addr(sKV), 16, K::kGroup);
        const uint64_t v0 = sdesc_sw128(smem_addr(sV), K::kV16Chunk, 1024);
        const uint64_t q0 = sdesc<K::kSwizzle>(smem_addr(sQ), 16, K::kGroup);
        int np = -1, left = 0;   // the next tile's part, its tiles from that one on
        bool first = true;       // the next tile is its part's first
        auto advance = [&]() {   // to the next tile; false at the end
            if (left == 0) {
                if (!take_part(sm, np + 1, part)) return false;
                ++np;
                left = part.tiles;
                first = true;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[np % kParts]));
            }
            --left;
            return true;
        };
        // A shared-memory access by the issuing warp holds back the products that follow, so
        // within a part it meets only named barriers: the warps of the values come to each
        // half's barrier once those and (the second half's) the next tile's keys are there, and
        // give the part's queries free once its first keys are.
        // Step T: the products of tile T's halves (none for T = -1), then S of tile T + 1.
        bool more = advance(), fresh = true;
#pragma unroll 1
        for (int T = -1; more || T >= 0; ++T) {
            if (T >= 0) {
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    named_bar_sync(kBarP + half, 224);
                    if (lane == 0) {
                        tc_fence_after();
                        const uint64_t vd = v0 + static_cast<uint64_t>((half % K::kV16Bufs * K::kV16Bytes) >> 4);
#pragma unroll
                        for (int kk = 0; kk < kHalf / 16; ++kk)
                            mma_ts(tmem + 128, tmem + kHalf * half + 8 * kk, vd + ((kk * 2048) >> 4), kIdescO,
                                   (!fresh || half > 0 || kk > 0) ? 1u : 0u);
                        mma_commit(smem_addr(&sm.o_half[half]));
                    }
                    __syncwarp();
                }
                if (!more) break;
            }
            if (lane == 0) {
                const int it = 4 * T + 4, st = it % kSlots;   // the keys' two slots are neighbours
                if (first) wait(&sm.q_full, np);   // (the part's first keys too)
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
                mma_commit(smem_addr(&sm.kv_empty[st + 1]));
                if (left == 0) mma_commit(smem_addr(&sm.q_empty));
            }
            __syncwarp();
            fresh = first;   // tile T + 1 is its part's first
            first = false;
            more = advance();
        }
        if (lane == 0) {
            mma_commit(smem_addr(&sm.all_done));
            mbar_wait_drain(smem_addr(&sm.all_done), 0, kDrainCycles);
        }
        __syncwarp();
    } else if (warp < 4) {
        // ----------------------------------------------------- queries and values
        const int t = threadIdx.x - 64;
        int T = 0;
        bool ok = true;
#pragma unroll 1
        for (int np = 0; take_part(sm, np, part); ++np) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[np % kParts]));
            if (np > 0) ok = __all_sync(0xffffffffu, ok && wait(&sm.q_empty, np - 1));
            cut_rows<D, E>(p, sm.q_next, sm.q_scale, sQ, part.req.start, part.req.n, part.h, part.row0);
            // All keys are waited for here, tile after tile, so that no wait can take an older phase
            // of their place for theirs (it looks at the parity; the first keys may land behind the
            // first values, so having those is not enough), and before S gives the place back.
            auto keys = [&](int ik) {
                return __all_sync(0xffffffffu, wait(&sm.kv_full[ik % kSlots], ik / kSlots) &&
                                                   wait(&sm.kv_full[ik % kSlots + 1], ik / kSlots));
            };
            if (ok) ok = keys(4 * T);
            fence_proxy_async_smem();
            mbar_arrive(smem_addr(&sm.q_full));
            // Values: a unit of 16 codes becomes two of 8 fp16 numbers.  A key's D / 16 units
            // are D / 16 threads', so that a warp reads whole rows.
            // (the threads of the upper 64 channels have the neighbouring row: 8 lanes' stores
            // then fall into different banks)
            constexpr int kPer = D / 16;
            const int vu = t % kPer, row0 = t / kPer ^ vu / 4;
#pragma unroll 1
            for (int i = 0; i < part.tiles; ++i, ++T) {
                const int sc = T % kScaleSlots;
                if (ok) ok = __all_sync(0xffffffffu, wait(&sm.scales_full[sc], T / kScaleSlots));
                const float ks = sm.scales[sc][lane & 7], vs = sm.scales[sc][8 + (lane & 7)];
                const bool gone = vs < 0.f, absent = __any_sync(0xffffffffu, gone);
                if (warp == 2) {
                    const uint32_t vb = __float_as_uint(vs);
                    float lvs = static_cast<float>(static_cast<int>(vb >> 23) - 127);
                    float inv = __uint_as_float((254u << 23) - vb);
                    if ((vb & 0x7fffffu) != 0 || vb < 0x00800000u || vb > 0x7e000000u) {
                        // not a power of two, or one without a normal inverse
                        lvs = log2f(vs);
                        inv = 1.f / vs;
                    }
                    if (lane < 8) sm.ready[sc][lane] = gone ? make_float4(0.f, 0.f, -1.f, 0.f) : make_float4(ks, lvs, inv, 0.f);
                    if (lane == 0) sm.absent[sc] = absent ? 1 : 0;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sm.ready_full[sc]));
                }
                const int kt = (part.tile0 + i) * kKeys;
                const bool edge = absent || kt < part.all_lo || kt + kKeys - 1 > part.all_hi;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const int it = 4 * T + 2 + half, st = it % kSlots;
                    if (ok) ok = __all_sync(0xffffffffu, wait(&sm.kv_full[st], it / kSlots));
                    // the place's last values have been multiplied (see there, kBarP)
                    const int o = K::kV16Bufs == 2 ? half : half ^ 1, use = K::kV16Bufs == 2 || half == 0 ? T - 1 : T;
                    if (use >= 0) wait_for_issuer(&sm.o_half[o], use);
                    if (ok) {
                        uint8_t* src = sKV + st * K::kSlotBytes;
                        uint8_t* dst = sV + half % K::kV16Bufs * K::kV16Bytes + vu / 4 * K::kV16Chunk;
                        if (edge) {
                            // 0 * NaN is NaN: no row's product may meet a NaN that it does not see.
                            // Values that no row sees count as zeros (their place may hold
                            // anything); where some rows see a NaN and others do not, it counts as
                            // zero too, and its channel becomes NaN at the part's end for the rows
                            // that see it.
#pragma unroll 1
                            for (int key = row0; key < kHalf; key += 64 / kPer) {
                                uint4* at = reinterpret_cast<uint4*>(src + unit_offset<D>(key, vu));
                                const int pos = kt + half * kHalf + key;
                                const bool hidden = sm.scales[sc][8 + half * 4 + key / 16] < 0.f ||
                                                    pos < part.lo_key || pos > part.hi_key || pos >= part.req.len;
                                if (hidden) {
                                    *at = make_uint4(0, 0, 0, 0);
                                } else if (pos < part.all_lo || pos > part.all_hi) {
                                    uint4 w = *at;
                                    const uint32_t a = nan_bytes(w.x), b = nan_bytes(w.y), e = nan_bytes(w.z),
                                                   f = nan_bytes(w.w);
                                    if (a | b | e | f) {
                                        w.x &= ~(a | (a - (a >> 7)));
                                        w.y &= ~(b | (b - (b >> 7)));
                                        w.z &= ~(e | (e - (e >> 7)));
                                        w.w &= ~(f | (f - (f >> 7)));
                                        *at = w;
                                        sm.poison[np & 1] = 1;
                                    }
                                }
                            }
                        }
                        uint4 w[kPer];
#pragma unroll
                        for (int j = 0; j < kPer; ++j)
                            w[j] = *reinterpret_cast<const uint4*>(src + unit_offset<D>(row0 + j * (64 / kPer), vu));
#pragma unroll
                        for (int j = 0; j < kPer; ++j) {
                            const int key = row0 + j * (64 / kPer);
                            uint4 x, y;
                            widen4(w[j].x, x.x, x.y);
                            widen4(w[j].y, x.z, x.w);
                            widen4(w[j].z, y.x, y.y);
                            widen4(w[j].w, y.z, y.w);
                            *swizzled_unit(dst, key, vu % 4 * 2) = x;
                            *swizzled_unit(dst, key, vu % 4 * 2 + 1) = y;
                        }
                    }
                    fence_proxy_async_smem();
                    named_bar_sync(kBarConv, 64);   // both warps have read the slot
                    if (t == 0 && ok) mbar_arrive(smem_addr(&sm.kv_empty[st]));   // (its copy has landed)
                    if (half == 1 && i + 1 < part.tiles && ok) ok = keys(4 * T + 4);   // for the issuer
                    named_bar_arrive(kBarP + half, 224);
                }
            }
        }
    } else {
        // -------------------------------------------------------------- softmax
        const int quad = warp - 4, row = quad * 32 + lane;   // TMEM lane
        const uint32_t tS0 = tmem + (static_cast<uint32_t>(quad * 32) << 16), tO = tS0 + 128;
        const int G = p.seq.group;
        int T = 0;   // tiles
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
            const int lo = first_key(p.seq.window, pos_row);
            if (np > 0) ok = __all_sync(0xffffffffu, ok && wait(&sm.q_empty, np - 1));
            cut_rows<D, E>(p, sm.q_next, sm.q_scale, sQ, part.req.start, part.req.n, part.h, part.row0);
            fence_proxy_async_smem();
            mbar_arrive(smem_addr(&sm.q_full));
            ok = __all_sync(0xffffffffu, ok && wait(&sm.q_full, np));
            const float rowc = sm.q_scale[row] * p.scale_log2;   // the row's scale, and the exponent's
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.q_empty));
            // a warp without rows leaves its part of P as it is (rows of O that nobody reads)
            const bool idle = part.row0 + quad * 32 >= part.req.n * G;
            float l = 0.f, ref = kNone;   // the exponents' offset: M - kShift
#pragma unroll 1
            for (int i = 0; i < part.tiles; ++i, ++T) {
                const int sc = T % kScaleSlots;
                const int kt = (part.tile0 + i) * kKeys;
                if (ok && !idle) ok = __all_sync(0xffffffffu, wait(&sm.ready_full[sc], T / kScaleSlots));
                const bool absent = sm.absent[sc] != 0;   // a block on a page that the cache does not have, or behind the last key
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const uint32_t tS = tS0 + kHalf * half;
                    const int kb = kt + kHalf * half;
                    const float4* ready = &sm.ready[sc][4 * half];
                    const bool edge = absent || kb < part.all_lo || kb + kHalf - 1 > part.all_hi;
                    if (!idle && half == 0) wait_for_issuer(&sm.s_full, T);
                    if (ok && !idle) {
                        tc_fence_after();
                        if (edge) {
                            // hidden keys' products become -inf
                            const int clo = lo - kb, chi = min(hi, part.req.len - 1) - kb;
#pragma unroll 1
                            for (int c0 = 0; c0 < kHalf; c0 += 16) {
                                const bool gone = ready[c0 / 16].z < 0.f;
                                uint32_t x[16];
                                tmem_ld16(tS + c0, x);
                                tmem_ld_wait();
                                reg_fence(x);
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    if (c0 + j < clo || c0 + j > chi || gone) x[j] = 0xff800000u;
                                tmem_st16(tS + c0, x);
                            }
                            tmem_st_wait();
                        }
                        uint32_t h[32];
                        float sum[4];
                        // Weights 2^(t - M + kRowsShift) (M = 0 of a row that has no reference yet).  They
                        // are computed before it is known that no row's reference has to move, so
                        // that the exponentials do not wait for the maxima; where one has, they
                        // are computed again from the products.
#pragma unroll 1
                        for (bool again = false;; again = true) {
                            const bool none = ref == kNone;
                            const float base = none ? 0.f : ref;
                            float s[64];
                            tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                            tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
                            tmem_ld_wait();
                            reg_fence(*reinterpret_cast<uint32_t(*)[64]>(&s[0]));
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                const float4 rd = ready[b];
                                const float off = rd.y - base;
                                float kc = rd.x * rowc;
                                if (kc < 1e-30f) kc = 1e-30f;   // (0 * -inf is NaN; no product is that large)
                                const uint64_t c2 = f2_pack(kc, kc), o2 = f2_pack(off, off);
#pragma unroll
                                for (int c = 16 * b; c < 16 * b + 16; c += 2) {
                                    const float2 e = f2_unpack(f2_fma(f2_pack(s[c], s[c + 1]), c2, o2));
                                    s[c] = e.x;
                                    s[c + 1] = e.y;
                                }
                            }
                            float top4[4];
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                uint64_t sum2[2];
                                top4[b] = s[16 * b];
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const int c = 16 * b + 2 * j;
                                    const float w0 = ex2_approx(s[c]), w1 = ex2_approx(s[c + 1]);
                                    top4[b] = fmax3(top4[b], s[c], s[c + 1]);
                                    const uint64_t w2 = f2_pack(w0, w1);
                                    sum2[j & 1] = j < 2 ? w2 : f2_add(sum2[j & 1], w2);
                                    h[8 * b + j] = pack2<kElemF16>(w0, w1);
                                }
                                const float2 both = f2_unpack(f2_add(sum2[0], sum2[1]));
                                sum[b] = both.x + both.y;
                            }
                            const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                            const bool moves = none ? top > kNegInf : top > kRowsShift + kRowsGrow;
                            if (again || !__any_sync(0xffffffffu, moves)) break;
                            // the row's reference moves up to its largest key
                            const float by = moves ? kRowsShift - top : 0.f;
                            const float f = none ? 1.f : ex2_approx(by);
                            l *= f;
                            if (moves) ref = base - by;
                            if (i > 0 || half > 0) {
                                // The last tile's products were complete before this tile's S; the
                                // first half's is waited for.
                                if (half == 1) ok = __all_sync(0xffffffffu, wait(&sm.o_half[0], T));
                                tc_fence_after();
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
#pragma unroll
                        for (int b = 0; b < 4; ++b) l = fmaf(sum[b], ready[b].z, l);
                        tmem_st32(tS, h);
                        tmem_st_wait();
                        tc_fence_before();
                    }
                    named_bar_signal(kBarP + half, 224, !idle);
                }
            }
            // ------------------------------------------------ the part's end
            wait_for_issuer(&sm.o_half[1], T - 1);   // (a warp may have no rows in the next part: kBarP)
            tc_fence_after();
            bool poison = false;
            if (part.tile0 * kKeys < part.all_lo || (part.tile0 + part.tiles) * kKeys - 1 > part.all_hi) {
                // (parts with no such edge set no poison)
                named_bar_sync(kBarRows, 128);
                poison = sm.poison[np & 1] != 0;
                named_bar_sync(kBarRows, 128);
                if (row == 0) sm.poison[np & 1] = 0;
            }
            if (ok) {
                const bool whole = part.whole;
                const float mul = !whole ? 1.f : l != 0.f ? 1.f / l : 0.f;   // (NaN divides on)
                const long long slot = (2LL * blockIdx.x + (part.begins ? 1 : 0)) * kRows + row;
                const bool in = real && fa_index_ok(token, p.seq.total_tokens, p.status);
                uint16_t* out = static_cast<uint16_t*>(p.o) + (token * p.seq.Hq + head) * D;
                float* partial = p.part_o + slot * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t x[32];
                    tmem_ld32(tO + c, x);
                    tmem_ld_wait();
                    reg_fence(x);
                    if (in && whole) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint32_t y[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                y[j] = pack2<E>(__uint_as_float(x[8 * u + 2 * j]) * mul,
                                                __uint_as_float(x[8 * u + 2 * j + 1]) * mul);
                            *reinterpret_cast<uint4*>(out + c + 8 * u) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    } else if (in) {
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            *reinterpret_cast<uint4*>(partial + c + 4 * u) =
                                make_uint4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
                    }
                }
                if (poison && in) spoil_row<D>(p, part, lo, hi, whole ? out : nullptr, whole ? nullptr : partial);
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
