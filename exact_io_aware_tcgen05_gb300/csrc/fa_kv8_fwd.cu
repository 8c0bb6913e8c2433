// fa_kv8_fwd.cu -- attention of new tokens over the paged 8-bit cache (fa_fwd_kv8 in
// include/fa.h) on sm_103a.
//
// A request's rows are its (new token, head of the group) pairs: they share a key/value
// head and take one pass over its keys together, up to C = 8 or 16 rows.  (Requests with more
// rows go to the kernel of fa_kv8_rows.cu; this file launches both.)  With so few rows the cache's bytes bound the pass (16 operations a byte at 8 rows and d = 128, too
// many for the CUDA cores, few for the tensor cores), so nothing is done to a code but to
// load it: TMA copies pages into shared memory and tcgen05 (kind::f8f6f4) multiplies them
// as they are.  The products are transposed, keys and channels on the 128 rows of an MMA
// tile, the few query rows on its columns:
//   S^T [128 keys x C] = K [128 x d] Q^T         K as stored, K-major
//   O^T [d x C]       += V^T [d x 128] P^T       V as stored, read MN-major
// so that a tile costs 128 x C products, every lane of a softmax warp has a key of its own
// (with its own scales, mask and page), and the running maxima are over lanes.
//
// Exactness.  The 8-bit products are exact and summed in fp32, but q and P have more bits
// than a code, so each goes in as a sum of codes:
//   q   each row times a power of two, so that its largest element is in (224, 448], as 2
//       (bf16) or 3 (fp16) e4m3 pieces of 4 bits, each piece the rounding of what the ones
//       before it left.  The last piece's least step is 2^-9, so an element whose last bit is
//       2^-9 or more is exact (elements of 2^-2 or more for bf16's 8 bits, of 2 or more for
//       fp16's 11), and a smaller one is off by 2^-10 at most, 2^-17.8 of the row's largest;
//   P   as fp16 (11 bits), cut into e5m2 pieces of 3 bits (the high byte of an fp16 number
//       is an e5m2 number): 3 pieces for bf16 outputs, the last one rounded (9 bits, one
//       more than bf16 holds), 4 for fp16 (all 11).  e5m2 rather than e4m3 because long
//       contexts need its range: weights are kept down to 2^-28 of the largest.
// V's scale joins the exponent: with t_j = s_j + log2(v_scale_j) and M the running maximum
// of t (or a little less, see kGrow), the weights 2^(t_j - M) are near 1 at most whatever the
// scales, and the sum of the probabilities is that of 2^(t_j - M) / v_scale_j.  In 32 bits that
// bounds V's scales.  With R = log2(largest / least scale), a key whose t is 123 or more below
// the largest (as far as a weight, or the factor that moves a reference, stays a normal number)
// has at most 2^(R - 123) of the probability of the key with the largest, so n such keys are
// nothing beside it (2^-24) up to R = 99 - log2(n); and a sum of n weights of up to 2^15 over
// scales of 2^-80 or more stays below 2^(95 + log2(n)).
//
// Work split.  The key tiles of all items (request, key/value head, C rows) lie one behind
// the other and every CTA, two per SM, takes an equal share of them (kItemCost more tiles
// stand for an item's fixed cost), wherever items begin and end; a CTA's share begins and
// ends inside at most two items, whose parts go to the workspace, and a second small
// kernel, launched with this one (programmatic dependence), joins them.  All lengths are
// read on the device, and the CTAs find their shares themselves.
//
// One CTA: 8 warps,
//   warp 0       producer: pages by TMA, K and V in turn through one ring of slots, the
//                tile's 16 scales by 4-byte asynchronous copies
//   warp 1       tcgen05 issuer; owns the TMEM allocation.  S^T of the next tile is issued
//                before the weights of this one are ready (two S^T buffers)
//   warp 2       the items' queries: scaled, cut into pieces, into shared memory
//   warp 3       relay: waits for what the issuer's next products read, so that the issuer
//                itself meets only named barriers (a shared-memory access by the issuing warp
//                holds the products that follow back)
//   warps 4..7   softmax: a lane has a key
// The second CTA of the SM works while this one waits at the ends of items.
//
// Measured (one GB300; bytes of the codes and scales that are seen): 2 requests of 131072 tokens
// (Hkv 16, d = 128) 163 us, 97 % of the measured copy rate; 64 requests of up to 8192 (Hkv 8)
// 79 us, 84 %; 128 of up to 2048 at d = 64, fp16, pages of 16, 41 us, 36 %; one request of 1000
// 10 us on the GPU, 24 to 32 for the whole call from Python, whose host side is the longer one.
// With 16 rows in place of 8 a tile's softmax takes twice the instructions and keeps some 50
// bytes a thread in local memory: 64 requests of up to 8192 with 16 heads a group 93 us (60 % of
// the measured copy rate; 67 us, 79 %, with 8 heads; 113 us with 17, in the 128-row kernel), 128
// of up to 2048 at d = 64, fp16, 69 us (40 with 8).  Long contexts are bound by the cache's bytes.
// Short ones are bound by a tile's and an item's instructions in the warps that handle them, at
// d = 64 twice as many for each byte: the producer has some 2000 cycles of work a tile
// (fa_kv8_work.cuh), the softmax 1700, and an item's start and end 5000.  A third CTA per SM (80
// registers a thread) took 59 us in place of 44 there, items of 32 rows in this kernel more than
// the 128-row kernel for the same rows.
// One request: two launches, the search for the shares, one item's chain and the join.
#include "fa_kv8_work.cuh"

#include <algorithm>

namespace fa {
namespace {

using namespace kv8;

// --------------------------------------------------------------------- configuration

template <int D, int E, int C>
struct Kv8Cfg {
    static constexpr int kQ = E == kElemBf16 ? 2 : 3;    // pieces of q
    static constexpr int kP = E == kElemBf16 ? 3 : 4;    // pieces of P
    // With few columns an MMA costs the reading of its 128 rows, so the pieces of q and of P
    // go side by side into one MMA of more columns (a multiple of 16, the rest zeros) and
    // are added up when read.
    static constexpr int kSCols = (kQ * C + 15) / 16 * 16;
    static constexpr int kPCols = (kP * C + 15) / 16 * 16;
    static constexpr int kTmemUsed = 2 * kSCols + kPCols;
    static constexpr int kTmemCols = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : 256;
    static_assert(kTmemUsed <= 256, "TMEM columns, two CTAs per SM");
    static constexpr int kSlotBytes = kKeys * D;         // K or V of a tile
    static constexpr int kQBytes = kSCols * D;           // one item's queries
    static constexpr int kPBytes = kPCols * kKeys;       // a tile's weights
    static constexpr int kSwizzle = D == 128 ? 2 : 4;    // descriptor code of the D-byte swizzle
    static constexpr int kGroup = 8 * D;                 // bytes of 8 rows
};

template <int C>
struct Kv8Smem {   // behind the tiles
    float scales[kScaleSlots][16];   // of a tile: K's 8 blocks, V's 8 (V < 0: hidden)
    alignas(16) float q_scale[2][C];
    int row_pos[2][C];               // position of the row's token; INT_MIN: no row
    long long out_at[2][C], lse_at[2][C];
    float wmax[2][4][C];             // [tile parity][warp]
    alignas(16) float ref[4][C];     // [warp]
    alignas(16) float fac[4][C];
    float part_sum[2][4][C];         // [part parity][warp]
    int3 window[kWindow];
    Share share;
    Part parts[kParts];
    long long warp_sums[kThreads / 32];
    uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots], scales_full[kScaleSlots];
    uint64_t part_full[kParts], part_empty[kParts];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], pv_done[2];  // [tile parity]
    uint64_t all_done;
    uint32_t tmem;
    int abort;
    int poison[2];                   // [part parity] NaN found among values that only some rows see
};

template <int D, int E, int C>
constexpr int kv8_slots() {
    using K = Kv8Cfg<D, E, C>;
    const int left = kCtaSmem - 1024 - 2 * (K::kQBytes + K::kPBytes) - static_cast<int>(sizeof(Kv8Smem<C>));
    const int n = left / K::kSlotBytes;
    return n < kMaxSlots ? n : kMaxSlots;
}

template <int D, int E, int C>
constexpr int kv8_smem_bytes() {
    using K = Kv8Cfg<D, E, C>;
    return 1024 + kv8_slots<D, E, C>() * K::kSlotBytes + 2 * (K::kQBytes + K::kPBytes) +
           static_cast<int>(sizeof(Kv8Smem<C>));
}

// named barriers (0 is __syncthreads)
constexpr int kBarP = 1;      // weights written, or not fitting; the softmax warps and the issuer
constexpr int kBarK = 3;      // the next tile's keys (and queries) and this one's values are there
constexpr int kBarMax = 2;    // the softmax warps' maxima (or a part's sums) written

// Sums of v[0 .. N) over the warp's lanes, by halving: lane l ends with the sum of column
// l / (32 / N) in v[0].
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N], int lane) {
    int width = N;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (width > 1) {
            // the upper half of the lanes keeps the upper half of the columns
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i < width / 2) {
                    const float give = up ? v[i] : v[i + width / 2];
                    const float keep = up ? v[i + width / 2] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            }
            width /= 2;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
}

// 8 TMEM columns, several sets added up.
template <int SETS>
__device__ __forceinline__ void load_sum8(uint32_t addr, int stride, float (&v)[8]) {
    uint32_t r[SETS][8];
#pragma unroll
    for (int i = 0; i < SETS; ++i)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[i][0]), "=r"(r[i][1]), "=r"(r[i][2]), "=r"(r[i][3]), "=r"(r[i][4]),
                       "=r"(r[i][5]), "=r"(r[i][6]), "=r"(r[i][7])
                     : "r"(addr + i * stride));
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < SETS; ++i) reg_fence(r[i]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        v[c] = __uint_as_float(r[0][c]);
#pragma unroll
        for (int i = 1; i < SETS; ++i) v[c] += __uint_as_float(r[i][c]);
    }
}

// A key's weights into its rows of the P operand, cut into KP e5m2 pieces: an fp16 number's
// high byte is its leading 3 bits as e5m2, and what is left is an fp16 number again.  The
// last of 3 pieces is rounded; the fourth is all that is left.  The pieces' columns lie one
// behind the other in blocks of 16 (kKeys * 16 bytes each), zeros behind the last.
template <int KP, int C>
__device__ __forceinline__ void store_weights(uint8_t* at, const float (&w)[C]) {
    uint32_t h[C / 2], words[(KP * C + 15) / 16 * 4];
#pragma unroll
    for (int j = 0; j < C / 2; ++j) h[j] = pack2<kElemF16>(w[2 * j], w[2 * j + 1]);
#pragma unroll
    for (int j = KP * C / 4; j < (KP * C + 15) / 16 * 4; ++j) words[j] = 0;
#pragma unroll
    for (int q = 0; q < KP; ++q) {
#pragma unroll
        for (int j = 0; j < C / 2; ++j)
            if (KP == 3 && q == 2) h[j] += 0x00800080u;
#pragma unroll
        for (int j = 0; j < C / 4; ++j) words[q * (C / 4) + j] = __byte_perm(h[2 * j], h[2 * j + 1], 0x7531);
#pragma unroll
        for (int j = 0; j < C / 2; ++j)
            if (q + 1 < KP) h[j] = sub_f16x2(h[j], h[j] & 0xff00ff00u);
    }
#pragma unroll
    for (int b = 0; b < (KP * C + 15) / 16; ++b)
        *reinterpret_cast<uint4*>(at + b * kKeys * 16) =
            make_uint4(words[4 * b], words[4 * b + 1], words[4 * b + 2], words[4 * b + 3]);
}

// Which of the columns n0 .. n0 + 7 see a NaN code in this channel of a value that other
// columns do not see, among the part's keys (a bit each).  Rare: the codes are read again.
template <int D, int C>
__device__ __noinline__ uint32_t find_nan(const Kv8FwdParams& p, const Part& part, const Kv8Smem<C>& sm,
                                          int buf, int n0, int channel) {
    uint32_t spoilt = 0;
    const int first = part.tile0 * kKeys, past = first + part.tiles * kKeys;
    for (int j = max(first, part.lo_key); j < min(past, part.hi_key + 1); ++j) {
        if (j >= part.all_lo && j <= part.all_hi) {
            j = part.all_hi;   // seen by all: the product has it
            continue;
        }
        const int id = p.table[static_cast<long long>(part.b) * p.width + (j >> p.page_log2)];
        if (id < 0 || id >= p.num_pages) continue;
        const long long r = ((static_cast<long long>(id) * p.seq.Hkv + part.h) << p.page_log2) +
                            (j & ((1 << p.page_log2) - 1));
        if ((p.v8[r * D + channel] & 0x7f) != 0x7f) continue;
        for (int n = 0; n < 8; ++n) {
            const int rp = sm.row_pos[buf][n0 + n];
            if (j <= rp && (p.seq.window <= 0 || rp - j < p.seq.window)) spoilt |= 1u << n;
        }
    }
    return spoilt;
}

// F32: O in fp32 (one of two parts that another kernel joins)
template <int D, int E, int C, bool F32>
__global__ void __launch_bounds__(kThreads, 2) fa_fwd_kv8_kernel(const __grid_constant__ Kv8FwdParams p) {
    using K = Kv8Cfg<D, E, C>;
    constexpr int kSlots = kv8_slots<D, E, C>();
    static_assert(kSlots >= 4 && kSlots / 2 + 2 < kScaleSlots, "ring of key/value tiles");
    // S^T: K e4m3 (K-major) times q's pieces e4m3 (K-major); O^T: V e4m3 (MN-major) times P's
    // pieces e5m2 (MN-major; operand format code 1)
    constexpr uint32_t kIdescS = idesc_f32acc(kKeys, K::kSCols, false, false, kElemFp8);
    constexpr uint32_t kIdescO = idesc_f32acc(128, K::kPCols, true, true, kElemFp8) | (1u << 10);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sKV = smem;                                  // [slots]
    uint8_t* sQ = smem + kSlots * K::kSlotBytes;          // [2][pieces and rows][D]
    uint8_t* sP = sQ + 2 * K::kQBytes;                    // [2][blocks of 16 columns][keys][16]
    Kv8Smem<C>& sm = *reinterpret_cast<Kv8Smem<C>*>(sP + 2 * K::kPBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    grid_launch_dependents();

    if (threadIdx.x == 0) {
        sm.abort = 0;
        sm.poison[0] = sm.poison[1] = 0;
#pragma unroll 1
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_addr(&sm.kv_full[i]), 1);
            mbar_init(smem_addr(&sm.kv_empty[i]), 1);
        }
#pragma unroll 1
        for (int i = 0; i < kScaleSlots; ++i) mbar_init(smem_addr(&sm.scales_full[i]), 32);
        for (int i = 0; i < kParts; ++i) {
            mbar_init(smem_addr(&sm.part_full[i]), 1);
            mbar_init(smem_addr(&sm.part_empty[i]), 7);   // every warp but the producer
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sm.q_full[i]), 32);
            mbar_init(smem_addr(&sm.q_empty[i]), 5);    // the last S^T of the part, 4 softmax warps
            mbar_init(smem_addr(&sm.s_full[i]), 1);
            mbar_init(smem_addr(&sm.pv_done[i]), 1);
        }
        mbar_init(smem_addr(&sm.all_done), 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&sm.tmem), K::kTmemCols);
        tmem_relinquish();
    }
    if constexpr (K::kSCols > K::kQ * C) {   // the columns behind the pieces
        constexpr int kPad = (K::kSCols - K::kQ * C) * D / 16;
        for (int i = threadIdx.x; i < 2 * kPad; i += kThreads)
            *reinterpret_cast<uint4*>(sQ + i / kPad * K::kQBytes + K::kQ * C * D + i % kPad * 16) =
                make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    // what the kernels before this one wrote is there from here on
    grid_dependency_wait();
    find_share<C>(p, sm);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const uint32_t colO = tmem + 2 * K::kSCols;

    auto wait = [&](uint64_t* bar, int phase) { return wait_for(p, sm, bar, phase); };
    auto take = [&](int np, Part& part) { return take_part(sm, np, part); };
    Part part;

    if (warp == 0) {
        produce<D, C, kKeys, kSlots, F32>(p, sm, sKV);
    } else if (warp == 1) {
        // --------------------------------------------------------------- issuer
        // Walks the tiles of all parts one behind the other, one tile ahead with S^T.  After
        // an abort it goes on issuing on stale data, so that every barrier's phases still
        // complete.
        const uint64_t kv0 = sdesc<K::kSwizzle>(smem_addr(sKV), 16, K::kGroup);
        // V: the second half of the 128 rows of the product at d = 64 reads the next keys'
        // channels and is not used
        const uint64_t v0 = sdesc<K::kSwizzle>(smem_addr(sKV), K::kGroup, K::kGroup);
        const uint64_t qd0 = sdesc<K::kSwizzle>(smem_addr(sQ), 16, K::kGroup);
        const uint64_t pd0 = sdesc<0>(smem_addr(sP), 128, kKeys * 16);
        int np = -1, left = 0;   // the part of the next tile, its tiles from that one on
        bool first = true;
        auto advance = [&]() {   // to the next tile; false at the end
            if (left == 0) {
                if (!take(np + 1, part)) return false;
                ++np;
                left = part.tiles;
                first = true;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[np % kParts]));
            }
            --left;
            return true;
        };
        bool more = advance(), fresh = true;
        if (more) named_bar_sync(kBarK, 64);
        // Step T: S^T of tile T + 1, then (for T >= 0) the product with tile T's weights.
#pragma unroll 1
        for (int T = -1; more || T >= 0; ++T) {
            if (lane == 0 && more) {
                const int st = (2 * T + 2) % kSlots, buf = (T + 1) & 1;
                tc_fence_after();
                const uint64_t kd = kv0 + static_cast<uint64_t>((st * K::kSlotBytes) >> 4);
                const uint64_t qd = qd0 + static_cast<uint64_t>(((np & 1) * K::kQBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                    mma_ss_f8(tmem + buf * K::kSCols, kd + 2 * kk, qd + 2 * kk, kIdescS, kk > 0 ? 1u : 0u);
                mma_commit(smem_addr(&sm.s_full[buf]));
                mma_commit(smem_addr(&sm.kv_empty[st]));
                if (left == 0) mma_commit(smem_addr(&sm.q_empty[np & 1]));
            }
            __syncwarp();
            if (T >= 0) {
#pragma unroll 1
                while (!named_bar_all(kBarP, 160, true)) {}   // until the weights fit
                if (lane == 0) {
                    const int st = (2 * T + 1) % kSlots;
                    tc_fence_after();
                    const uint64_t vd = v0 + static_cast<uint64_t>((st * K::kSlotBytes) >> 4);
                    const uint64_t pd = pd0 + static_cast<uint64_t>(((T & 1) * K::kPBytes) >> 4);
#pragma unroll
                    for (int kk = 0; kk < kKeys / 32; ++kk)
                        mma_ss_f8(colO, vd + ((kk * 32 * D) >> 4), pd + ((kk * 512) >> 4), kIdescO,
                                  (!fresh || kk > 0) ? 1u : 0u);
                    mma_commit(smem_addr(&sm.pv_done[T & 1]));
                    mma_commit(smem_addr(&sm.kv_empty[st]));
                }
                __syncwarp();
                if (!more) break;
            }
            fresh = first;   // tile T + 1 is its part's first
            first = false;
            more = advance();
            named_bar_sync(kBarK, 64);   // keys of tile T + 2, values of tile T + 1
        }
        if (lane == 0) {
            mma_commit(smem_addr(&sm.all_done));
            mbar_wait_drain(smem_addr(&sm.all_done), 0, kDrainCycles);
        }
        __syncwarp();
    } else if (warp == 2) {
        // -------------------------------------------------------------- queries
        constexpr int kLanes = D / 8;         // threads of a row
        constexpr int kRows = 32 / kLanes;    // rows at a time
        const int t = lane, sub = t % kLanes;
        bool ok = true;
#pragma unroll 1
        for (int np = 0; take(np, part); ++np) {
            const int buf = np & 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[np % kParts]));
            if (np >= 2) ok = __all_sync(0xffffffffu, ok && wait(&sm.q_empty[buf], (np >> 1) - 1));
            if (ok) {
                uint8_t* dst = sQ + buf * K::kQBytes;
                const int G = p.seq.group, rows = part.req.n * G;
                constexpr int kPasses = C / kRows;
                uint4 w[kPasses];
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int n = t / kLanes + i * kRows;
                    const int tok = small_div(n, G, p.group_inv);   // (a request's rows are one item)
                    const long long token = part.req.start + tok;
                    const int head = part.h * G + n - tok * G;
                    w[i] = make_uint4(0, 0, 0, 0);
                    if (n < rows)
                        w[i] = *reinterpret_cast<const uint4*>(
                            static_cast<const uint16_t*>(p.q) + token * p.q_stride + head * D + sub * 8);
                    if (sub == 0) {
                        sm.row_pos[buf][n] = n < rows ? part.req.len - part.req.n + tok : INT_MIN;
                        sm.out_at[buf][n] = (token * p.seq.Hq + head) * D;
                        sm.lse_at[buf][n] = row_stat_index(p.seq, part.b, head, part.req.start, tok);
                    }
                }
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int n = t / kLanes + i * kRows;
                    const float scale = cut_queries<D, E, K::kQ>(
                        w[i], dst + unit_offset<D>(n, sub >> 1) + (sub & 1) * 8, C * D);
                    if (sub == 0) sm.q_scale[buf][n] = scale;
                }
            }
            fence_proxy_async_smem();
            // (after an abort the rows' places are not written: nobody may take them for these)
            if (ok) mbar_arrive(smem_addr(&sm.q_full[buf]));
        }
    } else if (warp == 3) {
        // ---------------------------------------------------------------- relay
        int T = 0;
#pragma unroll 1
        for (int np = 0; take(np, part); ++np) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[np % kParts]));
#pragma unroll 1
            for (int i = 0; i < part.tiles; ++i, ++T) {
                if (lane == 0) {
                    if (T > 0) wait(&sm.kv_full[(2 * T - 1) % kSlots], (2 * T - 1) / kSlots);
                    wait(&sm.kv_full[(2 * T) % kSlots], (2 * T) / kSlots);
                    wait(&sm.scales_full[T % kScaleSlots], T / kScaleSlots);
                    if (i == 0) wait(&sm.q_full[np & 1], np >> 1);
                }
                __syncwarp();
                named_bar_sync(kBarK, 64);
            }
        }
        if (T > 0) {
            if (lane == 0) wait(&sm.kv_full[(2 * T - 1) % kSlots], (2 * T - 1) / kSlots);
            __syncwarp();
            named_bar_sync(kBarK, 64);
        }
    } else {
        // -------------------------------------------------------------- softmax
        const int quad = warp - 4, key = quad * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t tO = colO + lane_addr;
        int T = 0;
        bool ok = true;
#pragma unroll 1
        for (int np = 0; take(np, part); ++np) {
            const int buf = np & 1;
            ok = __all_sync(0xffffffffu, ok && wait(&sm.q_full[buf], np >> 1));
            float l[C], ref = kNegInf;   // lane n keeps column n's reference
#pragma unroll
            for (int n = 0; n < C; ++n) l[n] = 0.f;
            const int nrows = min(C, part.req.n * p.seq.group - part.row0);
#pragma unroll 1
            for (int i = 0; i < part.tiles; ++i, ++T) {
                const int sc = T % kScaleSlots;
                // (the relay waited for the scales before it let S^T be issued)
                if (ok) ok = __all_sync(0xffffffffu, wait(&sm.s_full[T & 1], T >> 1));
                float v[C], kc = 0.f, lvs = 0.f, inv_vs = 0.f;
                uint32_t seen = ~0u;   // a bit per column
                const float4* qs = reinterpret_cast<const float4*>(sm.q_scale[buf]);
                const float4* rf = reinterpret_cast<const float4*>(sm.ref[quad]);
                if (ok) {
                    tc_fence_after();
                    const int kb = (part.tile0 + i) * kKeys, pos = kb + key;
                    float ks = sm.scales[sc][key / 16], vs = sm.scales[sc][8 + key / 16];
                    const bool hidden = vs < 0.f || pos < part.lo_key || pos > part.hi_key ||
                                        pos >= part.req.len;
                    const bool edge = kb < part.all_lo || kb + kKeys - 1 > part.all_hi;
#pragma unroll
                    for (int cc = 0; cc < C; cc += 8)
                        if (cc < nrows)
                            load_sum8<K::kQ>(tmem + lane_addr + (T & 1) * K::kSCols + cc, C,
                                             *reinterpret_cast<float(*)[8]>(&v[cc]));
                    tc_fence_before();
                    if (hidden) {
                        ks = 0.f;
                        vs = 1.f;
                    }
                    const uint32_t vb = __float_as_uint(vs);
                    lvs = static_cast<float>(static_cast<int>(vb >> 23) - 127);
                    inv_vs = __uint_as_float((254u << 23) - vb);
                    if ((vb & 0x7fffffu) != 0 || vb < 0x00800000u || vb > 0x7e000000u) {
                        // not a power of two, or one without a normal inverse
                        lvs = log2f(vs);
                        inv_vs = 1.f / vs;
                    }
                    kc = ks * p.scale_log2;
                    if (edge || __any_sync(0xffffffffu, hidden)) {
                        const bool some = !hidden && (pos < part.all_lo || pos > part.all_hi);
                        seen = hidden ? 0u : ~0u;
                        if (some) {
#pragma unroll
                            for (int n = 0; n < C; ++n) {
                                const int rp = sm.row_pos[buf][n];
                                if (pos > rp || (p.seq.window > 0 && rp - pos >= p.seq.window)) seen &= ~(1u << n);
                            }
                        }
                        // 0 * NaN is NaN: no row's product may meet a NaN that it does not
                        // see.  (The values have to be there to be looked at.)
                        const int vi = 2 * T + 1;
                        ok = __all_sync(0xffffffffu, wait(&sm.kv_full[vi % kSlots], vi / kSlots));
                        uint4* vrow = reinterpret_cast<uint4*>(sKV + (vi % kSlots) * K::kSlotBytes + key * D);
                        if (hidden) {
#pragma unroll
                            for (int u = 0; u < D / 16; ++u) vrow[u] = make_uint4(0, 0, 0, 0);
                        } else if (some) {
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
                                    sm.poison[buf] = 1;
                                }
                            }
                        }
                    }
                }
                // The weights 2^(t - M + kShift); at the part's first tile, and where one is
                // too large, new references come first.  The fence and the barrier hand
                // them to the issuer.
                float w[C];
                bool fits = i > 0;
#pragma unroll 1
                for (int attempt = 0;; ++attempt) {
                    if (ok && (attempt > 0 || i > 0)) {
                        float top = kNegInf;
#pragma unroll
                        for (int n4 = 0; n4 < C; n4 += 4)
                            if (n4 < nrows) {
                                const float4 q4 = qs[n4 / 4], r4 = rf[n4 / 4];
                                const float qq[4] = {q4.x, q4.y, q4.z, q4.w}, rr[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    float e = fmaf(v[n4 + j], kc * qq[j], lvs - rr[j]);
                                    if (!((seen >> (n4 + j)) & 1u)) e = kNegInf;
                                    top = fmaxf(top, e);
                                    w[n4 + j] = ex2_approx(e);
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 4; ++j) w[n4 + j] = 0.f;
                            }
                        fits = attempt > 0 || top <= kShift + kGrow;
                        // (tile T - 2's product was complete before this tile's S^T was)
                        store_weights<K::kP, C>(sP + (T & 1) * K::kPBytes + key * 16, w);
                        tc_fence_before();
                        fence_proxy_async_smem();
                    }
                    if ((i > 0 || attempt > 0) && named_bar_all(kBarP, 160, !ok || fits)) break;
                    // the maxima over the tile's keys
                    float mine = kNegInf;
                    if (ok) {
#pragma unroll
                        for (int n4 = 0; n4 < C; n4 += 4)
                            if (n4 < nrows) {
#pragma unroll
                                for (int n = n4; n < n4 + 4; ++n) {
                                    const float m = warp_max((seen >> n) & 1u ? fmaf(v[n], kc * sm.q_scale[buf][n], lvs)
                                                                              : kNegInf);
                                    if (lane == n) mine = m;
                                }
                            }
                        if (lane < C) sm.wmax[T & 1][quad][lane] = mine;
                    }
                    named_bar_sync(kBarMax, 128);
                    if (ok) {
                        // every warp comes to the same references
                        if (lane < C) {
                            const auto& wm = sm.wmax[T & 1];
                            const float m = fmaxf(fmaxf(wm[0][lane], wm[1][lane]), fmaxf(wm[2][lane], wm[3][lane]));
                            float f = 1.f;
                            if (m > ref) {
                                f = ex2_approx(ref - m);
                                ref = m;
                            }
                            sm.fac[quad][lane] = f;
                            sm.ref[quad][lane] = ref == kNegInf ? kNone : ref - kShift;
                        }
                        __syncwarp();
                        if (i > 0) {
                            ok = __all_sync(0xffffffffu, wait(&sm.pv_done[(T - 1) & 1], (T - 1) >> 1));
                            tc_fence_after();
#pragma unroll
                            for (int n = 0; n < C; ++n) l[n] *= sm.fac[quad][n];
#pragma unroll 1
                            for (int cc = 0; cc < K::kPCols; cc += 16) {
                                uint32_t r[16];
                                tmem_ld16(tO + cc, r);
                                tmem_ld_wait();
                                reg_fence(r);
                                const float* fc = &sm.fac[quad][cc % C];
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    r[j] = __float_as_uint(__uint_as_float(r[j]) * fc[C < 16 ? j % C : j]);
                                tmem_st16(tO + cc, r);
                            }
                            tmem_st_wait();
                        }
                    }
                }
                if (ok) {
#pragma unroll
                    for (int n = 0; n < C; ++n) l[n] = fmaf(w[n], inv_vs, l[n]);
                }
            }
            // ------------------------------------------------ the part's end
            // (The last tile's scores were issued before the product of the tile before it, so
            // that one may be running still.  A wait looks at a phase's parity: with one barrier
            // for all products it could take the one before those two for the last.)
            if (ok) ok = __all_sync(0xffffffffu, wait(&sm.pv_done[(T - 1) & 1], (T - 1) >> 1));
            tc_fence_after();
            warp_sums(l, lane);
            constexpr int kSame = 32 / C;   // lanes that hold the same column's sum
            if (lane % kSame == 0) sm.part_sum[buf][quad][lane / kSame] = l[0];
            named_bar_sync(kBarMax, 128);
            const bool poison = sm.poison[buf] != 0;
            if (ok) {
                // lane n: column n's sum, and what its accumulators are multiplied by
                const long long slot = 2LL * blockIdx.x + (part.begins ? 1 : 0);
                if (lane < C) {
                    const float sum = (sm.part_sum[buf][0][lane] + sm.part_sum[buf][1][lane]) +
                                      (sm.part_sum[buf][2][lane] + sm.part_sum[buf][3][lane]);
                    sm.fac[quad][lane] = !part.whole ? 1.f : sum != 0.f ? 1.f / sum : 0.f;   // (NaN divides on)
                    if (quad == 0 && lane < nrows) {
                        if (!part.whole)
                            p.part_stat[slot * C + lane] = make_float2(ref, sum);
                        else if (fa_index_ok(sm.out_at[buf][lane], static_cast<long long>(p.seq.total_tokens) * p.seq.Hq * D, p.status))
                            p.lse[sm.lse_at[buf][lane]] =
                                sum != 0.f ? ((ref == kNegInf ? 0.f : ref) - kShift + log2f(sum)) * kLn2 : kNegInf;
                    }
                }
                __syncwarp();
#pragma unroll 1
                for (int n0 = 0; n0 < nrows; n0 += 8) {
                    float o[8];
                    load_sum8<K::kP>(tO + n0, C, o);
                    uint32_t spoilt = 0;   // columns of these 8 that see a NaN in this channel
                    if (poison && key < D) spoilt = find_nan<D, C>(p, part, sm, buf, n0, key);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int n = n0 + j;
                        float x = o[j] * sm.fac[quad][n];
                        if ((spoilt >> j) & 1u) x = __uint_as_float(0x7fc00000u);
                        if (n >= nrows || key >= D) continue;
                        if (part.whole) {
                            const long long at = sm.out_at[buf][n] + key;
                            if (fa_index_ok(at, static_cast<long long>(p.seq.total_tokens) * p.seq.Hq * D, p.status)) {
                                if (F32) static_cast<float*>(p.o)[at] = x;
                                else static_cast<uint16_t*>(p.o)[at] = static_cast<uint16_t>(pack2<E>(x, 0.f));
                            }
                        } else {
                            p.part_o[(slot * C + n) * D + key] = x;
                        }
                    }
                }
            }
            tc_fence_before();
            if (poison) {   // (uniform) taken back once all have read it; not set again before part np + 2
                named_bar_sync(kBarMax, 128);
                if (key == 0) sm.poison[buf] = 0;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_addr(&sm.q_empty[buf]));
                mbar_arrive(smem_addr(&sm.part_empty[np % kParts]));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, K::kTmemCols);
}

// Joins the parts of the item that begins at the end of CTA c's share, c = blockIdx.x: a warp
// per row, 8 rows a block (16 rows a warp, one behind the other, took 36 us behind a chunk of
// 2048 tokens: a row's loads wait for one another, so rows have to be on their way together).
// Its lanes take 32 parts' references and sums at a time, then the warp adds those parts'
// accumulators up in their order; the first two parts' (there are always two) are on their way
// before their weights are known.
template <int D, int E, bool F32>
__device__ __forceinline__ void join_parts(const Kv8FwdParams& p) {
    const int cta = blockIdx.x;
    const Kv8Join j = p.joins[cta];
    if (j.last <= cta) return;
    const int C = p.columns, G = p.seq.group, lane = threadIdx.x & 31;
    const int n = blockIdx.y * 8 + (threadIdx.x >> 5);
    if (j.row0 + n >= j.n * G) return;
    constexpr int kPer = D / 32;   // channels of a lane, side by side
    using Vec = std::conditional_t<kPer == 4, float4, float2>;
    // the parts: this CTA's second slot, the first slots of the ones behind it
    const int parts = j.last - cta + 1;
    auto row_of = [&](int part) { return (2LL * (cta + part) + (part == 0 ? 1 : 0)) * C + n; };
    auto load = [&](int part, float (&x)[kPer]) {
        *reinterpret_cast<Vec*>(x) = *reinterpret_cast<const Vec*>(p.part_o + row_of(part) * D + kPer * lane);
    };
    alignas(16) float early[2][kPer];
#pragma unroll
    for (int q = 0; q < 2; ++q) load(q, early[q]);
    float m = kNegInf, sum = 0.f;
    alignas(16) float o[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) o[c] = 0.f;
#pragma unroll 1
    for (int p0 = 0; p0 < parts; p0 += 32) {
        float2 st = make_float2(kNegInf, 0.f);
        if (p0 + lane < parts) st = p.part_stat[row_of(p0 + lane)];
        const float top = fmaxf(m, warp_max(st.x)), ref = top == kNegInf ? 0.f : top;
        const float old = ex2_approx(m - ref), mine = ex2_approx(st.x - ref);
        float s = mine * st.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        sum = old * sum + s;
#pragma unroll
        for (int c = 0; c < kPer; ++c) o[c] *= old;
        const int here = min(32, parts - p0);
        int q = 0;
        if (p0 == 0) {
#pragma unroll
            for (; q < 2; ++q) {
                const float f = __shfl_sync(0xffffffffu, mine, q);
#pragma unroll
                for (int c = 0; c < kPer; ++c) o[c] = fmaf(f, early[q][c], o[c]);
            }
        }
#pragma unroll 8
        for (; q < here; ++q) {
            const float f = __shfl_sync(0xffffffffu, mine, q);
            alignas(16) float x[kPer];
            load(p0 + q, x);
#pragma unroll
            for (int c = 0; c < kPer; ++c) o[c] = fmaf(f, x[c], o[c]);
        }
        m = top;
    }
    const int r = j.row0 + n, tok = r / G, head = j.h * G + r % G;
    const long long row = j.start + tok;
    if (!fa_index_ok(row, p.seq.total_tokens, p.status)) return;
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int c = 0; c < kPer; ++c) o[c] *= inv;
    const long long at = (row * p.seq.Hq + head) * D + kPer * lane;
    if (F32) {
        *reinterpret_cast<Vec*>(static_cast<float*>(p.o) + at) = *reinterpret_cast<Vec*>(o);
    } else {
#pragma unroll
        for (int c = 0; c < kPer; c += 2)
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + at + c) = pack2<E>(o[c], o[c + 1]);
    }
    if (lane == 0)
        p.lse[row_stat_index(p.seq, j.b, head, j.start, tok)] =
            sum != 0.f ? ((m == kNegInf ? 0.f : m) - kShift + log2f(sum)) * kLn2 : kNegInf;
}

template <int D, int E>
__global__ void __launch_bounds__(256) fa_fwd_kv8_join_kernel(const __grid_constant__ Kv8FwdParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    join_parts<D, E, false>(p);
}

// The joins of the pass over shared prefixes (z = 0) and of that over the requests' own keys.
template <int D, int E>
__global__ void __launch_bounds__(256) fa_kv8_prefix_parts_kernel(const __grid_constant__ Kv8FwdParams p0,
                                                                  const __grid_constant__ Kv8FwdParams p1) {
    grid_launch_dependents();
    grid_dependency_wait();
    const Kv8FwdParams& p = blockIdx.z == 0 ? p0 : p1;
    if (static_cast<int>(blockIdx.x) < p.ctas && 8 * static_cast<int>(blockIdx.y) < p.columns) join_parts<D, E, true>(p);
}

template <int D, int E, int C, bool F32>
cudaError_t launch_attend(const Kv8FwdParams& p, cudaStream_t stream) {
    constexpr int smem = kv8_smem_bytes<D, E, C>();
    static_assert(smem <= kCtaSmem, "shared memory per CTA");
    auto kern = fa_fwd_kv8_kernel<D, E, C, F32>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, p.ctas, kThreads, smem, stream, p);
}

template <int D, int E, bool F32>
cudaError_t launch_main(const Kv8FwdParams& p, cudaStream_t stream) {
    return p.columns == 8    ? launch_attend<D, E, 8, F32>(p, stream)
           : p.columns == 16 ? launch_attend<D, E, 16, F32>(p, stream)
                             : launch_fwd_kv8_rows(p, D, stream);
}

template <int D, int E>
cudaError_t launch_both(const Kv8FwdParams& p, const cudaEvent_t* ev, cudaStream_t stream) {
    cudaError_t e = ev ? cudaEventRecord(ev[0], stream) : cudaSuccess;
    if (e == cudaSuccess) e = launch_main<D, E, false>(p, stream);
    if (e == cudaSuccess && ev) e = cudaEventRecord(ev[1], stream);
    if (e != cudaSuccess) return e;
    e = launch_dependent(fa_fwd_kv8_join_kernel<D, E>, dim3(p.ctas, p.columns / 8), 256, 0, stream, p);
    if (e == cudaSuccess && ev) e = cudaEventRecord(ev[2], stream);
    return e;
}

// Attention with shared prefixes is two passes, a group's rows as one request over its prefix and the
// requests' own keys, whose O and LSE (fp32) this joins:
//   LSE = log sum_i exp(LSE_i),  O = sum_i exp(LSE_i - LSE) O_i.
// A warp has a row.  A row behind the last request is left as it was, one outside all groups has no first
// part.  Measured (one GB300, bf16, Hq 32, Hkv 8, d = 128, all four kernels): 64 single tokens behind 8192
// shared ones 59 us from call to call, 55 in a graph, some 10 of them until the first products over the prefix,
// 12 in the joins of split items, 4 here (bound by latency: 3 MB).  Both passes on the GPU at once, a CTA per SM
// each, took as long.  With few requests to a group or short prefixes that is slower than reading the prefix
// once for each request (fa.h says from where on sharing pays).
template <int D, int E>
__global__ void __launch_bounds__(256) fa_kv8_prefix_join_kernel(const Kv8PrefixJoinParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(p.seq.total_tokens) * p.seq.Hq) return;
    const int token = static_cast<int>(row / p.seq.Hq), h = static_cast<int>(row - static_cast<long long>(token) * p.seq.Hq);
    long long at;   // of its LSE, as in fa_fwd
    if (p.seq.cu_seqlens) {
        if (token < p.seq.cu_seqlens[0] || token >= p.seq.cu_seqlens[p.seq.B]) return;
        at = static_cast<long long>(h) * p.seq.total_tokens + token;
    } else {
        at = (static_cast<long long>(token / p.seq.N) * p.seq.Hq + h) * p.seq.N + token % p.seq.N;
    }
    if (!fa_index_ok(at, static_cast<long long>(p.seq.total_tokens) * p.seq.Hq, p.status)) return;
    const bool grouped = token >= p.prefix_cu[0] && token < p.prefix_cu[p.groups];
    const float l0 = grouped ? p.lse[0][static_cast<long long>(h) * p.seq.total_tokens + token] : kNegInf;
    const float l1 = p.lse[1][at];
    const float top = fmaxf(l0, l1), ref = top == kNegInf ? 0.f : top;
    const float w0 = expf(l0 - ref), w1 = expf(l1 - ref), sum = w0 + w1;
    const float inv = sum > 0.f ? 1.f / sum : sum;   // (NaN stays; 0: nothing seen)
    const float f0 = w0 * inv, f1 = w1 * inv;
    constexpr int kPer = D / 32;
    using Vec = std::conditional_t<kPer == 4, float4, float2>;
    alignas(16) float x[kPer], y[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = 0.f;
    if (grouped) *reinterpret_cast<Vec*>(x) = *reinterpret_cast<const Vec*>(p.part[0] + row * D + kPer * lane);
    *reinterpret_cast<Vec*>(y) = *reinterpret_cast<const Vec*>(p.part[1] + row * D + kPer * lane);
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = f0 * x[i] + f1 * y[i];
    uint32_t* out = static_cast<uint32_t*>(p.o) + (row * D + kPer * lane) / 2;
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) out[i] = pack2<E>(x[2 * i], x[2 * i + 1]);
    if (lane == 0) p.out_lse[at] = sum > 0.f || sum != sum ? ref + logf(sum) : kNegInf;
}

template <int D, int E>
cudaError_t launch_prefix(const Kv8FwdParams& p0, const Kv8FwdParams& p1, const Kv8PrefixJoinParams& j, cudaStream_t stream) {
    const long long grid = (static_cast<long long>(j.seq.total_tokens) * j.seq.Hq + 7) / 8;
    if (grid > INT_MAX) return cudaErrorInvalidValue;
    cudaError_t e = launch_main<D, E, true>(p0, stream);
    if (e == cudaSuccess) e = launch_main<D, E, true>(p1, stream);
    if (e == cudaSuccess)
        e = launch_dependent(fa_kv8_prefix_parts_kernel<D, E>,
                             dim3(std::max(p0.ctas, p1.ctas), std::max(p0.columns, p1.columns) / 8, 2), 256, 0, stream, p0, p1);
    if (e == cudaSuccess)
        e = launch_dependent(fa_kv8_prefix_join_kernel<D, E>, dim3(static_cast<unsigned>(grid)), 256, 0, stream, j);
    return e;
}

}  // namespace

cudaError_t launch_fwd_kv8(const Kv8FwdParams& p, int d, const cudaEvent_t* ev, cudaStream_t stream) {
    if (d == 128)
        return p.elem == kElemBf16Code ? launch_both<128, kElemBf16>(p, ev, stream)
                                       : launch_both<128, kElemF16>(p, ev, stream);
    return p.elem == kElemBf16Code ? launch_both<64, kElemBf16>(p, ev, stream)
                                   : launch_both<64, kElemF16>(p, ev, stream);
}

cudaError_t launch_fwd_kv8_prefix(const Kv8FwdParams& p0, const Kv8FwdParams& p1, const Kv8PrefixJoinParams& j, int d,
                                  cudaStream_t stream) {
    if (d == 128)
        return j.elem == kElemBf16Code ? launch_prefix<128, kElemBf16>(p0, p1, j, stream)
                                       : launch_prefix<128, kElemF16>(p0, p1, j, stream);
    return j.elem == kElemBf16Code ? launch_prefix<64, kElemBf16>(p0, p1, j, stream)
                                   : launch_prefix<64, kElemF16>(p0, p1, j, stream);
}

}  // namespace fa
