// bkv_window_tc.cu -- tensor-core (tcgen05 + TMA) kernel of the attention over
// E4M3 caches with a scale a block and head, and over windows whose first
// tokens stay visible: bf16 queries of head_dim 128, bf16 or E4M3 caches.
//
// For a stream (request, KV head, row group of at most 16 query rows) and a run
// of 128-position tiles of the request's span: an online softmax over s_j =
// scale q . k_j and o += p_j v_j ("Padding and Batching with Block KV", Cache
// Masking; Special Block and Slot Values).  A stream that one CTA finishes is
// written to `out` there; one that several share leaves partials for the merge.
//
// Design (sm_103a):
// * Schedule: the grid is P columns of one CTA per (KV head, row group); a column
//   takes an equal share of the requests' cost (bkv_window.cuh), its CTAs the same
//   positions of all heads together.
// * Keys are the MMA's rows: S^T[128 x 16] = K . Q^T and O^T[128 x 16] = V^T .
//   P^T, so that a decode step's few query rows fill the N side and a position is
//   a thread's.  With a position a thread, the scales of its block are two
//   registers: k's joins the score's factor, and v's the exponent: with s'_j =
//   s_j + log2 vs_j the weights that enter P V are p'_j = 2^(s'_j - ref), ref near
//   their running maximum (below), and the row sum is sum_j p'_j / vs_j.  The value
//   tile stays the codes that TMA brought.
// * E4M3 caches: both products in kind::f8f6f4 on the codes.  A query row is
//   divided by a power of two and split into two E4M3 parts (exact for elements
//   down to 2^-10 of the row's largest, within 2^-17 of it below), which are columns
//   [0, 16) and [16, 32) of one MMA, summed as they are read.
// * E4M3 weights have four parts, columns of one MMA whose sums are worth 1, 2^-5,
//   2^-14 and 2^-19.  A weight p' (256 at most) from 2^-6 on is hi + lo / 32, lo the
//   code of 32 times what hi leaves (8 at most: no code overflows); a smaller one is
//   that of 2^14 p', in the other two columns.  Both codes are normal numbers, or lo's
//   step is 2^-14, so that a weight keeps 2^-8 of itself down to 2^-20 and is within
//   2^-29 below: 2^-22 and 2^-31 of the row's largest, or, as a fresh reference is
//   2^5 in place of 2^2 where lengths may pass 2^22, 2^-25 and 2^-34.  What a row of n
//   keys loses by that is n 2^-31 (n 2^-34) of its largest weight at most, 2^-8 whatever
//   the length.  (Rounding errors of small weights have one sign where their keys' scores
//   are alike.  Two parts of one fixed step, 2^-9, lost all weights below 2^-15 of the
//   first maximum from the product and not from the sums: 30 to 50% of an output where
//   one key has 0.9 of the weight and 8192 share the rest.)  Row sums take fp32 weights.
// * bf16 caches: weights are rounded to bf16 (2^-8 of each), and the row sums take
//   the rounded ones.
// * O stays in tensor memory over a unit, one of each softmax warpgroup (even and
//   odd tiles), joined at the unit's end.  The reference that weights are taken
//   from, ref, is not the running maximum: it moves when a weight passes 2^8 (and
//   O is rescaled then), which a unit's first tiles do and few others.  A tile's
//   warps agree on it by a vote over a barrier, and work out their weights while
//   the others arrive.
// * P is MN-major: a position's 16 weights (or four parts of 8) are one 32-byte span,
//   four parts of 16 two, with no transposition and no bank conflicts.
// * Four S tiles let the S issuer run two tiles ahead of each warpgroup.
// * Warp roles (384 threads): 0 gathers K tiles, 2 V tiles through the block table
//   by 3-D TMA boxes (head_dim half, one head, rows of a block), 1 and 3 issue the
//   MMAs of S and of P V, 4-7 and 8-11 are two softmax warpgroups on alternate
//   tiles, the one that has a unit's last tile writes its output.  Warp 2 also
//   brings the queries, and splits them, so that no launch has to come before this
//   one.  K and V have rings of 96 KB each, or 64 (16 rows over E4M3 caches: five
//   stages in place of four were 3 us slower in the second case below).  Block
//   entries are loaded 32 segments ahead, a lane each, and a unit's queries with its
//   first ones; the scales follow by cp.async, whose arrival the tile's mask barrier
//   counts.
// * V rows that no query row of the group sees, and segments that were not loaded,
//   are zeroed before P V; a row that only some see is, too, if it is not finite,
//   and those that see it become NaN.  That lies behind the store of P, when the
//   V tile has landed anyway.
// * Every wait is bounded (~2 s), after which the CTA records 1 << 24 in
//   err_count, frees its tensor memory and exits.
//
// Bound by HBM where requests are long, and by what stands still at a request's
// start and end where they are short.  Device times (of 6.79 TB/s measured):
// * bf16, 256 requests of 9 to 16384, 4 tokens, window of 2048 and 4 first tokens,
//   32 / 8 heads, blocks of 16: 153 us, 5.9 TB/s; 32 of 8192: 6.6 TB/s with one
//   token, 6.4 with four.
// * E4M3, 8 requests of 4000 to 131071, 2 tokens, 64 / 8 heads: 99 us, 6.0 TB/s;
//   32 of 512 to 4096, one token, 32 / 8 heads: 28.6 us (26 where L2 holds them in
//   part), of which some 9 are the chain lengths -> table -> first tile and the last
//   unit's end with the merge.
// * One-tile requests, 16 rows: 3.0 us of a CTA each (bf16), 5.2 (E4M3: the query
//   split is one warp's).
// What a row needs once a unit (references, factors, sums) is one lane's a row, not
// every thread's: the unrolled code of 16 rows ran once a unit, at the rate that
// instructions come in, and took as long as four tiles (the first case 189 us in
// place of 156 then, the second 126 in place of 106).  Warps still wait 1.1 cycles an
// instruction issued for instructions.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "bkv_tc_cols.cuh"
#include "bkv_window.cuh"

namespace bkv {
namespace win {

using namespace tc;

constexpr int kTcTile = 128;
constexpr int kD = 128;
constexpr int kN = kTcRows;
constexpr int kTcThreads = 384;
constexpr int kWarpV = 2, kWarpS = 4;                // (1 and 3 issue MMAs)
constexpr int kHalfBytes = kTcTile * 128;            // a bf16 tile's half of head_dim
constexpr int kRing = 16;                            // tiles whose segment words and scales are kept
constexpr int kSTiles = 4;                           // S tiles in tensor memory, two a warpgroup
constexpr int kSets = 4, kQSets = 8;                 // exchanges, and units whose query scales are kept
constexpr uint32_t kColO = 32 * kSTiles;             // tensor memory: S tiles, O of both warpgroups, exchanges
constexpr int kTimeoutErr = 1 << 24;
// The softmax's reference moves when a weight passes 2^kPMax, so that O is seldom rescaled: weights are at most 256 <
// 448, E4M3's largest value.  Over E4M3 caches a fresh reference puts the largest weight at 2^kFresh, so that small ones
// have codes, and at 2^kFreshLong where a request may be longer than kLong: what the codes lose of its weights stays
// below 2^-8.  (8 requests of 4000 to 131071, 2 tokens, 64 / 8 heads: 99 us with 2^2, 101 with 2^3, 106 with 2^5, whose
// references move more often.)
constexpr float kPMax = 8.f, kFresh = 2.f, kFreshLong = 5.f;
constexpr int32_t kLong = 1 << 22;

// E4M3 weights: below kSmall a weight enters P V times kLift, in columns of its own, and a second part times 32.
constexpr float kSmall = 0.015625f, kLift = 16384.f;               // 2^-6, 2^14
constexpr float kLowered = 6.103515625e-05f, kSecond = 0.03125f;   // 2^-14, 2^-5: what the columns' sums are worth

template <int NQ, bool kF8>
struct TcCfg {
    // columns between two parts of the weights (NQ of them are used), and of O, which has four parts
    static constexpr int kPart = NQ == 16 ? 16 : 8;
    static constexpr int kOCols = kF8 ? 4 * kPart : 32;
    static constexpr uint32_t kColX = kColO + 2 * kOCols;             // 16 columns each
    static constexpr int kTmemCols = kColX + 16 * kSets <= 256 ? 256 : 512;
    static constexpr int kStages = !kF8 ? 3 : NQ == 16 ? 4 : 6;
    static constexpr int kSlot = kF8 ? kTcTile * 128 : 2 * kHalfBytes;
    static constexpr int kQBytes = 2 * kN * 128;                      // two halves (bf16) or parts (E4M3) of 16 rows
    static constexpr int kOffV = kStages * kSlot;
    static constexpr int kOffQ = 2 * kStages * kSlot;
    // a position's weights: a span of 32 bytes (16 bf16, or four E4M3 parts of 8), or two (four parts of 16)
    static constexpr int kPSpans = kF8 && NQ == 16 ? 2 : 1;
    static constexpr int kPBytes = kPSpans * kTcTile * 32;
    static constexpr int kOffP = kOffQ + 2 * kQBytes;
    static constexpr int kOffMax = kOffP + 2 * kPBytes;               // [warpgroup][2][16][4 warps] floats
    static constexpr int kOffRows = kOffMax + 4 * 4 * kN * 4;         // [softmax warp][3][16] floats
    static constexpr int kOffFlag = kOffRows + 8 * 3 * kN * 4;        // [warpgroup][2][4 warps] words
    static constexpr int kOffSum = kOffFlag + 2 * 2 * 4 * 4;          // [warpgroup][2][16][4] floats
    static constexpr int kOffXm = kOffSum + 4 * kN * 4 * 4;           // [set][16] (max, sum)
    static constexpr int kOffQs = kOffXm + kSets * kN * 8;            // [set][16] scores' factors
    static constexpr int kOffScale = kOffQs + kQSets * kN * 4;         // [kRing][2][16 segments]
    static constexpr int kOffMask = kOffScale + (kF8 ? kRing * 2 * 16 * 4 : 0);   // [kRing] loaded segments
    static constexpr int kOffBar = kOffMask + kRing * 4;
    static constexpr int kNumBars = 4 * kStages + 4 + 2 * kSTiles + 6 + kQSets + kSets + kRing;
    static constexpr int kOffTmem = kOffBar + kNumBars * 8;
    static constexpr int kOffAbort = kOffTmem + 4;
    static constexpr int kOffSums = kOffAbort + 4;                    // a word a warp: prefix sum's scratch
    static constexpr int kOffPre = (kOffSums + kTcThreads / 32 * 4 + 15) / 16 * 16;
    static constexpr int kOffLens = kOffPre + (kMaxReqs + 4) * 4;
    static constexpr int kOffRow = (kOffLens + kMaxReqs * 4 + 15) / 16 * 16;   // [16] where a group's rows stand in their request
    static constexpr int kSmem = kOffRow + kN * 4 + 1024;             // slack for 1024 alignment
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA exceeds the sm_103a limit");
    static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kOffBar % 8 == 0 && kOffScale % 16 == 0 && kOffRow % 16 == 0 &&
                      kOffQs % 16 == 0,
                  "alignment");
    static_assert(kStages + kSTiles < kRing, "a ring word is rewritten behind its readers");
    static_assert(kColX + 16 * kSets <= kTmemCols, "tensor memory");
};

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3])
                 : "memory");
}
template <int NQ>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const float (&v)[NQ]) {
    uint32_t w[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) w[i] = __float_as_uint(v[i]);
    if constexpr (NQ == 16) tmem_st16(taddr, w);
    else if constexpr (NQ == 8) tmem_st8(taddr, w);
    else tmem_st4(taddr, w);
}

// Shared-memory descriptors by their words: the upper ones are constants (128-byte swizzle with 8-row groups 1024 bytes
// apart; 32-byte swizzle with groups of 8 spans 256 bytes apart), the lower hold the address, so that an operand's next
// piece is an addition away.
constexpr uint32_t kDesc128 = 1024 >> 4 | 1u << 14 | 2u << 29, kDesc32 = 256 >> 4 | 1u << 14 | 6u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return saddr >> 4 | (lbo >> 4) << 16; }

template <bool kF8, uint32_t kHiA, uint32_t kHiB>
__device__ __forceinline__ void mma_words(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (kF8)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
            "setp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %6};\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kHiA), "n"(kHiB)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
            "setp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %6};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kHiA), "n"(kHiB)
            : "memory");
}

__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// Two numbers of at most 256 as E4M3 codes hi, hi' and the remainders' lo, lo', in half precision: x to 11 bits, hi to 4
// of them, lo to 4 of the rest.  kTimes32: the second parts are those of 32 times the remainder, which is 8 at most.
template <bool kTimes32>
__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x0, x1);
    const __nv_fp8x2_storage_t a = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(h), __NV_SATFINITE, __NV_E4M3);
    __half2 r = __hsub2(h, __half2(__nv_cvt_fp8x2_to_halfraw2(a, __NV_E4M3)));
    if constexpr (kTimes32) r = __hmul2(r, __half2half2(__ushort_as_half(0x5000)));   // (exact)
    hi = a;
    lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(r), __NV_SATFINITE, __NV_E4M3);
}

// Weights of a position; chunk c of a span's two of 16 bytes stands at c ^ (position / 4 & 1).
template <int W>
__device__ __forceinline__ void put_words(uint8_t *at, const uint32_t (&w)[W]) {
    if constexpr (W == 1) *reinterpret_cast<uint32_t *>(at) = w[0];
    else if constexpr (W == 2) *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Whether a phase is over, without mbarrier.try_wait's suspension.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void copy4_async(uint32_t dst, const float *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives when this thread's copies so far have landed (one of the barrier's count).
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Few rows' registers are held to what 512 threads could have: the merge's CTAs then wait beside this kernel's from its
// start on, and begin as it ends (one request of 700, E4M3: 9.5 -> 8.5 us; 16 rows take all 168 that 384 threads can have,
// and spill 8 bytes over E4M3 caches).
template <int NQ>
constexpr int kRegThreads = NQ <= 8 ? 512 : kTcThreads;

template <int NQ, bool kF8>
__global__ void __launch_bounds__(kRegThreads<NQ>, 1)
    window_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Args a) {
    using C = TcCfg<NQ, kF8>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *qs = reinterpret_cast<float *>(smem + C::kOffQs);
    volatile uint32_t *mask_words = reinterpret_cast<uint32_t *>(smem + C::kOffMask);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffAbort);
    int32_t *pre = reinterpret_cast<int32_t *>(smem + C::kOffPre);
    int32_t *lens = reinterpret_cast<int32_t *>(smem + C::kOffLens);
    const uint32_t bar0 = sbase + C::kOffBar;
    auto bar_kfull = [&](int s) { return bar0 + 8u * s; };
    auto bar_kempty = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto bar_vfull = [&](int s) { return bar0 + 8u * (2 * kStages + s); };
    auto bar_vempty = [&](int s) { return bar0 + 8u * (3 * kStages + s); };
    constexpr int kB = 4 * kStages;
    auto bar_qfull = [&](int b) { return bar0 + 8u * (kB + b); };
    auto bar_qempty = [&](int b) { return bar0 + 8u * (kB + 2 + b); };
    auto bar_sfull = [&](int i) { return bar0 + 8u * (kB + 4 + i); };
    auto bar_sfree = [&](int i) { return bar0 + 8u * (kB + 4 + kSTiles + i); };
    constexpr int kB2 = kB + 4 + 2 * kSTiles;
    auto bar_pfull = [&](int b) { return bar0 + 8u * (kB2 + b); };
    auto bar_ofull = [&](int b) { return bar0 + 8u * (kB2 + 2 + b); };
    auto bar_group = [&](int k) { return bar0 + 8u * (kB2 + 4 + k); };
    auto bar_qscale = [&](int i) { return bar0 + 8u * (kB2 + 6 + i); };
    auto bar_x = [&](int i) { return bar0 + 8u * (kB2 + 6 + kQSets + i); };
    auto bar_mask = [&](int m) { return bar0 + 8u * (kB2 + 6 + kQSets + kSets + m); };
    const uint32_t sm_k = sbase, sm_v = sbase + C::kOffV, sm_q = sbase + C::kOffQ, sm_p = sbase + C::kOffP;

    // what this CTA is: column q, KV head g, row group grp, and its rows
    const int HP = a.H_kv * a.groups;
    const int q = (int)blockIdx.x / HP, hp = (int)blockIdx.x - q * HP;
    const int g = hp / a.groups, grp = hp - g * a.groups;
    const int i0 = grp * a.NR;
    const int rows = min(a.NR, a.q_len * a.G - i0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar_kfull(s), 1);
            mbar_init(bar_kempty(s), 1);
            mbar_init(bar_vfull(s), 1);
            mbar_init(bar_vempty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_qfull(b), 1);
            mbar_init(bar_qempty(b), 1);
            mbar_init(bar_pfull(b), 4);
            mbar_init(bar_ofull(b), 1);
            mbar_init(bar_group(b), 4);
        }
        for (int i = 0; i < kSTiles; ++i) {
            mbar_init(bar_sfull(i), 1);
            mbar_init(bar_sfree(i), 4);
        }
        for (int i = 0; i < kQSets; ++i) mbar_init(bar_qscale(i), 1);
        for (int i = 0; i < kSets; ++i) mbar_init(bar_x(i), 4);
        for (int m = 0; m < kRing; ++m) mbar_init(bar_mask(m), kF8 ? 33 : 1);   // the word, and the lanes' copies
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    {
        // query rows past the group's, and P, start at zero
        uint4 *z = reinterpret_cast<uint4 *>(smem + C::kOffQ);
        for (int i = threadIdx.x; i < (C::kOffMax - C::kOffQ) / 16; i += kTcThreads) z[i] = make_uint4(0, 0, 0, 0);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(C::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    int32_t *row_at = reinterpret_cast<int32_t *>(smem + C::kOffRow);
    if (threadIdx.x >= 64 && threadIdx.x < 64 + kN) {
        const int i = i0 + min((int)threadIdx.x - 64, rows - 1), t = i / a.G;
        row_at[threadIdx.x - 64] = (t * a.H_q + g * a.G + (i - t * a.G)) * kD;
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();   // global memory is read from here on
    pdl_trigger();
    lay_out<kTcThreads>(a, pre, lens, reinterpret_cast<int32_t *>(smem + C::kOffSums));
    const uint32_t tmem = *tmem_slot;
    const int seg_rows = a.seg;                      // a power of two, 8 to 128
    const int nseg = kTcTile / seg_rows;
    const int seg_shift = 31 - __clz(seg_rows);
    Units units(pre, a.num_reqs, q, a.P);
    Unit x;
    const int64_t req_elems = (int64_t)a.q_len * a.H_q * kD;   // of q and out

    if (warp == 0 || warp == kWarpV) {
        // ================= TMA producers =================
        const bool is_v = warp == kWarpV;
        const bool count = !is_v && grp == 0 && a.err;   // bad entries count once a KV head
        // ---- queries (warp 2): unit us's rows, eight elements a lane, two rows at a time ----
        constexpr int kPairs = (NQ + 1) / 2;
        uint4 raw[kPairs];
        int32_t raw_at[kPairs];   // where this lane's eight elements stand in their request
        const int half = lane >> 4, col = lane & 15;
        if (is_v) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                raw_at[i] = row_at[2 * i + half] + 8 * col;
                raw[i] = make_uint4(0, 0, 0, 0);
            }
        }
        auto load_q = [&](int r) {
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) + r * req_elems;
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                if (2 * i < rows) raw[i] = __ldg(reinterpret_cast<const uint4 *>(src + raw_at[i]));
        };
        auto put_q = [&](int us) -> bool {
            const int b = us & 1;
            if (!mbar_wait_warp(bar_qempty(b), (uint32_t)((us >> 1) & 1) ^ 1u, abort_flag)) return false;
            uint8_t *dst = smem + C::kOffQ + b * C::kQBytes;
            if constexpr (kF8) {
                // A row is scaled by 2^-e, e = floor(log2 max) - 7, then x = hi + lo in E4M3: x has at most 8 significant
                // bits, so the remainder is exact where |x| >= 2^-2 and within 2^-10 (2^-17 of the largest) below.
                // (All pairs of rows side by side: one after the other is a chain of 700 cycles each.)
                uint32_t top[kPairs];
#pragma unroll
                for (int i = 0; i < kPairs; ++i)
                    top[i] = __vmaxu2(__vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu),
                                      __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) top[i] = __vmaxu2(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const int n = 2 * i + half;   // (an odd group's last row is written twice, to rows n and n + 1 < 16)
                    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                    // the largest as fp32 bits: NaN and infinity come out above every number
                    const uint32_t t = max(top[i] & 0xffffu, top[i] >> 16) << 16;
                    // (a row whose largest is subnormal is left as it is: its scores are 0 to fp32's own rounding)
                    const int e = t >= 0x00800000u && t < 0x7f800000u ? max((int)(t >> 23) - 127 - 7, -126) : 0;
                    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t h0, h1, l0, l1;
                        split2<false>(__uint_as_float(w[2 * k] << 16) * down, __uint_as_float(w[2 * k] & 0xffff0000u) * down, h0, l0);
                        split2<false>(__uint_as_float(w[2 * k + 1] << 16) * down,
                                      __uint_as_float(w[2 * k + 1] & 0xffff0000u) * down, h1, l1);
                        hi[k] = __byte_perm(h0, h1, 0x5410);
                        lo[k] = __byte_perm(l0, l1, 0x5410);
                    }
                    uint8_t *at = dst + n * 128 + (((col >> 1) ^ (n & 7)) << 4) + (col & 1) * 8;
                    *reinterpret_cast<uint2 *>(at) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2 *>(at + kN * 128) = make_uint2(lo[0], lo[1]);
                    // a row that is not finite makes its scores NaN (rows past the group's: 0)
                    if (col == 0)
                        qs[(us & (kQSets - 1)) * kN + n] =
                            n >= rows ? 0.f
                                      : t < 0x7f800000u ? a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23)
                                                        : __uint_as_float(0x7fffffffu);
                }
            } else {
                // 64 elements a half; 16-byte chunk c of row n at c ^ (n & 7)
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const int n = 2 * i + half;
                    *reinterpret_cast<uint4 *>(dst + (col >> 3) * (kN * 128) + n * 128 + (((col & 7) ^ (n & 7)) << 4)) = raw[i];
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar_qfull(b));
                if constexpr (kF8) mbar_arrive(bar_qscale(us & (kQSets - 1)));
            }
            return true;
        };
        // A chunk is 32 segments of a unit, a lane each.  The next one's block entries are loaded while this one's tiles
        // are issued: nothing looks at an entry before its chunk's turn.
        struct Chunk {
            int r, f, nt, c;   // the unit; the chunk's number in it
            int32_t entry;     // the segment's block entry, as it is in the table; INT32_MAX: past its columns
            int32_t off;       // the segment's first row in the block, and, in bit 31, that the block begins here in the
                               // span; -1: no segment
        };
        const int tiles = 32 / nseg;   // tiles a chunk
        auto fetch = [&](Chunk &w) {
            w.entry = 0;
            w.off = -1;
            const Span s = span_of(a, lens[w.r]);
            const int32_t seg = w.f * nseg + w.c * 32 + lane, v = seg << seg_shift;
            if (w.c * 32 + lane < w.nt * nseg && v < s.len) {
                const int32_t p = s.pos(v);
                // (a block is one segment, or, above 128 positions, several)
                const int32_t lb = a.bs == seg_rows ? p >> seg_shift : p / a.bs, off = p - lb * a.bs;
                const bool begins = off == 0 || (s.gap > 0 && v == s.sb && (s.sb == 0 || (s.sb - 1) / a.bs != lb));
                w.off = off | (begins ? INT32_MIN : 0);
                w.entry = lb < a.bt_cols ? __ldg(a.bt + (int64_t)w.r * a.bt_stride + lb) : INT32_MAX;
            }
        };
        auto next = [&](const Chunk &w, Chunk &n) -> bool {
            if ((w.c + 1) * tiles < w.nt) {
                n = w;
                ++n.c;
            } else {
                if (!units.next(x)) return false;
                n.r = x.r;
                n.f = x.f;
                n.nt = x.nt;
                n.c = 0;
                if (is_v) load_q(x.r);
            }
            fetch(n);
            return true;
        };
        if (is_v) {
            if (hp == 0 && lane == 0) a.ws_split[q] = units.split();
            // requests without a cached position
            for (int r = q; r < a.num_reqs; r += a.P)
                if (pre[r + 1] == pre[r])
                    for (int n = 0; n < rows; ++n)
                        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + r * req_elems + row_at[n] + 4 * lane) =
                            make_uint2(0, 0);
        }
        Chunk cur{0, 0, 0, 0, 0, -1}, nxt;
        bool have = next(cur, cur);
        Ring ring;
        int j = 0, us = 0;
        while (have && !*abort_flag) {
            if (is_v && cur.c == 0 && !put_q(us++)) break;   // (its registers go to the next unit's below)
            // the cache row that this lane's segment begins at (-1: nothing to load) and its block
            int32_t seg_row = -1, seg_blk = 0;
            if (cur.off != -1) {
                if (cur.entry >= a.total_blocks) {
                    if (count && cur.off < 0) atomicAdd(a.err, 1);   // at the block's first segment in the span
                } else if (cur.entry > 0) {
                    seg_blk = cur.entry;
                    seg_row = cur.entry * a.bs + (cur.off & INT32_MAX);
                }
            }
            const bool more = next(cur, nxt);
            const int nt = min(tiles, cur.nt - cur.c * tiles);
            for (int kt = 0; kt < nt; ++kt, ++j, ring.advance(kStages)) {
                const int s = ring.slot;
                const uint32_t bar_f = is_v ? bar_vfull(s) : bar_kfull(s);
                const int32_t row = __shfl_sync(0xffffffffu, seg_row, (kt * nseg + lane) & 31);
                const int32_t blk = __shfl_sync(0xffffffffu, seg_blk, (kt * nseg + lane) & 31);
                const bool load = lane < nseg && row >= 0;
                const uint32_t ballot = __ballot_sync(0xffffffffu, load);
                if (!mbar_wait_warp(is_v ? bar_vempty(s) : bar_kempty(s), ring.phase ^ 1u, abort_flag)) break;
                if (!is_v) {
                    // Tile j's word and scales: written only after the S MMA of tile j - kStages completed, which was
                    // issued after the softmax had read tile j - kStages - kSTiles's, so that the writer is at most
                    // kStages + kSTiles < kRing tiles ahead of the readers.
                    const int m = j & (kRing - 1);
                    if constexpr (kF8) {
                        if (load) {
                            const uint32_t dst = sbase + C::kOffScale + (uint32_t)(m * 32 + lane) * 4u;
                            const int64_t at = (int64_t)blk * a.H_kv + g;
                            copy4_async(dst, a.ks + at);
                            copy4_async(dst + 64u, a.vs + at);
                        }
                        copies_arrive(bar_mask(m));
                    }
                    if (lane == 0) {
                        mask_words[m] = ballot;
                        mbar_arrive(bar_mask(m));
                    }
                }
                if (lane == 0) mbar_arrive_expect_tx(bar_f, (uint32_t)__popc(ballot) * (uint32_t)seg_rows * (kF8 ? 128u : 256u));
                __syncwarp();
                if (load) {
                    const CUtensorMap *map = is_v ? &tmV : &tmK;
                    const uint32_t dst = (is_v ? sm_v : sm_k) + s * C::kSlot + lane * seg_rows * 128;
                    tma_load_3d(dst, map, bar_f, 0, g, row);
                    if constexpr (!kF8) tma_load_3d(dst + kHalfBytes, map, bar_f, 64, g, row);
                }
                __syncwarp();
            }
            cur = nxt;
            have = more;
        }
        if (*abort_flag) {   // let copies in flight land
            asm volatile("cp.async.wait_all;" ::: "memory");
            const unsigned long long t0 = global_ns();
            while (global_ns() - t0 < 200000ull) {
            }
        }
    } else if (warp == 1 || warp == 3) {
        // ================= MMA issuers (one thread each) =================
        if (lane == 0 && warp == 1) {
            constexpr uint32_t kIdesc = kF8 ? idesc_f16(128, 2 * kN, 0, 0) : idesc_bf16(128, kN, 0, 0);
            const uint32_t k_lo = desc_lo(sm_k, 16);
            int j = 0, us = 0;
            Ring ring;
            bool ok = true;
            for (; ok && units.next(x); ++us) {
                const int qb = us & 1;
                if (!mbar_wait(bar_qfull(qb), (uint32_t)(us >> 1) & 1u, abort_flag)) break;
                const uint32_t q_lo = desc_lo(sm_q + qb * C::kQBytes, 16);
                for (int jt = 0; jt < x.nt; ++jt, ++j, ring.advance(kStages)) {
                    const int b = j & (kSTiles - 1);
                    // K landed, and the softmax has read what was in this S tile
                    if (!mbar_wait(bar_kfull(ring.slot), ring.phase, abort_flag) ||
                        (j >= kSTiles && !mbar_wait(bar_sfree(b), (uint32_t)(j / kSTiles - 1) & 1u, abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + 32u * (uint32_t)b, k = k_lo + ring.slot * (C::kSlot >> 4);
                    if constexpr (kF8) {
#pragma unroll
                        for (int kk = 0; kk < kD / 32; ++kk)
                            mma_words<kF8, kDesc128, kDesc128>(d, k + 2 * kk, q_lo + 2 * kk, kIdesc, kk > 0);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < kD / 16; ++kk)
                            mma_words<kF8, kDesc128, kDesc128>(d, k + (kk >> 2) * (kHalfBytes >> 4) + (kk & 3) * 2,
                                                               q_lo + (kk >> 2) * (kN * 8) + (kk & 3) * 2, kIdesc, kk > 0);
                    }
                    mma_commit(bar_sfull(b));
                    mma_commit(bar_kempty(ring.slot));
                    if (jt == x.nt - 1) mma_commit(bar_qempty(qb));
                }
            }
        } else if (lane == 0) {
            constexpr uint32_t kIdesc = kF8 ? idesc_f16(128, C::kOCols, 1, 1) : idesc_bf16(128, kN, 1, 1);
            const uint32_t v_lo = desc_lo(sm_v, kF8 ? 16 : kHalfBytes);
            const uint32_t p_lo = desc_lo(sm_p, C::kPSpans == 2 ? kTcTile * 32 : 16);
            int j = 0;
            Ring ring;
            bool ok = true;
            while (ok && units.next(x)) {
                for (int jt = 0; jt < x.nt; ++jt, ++j, ring.advance(kStages)) {
                    const int b = j & 1;
                    if (!mbar_wait(bar_vfull(ring.slot), ring.phase, abort_flag) ||
                        !mbar_wait(bar_pfull(b), (uint32_t)((j >> 1) & 1), abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + kColO + (uint32_t)(C::kOCols * b), v = v_lo + ring.slot * (C::kSlot >> 4);
                    const uint32_t p = p_lo + b * (C::kPBytes >> 4);
                    const uint32_t more = jt >= 2;   // a warpgroup's first tile of a unit begins its O
                    // V^T and P^T MN-major: a row's 128 codes (64 bf16) are one 128-byte span, a position's weights one
                    // or two of 32 bytes
#pragma unroll
                    for (int kk = 0; kk < (kF8 ? kTcTile / 32 : kTcTile / 16); ++kk)
                        mma_words<kF8, kDesc128, kDesc32>(d, v + kk * (kF8 ? 256 : 128), p + kk * (kF8 ? 64 : 32), kIdesc,
                                                          more | (kk > 0));
                    mma_commit(bar_ofull(b));
                    mma_commit(bar_vempty(ring.slot));
                }
            }
        }
        __syncwarp();
    } else {
        // ================= softmax and output (two warpgroups of 128 threads) =================
        const int wg = (warp - kWarpS) >> 2, wq = warp & 3;
        const int row = 32 * wq + lane;                  // TMEM lane: position in the tile, and head_dim row
        const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
        const uint32_t o_col = tmem + lane_base + kColO + (uint32_t)(C::kOCols * wg);
        const int red_row = reduced_row<NQ>(lane);
        const bool red_writer = reduced_writer<NQ>(lane);
        const int flip = (row >> 2) & 1;
        uint8_t *p_hi = smem + C::kOffP + wg * C::kPBytes + row * 32 + 16 * flip, *p_lo = p_hi + 16 - 32 * flip;
        float *rm = reinterpret_cast<float *>(smem + C::kOffMax) + wg * 2 * 4 * kN;
        // What belongs to a query row and not to a position is worked out by one lane a row (lanes past NQ repeat others)
        // and handed to the warp through shared memory: three arrays of 16, a warp's own.  Every use of one ends with a
        // __syncwarp further on, before the next.
        float *warp_rows = reinterpret_cast<float *>(smem + C::kOffRows) + (warp - kWarpS) * 3 * kN;
        const int my_row = lane & (NQ - 1);
        auto hand_out = [&](int k, float mine) {
            if (lane < NQ) warp_rows[k * kN + lane] = mine;
        };
        auto take = [&](int k, float (&v)[NQ]) {   // behind a __syncwarp
#pragma unroll
            for (int n = 0; n < NQ; n += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(warp_rows + k * kN + n);
                v[n] = f.x, v[n + 1] = f.y, v[n + 2] = f.z, v[n + 3] = f.w;
            }
        };
        uint32_t moves = 0;
        uint32_t gphase = 0;
        // Bounded barrier of the warpgroup's four warps.
        auto group_arrive = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_group(wg));
        };
        auto group_wait = [&]() -> bool {
            bool r = false;
            for (int i = 0; i < 64 && !r; ++i) r = __all_sync(0xffffffffu, mbar_test(bar_group(wg), gphase));
            if (!r) r = mbar_wait_warp(bar_group(wg), gphase, abort_flag);
            gphase ^= 1u;
            return r;
        };
        auto group_sync = [&]() -> bool {
            group_arrive();
            return group_wait();
        };
        auto load_o = [&](float (&v)[NQ]) {
            tmem_ld_cols<NQ>(o_col, v);
            if constexpr (kF8) {   // the parts, each worth its power of two
                float part[NQ];
#pragma unroll 1
                for (int k = 1; k < 4; ++k) {
                    tmem_ld_cols<NQ>(o_col + (uint32_t)(C::kPart * k), part);
                    const float worth = (k & 1 ? kSecond : 1.f) * (k & 2 ? kLowered : 1.f);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) v[n] = fmaf(part[n], worth, v[n]);
                }
            }
        };
        const int tok_lo = i0 / a.G, tok_hi = (i0 + rows - 1) / a.G, head0 = i0 % a.G;
        const float fresh = !kF8 ? 0.f : a.max_ctx > kLong ? kFreshLong : kFresh;
        int j = 0, xs = 0, mu = 0;   // tile, exchange and own unit number
        Ring vring;
        bool ok = true;
        for (int us = 0; ok && units.next(x); ++us) {
            const bool both = x.nt > 1;   // a unit of one tile is one warpgroup's alone
            if (!both && (j & 1) != wg) {
                ++j;
                vring.advance(kStages);
                continue;
            }
            const Span s = span_of(a, lens[x.r]);
            // Positions at or below last_lo (and from first_hi on, or below `sinks`) are seen by every row of the
            // group, those past last_hi (or before first_lo) by none.
            const int32_t t_lo = s.L - a.q_len + tok_lo, t_hi = s.L - a.q_len + tok_hi;
            const int32_t last_lo = a.causal ? t_lo : s.L - 1, last_hi = a.causal ? t_hi : s.L - 1;
            const int32_t first_lo = a.window > 0 ? t_lo - a.window + 1 : INT32_MIN;
            const int32_t first_hi = a.window > 0 ? t_hi - a.window + 1 : INT32_MIN;
            // A row's weights are 2^(s - ref): ref is set at the first tile in which the row sees a key (bit n of
            // `have`) and moved when a weight passes 2^kPMax.
            float lsum[NQ], ref[NQ];
            uint32_t have = 0u;
            const uint32_t every = (1u << rows) - 1u;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                lsum[n] = 0.f;
                ref[n] = 0.f;
            }
            const float *cs = qs + (us & (kQSets - 1)) * kN;   // E4M3: the scores' factors, read in every tile
            if constexpr (kF8) {
                // A set is rewritten eight units on, behind the S MMAs of the sixth unit after this one: its last tile is at
                // least six behind this unit's last, and its S tile's last reader this warpgroup, past this unit.
                if (!mbar_wait_warp(bar_qscale(us & (kQSets - 1)), (uint32_t)(us / kQSets) & 1u, abort_flag)) break;
            }
            for (int jt = 0; jt < x.nt; ++jt, ++j, vring.advance(kStages)) {
                if ((j & 1) != wg) continue;
                const uint32_t par = (uint32_t)(j >> 1) & 1u;
                const int m = j & (kRing - 1), sb = j & (kSTiles - 1);
                if (!mbar_wait_warp(bar_sfull(sb), (uint32_t)(j / kSTiles) & 1u, abort_flag) ||
                    !mbar_wait_warp(bar_mask(m), (uint32_t)(j / kRing) & 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                const int seg = row >> seg_shift;
                const bool loaded = (mask_words[m] >> seg) & 1u;
                float ks = 1.f, lv = 0.f, rv = 1.f;
                if constexpr (kF8) {
                    const float *sc = reinterpret_cast<const float *>(smem + C::kOffScale) + m * 32 + seg;
                    ks = sc[0];
                    const float vs = fminf(fmaxf(sc[16], kScaleMin), kScaleMax);
                    lv = __log2f(vs);
                    rv = __fdividef(1.f, vs);
                }
                tc_fence_after();
                float sv[NQ];
                if constexpr (kF8) tmem_ld_sum2<NQ>(tmem + lane_base + 32u * (uint32_t)sb, sv);
                else tmem_ld_cols<NQ>(tmem + lane_base + 32u * (uint32_t)sb, sv);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_sfree(sb));   // S tile may be overwritten (by tile j + 4's)
                const int32_t v = (x.f + jt) * kTcTile + row;
                const int32_t p = s.pos(v);
                const bool in = loaded && v < s.len, sink = p < a.sinks;
                const bool any = in && p <= last_hi && (p >= first_lo || sink);
                const bool all = in && p <= last_lo && (p >= first_hi || sink);
                if constexpr (kF8) {
#pragma unroll
                    for (int n = 0; n < NQ; n += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(cs + n);
                        sv[n] = fmaf(sv[n], f.x * ks, lv - ref[n]);
                        sv[n + 1] = fmaf(sv[n + 1], f.y * ks, lv - ref[n + 1]);
                        sv[n + 2] = fmaf(sv[n + 2], f.z * ks, lv - ref[n + 2]);
                        sv[n + 3] = fmaf(sv[n + 3], f.w * ks, lv - ref[n + 3]);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NQ; ++n) sv[n] = fmaf(sv[n], a.scale_log2, -ref[n]);
                }
                const bool tile_all = __all_sync(0xffffffffu, all);
                if (!tile_all && !all) {
                    // rows that see a position, one by one: row n's token is at position t
                    int32_t t = t_lo, h = head0;
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        const bool see = any && p <= (a.causal ? t : s.L - 1) && (a.window == 0 || p > t - a.window || sink);
                        if (!see) sv[n] = -INFINITY;
                        if (++h == a.G) {
                            h = 0;
                            ++t;
                        }
                    }
                }
                // The weights as they go to P V (E4M3: NQ / 4 words of each part), and into the sums.
                uint32_t pw[kF8 ? NQ : NQ / 2];
                auto weigh = [&] {
                    if constexpr (kF8) {
#pragma unroll
                        for (int n = 0; n < NQ; n += 4) {
                            float w[4];
                            uint32_t low = 0u;   // a byte of ones for each small weight
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                w[i] = fast_exp2(sv[n + i]);
                                lsum[n + i] = fmaf(w[i], rv, lsum[n + i]);
                                const bool small = w[i] < kSmall;
                                if (small) w[i] *= kLift, low |= 0xffu << (8 * i);
                            }
                            uint32_t h0, h1, l0, l1;
                            split2<true>(w[0], w[1], h0, l0);
                            split2<true>(w[2], w[3], h1, l1);
                            const uint32_t hi = __byte_perm(h0, h1, 0x5410), lo = __byte_perm(l0, l1, 0x5410);
                            pw[n / 4] = hi & ~low;
                            pw[NQ / 4 + n / 4] = lo & ~low;
                            pw[NQ / 2 + n / 4] = hi & low;
                            pw[3 * NQ / 4 + n / 4] = lo & low;
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < NQ; n += 2) {
                            const __nv_bfloat162 b2 = __floats2bfloat162_rn(fast_exp2(sv[n]), fast_exp2(sv[n + 1]));
                            pw[n / 2] = *reinterpret_cast<const uint32_t *>(&b2);
                            lsum[n] += __uint_as_float(pw[n / 2] << 16);
                            lsum[n + 1] += __uint_as_float(pw[n / 2] & 0xffff0000u);
                        }
                    }
                };
                // Does a reference have to be set or moved?  The warpgroup's warps agree on it; a warp that sees no need
                // works out its weights while the others arrive.
                bool move = (have & every) != every, weighed = false;
                if (!move) {
                    float top = fmaxf(sv[0], sv[1]);
#pragma unroll
                    for (int n = 2; n < NQ; n += 2) top = max3(top, sv[n], sv[n + 1]);
                    const bool up = __any_sync(0xffffffffu, top > kPMax);
                    uint32_t *flags = reinterpret_cast<uint32_t *>(smem + C::kOffFlag) + (wg * 2 + (int)par) * 4;
                    if (lane == 0) flags[wq] = up;
                    group_arrive();
                    if (!up) {
                        weigh();
                        weighed = true;
                    }
                    if (!group_wait()) {
                        ok = false;
                        break;
                    }
                    const uint4 f = *reinterpret_cast<const uint4 *>(flags);
                    move = (f.x | f.y | f.z | f.w) != 0u;
                }
                if (move) {
                    if (weighed) {
                        // out of the sums again: a sum is off by its own rounding, and the same weights follow
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
                            lsum[n] -= kF8 ? fast_exp2(sv[n]) * rv : __bfloat162float(__float2bfloat16_rn(fast_exp2(sv[n])));
                    }
                    // (two sets of maxima in turn: one is written again behind the next move's barrier, which all
                    // passed after reading it)
                    float *tops = rm + (moves++ & 1u) * (4 * kN);
                    const float wmax = warp_reduce_rows<true, NQ>(sv, lane);
                    if (red_writer) tops[red_row * 4 + wq] = wmax;
                    if (!group_sync()) {
                        ok = false;
                        break;
                    }
                    const float4 t4 = *reinterpret_cast<const float4 *>(tops + my_row * 4);
                    const float top = fmaxf(max3(t4.x, t4.y, t4.z), t4.w);
                    const bool had = (have >> my_row) & 1u;
                    const bool to = had ? top > kPMax : top > -INFINITY;
                    const float down = to ? top - fresh : 0.f;
                    hand_out(0, down);
                    hand_out(1, had ? fast_exp2(-down) : 1.f);
                    const bool scale = have != 0u;   // there is something in the sums and in O
                    have |= __ballot_sync(0xffffffffu, to) & ((1u << NQ) - 1u);
                    __syncwarp();
                    float by[NQ];
                    take(0, by);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        ref[n] += by[n];
                        sv[n] -= by[n];
                    }
                    if (scale) {
                        if (!mbar_wait_warp(bar_ofull(wg), par ^ 1u, abort_flag)) {   // the last P V into O
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        float corr[NQ], o[NQ];
                        take(1, corr);
#pragma unroll
                        for (int n = 0; n < NQ; ++n) lsum[n] *= corr[n];
#pragma unroll 1
                        for (int k = 0; k < (kF8 ? 4 : 1); ++k) {
                            tmem_ld_cols<NQ>(o_col + (uint32_t)(C::kPart * k), o);
#pragma unroll
                            for (int n = 0; n < NQ; ++n) o[n] *= corr[n];
                            tmem_st_cols<NQ>(o_col + (uint32_t)(C::kPart * k), o);
                        }
                        tmem_st_wait();
                    }
                    weigh();
                }
                // P, once the last P V has read its buffer
                if (j >= 2 && !mbar_wait_warp(bar_ofull(wg), par ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                if constexpr (kF8 && NQ == 16) {
                    put_words(p_hi, reinterpret_cast<const uint32_t(&)[4]>(pw[0]));
                    put_words(p_lo, reinterpret_cast<const uint32_t(&)[4]>(pw[4]));
                    put_words(p_hi + kTcTile * 32, reinterpret_cast<const uint32_t(&)[4]>(pw[8]));
                    put_words(p_lo + kTcTile * 32, reinterpret_cast<const uint32_t(&)[4]>(pw[12]));
                } else if constexpr (kF8 && NQ == 8) {
                    put_words(p_hi, reinterpret_cast<const uint32_t(&)[4]>(pw[0]));
                    put_words(p_lo, reinterpret_cast<const uint32_t(&)[4]>(pw[4]));
                } else if constexpr (kF8) {
                    const uint32_t w0[4] = {pw[0], 0u, pw[1], 0u}, w1[4] = {pw[2], 0u, pw[3], 0u};
                    put_words(p_hi, w0);
                    put_words(p_lo, w1);
                } else if constexpr (NQ == 16) {
                    put_words(p_hi, reinterpret_cast<const uint32_t(&)[4]>(pw[0]));
                    put_words(p_lo, reinterpret_cast<const uint32_t(&)[4]>(pw[4]));
                } else {
                    put_words(p_hi, pw);
                }
                if (!tile_all) {
                    // V rows that must not reach P V, once the tile is there.  (Behind the wait for the warpgroup's last
                    // P V, above: the slot's tile before this one has been consumed by then, so that the parity cannot be
                    // answered by a phase before that.)
                    const int vslot = vring.slot;
                    if (!mbar_wait_warp(bar_vfull(vslot), vring.phase, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (!all) {
                        uint4 *vr = reinterpret_cast<uint4 *>(smem + C::kOffV + vslot * C::kSlot + row * 128);
                        // (code that seldom runs is kept short: sink windows of bf16 156 -> 153 us; over E4M3 caches, where
                        // 16 rows leave no registers for its counters, it was 107 -> 114)
                        constexpr int kParts = kF8 ? 1 : 2, kScan = kF8 ? 8 : 4, kClear = kF8 ? 8 : 1;
                        bool clear = !any;
                        if (any) {
                            // seen by some rows and not by others: not finite?
#pragma unroll 1
                            for (int h = 0; h < kParts; ++h)
#pragma unroll kScan
                                for (int c = 0; c < 8; ++c) {
                                    const uint4 w = vr[h * (kHalfBytes / 16) + ((c + lane) & 7)];
                                    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        if constexpr (kF8) clear |= __vcmpeq4(ws[i] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u;
                                        else clear |= (ws[i] & 0x7f80u) == 0x7f80u || (ws[i] & 0x7f800000u) == 0x7f800000u;
                                    }
                                }
                            if (clear) {
#pragma unroll
                                for (int n = 0; n < NQ; ++n)
                                    if (sv[n] != -INFINITY) lsum[n] = __uint_as_float(0x7fffffffu);
                            }
                        }
                        if (clear) {
#pragma unroll 1
                            for (int h = 0; h < kParts; ++h)
#pragma unroll kClear
                                for (int c = 0; c < 8; ++c) vr[h * (kHalfBytes / 16) + ((c + lane) & 7)] = make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_pfull(wg));
            }
            if (!ok) break;
            // row sums across the warpgroup, in two buffers in turn: one is written again behind the next unit's
            // barrier, which all passed after reading it
            float *sums = reinterpret_cast<float *>(smem + C::kOffSum) + (wg * 2 + (mu & 1)) * (kN * 4);
            ++mu;
            const float wsum = warp_reduce_rows<false, NQ>(lsum, lane);
            if (red_writer) sums[red_row * 4 + wq] = wsum;
            if (lane == 0) {
#pragma unroll
                for (int n = 0; n < NQ; n += 4)
                    *reinterpret_cast<float4 *>(warp_rows + n) = make_float4(ref[n], ref[n + 1], ref[n + 2], ref[n + 3]);
            }
            // the warpgroup's last tile here is j - 1 or j - 2
            const int last = (j - 1 - wg) >> 1;
            if (!group_sync()) break;
            const float4 s4 = *reinterpret_cast<const float4 *>(sums + my_row * 4);
            float my_sum = (s4.x + s4.y) + (s4.z + s4.w);
            float my_ref = (have >> my_row) & 1u ? warp_rows[my_row] : -INFINITY;   // no key, or none whose score is a number
            // The warpgroup of the unit's last tile finishes it; the other hands its part over through tensor memory and
            // goes on.  A set is written again four exchanges on, behind a P V that follows one of the other's tiles of
            // the exchange after this one, which it begins when it has read this.
            const bool finish = ((j - 1) & 1) == wg;
            const int set = xs & (kSets - 1);
            const uint32_t x_col = tmem + lane_base + C::kColX + 16u * (uint32_t)set;
            float2 *xm = reinterpret_cast<float2 *>(smem + C::kOffXm) + set * kN;
            const uint32_t x_par = (uint32_t)(xs >> 2) & 1u;
            if (both) ++xs;
            if (!mbar_wait_warp(bar_ofull(wg), (uint32_t)last & 1u, abort_flag)) break;
            tc_fence_after();
            float o[NQ];
            load_o(o);
            if (!finish) {
                tmem_st_cols<NQ>(x_col, o);
                if (row < NQ) xm[row] = make_float2(my_ref, my_sum);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_x(set));
                continue;
            }
            float f0 = 1.f, f1 = 0.f;
            float o1[NQ];
            if (both) {
                if (!mbar_wait_warp(bar_x(set), x_par, abort_flag)) break;
                tc_fence_after();
                tmem_ld_cols<NQ>(x_col, o1);
                const float2 ml = xm[my_row];
                const float mn = fmaxf(my_ref, ml.x);
                f0 = mn == -INFINITY ? 1.f : fast_exp2(my_ref - mn);
                f1 = mn == -INFINITY ? 1.f : fast_exp2(ml.x - mn);
                my_sum = my_sum * f0 + ml.y * f1;
                my_ref = mn;
            } else {
#pragma unroll
                for (int n = 0; n < NQ; ++n) o1[n] = 0.f;
            }
            if (x.whole) {
                const float inv = inverse(my_sum);
                f0 *= inv;
                f1 *= inv;
            }
            hand_out(1, f0);
            hand_out(2, f1);
            __syncwarp();
            float by[NQ];
            take(1, by);
#pragma unroll
            for (int n = 0; n < NQ; ++n) o[n] *= by[n];
            take(2, by);
#pragma unroll
            for (int n = 0; n < NQ; ++n) o[n] = fmaf(o1[n], by[n], o[n]);
            if (x.whole) {
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + x.r * req_elems + row;
#pragma unroll
                for (int n = 0; n < NQ; n += 4) {
                    const int4 to = *reinterpret_cast<const int4 *>(row_at + n);
                    if (n < rows) out[to.x] = __float2bfloat16_rn(o[n]);
                    if (n + 1 < rows) out[to.y] = __float2bfloat16_rn(o[n + 1]);
                    if (n + 2 < rows) out[to.z] = __float2bfloat16_rn(o[n + 2]);
                    if (n + 3 < rows) out[to.w] = __float2bfloat16_rn(o[n + 3]);
                }
            } else {
                const int64_t at = ((int64_t)hp * (2 * a.P) + x.slot) * a.NR;
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                    if (n < rows) a.ws_o[(at + n) * kD + row] = o[n];
                if (row < rows) *reinterpret_cast<float2 *>(a.ws_ml + (at + row) * 2) = make_float2(my_ref, my_sum);
            }
        }
    }

    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0 && a.err) atomicAdd(a.err, kTimeoutErr);
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
bool prepare_tc(const Args &a, TcLaunch *t) {
    if (a.dtype != BKV_BF16 || a.D != kD || a.NR > kN || a.max_ctx <= 0) return false;
    if (a.bs < 8 || !((kTcTile % a.bs == 0) || (a.bs % kTcTile == 0)) || a.H_kv > 65535) return false;
    if (a.total_blocks <= 0 || a.total_blocks * a.bs >= ((int64_t)1 << 31)) return false;
    if (!aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.q, 16) || !aligned(a.out, 8)) return false;
    if (!encode_fn()) return false;
    const uint64_t rows = (uint64_t)a.total_blocks * (uint64_t)a.bs;
    if (a.ks) {
        const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
        return encode_3d(&t->mk, a.k, kD, a.H_kv, rows, kD, (uint64_t)a.H_kv * kD, 128, 1, a.seg, u8) &&
               encode_3d(&t->mv, a.v, kD, a.H_kv, rows, kD, (uint64_t)a.H_kv * kD, 128, 1, a.seg, u8);
    }
    return encode_3d(&t->mk, a.k, kD, a.H_kv, rows, kD * 2, (uint64_t)a.H_kv * kD * 2, 64, 1, a.seg) &&
           encode_3d(&t->mv, a.v, kD, a.H_kv, rows, kD * 2, (uint64_t)a.H_kv * kD * 2, 64, 1, a.seg);
}

template <int NQ, bool kF8>
static int launch(const Args &a, const TcLaunch &t, cudaStream_t st) {
    auto kern = window_tc_kernel<NQ, kF8>;
    constexpr int smem = TcCfg<NQ, kF8>::kSmem;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return launch_status();
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    const cudaError_t e =
        launch_pdl(kern, dim3((unsigned)(a.P * a.H_kv * a.groups)), dim3(kTcThreads), smem, st, t.mk, t.mv, a);
    if (e != cudaSuccess) set_cuda_error(e);
    return launch_status();
}

// The softmax handles only the query rows that exist (4, 8 or 16 columns).
int launch_tc(const Args &a, const TcLaunch &t, cudaStream_t st) {
    if (a.ks) return a.NR <= 4 ? launch<4, true>(a, t, st) : a.NR <= 8 ? launch<8, true>(a, t, st) : launch<16, true>(a, t, st);
    return a.NR <= 4 ? launch<4, false>(a, t, st) : a.NR <= 8 ? launch<8, false>(a, t, st) : launch<16, false>(a, t, st);
}

}  // namespace win
}  // namespace bkv
