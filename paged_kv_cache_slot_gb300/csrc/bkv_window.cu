// bkv_window.cu -- attention over paged caches in two forms beside
// bkv_paged_decode's: E4M3 caches with a scale for each block of tokens and KV
// head, and sliding windows whose first tokens stay visible.  Entry points,
// planner, the CUDA-core kernel and the merge of shared streams (bf16 queries of
// head_dim 128 run the tcgen05 kernel of bkv_window_tc.cu).
//
// For a query row at position p of a request of length L ("Padding and
// Batching with Block KV", Cache Masking; a null or sentinel block entry
// contributes nothing):
//   s_j = scale q . k_j,  out = sum_j e^(s_j) v_j / sum_j e^(s_j)
// over the cached j <= p (or all j < L) with j > p - W or j < S.  E4M3 caches:
// k_j, v_j are the codes' values times the scale of their block and KV head.
// The window's first tokens are this library's reading of streaming attention;
// the pages print windows alone ("KV Caching with vLLM", Layer-specific cache
// specification).
//
// Only the blocks of [0, S) and of the window are read: a request's span
// (bkv_window.cuh) lays those two runs end to end, so that tiles waste nothing
// on the positions between them.
#include <math.h>

#include "bkv_eight.cuh"
#include "bkv_window.cuh"

namespace bkv {
namespace win {

static constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }

// ---------------------------------------------------------------------------
// CUDA-core kernel: any dtype, head_dim up to 256, block size and alignment.
//
// A CTA of four warps walks its column's units for one (KV head, row group).
// LP lanes hold a position's row, eight elements each, so a warp takes 32 / LP
// positions at a time and U of those a step.  A set of LP lanes sums its U NR scores
// across by halves: at each round a lane hands the other one the half that it does
// not keep, and ends with one or two scores of one query row, whose maximum, weights
// and sum are its own to keep; the weights go back through shared memory.  (Every
// lane with every score took log2 LP shuffles a score and all exponentials LP times:
// the first case below 196 us in place of 172 then.)  The sets are joined when the
// unit ends.
//
// Rows come by cp.async through a ring of kStages steps in shared memory, each
// lane copying exactly what it reads itself, so that the only wait is its own:
// what is in flight does not hang on the registers that the rows' arithmetic takes
// (12 KB a warp for bf16 rows and up to 4 query rows, 8 for fp32 ones; with 8 query
// rows 6 and 12; E4M3 7.5 and 4.5).
// An fp32 row is two runs of 16 bytes a lane (eight elements side by side asked for
// every sector twice: 809 us in place of 480 in the second case), and E4M3 scales
// are copied for a lane's own scores alone (for all U: the third 940 in place of 538).
// Where the rows stand is worked out for 32 positions at a time, a lane each, their
// block entries loaded that much ahead, and handed to the lanes that copy them by
// shuffles.  Multiply-adds go two an instruction.  What seldom runs is kept short, in
// loops that are not unrolled: the code of a step has to stay near (172 -> 140 us).
//
// 64 requests of 6000, 32 / 8 heads: bf16 heads of 64 140 us, 5.6 TB/s; fp32 heads of
// 128 480 us, 6.5 TB/s, near HBM's rate; E4M3 heads of 256 538 us, 2.9 TB/s: there, and
// with more query rows, bound by instructions at 12 warps an SM.  Small calls are bound
// by the chain of dependent loads and the code's first pass (13 requests of 33 to 5000
// in a window of 777, 15 / 5 heads of 64, fp32: 11.4 us).
// ---------------------------------------------------------------------------
constexpr int kCcThreads = 128;
constexpr int kCcTile = 64;

template <int NR>
constexpr int kCcPerSm = NR <= 4 ? 3 : 2;   // CTAs an SM is laid out for

// What a warp's ring holds a step, and a CTA's shared memory: the rings, and over them (a unit's steps are all read by
// then) the warps' outputs.
template <typename KV, int NR>
struct CcShape {
    static constexpr int U = NR <= 4 ? 4 : 2;
    static constexpr int kStages = sizeof(KV) * U == 16 ? 2 : 4;         // steps in a warp's ring
    static constexpr int kChunk = 8 * (int)sizeof(KV);                   // a lane's piece of a row
    static constexpr int kStep = U * 2 * kChunk * 32 + (sizeof(KV) == 1 ? 2 * 2 * 4 * 32 : 0);   // rows, and scales of two scores a lane
    static constexpr int kRing = 4 * kStages * kStep;
};
template <typename KV, int NR, int LP>
constexpr int kCcSmem = CcShape<KV, NR>::kRing > 4 * NR * 8 * LP * 4 ? CcShape<KV, NR>::kRing : 4 * NR * 8 * LP * 4;

__device__ __forceinline__ float two_to(float x) {   // 2^x, 2 units in the last place
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t shared_at(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// n bytes of `size` come from src, the others are 0.
template <int size>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, int n) {
    if constexpr (size == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(size), "r"(n) : "memory");
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

template <typename T, typename KV, int NR, int LP>
__global__ void __launch_bounds__(kCcThreads, kCcPerSm<NR>) window_cc_kernel(const Args a, const bool vec) {
    using S = CcShape<KV, NR>;
    constexpr int U = S::U, kStages = S::kStages;
    constexpr int PW = 32 / LP;          // positions a warp holds at once
    constexpr int DP = 8 * LP;
    constexpr bool kF8 = sizeof(KV) == 1;
    constexpr int kPiece = S::kChunk > 16 ? 16 : S::kChunk, kPieces = S::kChunk / kPiece;   // a copy, copies a chunk
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int32_t pre[kMaxReqs + 1], lens[kMaxReqs], sums[kCcThreads / 32];
    __shared__ float sm[4][NR], sl[4][NR];
    // A step has N scores a set of lanes.  Their sums over the lanes end with kOwn of them a lane, of one query row, which
    // keeps that row's maximum and sum with the row's other lanes; the weights go back to all lanes through shared memory
    // (two buffers in turn, so that one is written behind a __syncwarp that all passed after reading it).
    constexpr int N = U * NR, kOwn = N > LP ? N / LP : 1, kRowLanes = LP / NR;
    __shared__ __align__(16) float weights[4][2][PW][N];
    float(*so)[NR][DP] = reinterpret_cast<float(*)[NR][DP]>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = smem + warp * (kStages * S::kStep) + lane * kPiece;   // this lane's part of the warp's ring
    const uint32_t ring_s = shared_at(ring);
    // This lane's position of PW, and its elements: four from e0 on and four from e1 on, side by side but for fp32 rows,
    // of which they are two pieces that LP lanes copy as one run of the row each.
    constexpr bool kApart = sizeof(KV) == 4;
    const int sub = lane / LP, e0 = (lane % LP) * (kApart ? 4 : 8), e1 = e0 + (kApart ? 4 * LP : 4);
    const int own = (lane % LP) * N / LP, own_n = own / U, own_u = own % U;   // score n U + u: row n, position u
    const int row_lane = lane & -LP;                   // row n's first lane: row_lane + n kRowLanes
    const int ne = min(max(a.D - e0, 0), kApart ? 4 : 8), ne1 = min(max(a.D - e1, 0), 4);   // (ne counts both if side by side)
    auto load_row = [&](auto &x, const auto *row, bool whole) {
        if constexpr (kApart) {
            x.zero();
            if (whole) {
                const uint4 lo = ne > 0 ? __ldg(reinterpret_cast<const uint4 *>(row + e0)) : make_uint4(0, 0, 0, 0);
                const uint4 hi = ne1 > 0 ? __ldg(reinterpret_cast<const uint4 *>(row + e1)) : make_uint4(0, 0, 0, 0);
                x.w[0] = lo.x, x.w[1] = lo.y, x.w[2] = lo.z, x.w[3] = lo.w;
                x.w[4] = hi.x, x.w[5] = hi.y, x.w[6] = hi.z, x.w[7] = hi.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i < ne) x.w[i] = __float_as_uint(row[e0 + i]);
                    if (i < ne1) x.w[4 + i] = __float_as_uint(row[e1 + i]);
                }
            }
        } else {
            x.zero();
            if (ne > 0) x.load(row + e0, ne, whole);
        }
    };
    const int HP = a.H_kv * a.groups;
    const int q = (int)blockIdx.x / HP, hp = (int)blockIdx.x - q * HP;
    const int g = hp / a.groups, grp = hp - g * a.groups;
    const int i0 = grp * a.NR;
    const int rows = min(a.NR, a.q_len * a.G - i0);
    const int tok_lo = i0 / a.G, tok_hi = (i0 + rows - 1) / a.G;
    const int shift = (a.bs & (a.bs - 1)) == 0 ? 31 - __clz(a.bs) : -1;
    pdl_wait();
    pdl_trigger();
    lay_out<kCcThreads>(a, pre, lens, sums);
    Units units(pre, a.num_reqs, q, a.P);
    if (hp == 0 && threadIdx.x == 0) a.ws_split[q] = units.split();
    T *out = static_cast<T *>(a.out);
    auto out_row = [&](int r, int n) {
        const int t = (i0 + n) / a.G;
        return (((int64_t)r * a.q_len + t) * a.H_q + g * a.G + (i0 + n - t * a.G)) * a.D;
    };
    // requests without a cached position
    for (int r = q; r < a.num_reqs; r += a.P)
        if (pre[r + 1] == pre[r])
            for (int x = threadIdx.x; x < rows * a.D; x += kCcThreads) put(out + out_row(r, x / a.D) + x % a.D, 0.f);

    Unit x;
    while (units.next(x)) {
        const Span s = span_of(a, lens[x.r]);
        const int v_end = min((x.f + x.nt) * kCcTile, s.len);
        const int32_t *table = a.bt + (int64_t)x.r * a.bt_stride;
        constexpr int kStepPos = 4 * PW * U, kMine = PW * U;   // positions the CTA, and a warp of it, takes a step
        constexpr int kBatch = 32 / kMine;                      // steps whose places are worked out together
        const int v_first = x.f * kCcTile + warp * kMine;
        const int steps = (v_end - x.f * kCcTile + kStepPos - 1) / kStepPos;
        auto block_of = [&](int32_t p) { return shift >= 0 ? p >> shift : p / a.bs; };
        // Positions at or below last_lo (and from first_hi on, or below `sinks`) are seen by every row of the group.
        const int32_t t_lo = s.L - a.q_len + tok_lo, t_hi = s.L - a.q_len + tok_hi;
        const int32_t last_lo = a.causal ? t_lo : s.L - 1;
        const int32_t first_hi = a.window > 0 ? t_hi - a.window + 1 : INT32_MIN;
        // lane k of batch b: position k % kMine of step b kBatch + k / kMine
        auto span_at = [&](int b) { return v_first + (b * kBatch + lane / kMine) * kStepPos + lane % kMine; };
        auto fetch = [&](int b) -> int32_t {   // its block entry as it is in the table, 0 where there is none
            const int v = span_at(b);
            if (v >= v_end) return 0;
            const int32_t lb = block_of(s.pos(v));
            return lb < a.bt_cols ? __ldg(table + lb) : 0;
        };
        // where batch `b` stands: the row's first element of this head (-1: nothing there) and, E4M3, its scales; and,
        // as bits by lane, which positions are there, and are seen by every row
        int64_t place = -1;
        int64_t scale_at = -1;
        uint32_t there_bits = 0u, all_bits = 0u;
        auto locate = [&](int b, int32_t ent) {
            const bool there = ent > 0 && ent < a.total_blocks;
            const int32_t p = s.pos(span_at(b));
            place = -1;
            scale_at = -1;
            if (there) {
                place = (((int64_t)ent * a.bs + (p - block_of(p) * a.bs)) * a.H_kv + g) * a.D;
                scale_at = (int64_t)ent * a.H_kv + g;
            }
            there_bits = __ballot_sync(0xffffffffu, there);
            all_bits = __ballot_sync(0xffffffffu, there && p <= last_lo && (p >= first_hi || p < a.sinks));
        };
        // the rows (and scales) of step i, of the batch that was located last, into its ring slot; its positions that
        // are there, and, from bit 16 on, that every row sees
        auto issue = [&](int i) -> uint32_t {
            const uint32_t slot = (uint32_t)(i % kStages) * S::kStep;
            const int from = (i % kBatch) * kMine;
            constexpr int kRow = kPieces * 32 * kPiece;
            auto one = [&](int u, bool whole) {
                const int64_t at = __shfl_sync(0xffffffffu, place, from + u * PW + sub);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const KV *src = static_cast<const KV *>(kv ? a.v : a.k);
                    const uint32_t to = slot + (u * 2 + kv) * kRow;
                    if (whole) {
#pragma unroll
                        for (int c = 0; c < kPieces; ++c) {
                            const int n = at >= 0 && (c ? ne1 : ne) > 0 ? kPiece : 0;
                            copy_async<kPiece>(ring_s + to + c * (32 * kPiece), src + (n > 0 ? at + (c ? e1 : e0) : 0), n);
                        }
                    } else {
                        Eight<KV> e;
                        e.zero();
                        if (at >= 0) load_row(e, src + at, false);
#pragma unroll
                        for (int c = 0; c < kPieces; ++c)
#pragma unroll
                            for (int w = 0; w < kPiece / 4; ++w)
                                reinterpret_cast<uint32_t *>(ring + to + c * (32 * kPiece))[w] = e.w[c * (kPiece / 4) + w];
                    }
                }
            };
            if (vec) {
#pragma unroll
                for (int u = 0; u < U; ++u) one(u, true);
            } else {
#pragma unroll 1
                for (int u = 0; u < U; ++u) one(u, false);
            }
            if constexpr (kF8) {   // behind the rows, the scales of this lane's own scores
#pragma unroll
                for (int k = 0; k < kOwn; ++k) {
                    const int64_t sc = __shfl_sync(0xffffffffu, scale_at, from + (own_u + k) * PW + sub);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv)
                        copy_async<4>(ring_s + slot - lane * kPiece + U * 2 * S::kChunk * 32 + ((k * 2 + kv) * 32 + lane) * 4,
                                      (kv ? a.vs : a.ks) + (sc >= 0 ? sc : 0), sc >= 0 ? 4 : 0);
                }
            }
            constexpr uint32_t kBits = (1u << kMine) - 1u;
            return ((there_bits >> from) & kBits) | ((all_bits >> from) & kBits) << 16;
        };
        // bits of the steps in the ring, the next one to work on first
        uint32_t fifo[kStages];
        int32_t ent = fetch(0), ent_next = fetch(1);
        Eight<T> raw[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            raw[n].zero();
            if (n < rows) load_row(raw[n], static_cast<const T *>(a.q) + out_row(x.r, n), vec);
        }
#pragma unroll 1   // (code that runs once comes as slowly as it is long)
        for (int i = 0; i < kStages - 1; ++i) {
            if (i % kBatch == 0) {
                locate(i / kBatch, ent);
                ent = ent_next;
                ent_next = fetch(i / kBatch + 2);
            }
#pragma unroll
            for (int k = 0; k < kStages - 2; ++k) fifo[k] = fifo[k + 1];
            fifo[kStages - 2] = issue(i);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        float2 qv[NR][4], o[NR][4];
        float own_m = -INFINITY, own_l = 0.f;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = raw[n].two(i);
                qv[n][i] = make_float2(f.x * a.scale_log2, f.y * a.scale_log2);
                o[n][i] = make_float2(0.f, 0.f);
            }
        }
        const uint32_t full = (1u << rows) - 1u;
        // which of the rows see position p, as bits
        auto seen = [&](int32_t p) {
            uint32_t b = 0u;
            int32_t t = t_lo, h = i0 - tok_lo * a.G;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const bool last = p <= (a.causal ? t : s.L - 1);
                const bool near = a.window == 0 || p > t - a.window || p < a.sinks;
                b |= (last && near && n < rows) ? 1u << n : 0u;
                if (++h == a.G) {
                    h = 0;
                    ++t;
                }
            }
            return b;
        };
        for (int i = 0; i < steps; ++i) {
            {
                const int j = i + kStages - 1;
                if (j % kBatch == 0) {
                    locate(j / kBatch, ent);
                    ent = ent_next;
                    ent_next = fetch(j / kBatch + 2);
                }
                fifo[kStages - 1] = issue(j);
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
            const uint32_t here = fifo[0];
#pragma unroll
            for (int k = 0; k < kStages - 1; ++k) fifo[k] = fifo[k + 1];
            // every position of the step is there, and every row sees it
            constexpr uint32_t kBits = (1u << kMine) - 1u;
            const bool every = here == (kBits | kBits << 16);
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            const uint8_t *slot = ring + (i % kStages) * S::kStep;
            auto held = [&](int u, int kv) {
                Eight<KV> e;
                const uint8_t *src = slot + (u * 2 + kv) * kPieces * (32 * kPiece);
                if constexpr (kPiece == 8) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(src);
                    e.w[0] = w.x, e.w[1] = w.y;
                } else {
#pragma unroll
                    for (int c = 0; c < kPieces; ++c) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(src + c * (32 * kPiece));
                        e.w[4 * c] = w.x, e.w[4 * c + 1] = w.y, e.w[4 * c + 2] = w.z, e.w[4 * c + 3] = w.w;
                    }
                }
                return e;
            };
            float v[N];
            uint32_t see = 0u;   // bit u NR + n: row n sees position u
            if (!every) {
#pragma unroll 1
                for (int u = 0; u < U; ++u) {
                    const int k = u * PW + sub;
                    uint32_t bits = 0u;
                    if ((here >> k) & 1u) bits = (here >> (16 + k)) & 1u ? full : seen(s.pos(v_first + i * kStepPos + k));
                    see |= bits << (u * NR);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Eight<KV> k = held(u, 0);
                float2 acc[NR];
#pragma unroll
                for (int n = 0; n < NR; ++n) acc[n] = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 f = k.two(c);
#pragma unroll
                    for (int n = 0; n < NR; ++n) acc[n] = fma2(qv[n][c], f, acc[n]);
                }
#pragma unroll
                for (int n = 0; n < NR; ++n) v[n * U + u] = acc[n].x + acc[n].y;
            }
            // sums over the LP lanes: a lane hands over the half of its scores that the other one keeps
            {
                int have = N;
#pragma unroll
                for (int w = LP / 2; w > 0; w >>= 1) {
                    if (have > 1) {
                        have /= 2;
                        const bool upper = lane & w;
#pragma unroll
                        for (int k = 0; k < N / 2; ++k) {
                            if (k >= have) break;
                            const float keep = upper ? v[k + have] : v[k], give = upper ? v[k] : v[k + have];
                            v[k] = keep + __shfl_xor_sync(0xffffffffu, give, w);
                        }
                    } else {
                        v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
                    }
                }
            }
            const float *scales = reinterpret_cast<const float *>(slot - lane * kPiece + U * 2 * S::kChunk * 32) + lane;   // E4M3
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                if constexpr (kF8) v[k] *= scales[k * 64];
                if (!every && !((see >> ((own_u + k) * NR + own_n)) & 1u)) v[k] = -INFINITY;
                top = fmaxf(top, v[k]);
            }
            // a new maximum anywhere in the warp: all rescale (seldom, behind the first steps)
            if (__any_sync(0xffffffffu, top > own_m)) {
                top = fmaxf(top, own_m);
#pragma unroll
                for (int w = 1; w < kRowLanes; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                const float corr = top == -INFINITY ? 1.f : two_to(own_m - top);
                own_m = top;
                own_l *= corr;
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    const float by = __shfl_sync(0xffffffffu, corr, row_lane + n * kRowLanes);
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[n][c].x *= by, o[n][c].y *= by;
                }
            }
            float *wb = weights[warp][i & 1][sub];
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                float w = v[k] == -INFINITY ? 0.f : two_to(v[k] - own_m);
                own_l += w;
                if constexpr (kF8) {
                    w *= fminf(fmaxf(scales[k * 64 + 32], kScaleMin), kScaleMax);
                }
                wb[(own_u + k) * NR + own_n] = w;
            }
            __syncwarp();
            // a value that some rows do not see reaches only those that do, whatever it is
            auto values = [&](int u, uint32_t bits) {
                const Eight<KV> val = held(u, 1);
                float w[NR];
#pragma unroll
                for (int n = 0; n < NR; n += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(wb + u * NR + n);
                    w[n] = f.x, w[n + 1] = f.y, w[n + 2] = f.z, w[n + 3] = f.w;
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 f = val.two(c);
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        if ((bits >> n) & 1u) o[n][c] = fma2(make_float2(w[n], w[n]), f, o[n][c]);
                }
            };
            if (every) {
#pragma unroll
                for (int u = 0; u < U; ++u) values(u, ~0u);
            } else {
#pragma unroll 1
                for (int u = 0; u < U; ++u) values(u, see >> (u * NR));
            }
        }
        // Bad entries among the blocks that the unit begins, counted once a KV head: every block that the span
        // reads begins once in it, at its first position there.
        if (a.err && grp == 0) {
            for (int v = x.f * kCcTile + (int)threadIdx.x; v < v_end; v += kCcThreads) {
                const int32_t p = s.pos(v), lb = block_of(p);
                if (p != lb * a.bs && !(s.gap > 0 && v == s.sb && (s.sb == 0 || lb != block_of(s.sb - 1)))) continue;
                if (lb >= a.bt_cols || __ldg(table + lb) >= a.total_blocks) atomicAdd(a.err, 1);
            }
        }
        // join the warp's sets of lanes, then the warps
        auto join = [](float m0, float m1, float &f0, float &f1) {
            const float mn = fmaxf(m0, m1);
            f0 = mn == -INFINITY ? 1.f : exp2f(m0 - mn);
            f1 = mn == -INFINITY ? 1.f : exp2f(m1 - mn);
            return mn;
        };
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();   // every warp is through with its ring
        // (above 16 lanes a score stands in two)
#pragma unroll
        for (int w = LP > N ? LP / N : 1; w < kRowLanes; w <<= 1) own_l += __shfl_xor_sync(0xffffffffu, own_l, w);
        float m[NR], l[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            m[n] = __shfl_sync(0xffffffffu, own_m, row_lane + n * kRowLanes);
            l[n] = __shfl_sync(0xffffffffu, own_l, row_lane + n * kRowLanes);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int w = LP; w < 32; w <<= 1) {
                float f0, f1;
                const float mn = join(m[n], __shfl_xor_sync(0xffffffffu, m[n], w), f0, f1);
                l[n] = l[n] * f0 + __shfl_xor_sync(0xffffffffu, l[n], w) * f1;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    o[n][c].x = o[n][c].x * f0 + __shfl_xor_sync(0xffffffffu, o[n][c].x, w) * f1;
                    o[n][c].y = o[n][c].y * f0 + __shfl_xor_sync(0xffffffffu, o[n][c].y, w) * f1;
                }
                m[n] = mn;
            }
            if (lane < LP) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<float2 *>(&so[warp][n][c < 2 ? e0 + 2 * c : e1 + 2 * (c - 2)]) = o[n][c];
            }
            if (lane == 0) {
                sm[warp][n] = m[n];
                sl[warp][n] = l[n];
            }
        }
        __syncthreads();
        for (int y = threadIdx.x; y < rows * a.D; y += kCcThreads) {
            const int n = y / a.D, d = y - n * a.D;
            const float mn = fmaxf(fmaxf(sm[0][n], sm[1][n]), fmaxf(sm[2][n], sm[3][n]));
            float lsum = 0.f, acc = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float f = mn == -INFINITY ? 1.f : exp2f(sm[w][n] - mn);
                lsum = fmaf(f, sl[w][n], lsum);
                acc = fmaf(f, so[w][n][d], acc);
            }
            if (x.whole) {
                put(out + out_row(x.r, n) + d, acc * inverse(lsum));
            } else {
                const int64_t at = ((int64_t)hp * (2 * a.P) + x.slot) * a.NR + n;
                a.ws_o[at * a.D + d] = acc;
                if (d == 0) {
                    a.ws_ml[at * 2] = mn;
                    a.ws_ml[at * 2 + 1] = lsum;
                }
            }
        }
        __syncthreads();   // the rings are filled again
    }
}

// ---------------------------------------------------------------------------
// Merge of the streams that several columns share, one (column, KV head, row
// group) a CTA row: the at most one stream that column q begins and does not
// end.  A warp a query row.  Up to 32 parts and a head_dim of fours up to 128:
// lane k holds part k's maximum and sum, and four elements of eight parts at a
// time, so that up to 8 parts cost one round of loads behind the split's.  Bound
// by its launch and those two rounds.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 4;

template <typename T>
__global__ void __launch_bounds__(kMergeWarps * 32) window_merge_kernel(const Args a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int HP = a.H_kv * a.groups;
    const int q = (int)blockIdx.x / HP, hp = (int)blockIdx.x - q * HP;
    const int g = hp / a.groups, i0 = (hp - g * a.groups) * a.NR;
    const int n = blockIdx.y * kMergeWarps + warp, t = (i0 + n) / a.G;
    const int64_t in_req = ((int64_t)t * a.H_q + g * a.G + (i0 + n - t * a.G)) * a.D, req = (int64_t)a.q_len * a.H_q * a.D;
    const bool there = n < min(a.NR, a.q_len * a.G - i0);
    pdl_wait();
    pdl_trigger();
    const int2 e = a.ws_split[q];
    const int r = e.x, nch = e.y;
    if (nch == 0 || !there) return;
    auto at = [&](int c) { return ((int64_t)hp * (2 * a.P) + (c == 0 ? a.P + q : q + c)) * a.NR + n; };
    T *out = static_cast<T *>(a.out) + r * req + in_req;
    if (nch <= 32 && a.D <= 128 && a.D % 4 == 0) {
        const bool act = 4 * lane < a.D;
        const float2 ml = lane < nch ? *reinterpret_cast<const float2 *>(a.ws_ml + at(lane) * 2) : make_float2(-INFINITY, 0.f);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float w = 0.f, inv = 0.f;
        for (int c = 0; c < nch; c += 8) {
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = act && c + k < nch ? *reinterpret_cast<const float4 *>(a.ws_o + at(c + k) * a.D + 4 * lane)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
            if (c == 0) {
                float M = ml.x;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                w = M == -INFINITY ? 1.f : exp2f(ml.x - M);
                float l = w * ml.y;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                inv = inverse(l);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, (c + k) & 31);
                acc.x = fmaf(wk, v[k].x, acc.x), acc.y = fmaf(wk, v[k].y, acc.y);
                acc.z = fmaf(wk, v[k].z, acc.z), acc.w = fmaf(wk, v[k].w, acc.w);
            }
        }
        if (act) {
            put(out + 4 * lane, acc.x * inv);
            put(out + 4 * lane + 1, acc.y * inv);
            put(out + 4 * lane + 2, acc.z * inv);
            put(out + 4 * lane + 3, acc.w * inv);
        }
        return;
    }
    float M = -INFINITY;
    for (int c = lane; c < nch; c += 32) M = fmaxf(M, a.ws_ml[at(c) * 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int d0 = 0; d0 < a.D; d0 += 128) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f}, lsum = 0.f;
        for (int c0 = 0; c0 < nch; c0 += 32) {
            const int c = c0 + lane;
            const float2 ml = c < nch ? *reinterpret_cast<const float2 *>(a.ws_ml + at(c) * 2) : make_float2(-INFINITY, 0.f);
            const float w = M == -INFINITY ? 1.f : exp2f(ml.x - M);
            lsum = fmaf(w, ml.y, lsum);
#pragma unroll 8
            for (int k = 0; k < min(32, nch - c0); ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, k);
                const float *src = a.ws_o + at(c0 + k) * a.D;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = d0 + 32 * i + lane;
                    if (d < a.D) acc[i] = fmaf(wk, src[d], acc[i]);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
        const float inv = inverse(lsum);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = d0 + 32 * i + lane;
            if (d < a.D) put(out + d, acc[i] * inv);
        }
    }
}

// ---------------------------------------------------------------------------
// Planner
// ---------------------------------------------------------------------------
struct Split {
    int32_t NR, groups, P;
    int64_t rows() const { return (int64_t)2 * P * groups * NR; }   // partial rows a KV head
};

// Rows in equal groups of at most `most`; columns that fill `resident` CTAs, or, where one column nearly does, about
// four waves of them.
static Split make_split(int64_t nq, int64_t H_kv, int most, int64_t resident) {
    Split s;
    s.groups = (int32_t)ceil_div<int64_t>(nq, most);
    s.NR = (int32_t)ceil_div<int64_t>(nq, s.groups);
    s.groups = (int32_t)ceil_div<int64_t>(nq, s.NR);
    const int64_t HP = H_kv * s.groups;
    const int64_t P = 2 * HP <= resident ? resident / HP : ceil_div<int64_t>(4 * resident, HP);
    s.P = (int32_t)P;
    return s;
}

constexpr int kCcRows = 8;

struct Plan {
    Split tc, cc;
    size_t o_off, ml_off, ws_bytes;
};

static bool make_plan(int32_t num_reqs, int32_t q_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                      int32_t block_size, int32_t max_context_len, Plan *p) {
    if (num_reqs <= 0 || q_len <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        max_context_len < 0 || num_q_heads % num_kv_heads != 0 || block_size > 65536)
        return false;
    // the whole cost of a launch (kMaxReqs times the tiles of 64 positions and the ends) stays within int32
    if (max_context_len > 1 << 26) return false;
    const int64_t nq = (int64_t)q_len * (num_q_heads / num_kv_heads);
    const int64_t sms = current_sm_count();
    if (nq > 65536 || nq * num_kv_heads > (1 << 24)) return false;
    p->tc = make_split(nq, num_kv_heads, kTcRows, sms);
    const int64_t per_sm = nq <= 4 ? kCcPerSm<4> : kCcPerSm<kCcRows>;
    p->cc = make_split(nq, num_kv_heads, kCcRows, per_sm * sms);
    int64_t rows = p->cc.rows(), P = p->cc.P;
    if (head_dim == 128) {
        rows = p->tc.rows() > rows ? p->tc.rows() : rows;
        P = p->tc.P > P ? p->tc.P : P;
    }
    rows *= num_kv_heads;
    p->ml_off = (size_t)ceil_div<int64_t>(P * 8, 256) * 256;
    p->o_off = p->ml_off + (size_t)ceil_div<int64_t>(rows * 8, 256) * 256;
    p->ws_bytes = p->o_off + (size_t)rows * head_dim * 4;
    return true;
}

template <typename T, typename KV, int NR, int LP>
static int launch_cc(const Args &a, bool vec, cudaStream_t st) {
    auto kern = window_cc_kernel<T, KV, NR, LP>;
    constexpr int smem = kCcSmem<KV, NR, LP>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return launch_status();
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)(a.P * a.H_kv * a.groups)), dim3(kCcThreads), smem, st, a, vec);
    if (e != cudaSuccess) set_cuda_error(e);
    return launch_status();
}

template <typename T, typename KV, int NR>
static int launch_cc_lanes(const Args &a, bool vec, cudaStream_t st) {
    if (a.D <= 64) return launch_cc<T, KV, NR, 8>(a, vec, st);
    if (a.D <= 128) return launch_cc<T, KV, NR, 16>(a, vec, st);
    return launch_cc<T, KV, NR, 32>(a, vec, st);
}

template <typename T, typename KV>
static int launch_cc_rows(const Args &a, cudaStream_t st) {
    const bool vec = a.D % 8 == 0 && aligned(a.q, 16) && aligned(a.k, 16) && aligned(a.v, 16);
    return a.NR <= 4 ? launch_cc_lanes<T, KV, 4>(a, vec, st) : launch_cc_lanes<T, KV, kCcRows>(a, vec, st);
}

static int partition_cc(const Args &a, cudaStream_t st) {
    if (a.ks) {
        return a.dtype == BKV_BF16 ? launch_cc_rows<__nv_bfloat16, __nv_fp8_e4m3>(a, st)
                                   : launch_cc_rows<float, __nv_fp8_e4m3>(a, st);
    }
    return a.dtype == BKV_BF16 ? launch_cc_rows<__nv_bfloat16, __nv_bfloat16>(a, st) : launch_cc_rows<float, float>(a, st);
}

static int merge(const Args &a, cudaStream_t st) {
    const dim3 grid((unsigned)(a.P * a.H_kv * a.groups), (unsigned)ceil_div<int32_t>(a.NR, kMergeWarps));
    const cudaError_t e = a.dtype == BKV_BF16
                              ? launch_pdl(window_merge_kernel<__nv_bfloat16>, grid, dim3(kMergeWarps * 32), 0, st, a)
                              : launch_pdl(window_merge_kernel<float>, grid, dim3(kMergeWarps * 32), 0, st, a);
    if (e != cudaSuccess) set_cuda_error(e);
    return launch_status();
}

static int attend(const void *q, const void *k_cache, const void *v_cache, const float *k_scales, const float *v_scales,
                  bool fp8, const int32_t *block_table, int64_t bt_stride, int32_t bt_cols, const int32_t *context_lens,
                  int32_t max_context_len, int32_t num_reqs, int32_t q_len, int32_t num_q_heads, int32_t num_kv_heads,
                  int32_t head_dim, int32_t block_size, int64_t total_blocks, float softmax_scale, int mask_mode,
                  int32_t sliding_window, int32_t num_sinks, int dtype, void *out, void *workspace,
                  size_t workspace_bytes, int32_t *err_count, cudaStream_t stream) {
    if (dtype != BKV_BF16 && dtype != BKV_F32) return BKV_ERR_UNSUPPORTED;
    if (head_dim > 256 || head_dim % 2 != 0) return BKV_ERR_UNSUPPORTED;
    if (mask_mode != BKV_MASK_CAUSAL && mask_mode != BKV_MASK_ALL) return BKV_ERR_INVALID_ARG;
    if (sliding_window < 0 || num_sinks < 0) return BKV_ERR_INVALID_ARG;
    if (bt_cols < 0 || bt_stride < bt_cols || total_blocks < 0) return BKV_ERR_INVALID_ARG;
    Plan plan;
    if (!make_plan(num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, &plan))
        return BKV_ERR_INVALID_ARG;
    if (!q || !out || !context_lens || (bt_cols > 0 && !block_table)) return BKV_ERR_INVALID_ARG;
    if (max_context_len > 0 && (!k_cache || !v_cache || (fp8 && (!k_scales || !v_scales)))) return BKV_ERR_INVALID_ARG;
    if (workspace_bytes < plan.ws_bytes || !workspace || !aligned(workspace, 32)) return BKV_ERR_INVALID_ARG;
    if (!(softmax_scale > 0.f)) softmax_scale = 1.0f / sqrtf((float)head_dim);
    Args a{};
    a.k = k_cache;
    a.v = v_cache;
    a.ks = fp8 ? k_scales : nullptr;
    a.vs = fp8 ? v_scales : nullptr;
    a.bt_stride = bt_stride;
    a.bt_cols = bt_cols;
    a.max_ctx = max_context_len;
    a.q_len = q_len;
    a.H_q = num_q_heads;
    a.H_kv = num_kv_heads;
    a.D = head_dim;
    a.bs = block_size;
    a.G = num_q_heads / num_kv_heads;
    a.total_blocks = total_blocks;
    a.scale_log2 = softmax_scale * kLog2e;
    a.causal = mask_mode == BKV_MASK_CAUSAL;
    a.window = sliding_window < max_context_len ? sliding_window : 0;   // (a window that reaches every position is none)
    a.sinks = num_sinks;
    a.dtype = dtype;
    a.err = err_count;
    char *ws = static_cast<char *>(workspace);
    a.ws_split = reinterpret_cast<int2 *>(ws);
    a.ws_ml = reinterpret_cast<float *>(ws + plan.ml_off);
    a.ws_o = reinterpret_cast<float *>(ws + plan.o_off);
    const size_t e = dtype == BKV_BF16 ? 2 : 4;
    const int64_t req_elems = (int64_t)q_len * num_q_heads * head_dim;
    // requests whose lengths a CTA keeps at a time; more go in launches behind one another, which share the workspace
    for (int64_t r0 = 0; r0 < num_reqs; r0 += kMaxReqs) {
        a.num_reqs = (int32_t)(num_reqs - r0 < kMaxReqs ? num_reqs - r0 : kMaxReqs);
        a.q = static_cast<const char *>(q) + (size_t)r0 * req_elems * e;
        a.out = static_cast<char *>(out) + (size_t)r0 * req_elems * e;
        a.bt = block_table ? block_table + r0 * bt_stride : nullptr;
        a.ctx = context_lens + r0;
        TcLaunch t;
        a.seg = block_size < 128 ? block_size : 128;
        a.tile = 128;
        a.NR = plan.tc.NR;
        a.groups = plan.tc.groups;
        a.P = plan.tc.P;
        const bool tc = prepare_tc(a, &t);
        if (!tc) {
            a.seg = 1;
            a.tile = kCcTile;
            a.NR = plan.cc.NR;
            a.groups = plan.cc.groups;
            a.P = plan.cc.P;
        }
        int rc = tc ? launch_tc(a, t, stream) : partition_cc(a, stream);
        if (rc != BKV_OK) return rc;
        rc = merge(a, stream);
        if (rc != BKV_OK) return rc;
    }
    return BKV_OK;
}

}  // namespace win
}  // namespace bkv

extern "C" size_t bkv_paged_decode_window_workspace_size(int32_t num_reqs, int32_t q_len, int32_t num_q_heads,
                                                         int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                                         int32_t max_context_len) {
    bkv::win::Plan p;
    if (head_dim > 256 || head_dim % 2 != 0 ||
        !bkv::win::make_plan(num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, &p))
        return 0;
    return p.ws_bytes;
}

extern "C" int bkv_paged_decode_sink(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
                                     int64_t bt_stride, int32_t bt_cols, const int32_t *context_lens,
                                     int32_t max_context_len, int32_t num_reqs, int32_t q_len, int32_t num_q_heads,
                                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t total_blocks,
                                     float softmax_scale, int mask_mode, int32_t sliding_window, int32_t num_sinks,
                                     int dtype, void *out, void *workspace, size_t workspace_bytes, int32_t *err_count,
                                     bkv_stream_t stream) {
    return bkv::win::attend(q, k_cache, v_cache, nullptr, nullptr, false, block_table, bt_stride, bt_cols, context_lens,
                            max_context_len, num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                            total_blocks, softmax_scale, mask_mode, sliding_window, num_sinks, dtype, out, workspace,
                            workspace_bytes, err_count, (cudaStream_t)stream);
}

extern "C" int bkv_paged_decode_fp8_blocks(const void *q, const uint8_t *k_cache, const uint8_t *v_cache,
                                           const float *k_scales, const float *v_scales, const int32_t *block_table,
                                           int64_t bt_stride, int32_t bt_cols, const int32_t *context_lens,
                                           int32_t max_context_len, int32_t num_reqs, int32_t q_len,
                                           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                           int32_t block_size, int64_t total_blocks, float softmax_scale, int mask_mode,
                                           int32_t sliding_window, int32_t num_sinks, int dtype, void *out,
                                           void *workspace, size_t workspace_bytes, int32_t *err_count,
                                           bkv_stream_t stream) {
    return bkv::win::attend(q, k_cache, v_cache, k_scales, v_scales, true, block_table, bt_stride, bt_cols,
                            context_lens, max_context_len, num_reqs, q_len, num_q_heads, num_kv_heads, head_dim,
                            block_size, total_blocks, softmax_scale, mask_mode, sliding_window, num_sinks, dtype, out,
                            workspace, workspace_bytes, err_count, (cudaStream_t)stream);
}
