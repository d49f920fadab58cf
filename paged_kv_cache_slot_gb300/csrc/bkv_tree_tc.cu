// bkv_tree_tc.cu -- tensor-core (tcgen05 + TMA) kernel of the attention of
// drafted trees: bf16, head_dim 128, any tree and any group size up to 128.
//
// For a stream (request, KV head, token group) and a run of its 128-position
// tiles: S = Q K^T, an online softmax under the tree's mask, O += P V ("Padding
// and Batching with Block KV", Cache Masking).  The cache is read once for all
// the rows of a group; a stream that one CTA finishes is written to `out`
// there, one that several CTAs share leaves partials for the merge.
//
// Design (sm_103a):
// * Schedule: the grid is P columns of one CTA per (KV head, token group).  The
//   requests are laid end to end by cost: a tile of positions costs 1, a
//   request's end kEndCost behind its tiles.  With C the whole cost, column q <
//   peff = min(P, ceil(C / kMinCost)) takes the tiles in [q C / peff, (q + 1)
//   C / peff): shares of equal cost whatever the lengths, their numbers of tiles
//   differing by the ends in them (a share may be an end alone, without a tile);
//   columns from peff on have nothing.  A column's CTAs read the same positions
//   of all heads together.
// * A query tile is 128 / G tokens times the G heads, rows (token, head): one
//   3-D TMA box of q.  A group of at most one query tile runs its key tiles
//   alternately on two softmax streams with their own S, P and O (columns of
//   tensor memory), so that one stream's softmax runs beside the other's MMAs;
//   their O are joined when the unit ends.  A group of two query tiles gives
//   each its own stream, and every K and V tile serves both.
// * Warp roles (384 threads): warp 0 loads Q and gathers K tiles, warp 2 gathers
//   V tiles (rings of two or three 32 KB slots each, as the queries leave room),
//   warps 1 and 3 issue the MMAs, one thread each; four softmax warps a stream,
//   one query row a thread.  A row's 128 scores stay in its thread's registers
//   between the max and the weights: the lanes' quarters are tied to the SM's
//   four partitions, so two warps a row would share one exponential unit anyway
//   (128 rows of a tile take 1024 cycles of it) and pay for exchanging their
//   maxima.  Quarters without rows mend the V tiles instead (below).
// * P (bf16, two per column) goes over its own S columns and enters P V from
//   tensor memory.  bf16 since the tensor cores take both operands of a product
//   in one type and V is bf16: each weight is off by 2^-8 of itself at most, at
//   random, while the sum l is of the fp32 weights.  Outputs' errors against 64
//   bits, all of a case over its norm: 0.0019 with 4 tokens of 4 heads, 0.0022
//   and 0.0023 with 16 and 61 tokens, where fp32 weights leave 0.0017, the
//   outputs' own rounding.  The running max is a lazy reference (it moves when a tile's
//   max passes it by 8 in log2 units), so O is seldom rescaled.
// * Masks: tiles wholly before the tree and without null entries take no
//   per-key tests.  V rows that were not loaded, or lie at or past the cache
//   end, are zeroed in shared memory before P V; a V row of the tree that is not
//   finite is zeroed too and remembered, and rows that see it become NaN.
// * Every wait is bounded (~2 s), after which the CTA records 1 << 24 in
//   err_count, frees its tensor memory and exits.
//
// Measured (device time of a call with its merge; 128-element heads, bf16): 256
// requests of 9 to 8192 positions, 4 tokens of 32 / 8 heads (16 rows a group)
// 217 us, 5.9 TB/s of K and V; 32 of 512 to 4096, 16 tokens (64 rows) 51 us, 4.6
// TB/s: 9 us of it launches, the first tiles and the merge; 8 of 1000 to 16693,
// 61 tokens of 64 / 8 heads (488 rows) 105 us, 0.84 PFLOP/s of the products
// that the rows need: there the two streams' softmaxes take turns at the
// exponential units with the products, and neither pipe is kept full.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "bkv_tc_ptx.cuh"
#include "bkv_tree.cuh"

namespace bkv {
namespace ttc {

using namespace tc;

constexpr int kTile = kTreeTile;
constexpr int kD = 128;
constexpr int kHalfBytes = kTile * 128;
constexpr int kTileBytes = 2 * kHalfBytes;
constexpr int kThreads = 384;   // K producer, MMA issuers (1 and 3), V producer; 2 x 4 softmax warps
constexpr int kWarpV = 2;
constexpr int kWarpS = 4;   // first softmax warp
constexpr int kTmemCols = 512;   // S and P of streams 0, 1, O of streams 0, 1 (128 columns each)
constexpr int kTimeoutErr = 1 << 24;
constexpr int kMaxReqs = 2048;
constexpr float kSlack = 8.f;
// Tiles that a unit's end takes as long as, and what a column takes of both at least (fewer columns leave fewer
// partials): 256 requests of 9 to 8192 positions 217 us, 221 with 3 or without the least, 227 with 1 or 4; 3 requests
// of up to 13459, 12 tokens of 16 / 2 heads: 18.3 us, 22.8 without the least.
constexpr int kEndCost = 2, kMinCost = 2;

constexpr int kMaxStages = 3;                             // slots of a ring, at most
constexpr int kOffMask = 0;                               // 8 words: loaded segments per tile (ring)
constexpr int kOffPoison = kOffMask + 8 * 4;              // 8 x 32 bytes: V rows of the tile that are not finite
constexpr int kOffBar = kOffPoison + 8 * 32;
constexpr int kNumBars = 2 * 8 + 2 * kMaxStages + 4 + 2 + 2 + 2 + 8 + 4;
constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
constexpr int kOffAbort = kOffTmemSlot + 4;
constexpr int kOffAnyBad = kOffAbort + 4;                 // a V row that was not finite has been met
constexpr int kOffSums = kOffAnyBad + 4;                  // [warps] prefix sum's scratch
constexpr int kOffPre = (kOffSums + kThreads / 32 * 4 + 15) / 16 * 16;   // [kMaxReqs + 1] tiles before request r
constexpr int kOffFill = kOffPre + (kMaxReqs + 4) * 4;    // [kMaxReqs] positions of its last tile, less one
// Sets of the streams' exchange at a unit's end, used in turn: a stream with no tile of the next unit, or one, writes
// its next entries while its partner may still read the last; before it writes the ones after those, the barrier of the
// unit between has seen the partner past them.  (A second barrier phase in place of the second set: 256 requests of 9 to
// 8192 positions 217 -> 220 us, 700 of 9 to 200 194 -> 200.)
constexpr int kXmSets = 2;
constexpr int kOffXm = kOffFill + kMaxReqs;               // [set][stream][row] running max, weight sum
// queries, then the K and V rings: what a launch needs of the rest (see ring_shape)
constexpr int kOffQ = (kOffXm + kXmSets * 2 * kTile * 8 + 1023) / 1024 * 1024;
constexpr int kSmemMax = 227 * 1024 - 1024;               // less the slack for 1024 alignment

// A ring slot and its phase parity.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void advance(int n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

__host__ __device__ constexpr uint32_t col_s(int x) { return 128u * (uint32_t)x; }
__host__ __device__ constexpr uint32_t col_o(int x) { return 256u + 128u * (uint32_t)x; }

// 32 bytes of one row (a whole sector: a thread's rows lie apart, and 16-byte
// stores would touch each line twice as often).
__device__ __forceinline__ void store32(void *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 32 fp32 columns of this thread's lane, without the wait; use32 after it keeps
// the compiler from reading them earlier.
__device__ __forceinline__ void tmem_ld32_nw(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void use32(float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(v[i]));
}

__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// Max of 32 values, three at a time.
__device__ __forceinline__ float max32(const float (&v)[32]) {
    float t[11];
#pragma unroll
    for (int i = 0; i < 10; ++i) t[i] = max3(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
    t[10] = fmaxf(v[30], v[31]);
    return max3(max3(max3(t[0], t[1], t[2]), max3(t[3], t[4], t[5]), max3(t[6], t[7], t[8])), t[9], t[10]);
}

// Two fp32 operations in one instruction, each rounded as the single one.
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %5};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// One unit: tiles [f, f + nt) of request r.  whole: they are all of its tiles.
struct Unit {
    int r, L, f, nt, slot;
    bool whole;
};

// Walks this CTA's units.  pre[r] is the cost of the requests before r: a tile
// costs 1 and a unit's end (the last softmax, the wait for the last P V, the
// output: nothing else runs meanwhile) kEndCost, laid behind the request's
// tiles.  Column q takes the tiles in its share of the whole cost.
struct Units {
    const int32_t *pre;
    const uint8_t *fill;
    int r, q, t, t1, P;
    // Columns that share a cost of C.
    __device__ static int64_t columns(int64_t C, int64_t P) {
        const int64_t most = (C + kMinCost - 1) / kMinCost;
        return most < P ? most : P;
    }
    __device__ Units(const TreeArgs &a, const int32_t *pre_, const uint8_t *fill_, int q_) {
        pre = pre_;
        fill = fill_;
        q = q_;
        P = a.P;
        const int64_t C = pre[a.num_reqs];
        const int64_t peff = columns(C, a.P);
        t = (int)(q < peff ? C * q / peff : C);
        t1 = (int)(q < peff ? C * (q + 1) / peff : C);
        int lo = 0, hi = a.num_reqs;   // first request whose cost ends after t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid + 1] > t) hi = mid;
            else lo = mid + 1;
        }
        r = lo;
    }
    // The stream that this column begins and does not end (before next() is called): its request and how
    // many columns share it; 0 without one.
    __device__ int2 split(const TreeArgs &a) const {
        if (t >= t1) return make_int2(0, 0);
        int r1 = r;
        while (pre[r1 + 1] < t1) ++r1;   // the request that the share ends in
        const int s = pre[r1], e = pre[r1 + 1] - kEndCost;   // its tiles
        if (s < t || s >= t1 || e <= t1) return make_int2(0, 0);
        const int64_t C = pre[a.num_reqs], peff = columns(C, a.P);
        const int q1 = (int)((e * peff - 1) / C);   // the column of its last tile
        return make_int2(r1, q1 - q + 1);
    }
    __device__ bool next(Unit &x) {
        for (; t < t1; ++r) {
            const int s = pre[r], e = pre[r + 1] - kEndCost;
            if (pre[r + 1] <= t) continue;   // no tiles (or passed)
            const int lo = t, hi = t1 < e ? t1 : e;
            t = pre[r + 1];
            if (lo >= hi) continue;   // only the end's share of the request is this column's
            x.r = r;
            x.f = lo - s;
            x.nt = hi - lo;
            x.L = (e - s - 1) * kTile + fill[r] + 1;
            x.whole = lo == s && hi == e;
            x.slot = lo == s ? P + q : q;
            ++r;
            return true;
        }
        return false;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ CUtensorMap tmQ, const TreeArgs a, const TreeShape sh) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    volatile uint32_t *mask_words = reinterpret_cast<uint32_t *>(smem + kOffMask);
    uint8_t *poison = smem + kOffPoison;   // [tile & 7][32], four rows a byte
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffTmemSlot);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffAbort);
    int32_t *warp_sums = reinterpret_cast<int32_t *>(smem + kOffSums);
    volatile int *any_bad = reinterpret_cast<volatile int *>(smem + kOffAnyBad);
    int32_t *pre = reinterpret_cast<int32_t *>(smem + kOffPre);
    uint8_t *fill = smem + kOffFill;
    const uint32_t bar0 = sbase + kOffBar;
    // Tile j's K and V have landed: by tile, not by slot.  Where the tiles alternate, an MMA thread looks at its
    // own stream's only, and a parity answers at once for a phase whose predecessor it has not seen end; of
    // eight barriers each belongs to one stream (8 is even).
    auto bar_kfull = [&](int j) { return bar0 + 8u * (j & 7); };
    auto bar_vfull = [&](int j) { return bar0 + 8u * (8 + (j & 7)); };
    auto phase_of = [](int j) { return (uint32_t)(j >> 3) & 1u; };
    auto bar_kempty = [&](int s) { return bar0 + 8u * (16 + s); };
    auto bar_vempty = [&](int s) { return bar0 + 8u * (16 + kMaxStages + s); };
    constexpr int kB = 16 + 2 * kMaxStages;
    auto bar_qfull = [&](int b) { return bar0 + 8u * (kB + b); };
    auto bar_qempty = [&](int b) { return bar0 + 8u * (kB + 2 + b); };
    auto bar_sfull = [&](int x) { return bar0 + 8u * (kB + 4 + x); };
    auto bar_pfull = [&](int x) { return bar0 + 8u * (kB + 6 + x); };
    const uint32_t bar_ofull = bar0 + 8u * (kB + 8);
    const uint32_t bar_oempty = bar0 + 8u * (kB + 9);
    auto bar_mask = [&](int m) { return bar0 + 8u * (kB + 10 + m); };
    // the two streams' warps of a lane quarter: their entries of a unit are written
    auto bar_pair = [&](int qw) { return bar0 + 8u * (kB + 18 + qw); };
    const int seg_rows = sh.seg_rows, tok_per_tile = sh.tok_per_tile, box_tok = sh.box_tok;
    const int nK = sh.k_stages, nV = sh.v_stages;
    const int off_v = kOffQ + sh.q_bytes + nK * kTileBytes;
    const uint32_t sm_q = sbase + kOffQ;
    const uint32_t sm_k = sm_q + sh.q_bytes;
    const uint32_t sm_v = sbase + off_v;

    // what this CTA is: column q, KV head g, token group p, and its rows
    const int G = a.G;
    const int HP = a.H_kv * a.groups;
    const int q = (int)blockIdx.x / HP, hp = (int)blockIdx.x - q * HP;
    const int g = hp / a.groups, p = hp - g * a.groups;
    const int tok0 = p * a.TS;
    const int ntok = min(a.TS, a.T - tok0);
    const bool dual = ntok > tok_per_tile;   // two query tiles, every key tile for both
    const int rows0 = (dual ? tok_per_tile : ntok) * G;
    const int rows1 = dual ? (ntok - tok_per_tile) * G : rows0;
    const int aq0 = (rows0 + 31) >> 5, aq1 = (rows1 + 31) >> 5;   // lane quarters with rows
    // units whose queries fit (a group of two tiles takes both buffers)
    const int nbuf = dual ? 1 : sh.q_buffers;

    if (threadIdx.x == 0) {
        for (int j = 0; j < 8; ++j) {
            mbar_init(bar_kfull(j), 1);
            mbar_init(bar_vfull(j), 1);
            mbar_init(bar_mask(j), 1);
        }
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(bar_kempty(s), 1);
            mbar_init(bar_vempty(s), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar_qfull(x), 1);
            mbar_init(bar_qempty(x), dual ? 1 : 2);
            mbar_init(bar_sfull(x), 1);
            mbar_init(bar_pfull(x), (!dual || x == 0) ? 4 : aq1);
        }
        mbar_init(bar_ofull, dual ? 2 : 4);
        mbar_init(bar_oempty, aq0 + aq1);
        for (int qw = 0; qw < 4; ++qw) mbar_init(bar_pair(qw), 2);
        *abort_flag = 0;
        *any_bad = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        prefetch_tmap(&tmQ);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();   // global memory is read from here on
    pdl_trigger();
    // costs of the requests and their exclusive prefix sum: a run of requests a thread
    {
        const int n = a.num_reqs, per = (n + kThreads - 1) / kThreads;
        const int lo = min(n, (int)threadIdx.x * per), hi = min(n, lo + per);
        int32_t sum = 0;
        for (int r = lo; r < hi; ++r) {
            const int32_t c = __ldg(a.ctx + r);
            const int32_t L = tree_len(a, c);
            if (c > a.max_ctx && blockIdx.x == 0 && a.err) atomicAdd(a.err, 1);
            fill[r] = (uint8_t)((L - 1) & (kTile - 1));
            const int32_t cost = L > 0 ? (L + kTile - 1) / kTile + kEndCost : 0;
            pre[r] = cost;
            sum += cost;
        }
        int32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) warp_sums[warp] = inc;
        __syncthreads();
        int32_t run = inc - sum;
        for (int w = 0; w < warp; ++w) run += warp_sums[w];
        for (int r = lo; r < hi; ++r) {
            const int32_t cost = pre[r];
            pre[r] = run;
            run += cost;
        }
        if (threadIdx.x == kThreads - 1) pre[n] = run;
    }
    __syncthreads();
    const uint32_t tmem = *tmem_slot;
    const int nseg = kTile / seg_rows;
    const int seg_shift = 31 - __clz(seg_rows);
    const uint32_t all_seg = (1u << nseg) - 1u;   // at most 16 segments

    // V rows of a tile that must not reach P V are zeroed: not loaded, at or past the cache end (row lim), or
    // of the tree (from row fst) and not finite, which is remembered.  Warp wi of the nw that share a tile.
    auto fix_v = [&](int slot, int jj, uint32_t mword, int fst, int lim, int wi, int nw) {
        fst = max(fst, 0);
        uint4 *v0 = reinterpret_cast<uint4 *>(smem + off_v + slot * kTileBytes);   // 8 a row
        uint4 *v1 = v0 + kHalfBytes / 16;
        auto zero_rows = [&](int r0, int r1) {
#pragma unroll 4
            for (int e = 8 * r0 + 32 * wi + lane; e < 8 * r1; e += 32 * nw)
                v0[e] = v1[e] = make_uint4(0, 0, 0, 0);
        };
        for (uint32_t miss = ~mword & all_seg; miss; miss &= miss - 1) {
            const int r0 = (__ffs(miss) - 1) * seg_rows;
            if (r0 < lim) zero_rows(r0, r0 + seg_rows);
        }
        if (fst < kTile) {
            zero_rows(lim, kTile);
            // the tree's rows: four at a time, eight lanes a row (16 bytes of each half)
            const int g0 = fst >> 2, g1 = (min(lim, kTile) + 3) >> 2;
            uint8_t *bad_rows = poison + (jj & 7) * 32;
            if (wi == 0 && (lane < g0 || lane >= g1)) bad_rows[lane] = 0;
            for (int i = g0 + wi; i < g1; i += nw) {
                const int e = 32 * i + lane, vrow = 4 * i + (lane >> 3);
                const uint4 p0 = v0[e], p1 = v1[e];
                const uint32_t ws[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
                bool bad = false;
#pragma unroll
                for (int h = 0; h < 8; ++h)   // an exponent of all ones in either half
                    bad |= (ws[h] & 0x7f80u) == 0x7f80u || (ws[h] & 0x7f800000u) == 0x7f800000u;
                bad &= vrow >= fst && vrow < lim && ((mword >> (vrow >> seg_shift)) & 1u);
                const uint32_t m8 = __ballot_sync(0xffffffffu, bad);
                uint32_t rows = 0u;
                if (m8) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) rows |= ((m8 >> (8 * h)) & 0xffu) ? 1u << h : 0u;
                    if ((rows >> (lane >> 3)) & 1u) v0[e] = v1[e] = make_uint4(0, 0, 0, 0);
                    if (lane == 0) *any_bad = 1;
                }
                if (lane == 0) bad_rows[i] = (uint8_t)rows;
            }
        }
        fence_proxy_async();
    };

    // A row's scores need more registers than the launch gives each thread (168): the first warpgroup hands
    // some of its own over (4 x 32 x 96 + 8 x 32 x 200 of 12 x 32 x 168).
    if (warp < kWarpS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == 0 || warp == kWarpV) {
            // ================= TMA producers (warp 0: Q and K, warp 2: V) =================
            const bool is_v = warp == kWarpV;
            const bool count = !is_v && p == 0 && a.err;   // bad entries count once a KV head
            const int stages = is_v ? nV : nK;
            Ring ring;
            int j = 0, uq = 0;
            Units units(a, pre, fill, q);
            Unit x;
            for (; !*abort_flag && units.next(x); ++uq) {
                if (!is_v) {
                    const int b = nbuf == 2 ? uq & 1 : 0;
                    if (!mbar_wait_warp(bar_qempty(b), (uint32_t)((nbuf == 2 ? uq >> 1 : uq) & 1) ^ 1u, abort_flag)) break;
                    if (lane == 0) {
                        const uint32_t bytes = (uint32_t)(box_tok * G) * 256u;
                        mbar_arrive_expect_tx(bar_qfull(b), dual ? 2 * bytes : bytes);
                        for (int xb = 0; xb < (dual ? 2 : 1); ++xb) {
                            const int tq = x.r * a.T + tok0 + xb * tok_per_tile;
                            const uint32_t dq = sm_q + (b + xb) * 2 * sh.q_half;
                            tma_load_3d(dq, &tmQ, bar_qfull(b), 0, g * G, tq);
                            tma_load_3d(dq + sh.q_half, &tmQ, bar_qfull(b), 64, g * G, tq);
                        }
                    }
                }
                // block entry of this lane's segment of key tile kt: the cache row to load, or -1
                auto entry = [&](int kt) -> int64_t {
                    if (lane >= nseg) return -1;
                    const int32_t p0 = kt * kTile + lane * seg_rows;
                    if (p0 >= x.L) return -1;
                    const int32_t lb = p0 / a.bs;
                    const int32_t off = p0 - lb * a.bs;
                    const int64_t e = lb < a.bt_cols ? __ldg(a.bt + (int64_t)x.r * a.bt_stride + lb) : a.total_blocks;
                    if (e >= a.total_blocks) {
                        if (count && off == 0) atomicAdd(a.err, 1);
                        return -1;
                    }
                    return e > 0 ? e * a.bs + off : -1;
                };
                int64_t row_cur = entry(x.f);
                for (int kt = 0; kt < x.nt; ++kt, ++j) {
                    const int64_t row_nxt = kt + 1 < x.nt ? entry(x.f + kt + 1) : -1;   // in flight meanwhile
                    const int s = ring.slot;
                    const uint32_t bar_e = is_v ? bar_vempty(s) : bar_kempty(s);
                    const uint32_t bar_f = is_v ? bar_vfull(j) : bar_kfull(j);
                    if (!mbar_wait_warp(bar_e, ring.phase ^ 1u, abort_flag)) break;
                    ring.advance(stages);
                    const bool load = row_cur >= 0;
                    const uint32_t ballot = __ballot_sync(0xffffffffu, load);
                    if (lane == 0) {
                        // a word is rewritten 8 tiles on; its readers are at most 5 tiles behind
                        if (!is_v) {
                            mask_words[j & 7] = ballot;
                            mbar_arrive(bar_mask(j & 7));
                        }
                        mbar_arrive_expect_tx(bar_f, (uint32_t)__popc(ballot) * (uint32_t)seg_rows * 256u);
                    }
                    __syncwarp();
                    if (load) {
                        const uint32_t dst = (is_v ? sm_v : sm_k) + s * kTileBytes + lane * seg_rows * 128;
                        const CUtensorMap *map = is_v ? &tmV : &tmK;
                        tma_load_3d(dst, map, bar_f, 0, g, (int)row_cur);
                        tma_load_3d(dst + kHalfBytes, map, bar_f, 64, g, (int)row_cur);
                    }
                    __syncwarp();
                    row_cur = row_nxt;
                }
            }
            if (*abort_flag) {   // let copies in flight land
                const unsigned long long t0 = global_ns();
                while (global_ns() - t0 < 200000ull) {
                }
            }
        } else {
            // ================= MMA issuers (one thread each) =================
            // A stream's tiles in turn: O += P V of its last one, then S of the next over the same columns (one
            // thread's MMAs run in issue order).  Where the tiles alternate each stream has its own thread, so
            // that one's barriers are waited for while the other's products run (32 requests of 512 to 4096
            // positions, 16 tokens of 32 / 8 heads: 51.3 us, 53.7 with one thread).  Two query tiles share every K
            // and V tile, and two threads drift apart over them: there warp 1 issues both (8 requests of 1000 to
            // 16693 positions, 61 tokens of 64 / 8 heads: 105 us, 118 with two threads).
            if (lane == 0 && (!dual || warp == 1)) {
                constexpr uint32_t kIdescS = idesc_bf16(128, 128, 0, 0);   // Q (K-major) x K (K-major)
                constexpr uint32_t kIdescO = idesc_bf16(128, 128, 0, 1);   // P (TMEM) x V (MN-major)
                uint32_t pphase = 0u;   // bit x: P of stream x
                // O_xb += P_xb V(tile): `first` overwrites O_xb, once the unit before has been read out
                auto issue_pv = [&](int xb, int tile, int slot, bool first, int unit) -> bool {
                    if (!mbar_wait(bar_vfull(tile), phase_of(tile), abort_flag) ||
                        !mbar_wait(bar_pfull(xb), (pphase >> xb) & 1u, abort_flag))
                        return false;
                    pphase ^= 1u << xb;
                    if (first && unit > 0 && !mbar_wait(bar_oempty, (uint32_t)((unit - 1) & 1), abort_flag)) return false;
                    tc_fence_after();
                    const uint32_t v_base = sm_v + slot * kTileBytes;
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_bf16_ts(tmem + col_o(xb), tmem + col_s(xb) + 8u * (uint32_t)kk,
                                    sdesc(v_base + kk * 2048, kHalfBytes, 1024), kIdescO, (first && kk == 0) ? 0u : 1u);
                    return true;
                };
                auto issue_s = [&](int xb, int slot, int qb) {
                    const uint32_t k_base = sm_k + slot * kTileBytes;
                    const uint32_t q_base = sm_q + qb * 2 * sh.q_half;
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk)
                        // (rows of the query tile past the group's: whatever lies there, their scores are not used)
                        mma_bf16(tmem + col_s(xb), sdesc(q_base + (kk >> 2) * sh.q_half + (kk & 3) * 32, 16, 1024),
                                 sdesc(k_base + (kk >> 2) * kHalfBytes + (kk & 3) * 32, 16, 1024), kIdescS,
                                 kk > 0 ? 1u : 0u);
                    mma_commit(bar_sfull(xb));
                };
                // This thread's part of the unit is settled.  The plain arrival carries the softmax warps' own
                // shared-memory writes (acquired with P) on to the other warps.
                auto finish = [&]() {
                    mma_commit(bar_ofull);
                    mbar_arrive(bar_ofull);
                };
                Units units(a, pre, fill, q);
                Unit x;
                Ring kr, vr;   // slots of the next K tile; of the next V tile (dual), or K's tile (alternating)
                int j = 0;
                bool ok = true;
                if (!dual) {
                    const int xb = warp == 1 ? 0 : 1;   // has the tiles j of its parity
                    // the tile whose P V is still to come: its number, V slot, and what it is in its unit
                    bool pend = false, pend_first = false, pend_last = false;
                    int pend_tile = 0, pend_slot = 0, pend_unit = 0;
                    auto settle = [&]() -> bool {
                        if (!pend) return true;
                        pend = false;
                        if (!issue_pv(xb, pend_tile, pend_slot, pend_first, pend_unit)) return false;
                        mma_commit(bar_vempty(pend_slot));
                        if (pend_last) finish();
                        return true;
                    };
                    for (int uq = 0; ok && units.next(x); ++uq) {
                        const int b = nbuf == 2 ? uq & 1 : 0;
                        const uint32_t qphase = (uint32_t)((nbuf == 2 ? uq >> 1 : uq) & 1);
                        bool had = false;
                        for (int kt = 0; kt < x.nt; ++kt, ++j, kr.advance(nK), vr.advance(nV)) {
                            if ((j & 1) != xb) continue;
                            ok = settle() && (had || mbar_wait(bar_qfull(b), qphase, abort_flag)) &&
                                 mbar_wait(bar_kfull(j), phase_of(j), abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            issue_s(xb, kr.slot, b);
                            mma_commit(bar_kempty(kr.slot));
                            pend = true;
                            pend_first = !had;
                            pend_last = kt + 2 >= x.nt;
                            pend_unit = uq;
                            pend_tile = j;
                            pend_slot = vr.slot;
                            had = true;
                            if (pend_last) mma_commit(bar_qempty(b));
                        }
                        if (ok && !had) {   // no tile of the unit is this stream's: only its part of the barriers
                            ok = settle() && mbar_wait(bar_qfull(b), qphase, abort_flag) &&
                                 (uq == 0 || mbar_wait(bar_oempty, (uint32_t)((uq - 1) & 1), abort_flag));
                            if (ok) {
                                mbar_arrive(bar_qempty(b));
                                finish();
                            }
                        }
                    }
                    if (ok) settle();
                } else {
                    // per key tile: O_A += P_A V(-1), S_A; O_B += P_B V(-1), S_B
                    for (int uq = 0; ok && units.next(x); ++uq) {
                        ok = mbar_wait(bar_qfull(0), (uint32_t)(uq & 1), abort_flag);
                        for (int kt = 0; ok && kt <= x.nt; ++kt) {
                            if (kt < x.nt && !mbar_wait(bar_kfull(j + kt), phase_of(j + kt), abort_flag)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll
                            for (int xb = 0; xb < 2; ++xb) {
                                if (kt > 0 && !issue_pv(xb, j + kt - 1, vr.slot, kt == 1, uq)) {
                                    ok = false;
                                    break;
                                }
                                if (kt < x.nt) issue_s(xb, kr.slot, xb);
                            }
                            if (!ok) break;
                            if (kt > 0) {
                                mma_commit(bar_vempty(vr.slot));
                                vr.advance(nV);
                            }
                            if (kt < x.nt) {
                                mma_commit(bar_kempty(kr.slot));
                                kr.advance(nK);
                                if (kt == x.nt - 1) mma_commit(bar_qempty(0));
                            } else {
                                finish();
                            }
                        }
                        j += x.nt;
                    }
                }
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ====== softmax: stream xb, lane quarter qw, one query row a thread ======
        // the merge's table, and the rows of requests without a position
        if (hp == 0 && threadIdx.x == 32 * kWarpS) a.ws_split[q] = Units(a, pre, fill, q).split(a);
        for (int r = q; r < a.num_reqs; r += a.P) {
            if (pre[r + 1] > pre[r]) continue;
            for (int e = (int)threadIdx.x - 32 * kWarpS; e < ntok * G * (kD / 8); e += 256) {
                const int row = e / (kD / 8), t = tok0 + row / G, h = g * G + row % G;
                reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                          (((int64_t)r * a.T + t) * a.H_q + h) * kD)[e % (kD / 8)] = make_uint4(0, 0, 0, 0);
            }
        }
        const int xb = (warp - kWarpS) >> 2;
        const int qw = warp & 3;
        const int aq = xb ? aq1 : aq0;
        const bool fixes = !dual || xb == 0;   // V serves both query tiles: the first one's stream mends it
        Ring vr;             // the V slot of the tile at hand
        int j = 0;           // tiles of this CTA before the unit
        int ns = 0;          // S tiles of this stream seen so far
        bool ok = true;
        Units units(a, pre, fill, q);
        Unit x;
        if (qw >= aq) {
            // a quarter without rows: it mends the stream's V tiles beside the softmax
            while (fixes && ok && units.next(x)) {
                for (int kt = 0; kt < x.nt; ++kt, ++j, vr.advance(nV)) {
                    if (!dual && (j & 1) != xb) continue;
                    if (!mbar_wait_warp(bar_sfull(xb), (uint32_t)(ns & 1), abort_flag) ||
                        !mbar_wait_warp(bar_mask(j & 7), (uint32_t)((j >> 3) & 1), abort_flag)) {
                        ok = false;
                        break;
                    }
                    ++ns;
                    const uint32_t mword = mask_words[j & 7];
                    const int k0 = (x.f + kt) * kTile;
                    if (mword != all_seg || k0 + kTile > x.L - a.T) {
                        if (!mbar_wait_warp(bar_vfull(j), phase_of(j), abort_flag)) {
                            ok = false;
                            break;
                        }
                        fix_v(vr.slot, j, mword, x.L - a.T - k0, x.L - k0, qw - aq, 4 - aq);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_pfull(xb));
                }
            }
        } else {
            const int row = 32 * qw + lane;
            const int nrows = xb ? rows1 : rows0;
            const bool valid = row < nrows;
            const int tok = tok0 + (dual ? xb * tok_per_tile : 0) + min(row, nrows - 1) / G;
            const int hh = valid ? row % G : 0;
            const uint32_t lanes = tmem + ((uint32_t)(32 * qw) << 16);
            const uint32_t s_col = lanes + col_s(xb);
            float2 *xm = reinterpret_cast<float2 *>(smem + kOffXm);   // [set][stream][row]
            int no = 0;          // units finished so far
            while (ok && units.next(x)) {
                const int first = x.L - a.T;   // position of the tree's first token
                const uint32_t *mrow = a.mask + (int64_t)x.r * a.mask_stride + (int64_t)tok * a.mask_words;
                const int jb = j;
                j += x.nt;
                float m = -INFINITY, l = 0.f;
                bool any = false;   // this stream had a tile of the unit
                for (int kt = 0; kt < x.nt; ++kt, vr.advance(nV)) {
                    const int jj = jb + kt;
                    if (!dual && (jj & 1) != xb) continue;
                    const int k0 = (x.f + kt) * kTile;
                    const bool near = k0 + kTile > first;    // positions of the tree, or past the cache end
                    // what this row sees of the tile, as bits (the mask's words are on their way while the
                    // scores are waited for)
                    uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
                    if (near) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) vis[c] = tree_vis32(mrow, a.mask_words, first, x.L, k0 + 32 * c);
                    }
                    if (!mbar_wait_warp(bar_sfull(xb), (uint32_t)(ns & 1), abort_flag) ||
                        !mbar_wait_warp(bar_mask(jj & 7), (uint32_t)((jj >> 3) & 1), abort_flag)) {
                        ok = false;
                        break;
                    }
                    ++ns;
                    tc_fence_after();
                    const uint32_t mword = mask_words[jj & 7];
                    const bool full = !near && mword == all_seg;
                    if (mword != all_seg) {   // keys of entries that are not there
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t bits = mword >> ((32 * c) >> seg_shift);
                            uint32_t sb = 0u;
                            if (seg_rows >= 32) {
                                sb = (bits & 1u) ? 0xffffffffu : 0u;
                            } else {
                                const uint32_t ones = (1u << seg_rows) - 1u;
                                for (int i = 0; i < (32 >> seg_shift); ++i)
                                    if ((bits >> i) & 1u) sb |= ones << (i * seg_rows);
                            }
                            vis[c] &= sb;
                        }
                    }
                    // the row's 128 scores stay in registers: their max, then the weights
                    float sv[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32_nw(s_col + 32u * c, sv[c]);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c) use32(sv[c]);
                    if (!full) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int k = 0; k < 32; ++k) sv[c][k] = (vis[c] & (1u << k)) ? sv[c][k] : -INFINITY;
                    }
                    float top[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) top[c] = max32(sv[c]);
                    const float mt = fmaxf(max3(top[0], top[1], top[2]), top[3]) * a.scale_log2;
                    const bool bump = mt > m + kSlack;
                    const float mn = bump ? mt : m;
                    const float corr = bump ? fast_exp2(m - mn) : 1.f;
                    // the stream's last P V completed before this S did: rescale O
                    if (any && __any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll 1
                        for (int c = 0; c < 16; ++c) {
                            float ov[8];
                            uint32_t ow[8];
                            tmem_ld8(lanes + col_o(xb) + 8u * c, ov);
#pragma unroll
                            for (int k = 0; k < 8; ++k) ow[k] = __float_as_uint(ov[k] * corr);
                            tmem_st8(lanes + col_o(xb) + 8u * c, ow);
                        }
                    }
                    any = true;
                    // weights 2^(s scale - mn) (a masked score is -inf: 0), their sum, and P (bf16) over the
                    // first half of S's columns
                    const float nb = mn == -INFINITY ? 0.f : -mn;
                    float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            float2 e = fma2(make_float2(sv[c][k], sv[c][k + 1]), a.scale_log2, nb);
                            e.x = fast_exp2(e.x);
                            e.y = fast_exp2(e.y);
                            const __nv_bfloat162 pb = __floats2bfloat162_rn(e.x, e.y);
                            pk[k >> 1] = *reinterpret_cast<const uint32_t *>(&pb);
                            sum2 = add2(sum2, e);
                        }
                        tmem_st16(s_col + 16u * c, pk);
                    }
                    tmem_st_wait();
                    l = fmaf(l, corr, sum2.x + sum2.y);
                    m = mn;
                    if (!full && fixes && aq == 4) {
                        if (!mbar_wait_warp(bar_vfull(jj), phase_of(jj), abort_flag)) {
                            ok = false;
                            break;
                        }
                        fix_v(vr.slot, jj, mword, first - k0, x.L - k0, qw, 4);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_pfull(xb));
                }
                if (!ok) break;
                // ---- the unit's end ----
                const int srow = row + (dual ? xb * tok_per_tile * G : 0);   // row of the slot
                const int64_t prow = ((int64_t)hp * (2 * a.P) + x.slot) * a.NR + srow;
                float *po = a.ws_o + prow * kD;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) +
                                     (((int64_t)x.r * a.T + tok) * a.H_q + (int64_t)g * G + hh) * kD;
                float M = m, fa = 1.f, fb = 0.f, lsum = l;
                if (!dual) {
                    // the streams' parts of this row
                    float2 *xu = xm + no % kXmSets * 2 * kTile;
                    xu[xb * kTile + row] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_pair(qw));
                    if (!mbar_wait_warp(bar_pair(qw), (uint32_t)(no & 1), abort_flag)) break;
                    const float2 pa = xu[row], pb = xu[kTile + row];
                    M = fmaxf(pa.x, pb.x);
                    fa = pa.x == -INFINITY ? 0.f : fast_exp2(pa.x - M);
                    fb = pb.x == -INFINITY ? 0.f : fast_exp2(pb.x - M);
                    lsum = fa * pa.y + fb * pb.y;
                }
                // O of both streams is settled
                if (!mbar_wait_warp(bar_ofull, (uint32_t)(no & 1), abort_flag)) break;
                tc_fence_after();
                ++no;
                // a V row of the tree that was not finite makes the rows that see it NaN
                if (*any_bad) {
#pragma unroll 1
                    for (int c = 4 * max(0, (first >> 7) - x.f); c < 4 * x.nt; ++c) {
                        const uint8_t *bad_rows = poison + ((jb + (c >> 2)) & 7) * 32 + 8 * (c & 3);
                        uint32_t w = 0u;
                        for (int i = 0; i < 8; ++i) w |= (uint32_t)bad_rows[i] << (4 * i);
                        if (w && (w & tree_vis32(mrow, a.mask_words, first, x.L, x.f * kTile + 32 * c))) lsum = NAN;
                    }
                }
                const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
                auto put32 = [&](int c, const float (&ov)[32]) {   // columns [32 c, 32 c + 32)
                    if (!valid) return;
                    if (x.whole) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const __nv_bfloat162 h2 =
                                    __floats2bfloat162_rn(ov[16 * h + 2 * e] * inv, ov[16 * h + 2 * e + 1] * inv);
                                w[e] = *reinterpret_cast<const uint32_t *>(&h2);
                            }
                            store32(out + 32 * c + 16 * h, w);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) store32(po + 32 * c + k, reinterpret_cast<const uint32_t *>(ov + k));
                    }
                };
                if (dual) {
#pragma unroll 1
                    for (int c = 0; c < 4; c += 2) {
                        float oa[32], ob[32];
                        tmem_ld32_nw(lanes + col_o(xb) + 32u * c, oa);
                        tmem_ld32_nw(lanes + col_o(xb) + 32u * c + 32u, ob);
                        tmem_ld_wait();
                        use32(oa);
                        use32(ob);
                        put32(c, oa);
                        put32(c + 1, ob);
                    }
                } else {
                    // the quarter's two warps take half of the columns each (those of a stream without a tile
                    // in the unit may hold anything)
                    const bool use_a = x.nt > 1 || (jb & 1) == 0, use_b = x.nt > 1 || (jb & 1) == 1;
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        float oa[32], ob[32];
                        tmem_ld32_nw(lanes + col_o(0) + 64u * xb + 32u * h, oa);
                        tmem_ld32_nw(lanes + col_o(1) + 64u * xb + 32u * h, ob);
                        tmem_ld_wait();
                        use32(oa);
                        use32(ob);
#pragma unroll
                        for (int k = 0; k < 32; ++k) oa[k] = (use_a ? oa[k] * fa : 0.f) + (use_b ? ob[k] * fb : 0.f);
                        put32(2 * xb + h, oa);
                    }
                }
                if (!x.whole && valid && (dual || xb == 0))
                    *reinterpret_cast<float2 *>(a.ws_ml + prow * 2) = make_float2(M, lsum);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_oempty);
            }
        }
    }

    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0 && a.err) atomicAdd(a.err, kTimeoutErr);
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

static bool encode_3d(CUtensorMap *m, const void *base, uint64_t d1, uint64_t d2, uint32_t b1, uint32_t b2) {
    const cuuint64_t dims[3] = {kD, d1, d2};
    const cuuint64_t strides[2] = {kD * 2, d1 * kD * 2};
    const cuuint32_t box[3] = {64, b1, b2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared memory of a launch.  A query tile keeps only its own rows (whole
// swizzle atoms of 8); the rest goes to the rings, up to three slots each.  One
// query tile is kept twice unless a single one leaves another slot (33 to 72 rows
// and 97 on); two query tiles leave five slots, four from 97 rows each on.
static void ring_shape(const TreeArgs &a, TreeShape *s) {
    s->seg_rows = a.bs < kTile ? a.bs : kTile;
    s->tok_per_tile = kTile / a.G;
    s->box_tok = a.T < s->tok_per_tile ? a.T : s->tok_per_tile;
    s->q_half = (s->box_tok * a.G + 7) / 8 * 1024;
    s->q_buffers = 2;
    auto slots = [&](int buffers) { return (kSmemMax - kOffQ - buffers * 2 * s->q_half) / kTileBytes; };
    if (a.T <= s->tok_per_tile && slots(1) > slots(2) && slots(2) < 2 * kMaxStages) s->q_buffers = 1;
    s->q_bytes = s->q_buffers * 2 * s->q_half;
    int n = slots(s->q_buffers);
    n = n < 2 * kMaxStages ? n : 2 * kMaxStages;
    s->k_stages = n / 2;
    s->v_stages = n - n / 2;
    s->smem = kOffQ + s->q_bytes + n * kTileBytes + 1024;
}

}  // namespace ttc

bool prepare_tree_tc(const TreeArgs &a, TreeTc *t) {
    using namespace ttc;
    if (a.dtype != BKV_BF16 || a.D != kD || a.G < 1 || a.G > 128) return false;
    if (a.bs < 8 || !((kTile % a.bs == 0) || (a.bs % kTile == 0))) return false;
    if (a.num_reqs > kMaxReqs || (int64_t)a.num_reqs * a.T >= ((int64_t)1 << 31)) return false;
    if (a.total_blocks <= 0 || (int64_t)a.total_blocks * a.bs >= ((int64_t)1 << 31)) return false;
    // the costs' prefix stays within int32
    if ((int64_t)a.num_reqs * ((a.max_ctx + (int64_t)kTile - 1) / kTile + kEndCost) >= ((int64_t)1 << 31)) return false;
    if ((int64_t)a.P * a.H_kv * a.groups >= ((int64_t)1 << 31)) return false;
    if (!aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.q, 16) || !aligned(a.out, 32)) return false;
    if (!encode_fn()) return false;
    ring_shape(a, &t->sh);
    const uint64_t rows = (uint64_t)a.total_blocks * (uint64_t)a.bs;
    return encode_3d(&t->mk, a.k, a.H_kv, rows, 1, t->sh.seg_rows) &&
           encode_3d(&t->mv, a.v, a.H_kv, rows, 1, t->sh.seg_rows) &&
           encode_3d(&t->mq, a.q, a.H_q, (uint64_t)a.num_reqs * a.T, a.G, t->sh.box_tok);
}

int launch_tree_tc(const TreeArgs &a, const TreeTc &t, cudaStream_t st) {
    using namespace ttc;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(tree_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax + 1024);
        if (e != cudaSuccess) {
            set_cuda_error(e);
            (void)launch_status();   // clears the sticky status
            return BKV_ERR_CUDA;
        }
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    const cudaError_t e = launch_pdl(tree_tc_kernel, dim3((unsigned)(a.P * a.H_kv * a.groups)), dim3(kThreads),
                                     (size_t)t.sh.smem, st, t.mk, t.mv, t.mq, a, t.sh);
    if (e != cudaSuccess) set_cuda_error(e);
    return launch_status();
}

}  // namespace bkv
