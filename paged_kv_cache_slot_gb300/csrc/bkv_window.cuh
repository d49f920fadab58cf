// bkv_window.cuh -- shared declarations of the attention over E4M3 caches with
// a scale a block and head, and over windows whose first tokens stay visible.
#pragma once

#include <cuda.h>

#include "bkv_internal.cuh"

namespace bkv {
namespace win {

// Everything a launch needs; passed by value to its kernels.  Query row i of a
// KV head is token i / G, head g G + i % G; a row group is NR consecutive rows.
struct Args {
    const void *q;            // [num_reqs][q_len][H_q][D]
    const void *k, *v;
    const float *ks, *vs;     // E4M3 caches: scales [total_blocks][H_kv]; null otherwise
    const int32_t *bt;
    int64_t bt_stride;
    int32_t bt_cols;
    const int32_t *ctx;
    int32_t max_ctx;
    int32_t num_reqs, q_len, H_q, H_kv, D, bs, G;
    int64_t total_blocks;
    float scale_log2;         // softmax_scale * log2(e): scores are kept in base 2
    int32_t causal;
    int32_t window, sinks;    // window 0: none
    int32_t seg;              // positions that are read together, a power of two (see Span)
    int32_t tile;             // span positions a tile
    int32_t NR, groups;       // query rows a group, groups a KV head
    int32_t P;                // columns: each takes its share of the cost of all requests
    int dtype;
    // A column may end one stream that it did not begin (its partial: slot q of 2 P a KV head and group) and begin
    // one that it does not end (slot P + q).
    int2 *ws_split;           // [P] the latter: (request, columns that share it), (0, 0) without one
    float *ws_o;              // [slots][NR][D] unnormalised partial outputs
    float *ws_ml;             // [slots][NR][2] (running max in base 2, sum of weights)
    void *out;                // [num_reqs][q_len][H_q][D]
    int32_t *err;
};

// The positions that a request's queries read, laid end to end: the first
// `sb` (those that stay visible) and, behind them, the window's, with `gap`
// positions between left out; both begin and end at multiples of `seg`.
struct Span {
    int32_t L, sb, gap, len;
    __host__ __device__ int32_t pos(int32_t v) const { return v < sb ? v : v + gap; }
};
__host__ __device__ inline Span span_of(const Args &a, int32_t ctx) {
    Span s;
    s.L = ctx > a.max_ctx ? a.max_ctx : (ctx > 0 ? ctx : 0);
    s.sb = 0;
    s.gap = 0;
    if (a.window > 0) {
        const int64_t lo = (int64_t)s.L - a.q_len - a.window + 1;   // first position in the first token's window
        if (lo > 0) {
            const int32_t w = (int32_t)lo & -a.seg;
            const int32_t keep = a.sinks < s.L ? a.sinks : s.L;
            const int32_t sb = (keep + a.seg - 1) & -a.seg;
            if (sb < w) {
                s.sb = sb;
                s.gap = w - sb;
            }
        }
    }
    s.len = s.L - s.gap;
    return s;
}

// The schedule: requests end to end by cost.  A tile costs 1; a request's end
// (the last softmax, the wait for the last product, the output: nothing else
// runs beside them) kEndCost, laid behind its tiles.  A column takes at least
// kMinCost, so that few columns share a short request.
constexpr int kEndCost = 2, kMinCost = 2;
constexpr int kMaxReqs = 1024;   // requests a launch; more go in several
__host__ __device__ inline int64_t columns_of(int64_t cost, int64_t P) {
    const int64_t most = (cost + kMinCost - 1) / kMinCost;
    return most < P ? most : P;
}

// One unit: tiles [f, f + nt) of request r.  whole: they are all of its tiles.
struct Unit {
    int r, f, nt, slot;
    bool whole;
};

// Walks a column's units; pre[r] is the cost of the requests before r.
struct Units {
    const int32_t *pre;
    int r, q, t, t1, P, n;
    __host__ __device__ Units(const int32_t *pre_, int n_, int q_, int P_) {
        pre = pre_;
        n = n_;
        q = q_;
        P = P_;
        const int64_t C = pre[n], peff = columns_of(C, P);
        t = (int)(q < peff ? C * q / peff : C);
        t1 = (int)(q < peff ? C * (q + 1) / peff : C);
        int lo = 0, hi = n;   // first request whose cost ends after t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid + 1] > t) hi = mid;
            else lo = mid + 1;
        }
        r = lo;
    }
    // The stream that this column begins and does not end (before next() is called).
    __host__ __device__ int2 split() const {
        int2 none;
        none.x = none.y = 0;
        if (t >= t1) return none;
        int r1 = r;
        while (pre[r1 + 1] < t1) ++r1;   // the request that the share ends in
        const int s = pre[r1], e = pre[r1 + 1] - kEndCost;   // its tiles
        if (s < t || s >= t1 || e <= t1) return none;
        const int64_t C = pre[n], peff = columns_of(C, P);
        int2 x;
        x.x = r1;
        x.y = (int)((e * peff - 1) / C) - q + 1;   // up to the column of its last tile
        return x;
    }
    __host__ __device__ bool next(Unit &x) {
        for (; t < t1; ++r) {
            const int s = pre[r], e = pre[r + 1] - kEndCost;
            if (pre[r + 1] <= t) continue;   // no tiles (or passed)
            const int lo = t, hi = t1 < e ? t1 : e;
            t = pre[r + 1];
            if (lo >= hi) continue;   // only the end's share of the request is this column's
            x.r = r;
            x.f = lo - s;
            x.nt = hi - lo;
            x.whole = lo == s && hi == e;
            x.slot = lo == s ? P + q : q;
            ++r;
            return true;
        }
        return false;
    }
};

// Lengths of all requests and the exclusive prefix sum of their costs, over a
// CTA of kThreads; sums: a word a warp.  Ends with a barrier.
template <int kThreads>
__device__ __forceinline__ void lay_out(const Args &a, int32_t *pre, int32_t *lens, int32_t *sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = a.num_reqs, per = (n + kThreads - 1) / kThreads;
    const int lo = min(n, (int)threadIdx.x * per), hi = min(n, lo + per);
    int32_t sum = 0;
    for (int r = lo; r < hi; ++r) {
        const int32_t c = __ldg(a.ctx + r);
        if (c > a.max_ctx && blockIdx.x == 0 && a.err) atomicAdd(a.err, 1);
        const Span s = span_of(a, c);
        lens[r] = s.L;
        const int32_t cost = s.len > 0 ? (s.len + a.tile - 1) / a.tile + kEndCost : 0;
        pre[r] = cost;
        sum += cost;
    }
    int32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int32_t run = inc - sum;
    for (int w = 0; w < warp; ++w) run += sums[w];
    for (int r = lo; r < hi; ++r) {
        const int32_t cost = pre[r];
        pre[r] = run;
        run += cost;
    }
    if (threadIdx.x == kThreads - 1) pre[n] = run;
    __syncthreads();
}

// The reciprocal that turns a row's sums into its output: a row that saw no
// key is 0, one whose sum is NaN stays NaN.
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : __frcp_rn(l); }

// Scales of values that the writes make; others are held to this range.
constexpr float kScaleMin = 9.094947017729282e-13f, kScaleMax = 1099511627776.f;   // 2^-40, 2^40

// tcgen05 / TMA kernel (bkv_window_tc.cu): bf16 queries of head_dim 128.
struct TcLaunch {
    CUtensorMap mk, mv;
};
constexpr int kTcRows = 16;   // query rows a group, at most
bool prepare_tc(const Args &a, TcLaunch *t);
int launch_tc(const Args &a, const TcLaunch &t, cudaStream_t stream);

}  // namespace win
}  // namespace bkv
