// bkv_verify.cu -- verification of drafted tokens against the target model's
// probabilities, from given random numbers: a chain of drafts with the draft
// model's probabilities, or a tree of drafts without them.
//
// Chain: draft i (token x_i, drawn from q_i) is accepted while u_i q_i(x_i) <
// p_i(x_i); at the first rejection the next token is sampled from max(p_i -
// q_i, 0), after the last draft from p_len, so the tokens are distributed as
// the target's own.  Tree: at a node with row p, its children in index order
// are accepted when u_c rem < p(x_c), rem = 1 - the probabilities of the
// siblings rejected before; with no child accepted the next token is sampled
// from p without the rejected tokens.  The pages name speculative tokens
// ("Padding and Batching with Block KV", Cache Masking) and print nothing
// about their verification.
//
// A sample is the lowest v whose running sum of weights passes u times their
// whole sum.  Running sums over a vocabulary cross that border within
// rounding errors of one another, so weights are summed as integers in units
// of 2^-56: exact for probabilities from 2^-32 up (24 significant bits) and
// within 2^-57 below, associative, so the answer depends on no order, and
// sums below 256 fit 64 bits.
//
// Memory-bound: one row of p (chain: of q too) of V fp32 a request.  A
// cluster of CTAs shares a request's row; every CTA walks the drafts itself
// (a few gathers), sums its part by warps, the CTA totals go round the
// cluster, and the CTA whose part holds the border scans the part of the warp
// that does once more (from L2), a few elements a thread.
#include <cooperative_groups.h>

#include "bkv_internal.cuh"

namespace bkv {
namespace verify {

namespace cg = cooperative_groups;

constexpr int kMaxNodes = 1024;   // drafts (chain) or nodes (tree) a request
constexpr int kMaxWarps = 16;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 16;       // elements of each row in flight a lane

// CTA size, the CTAs an SM is built to hold, and how many of them an SM a launch
// may ask for before its clusters get narrower.  Chains stream two rows and are
// bound by bandwidth: small CTAs, about two waves, so that one's walk and border
// run beside another's sums (256 requests of 100003 tokens: 41 us, 5.0 TB/s; 45
// with one wave or four, 44 with three CTAs an SM, 58 with six and half of the
// loads in flight; 61.7 with 512 threads, before the sums by pairs).  Trees walk
// before they stream: large CTAs, one wave (64 requests of 131072 14.1 us, 18.2
// with three an SM; 22.2 with 256 threads, before the sums by pairs).
template <bool kChain>
struct Shape {
    static constexpr int kThreads = kChain ? 256 : 512;
    static constexpr int kWarps = kThreads / 32;
    static constexpr int kBuilt = kChain ? 4 : 2;
    static constexpr int kAsked = kChain ? 7 : 2;
};

struct Args {
    const float *p;
    int64_t p_req, p_row;      // strides: request, row
    const float *q;            // chain only
    int64_t q_req, q_row;
    const int64_t *tokens;     // chain [R][nodes], tree [R][nodes]
    const int32_t *parents;    // tree [R][nodes]
    const int32_t *lens;       // chain [R] or null
    const float *u, *us;       // accept [R][nodes], sample [R]
    int32_t nodes;             // chain: K drafts; tree: T nodes
    int32_t V;
    int64_t *out;              // chain [R][K + 1], tree [R][T]
    int32_t *path;             // tree [R][T]
    int32_t *count;            // [R]
    int32_t *err;
};

// A probability x in [0, 1] in units of 2^-56, as three integers h 2^34 + l 2^12
// + m: adding a constant whose last place is 2^-22 (then 2^-44, 2^-56) leaves
// the rounded multiple in the sum's low bits, and what it leaves over is exact,
// so three sums and their differences do what a conversion to a 64-bit integer
// would, at the full rate of fp32 additions (64-bit conversions run at 2 a
// clock and SM here: they bound this kernel at 140 us where the rows' bytes
// take 30, 256 requests of 100003 tokens).
struct Limbs {
    int32_t h, l, m;
};
constexpr float kC1 = 2.f, kC2 = 0x1.8p-21f, kC3 = 0x1.8p-33f;
__device__ __forceinline__ Limbs limbs(float x) {
    const float a = __fadd_rn(x, kC1);
    const float x1 = __fsub_rn(x, __fsub_rn(a, kC1));
    const float b = __fadd_rn(x1, kC2);
    const float x2 = __fsub_rn(x1, __fsub_rn(b, kC2));
    const float c = __fadd_rn(x2, kC3);
    return {__float_as_int(a) - __float_as_int(kC1), __float_as_int(b) - __float_as_int(kC2),
            __float_as_int(c) - __float_as_int(kC3)};
}
__device__ __forceinline__ long long whole_of(const Limbs &v) {
    return ((long long)v.h << 34) + ((long long)v.l << 12) + v.m;
}
// Below 0 and NaN: 0; above 1: 1.
__device__ __forceinline__ long long fixed(float p) { return whole_of(limbs(__saturatef(p))); }

// floor(u n) of a random number u in [0, 1), exactly: u n < m for integers is
// floor(u n) < m.  From 1 on (and NaN) u is the largest number below, 2^-64 off;
// below 0 it is 0.  u in units of 2^-64 makes floor(u n) the high word of a
// product.  Below 2^-40 the last of its 24 bits would fall out of those units:
// there they are of 2^-104, which hold every bit down to 2^-80, and below that
// u n < 2^-16 is 0 either way.
struct Unit {
    unsigned long long u;
    int shift;
    __device__ __forceinline__ explicit Unit(float x) {
        const bool tiny = x < 0x1p-40f;
        shift = tiny ? 40 : 0;
        u = x < 1.f ? __float2ull_rz(fmaxf(x, 0.f) * (tiny ? 0x1p104f : 0x1p64f)) : ~0ull;
    }
    __device__ __forceinline__ unsigned long long times(unsigned long long n) const { return __umul64hi(u, n) >> shift; }
};

// What token v weighs: its probability p, less the draft's q in a chain.
__device__ __forceinline__ unsigned long long weight(float p, float q) {
    const long long w = fixed(p) - fixed(q);
    return w > 0 ? w : 0;
}

// limbs() of two values in one instruction each step (every operation rounds
// as the single one): the sums' bits, with the constants still in them.
struct Limbs2 {
    uint32_t h[2], l[2], m[2];
};
__device__ __forceinline__ unsigned long long pair_of(float x, float y) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, float c) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(pair_of(c, c)));
    return r;
}
__device__ __forceinline__ unsigned long long sub2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(b), "l"(pair_of(-1.f, -1.f)), "l"(a));
    return r;
}
__device__ __forceinline__ void split2(unsigned long long a, uint32_t (&w)[2]) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(w[0]), "=r"(w[1]) : "l"(a));
}
__device__ __forceinline__ Limbs2 limbs2(float x, float y) {
    Limbs2 r;
    const unsigned long long v = pair_of(x, y);
    const unsigned long long a = add2(v, kC1);
    const unsigned long long v1 = sub2(v, add2(a, -kC1));
    const unsigned long long b = add2(v1, kC2);
    const unsigned long long v2 = sub2(v1, add2(b, -kC2));
    split2(a, r.h);
    split2(b, r.l);
    split2(add2(v2, kC3), r.m);
    return r;
}

// The weights of one round: N tokens of this lane from v, below v1 (all of
// them: kFull).  Their limbs fit 32 bits.
template <bool kResidual, int kVec, int N, bool kFull>
__device__ __forceinline__ long long round_sum(const float *pr, const float *qr, uint32_t v, uint32_t v1) {
    float x[N], y[N];
#pragma unroll
    for (int k = 0; k < N; k += kVec) {
        const bool in = kFull || v + 32 * k < v1;
        if constexpr (kVec == 4) {
            const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4 *>(x + k) = in ? __ldg(reinterpret_cast<const float4 *>(pr + v + 32 * k)) : z;
            if (kResidual)
                *reinterpret_cast<float4 *>(y + k) = in ? __ldg(reinterpret_cast<const float4 *>(qr + v + 32 * k)) : z;
        } else {
            x[k] = in ? __ldg(pr + v + 32 * k) : 0.f;
            if (kResidual) y[k] = in ? __ldg(qr + v + 32 * k) : 0.f;
        }
    }
    uint32_t h = 0, l = 0, m = 0;
    if constexpr (kResidual) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float xs = __saturatef(x[k]), ys = __saturatef(y[k]);
            const Limbs2 t = limbs2(xs, ys);
            if (xs > ys) {   // rounding keeps the order
                h += t.h[0] - t.h[1];
                l += t.l[0] - t.l[1];
                m += t.m[0] - t.m[1];
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const Limbs2 t = limbs2(__saturatef(x[k]), __saturatef(x[k + 1]));
            h += t.h[0] + t.h[1];
            l += t.l[0] + t.l[1];
            m += t.m[0] + t.m[1];
        }
        h -= N * __float_as_uint(kC1);
        l -= N * __float_as_uint(kC2);
        m -= N * __float_as_uint(kC3);
    }
    return whole_of({(int32_t)h, (int32_t)l, (int32_t)m});
}

// The weights of tokens [v0, v1), a warp's part, of this lane: four at a time
// where both rows start on 16 bytes (and v0 and v1 are whole fours), one
// otherwise; the elements of a round are loaded before the first is used, and
// what is left below a round takes no more of one than it needs.  (256 chains of
// 100003 tokens: 40.9 us, 44.6 with a value an instruction and a test a load.)
template <bool kResidual, int kVec>
__device__ __forceinline__ unsigned long long part_sum(const float *pr, const float *qr, int64_t v0, int64_t v1,
                                                       int lane) {
    long long sum = 0;
    uint32_t v = (uint32_t)min(v0, v1) + lane * kVec;   // (below 2^31 + 2^12)
    const uint32_t end = (uint32_t)v1;
    for (; v - lane * kVec + 32 * kUnroll <= end; v += 32 * kUnroll)
        sum += round_sum<kResidual, kVec, kUnroll, true>(pr, qr, v, end);
    const uint32_t rest = end - min(v - lane * kVec, end);
    if (rest > 32 * kUnroll / 2) sum += round_sum<kResidual, kVec, kUnroll, false>(pr, qr, v, end);
    else if (rest > 32 * kUnroll / 4) sum += round_sum<kResidual, kVec, kUnroll / 2, false>(pr, qr, v, end);
    else if (rest > 0) sum += round_sum<kResidual, kVec, kUnroll / 4, false>(pr, qr, v, end);
    return (unsigned long long)sum;
}

struct Shared {
    long long fx[kMaxNodes];             // tree: the nodes' probabilities in units of 2^-56
    float u[kMaxNodes];
    int32_t tok[kMaxNodes], par[kMaxNodes];
    int32_t next[kMaxNodes];             // tree: the child taken, kMaxNodes: none
    int32_t path[kMaxNodes];             // tree: the accepted path
    int32_t ex[kMaxNodes];               // tree: the rejected children of the stop node
    int32_t n, cur, nex;                 // accepted drafts, stop row, rejected children
    unsigned long long seg[kMaxWarps];      // sums of the warps' parts
    unsigned long long run[kMaxWarps];      // and of the warps' shares of the part with the border
    unsigned long long tot[2][kMaxCluster];
};

template <bool kChain>
__global__ void __launch_bounds__(Shape<kChain>::kThreads, Shape<kChain>::kBuilt) verify_kernel(const Args a) {
    constexpr int kThreads = Shape<kChain>::kThreads, kWarps = Shape<kChain>::kWarps;
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int64_t r = blockIdx.x / cs;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a CTA's shared memory may be written by the others only once it runs: the wait is behind the walk
    asm volatile("barrier.cluster.arrive;" ::: "memory");
    pdl_wait();
    pdl_trigger();
    const int64_t *tokens = a.tokens + r * a.nodes;
    const float *P = a.p + r * a.p_req;
    const float *Q = kChain ? a.q + r * a.q_req : nullptr;

    // ---- which drafts stand: every CTA of the cluster for itself ----
    int len = a.nodes;
    if (kChain && a.lens) {
        const int l = __ldg(a.lens + r);
        len = min(max(l, 0), a.nodes);
        if (l != len && threadIdx.x == 0 && rank == 0 && a.err) atomicAdd(a.err, 1);
    }
    if (threadIdx.x == 0) {
        s.n = kChain ? len : 0;
        s.cur = 0;
        s.nex = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < len; i += kThreads) {
        const int64_t x = __ldg(tokens + i);
        const float u = __ldg(a.u + r * a.nodes + i);
        const bool in = x >= 0 && x < a.V;
        if (kChain) {
            bool ok = false;
            if (in) {
                const double q = Q[i * a.q_row + x], p = P[i * a.p_row + x];
                ok = (double)u * q < p;
            } else if (rank == 0 && a.err) {
                atomicAdd(a.err, 1);
            }
            s.tok[i] = (int32_t)x;
            if (!ok) atomicMin(&s.n, i);
        } else {
            // the root's token was settled before; other nodes hang under an earlier one, or are padding
            const int32_t par = i > 0 ? __ldg(a.parents + r * a.nodes + i) : -1;
            const bool node = par >= 0 && par < i;
            if (i > 0 && rank == 0 && a.err && ((!node && par != -1) || (node && !in))) atomicAdd(a.err, 1);
            s.par[i] = node ? par : -1;
            s.next[i] = kMaxNodes;
            s.tok[i] = in ? (int32_t)x : -1;
            s.u[i] = in ? u : INFINITY;   // no child: its test fails whatever its number
            s.fx[i] = node && in ? fixed(P[par * a.p_row + x]) : 0;
        }
    }
    __syncthreads();
    if (!kChain) {
        // A child is put to the test only when all its older siblings failed theirs, so each node's test
        // stands by itself: its rem is 1 less its older siblings' probabilities, in their order, a token
        // counted once.  next[a] = the first child of a that passes.
        // Eight lanes a node.
        const int sub = lane & 7;
        for (int c0 = 0; c0 < len; c0 += kThreads / 8) {
            const int c = c0 + (int)threadIdx.x / 8;
            const int par = c < len ? s.par[c] : -1, x = c < len ? s.tok[c] : -1;
            bool dup = false;
            if (par >= 0)
                for (int j = 1 + sub; j < c; j += 8) dup |= (s.par[j] == par) & (s.tok[j] == x);
            const unsigned any = __ballot_sync(0xffffffffu, dup);
            if (sub == 0 && ((any >> lane) & 0xffu)) {   // it is never taken and weighs nothing
                s.fx[c] = 0;
                s.u[c] = INFINITY;
            }
        }
        __syncthreads();
        for (int c0 = 0; c0 < len; c0 += kThreads / 8) {
            const int c = c0 + (int)threadIdx.x / 8;
            const int par = c < len ? s.par[c] : -1;
            long long out_of_it = 0;
            if (par >= 0)
                for (int j = 1 + sub; j < c; j += 8) out_of_it += s.par[j] == par ? s.fx[j] : 0;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) out_of_it += __shfl_xor_sync(0xffffffffu, out_of_it, o);
            if (sub == 0 && par >= 0) {
                const long long rem = max((1ll << 56) - out_of_it, 0ll);
                const float u = s.u[c];
                // (fp64 runs at 2 a clock and SM here; a u outside [0, 1) and NaN take it)
                const bool ok = u >= 0.f && u < 1.f ? (long long)Unit(u).times(rem) < s.fx[c]
                                                    : (double)u * (double)rem < (double)s.fx[c];
                if (ok) atomicMin(&s.next[par], c);
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int cur = 0, n = 0;
            s.path[0] = 0;
            while (s.next[cur] < len) {
                cur = s.next[cur];
                s.path[++n] = cur;
            }
            s.n = n;
            s.cur = cur;
        }
        __syncthreads();
        // the stop node's children all failed: their tokens are left out of the sample
        for (int c = threadIdx.x; c < len; c += kThreads)
            if (s.par[c] == s.cur && s.fx[c] > 0) s.ex[atomicAdd(&s.nex, 1)] = c;
    }
    __syncthreads();
    const int n = s.n;
    const int cur = kChain ? n : s.cur;
    const bool residual = kChain && n < len;
    int64_t *out = a.out + r * (kChain ? a.nodes + 1 : a.nodes);
    if (rank == 0 && threadIdx.x == 0) out[n] = -1;   // until the sample is found, behind the cluster barrier

    // ---- sample the next token ----
    const float *pr = P + cur * a.p_row;
    const float *qr = residual ? Q + cur * a.q_row : nullptr;
    const int part = (int)((((int64_t)a.V + cs * kWarps - 1) / (cs * kWarps) + 127) / 128 * 128);   // a warp's elements
    const int64_t v0 = ((int64_t)rank * kWarps + warp) * part;
    const int64_t v1 = min((int64_t)a.V, v0 + part);
    const float us = __ldg(a.us + r);
    const Unit U(us);
    asm volatile("barrier.cluster.wait;" ::: "memory");   // every CTA of the cluster has started
    // pass 0: the residual weights; where they are all 0, pass 1: the row itself
    for (int pass = 0; pass < 2; ++pass) {
        const bool plain = pass == 1;
        const float *qq = plain ? nullptr : qr;
        const bool fours = ((reinterpret_cast<uintptr_t>(pr) | reinterpret_cast<uintptr_t>(qq)) & 15) == 0 && a.V % 4 == 0;
        unsigned long long sum;
        if (kChain && qq) sum = fours ? part_sum<true, 4>(pr, qq, v0, v1, lane) : part_sum<true, 1>(pr, qq, v0, v1, lane);
        else sum = fours ? part_sum<false, 4>(pr, qq, v0, v1, lane) : part_sum<false, 1>(pr, qq, v0, v1, lane);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const int nex = plain ? 0 : s.nex;
        if (!kChain)
            for (int e = 0; e < nex; ++e) {
                const int v = s.tok[s.ex[e]];
                if (v >= v0 && v < v1) sum -= s.fx[s.ex[e]];
            }
        if (lane == 0) s.seg[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            unsigned long long t = lane < kWarps ? s.seg[lane] : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            if (lane < cs) *cluster.map_shared_rank(&s.tot[pass][rank], lane) = t;
        }
        cluster.sync();
        unsigned long long whole = 0, before = 0;
        for (int c = 0; c < cs; ++c) {
            if (c < rank) before += s.tot[pass][c];
            whole += s.tot[pass][c];
        }
        if (whole == 0) {
            if (pass == 1 && rank == 0 && threadIdx.x == 0 && a.err) atomicAdd(a.err, 1);   // a row without any weight
            continue;
        }
        const unsigned long long border = U.times(whole);   // floor(u * whole) < whole
        // the CTA whose part holds the border: its threads scan the warp's part that does, together
        if (border < before || border - before >= s.tot[pass][rank]) break;
        int w = 0;
        while (border - before >= s.seg[w]) before += s.seg[w++];
        const int64_t s0 = ((int64_t)rank * kWarps + w) * part;
        const int64_t s1 = min((int64_t)a.V, s0 + part);
        const int each = (part + kThreads - 1) / kThreads;
        const int64_t e0 = s0 + (int64_t)threadIdx.x * each;
        const int64_t e1 = min(s1, e0 + each);
        auto at = [&](int64_t v) { return weight(pr[v], qq ? qq[v] : 0.f); };
        unsigned long long mine = 0;
        for (int64_t v = e0; v < e1; ++v) mine += at(v);
        if (!kChain)
            for (int e = 0; e < nex; ++e) {
                const int v = s.tok[s.ex[e]];
                if (v >= e0 && v < e1) mine -= s.fx[s.ex[e]];
            }
        unsigned long long inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) s.run[warp] = inc;
        __syncthreads();
        unsigned long long run = before + inc - mine;
        for (int i = 0; i < warp; ++i) run += s.run[i];
        if (border >= run && border - run < mine)
            for (int64_t v = e0; v < e1; ++v) {
                bool out_of_it = false;
                if (!kChain)
                    for (int e = 0; e < nex; ++e) out_of_it |= s.tok[s.ex[e]] == v;
                if (!out_of_it) run += at(v);
                if (run > border) {
                    out[n] = v;
                    break;
                }
            }
        break;
    }
    if (rank == 0) {
        if (threadIdx.x == 0) a.count[r] = n;
        if (kChain) {
            for (int i = threadIdx.x; i <= a.nodes; i += kThreads)
                if (i != n) out[i] = i < n ? s.tok[i] : -1;
        } else {
            for (int i = threadIdx.x; i < len; i += kThreads) {
                a.path[r * a.nodes + i] = i <= n ? s.path[i] : -1;
                if (i != n) out[i] = i < n ? s.tok[s.path[i + 1]] : -1;
            }
        }
    }
}

template <bool kChain>
static int launch(const Args &a, int32_t num_reqs, cudaStream_t st) {
    // few requests: a wide cluster each, so that a row is read by many SMs; many: narrower ones
    int cs = kMaxCluster;
    while (cs > 1 && (int64_t)num_reqs * cs > Shape<kChain>::kAsked * current_sm_count()) cs /= 2;
    if ((int64_t)num_reqs * cs > 0x7fffffff) return BKV_ERR_INVALID_ARG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_reqs * cs));
    cfg.blockDim = dim3(Shape<kChain>::kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<kChain>, a);
    if (e != cudaSuccess) set_cuda_error(e);
    return launch_status();
}

}  // namespace verify
}  // namespace bkv

extern "C" int bkv_verify_draft_chain(const float *target_probs, int64_t target_req_stride, int64_t target_row_stride,
                                      const float *draft_probs, int64_t draft_req_stride, int64_t draft_row_stride,
                                      const int64_t *draft_tokens, const int32_t *draft_lens, const float *accept_u,
                                      const float *sample_u, int32_t num_reqs, int32_t num_drafts, int32_t vocab_size,
                                      int64_t *out_tokens, int32_t *num_accepted, int32_t *err_count,
                                      bkv_stream_t stream) {
    using namespace bkv::verify;
    if (num_reqs < 0 || num_drafts < 0 || vocab_size <= 0) return BKV_ERR_INVALID_ARG;
    if (num_drafts > kMaxNodes) return BKV_ERR_UNSUPPORTED;
    if (target_row_stride < vocab_size || target_req_stride < 0 ||
        (num_drafts > 0 && (draft_row_stride < vocab_size || draft_req_stride < 0)))
        return BKV_ERR_INVALID_ARG;
    if (num_reqs == 0) return BKV_OK;
    if (!target_probs || !sample_u || !out_tokens || !num_accepted ||
        (num_drafts > 0 && (!draft_probs || !draft_tokens || !accept_u)))
        return BKV_ERR_INVALID_ARG;
    const Args a{target_probs, target_req_stride, target_row_stride, draft_probs, draft_req_stride, draft_row_stride,
                 draft_tokens, nullptr, draft_lens, accept_u, sample_u, num_drafts, vocab_size, out_tokens, nullptr,
                 num_accepted, err_count};
    return launch<true>(a, num_reqs, (cudaStream_t)stream);
}

extern "C" int bkv_verify_draft_tree(const float *target_probs, int64_t target_req_stride, int64_t target_row_stride,
                                     const int64_t *draft_tokens, const int32_t *parents, const float *accept_u,
                                     const float *sample_u, int32_t num_reqs, int32_t num_nodes, int32_t vocab_size,
                                     int64_t *out_tokens, int32_t *path, int32_t *num_accepted, int32_t *err_count,
                                     bkv_stream_t stream) {
    using namespace bkv::verify;
    if (num_reqs < 0 || num_nodes <= 0 || vocab_size <= 0) return BKV_ERR_INVALID_ARG;
    if (num_nodes > kMaxNodes) return BKV_ERR_UNSUPPORTED;
    if (target_row_stride < vocab_size || target_req_stride < 0) return BKV_ERR_INVALID_ARG;
    if (num_reqs == 0) return BKV_OK;
    if (!target_probs || !draft_tokens || !parents || !accept_u || !sample_u || !out_tokens || !path || !num_accepted)
        return BKV_ERR_INVALID_ARG;
    const Args a{target_probs, target_req_stride, target_row_stride, nullptr, 0, 0, draft_tokens, parents, nullptr,
                 accept_u, sample_u, num_nodes, vocab_size, out_tokens, path, num_accepted, err_count};
    return launch<false>(a, num_reqs, (cudaStream_t)stream);
}
