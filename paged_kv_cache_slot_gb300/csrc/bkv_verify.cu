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
// sums up to 256 fit 64 bits.  (Conversions to 64-bit integers run at 16 a
// clock and SM; fp64 additions at 2.)
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

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxNodes = 1024;   // drafts (chain) or nodes (tree) a request
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 8;        // elements of each row in flight a lane

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

// A probability in units of 2^-56 (below 0 and NaN: 0; above 1: 1).
__device__ __forceinline__ long long fixed(float x) { return __float2ll_rn(__saturatef(x) * 72057594037927936.f); }

// What token v weighs: its probability p, less the draft's q in a chain.
__device__ __forceinline__ unsigned long long weight(float p, float q) {
    const long long w = fixed(p) - fixed(q);
    return w > 0 ? w : 0;
}

struct Shared {
    float p[kMaxNodes], u[kMaxNodes];
    int32_t tok[kMaxNodes], par[kMaxNodes];
    int32_t ex[kMaxNodes];               // tree: rejected children's tokens at the stop node
    int32_t n, cur, nex;                 // accepted drafts, stop row, rejected tokens
    unsigned long long seg[kWarps];      // sums of the warps' parts
    unsigned long long run[kWarps];      // and of the warps' shares of the part with the border
    unsigned long long tot[2][kMaxCluster];
};

template <bool kChain>
__global__ void __launch_bounds__(kThreads) verify_kernel(const Args a) {
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int64_t r = blockIdx.x / cs;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
            s.tok[i] = in ? (int32_t)x : -1;
            s.u[i] = u;
            s.p[i] = node && in ? P[par * a.p_row + x] : 0.f;
        }
    }
    __syncthreads();
    if (!kChain && warp == 0) {
        // One pass over the nodes in index order: the children of the current node follow it, and a
        // child taken becomes the current node.  Lane 0's verdict goes round the warp.
        int cur = 0, n = 0, nex = 0;
        double rem = 1.0;
        int32_t *path = a.path + r * a.nodes;
        if (rank == 0 && lane == 0) path[0] = 0;
        for (int base = 0; base < len; base += 32) {
            const int c = base + lane;
            const int par = c < len ? s.par[c] : -1;
            unsigned todo = __ballot_sync(0xffffffffu, c > 0 && par == cur);
            while (todo) {
                const int l = __ffs(todo) - 1;
                const int cc = base + l;
                const int x = s.tok[cc];
                bool dup = false;   // a token counts once under a node
                for (int e = lane; e < nex; e += 32) dup |= s.ex[e] == x;
                dup = __any_sync(0xffffffffu, dup);
                const float pf = fminf(fmaxf(s.p[cc], 0.f), 1.f);
                const double p = dup ? 0.0 : (double)pf;
                if ((double)s.u[cc] * fmax(rem, 0.0) < p) {
                    cur = cc;
                    ++n;
                    nex = 0;
                    rem = 1.0;
                    if (rank == 0 && lane == 0) {
                        path[n] = cc;
                        a.out[r * a.nodes + n - 1] = x;
                    }
                    todo = __ballot_sync(0xffffffffu, c > cc && par == cur);
                } else {
                    rem -= p;
                    if (x >= 0 && !dup) {
                        if (lane == 0) s.ex[nex] = x;
                        ++nex;
                        __syncwarp();
                    }
                    todo &= todo - 1;
                }
            }
        }
        if (lane == 0) {
            s.n = n;
            s.cur = cur;
            s.nex = nex;
        }
        if (rank == 0) {
            for (int i = n + 1 + lane; i < len; i += 32) {
                path[i] = -1;
                a.out[r * a.nodes + i] = -1;
            }
        }
    }
    __syncthreads();
    const int n = s.n;
    const int cur = kChain ? n : s.cur;
    const bool residual = kChain && n < len;
    int64_t *out = a.out + r * (kChain ? a.nodes + 1 : a.nodes);
    if (rank == 0) {
        if (threadIdx.x == 0) {
            a.count[r] = n;
            out[n] = -1;   // until a warp finds the sample (it writes behind the cluster barrier)
        }
        if (kChain)
            for (int i = threadIdx.x; i <= a.nodes; i += kThreads)
                if (i != n) out[i] = i < n ? s.tok[i] : -1;
    }

    // ---- sample the next token ----
    const float *pr = P + cur * a.p_row;
    const float *qr = residual ? Q + cur * a.q_row : nullptr;
    const int part = (int)((((int64_t)a.V + cs * kWarps - 1) / (cs * kWarps) + 31) / 32 * 32);   // a warp's elements
    const int64_t v0 = ((int64_t)rank * kWarps + warp) * part;
    const int64_t v1 = min((int64_t)a.V, v0 + part);
    const float us = __ldg(a.us + r);
    // u in units of 2^-64; u >= 1 (and NaN) take the border to the whole sum's end, u < 0 to its start
    const unsigned long long U = us < 1.f ? __float2ull_rz(fmaxf(us, 0.f) * 18446744073709551616.f) : ~0ull;
    // pass 0: the residual weights; where they are all 0, pass 1: the row itself
    for (int pass = 0; pass < 2; ++pass) {
        const bool plain = pass == 1;
        const float *qq = plain ? nullptr : qr;
        unsigned long long sum = 0;
        for (int64_t base = v0 + lane; base < v1; base += 32 * kUnroll) {
            // every load of the round before the first conversion
            float x[kUnroll], y[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int64_t v = base + 32 * k;
                x[k] = v < v1 ? pr[v] : 0.f;
                y[k] = v < v1 && qq ? qq[v] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) sum += weight(x[k], y[k]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const int nex = plain ? 0 : s.nex;
        if (!kChain)
            for (int e = 0; e < nex; ++e)
                if (s.ex[e] >= v0 && s.ex[e] < v1) sum -= fixed(pr[s.ex[e]]);
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
        const unsigned long long border = __umul64hi(U, whole);   // floor(u * whole) < whole
        // the CTA whose part holds the border: its threads scan the warp's part that does, together
        if (border < before || border - before >= s.tot[pass][rank]) break;
        int w = 0;
        while (border - before >= s.seg[w]) before += s.seg[w++];
        const int64_t s0 = ((int64_t)rank * kWarps + w) * part;
        const int64_t s1 = min((int64_t)a.V, s0 + part);
        const int each = (part + kThreads - 1) / kThreads;
        const int64_t e0 = s0 + (int64_t)threadIdx.x * each;
        const int64_t e1 = min(s1, e0 + each);
        auto at = [&](int64_t v) -> unsigned long long {
            if (!kChain)
                for (int e = 0; e < nex; ++e)
                    if (s.ex[e] == v) return 0;
            return weight(pr[v], qq ? qq[v] : 0.f);
        };
        unsigned long long mine = 0;
        for (int64_t v = e0; v < e1; ++v) mine += at(v);
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
                run += at(v);
                if (run > border) {
                    out[n] = v;
                    break;
                }
            }
        break;
    }
}

template <bool kChain>
static int launch(const Args &a, int32_t num_reqs, cudaStream_t st) {
    // few requests: a wide cluster each, so that a row is read by many SMs
    const int cs = kMaxCluster;
    if ((int64_t)num_reqs * cs > 0x7fffffff) return BKV_ERR_INVALID_ARG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_reqs * cs));
    cfg.blockDim = dim3(kThreads);
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
