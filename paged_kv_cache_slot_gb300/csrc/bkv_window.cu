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
// positions at a time and U of those at once (their loads in flight together;
// the positions' block entries come one step ahead).  Each set of LP lanes
// keeps its own running maximum, sum and output for the NR query rows, and the
// sets are joined when the unit ends.
//
// Bound by the loads in flight and, from 8 query rows on, by issue slots: a
// position costs 16 multiply-adds a lane and row, log2(LP) shuffles and an
// exponential.
// ---------------------------------------------------------------------------
constexpr int kCcThreads = 128;
constexpr int kCcTile = 64;
constexpr int kCcPerSm = 2;   // CTAs an SM is laid out for

template <typename T, typename KV, int NR, int LP>
__global__ void __launch_bounds__(kCcThreads, kCcPerSm) window_cc_kernel(const Args a, const bool vec) {
    constexpr int U = sizeof(KV) == 4 || NR > 4 ? 2 : 4;
    constexpr int PW = 32 / LP;          // positions a warp holds at once
    constexpr int DP = 8 * LP;
    constexpr bool kF8 = sizeof(KV) == 1;
    __shared__ int32_t pre[kMaxReqs + 1], lens[kMaxReqs], sums[kCcThreads / 32];
    __shared__ float so[4][NR][DP], sm[4][NR], sl[4][NR];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / LP, e0 = (lane % LP) * 8;   // this lane's position of PW, and elements
    const int ne = min(max(a.D - e0, 0), 8);
    const int HP = a.H_kv * a.groups;
    const int q = (int)blockIdx.x / HP, hp = (int)blockIdx.x - q * HP;
    const int g = hp / a.groups, grp = hp - g * a.groups;
    const int i0 = grp * a.NR;
    const int rows = min(a.NR, a.q_len * a.G - i0);
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
        float qv[NR][8], o[NR][8], m[NR], l[NR];
        int32_t tp[NR];   // a row's own position
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int nn = min(n, rows - 1);
            tp[n] = s.L - a.q_len + (i0 + nn) / a.G;
            Eight<T> raw;
            raw.zero();
            if (n < rows && ne > 0) raw.load(static_cast<const T *>(a.q) + out_row(x.r, n) + e0, ne, vec);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = raw.two(i);
                qv[n][2 * i] = f.x * a.scale_log2;
                qv[n][2 * i + 1] = f.y * a.scale_log2;
            }
            m[n] = -INFINITY;
            l[n] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[n][i] = 0.f;
        }
        // Bad entries among the blocks that the unit begins, counted once a KV head: every block that the span
        // reads begins once in it, at its first position there.
        if (a.err && grp == 0) {
            for (int v = x.f * kCcTile + (int)threadIdx.x; v < v_end; v += kCcThreads) {
                const int32_t p = s.pos(v);
                if (p % a.bs != 0 && !(s.gap > 0 && v == s.sb && (s.sb == 0 || p / a.bs != (s.sb - 1) / a.bs))) continue;
                const int32_t lb = p / a.bs;
                if (lb >= a.bt_cols || __ldg(a.bt + (int64_t)x.r * a.bt_stride + lb) >= a.total_blocks) atomicAdd(a.err, 1);
            }
        }
        // which of the rows see position p, as bits
        auto seen = [&](int32_t p) {
            uint32_t b = 0u;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const bool last = p <= (a.causal ? tp[n] : s.L - 1);
                const bool near = a.window == 0 || p > tp[n] - a.window || p < a.sinks;
                b |= (last && near && n < rows) ? 1u << n : 0u;
            }
            return b;
        };
        // where position v of the span is cached: row of the cache, or -1
        auto entry = [&](int v, int32_t &p) -> int64_t {
            p = -1;
            if (v >= v_end) return -1;
            p = s.pos(v);
            const int32_t lb = p / a.bs;
            const int64_t b = lb < a.bt_cols ? __ldg(a.bt + (int64_t)x.r * a.bt_stride + lb) : 0;
            return b > 0 && b < a.total_blocks ? b * a.bs + (p - lb * a.bs) : -1;
        };
        const int step = 4 * PW * U;
        int v0 = x.f * kCcTile + warp * PW * U;
        int64_t row[U];
        int32_t pos[U];
#pragma unroll
        for (int u = 0; u < U; ++u) row[u] = entry(v0 + u * PW + sub, pos[u]);
        for (; v0 < v_end; v0 += step) {
            Eight<KV> kr[U], vr[U];
            float ks[U], vs[U];
            uint32_t see[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                see[u] = row[u] >= 0 ? seen(pos[u]) : 0u;
                kr[u].zero();
                vr[u].zero();
                ks[u] = vs[u] = 1.f;
                if (see[u]) {
                    const int64_t at = (row[u] * a.H_kv + g) * a.D + e0;
                    if (ne > 0) {
                        kr[u].load(static_cast<const KV *>(a.k) + at, ne, vec);
                        vr[u].load(static_cast<const KV *>(a.v) + at, ne, vec);
                    }
                    if constexpr (kF8) {
                        const int64_t b = row[u] / a.bs * a.H_kv + g;
                        ks[u] = __ldg(a.ks + b);
                        vs[u] = fminf(fmaxf(__ldg(a.vs + b), kScaleMin), kScaleMax);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) row[u] = entry(v0 + step + u * PW + sub, pos[u]);
            float sc[U][NR];
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int n = 0; n < NR; ++n) sc[u][n] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = kr[u].two(i);
#pragma unroll
                    for (int n = 0; n < NR; ++n) sc[u][n] = fmaf(qv[n][2 * i + 1], f.y, fmaf(qv[n][2 * i], f.x, sc[u][n]));
                }
#pragma unroll
                for (int n = 0; n < NR; ++n) {
#pragma unroll
                    for (int w = LP / 2; w > 0; w >>= 1) sc[u][n] += __shfl_xor_sync(0xffffffffu, sc[u][n], w);
                    sc[u][n] = (see[u] >> n) & 1u ? sc[u][n] * ks[u] : -INFINITY;
                }
            }
            // a value that some rows see and others do not reaches only the former, whatever it is
            const uint32_t full = (1u << rows) - 1u;
            bool mixed = false;
#pragma unroll
            for (int u = 0; u < U; ++u) mixed |= see[u] != 0u && see[u] != full;
            mixed = __any_sync(0xffffffffu, mixed);
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                float mn = m[n];
#pragma unroll
                for (int u = 0; u < U; ++u) mn = fmaxf(mn, sc[u][n]);
                const float corr = mn == -INFINITY ? 1.f : exp2f(m[n] - mn);
                m[n] = mn;
                l[n] *= corr;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    sc[u][n] = sc[u][n] == -INFINITY ? 0.f : exp2f(sc[u][n] - mn);
                    l[n] += sc[u][n];
                    if constexpr (kF8) sc[u][n] *= vs[u];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) o[n][i] *= corr;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = vr[u].two(i);
                    if (!mixed) {
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            o[n][2 * i] = fmaf(sc[u][n], f.x, o[n][2 * i]);
                            o[n][2 * i + 1] = fmaf(sc[u][n], f.y, o[n][2 * i + 1]);
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < NR; ++n)
                            if ((see[u] >> n) & 1u) {
                                o[n][2 * i] = fmaf(sc[u][n], f.x, o[n][2 * i]);
                                o[n][2 * i + 1] = fmaf(sc[u][n], f.y, o[n][2 * i + 1]);
                            }
                    }
                }
        }
        // join the warp's sets of lanes, then the warps
        auto join = [](float m0, float m1, float &f0, float &f1) {
            const float mn = fmaxf(m0, m1);
            f0 = mn == -INFINITY ? 1.f : exp2f(m0 - mn);
            f1 = mn == -INFINITY ? 1.f : exp2f(m1 - mn);
            return mn;
        };
        __syncthreads();   // the last unit's sums have been read
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int w = LP; w < 32; w <<= 1) {
                float f0, f1;
                const float mn = join(m[n], __shfl_xor_sync(0xffffffffu, m[n], w), f0, f1);
                l[n] = l[n] * f0 + __shfl_xor_sync(0xffffffffu, l[n], w) * f1;
#pragma unroll
                for (int i = 0; i < 8; ++i) o[n][i] = o[n][i] * f0 + __shfl_xor_sync(0xffffffffu, o[n][i], w) * f1;
                m[n] = mn;
            }
            if (lane < LP) {
#pragma unroll
                for (int i = 0; i < 8; ++i) so[warp][n][e0 + i] = o[n][i];
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
    }
}

// ---------------------------------------------------------------------------
// Merge of the streams that several columns share, one (column, KV head, row
// group) a CTA row: the at most one stream that column q begins and does not
// end.  A warp a query row; the lanes hold the parts' maxima and sums, then
// the row's elements.  Bound by its launch and one chain of loads.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 4;

template <typename T>
__global__ void __launch_bounds__(kMergeWarps * 32) window_merge_kernel(const Args a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int HP = a.H_kv * a.groups;
    const int q = (int)blockIdx.x / HP, hp = (int)blockIdx.x - q * HP;
    const int2 e = a.ws_split[q];
    const int r = e.x, nch = e.y;
    if (nch == 0) return;
    const int g = hp / a.groups, i0 = (hp - g * a.groups) * a.NR;
    const int n = blockIdx.y * kMergeWarps + warp;
    if (n >= min(a.NR, a.q_len * a.G - i0)) return;
    auto at = [&](int c) { return ((int64_t)hp * (2 * a.P) + (c == 0 ? a.P + q : q + c)) * a.NR + n; };
    float M = -INFINITY;
    for (int c = lane; c < nch; c += 32) M = fmaxf(M, a.ws_ml[at(c) * 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const int t = (i0 + n) / a.G;
    T *out = static_cast<T *>(a.out) + (((int64_t)r * a.q_len + t) * a.H_q + g * a.G + (i0 + n - t * a.G)) * a.D;
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
    p->cc = make_split(nq, num_kv_heads, kCcRows, kCcPerSm * sms);
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
    const cudaError_t e = launch_pdl(window_cc_kernel<T, KV, NR, LP>, dim3((unsigned)(a.P * a.H_kv * a.groups)),
                                     dim3(kCcThreads), 0, st, a, vec);
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
    a.window = sliding_window;
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
