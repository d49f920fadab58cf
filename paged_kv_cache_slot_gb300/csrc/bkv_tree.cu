// bkv_tree.cu -- attention of drafted trees over the paged cache: planner,
// the CUDA-core kernel, the merge of split streams and the ABI entry points.
//
// Request r has T tree tokens, the last T of its L cached positions.  Token t
// sees the committed positions [0, L - T) and those of the tree's own that its
// mask row names (its ancestors and itself, as the caller builds it):
//   out_t = sum_j softmax_j(scale q_t . k_j) v_j, 0 where no key is seen.
// "Padding and Batching with Block KV", Cache Masking: mask_cache over the
// committed positions, mask_active between this step's tokens, here any mask;
// Special Block and Slot Values: null and sentinel entries contribute nothing.
//
// Every query row of a KV head (T * G) shares each K and V row, so the cache
// is read once: memory-bound up to about 280 rows a KV head in bf16 (4 D
// operations a row against 4 D bytes a position and head, at the measured
// rates), bound by the multiply-adds in fp32 from a few rows on.
#include <cuda_bf16.h>
#include <math.h>

#include "bkv_tree.cuh"

namespace bkv {
namespace tree {

static constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxT = 256;       // tree tokens a request
constexpr int kMaxCtx = 1 << 30; // positions a request: sums of one and a tile or a block stay within int32
constexpr int kBK = 32;          // keys a tile of the CUDA-core kernel
constexpr int kThreads = 128;
constexpr int kCcEnd = 1;        // tiles of the CUDA-core kernel that a unit's start and end take as long as

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ void unpack(const uint4 &w, float (&f)[8]) {   // eight bf16
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4 &w, float (&f)[4]) {   // four fp32
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void store_out(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store_out(float *p, float x) { *p = x; }

// Four of a row, at a multiple of four of their size.
__device__ __forceinline__ void store4(float *p, const float4 &v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float4 &v) {
    __nv_bfloat162 w[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(w);
}

// Two fp32 multiply-adds in one instruction (each rounded as fmaf's), on pairs
// of consecutive elements: half the issue slots of the products.
struct __align__(8) Pair {
    float x, y;
};
__device__ __forceinline__ unsigned long long bits(const Pair &p) {
    unsigned long long u;
    asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(p.x), "f"(p.y));
    return u;
}
__device__ __forceinline__ Pair fma2(const Pair &a, const Pair &b, const Pair &c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    Pair r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}

// ---------------------------------------------------------------------------
// CUDA-core kernel: any dtype, head_dim <= DP, any block size.  CTA = (column,
// KV head; BR query rows).  The schedule is the tensor-core kernel's: the
// requests' tiles of 32 positions laid end to end, a column an equal share of
// them, whatever the lengths.  A CTA finds its share by a scan over the lengths.
// Tiles go through shared memory as fp32.  A warp's share of S is keys by rows,
// of O elements by rows, each as wide as it can be in keys and elements: a
// thread's own keys and elements take four cycles of the shared memory each
// load, the rows' values, which eight lanes share, one.  S crosses shared
// memory to the eight lanes that own a row (its max and sum are three
// shuffles), the weights cross it back.
// Bound by shared memory and the multiply-adds in turn (a few warps an SM, by
// their registers; with more rows a thread they would balance) and, in small
// calls, by the chain length -> table -> keys.  13 requests of 33 to 2500
// positions, 11 tokens of 15 / 5 heads of 64, fp32: 28.4 us (32.3 with the keys
// of a tile shared by no warps and equal runs of positions; 16 of 35 to 268
// positions, 4 tokens of 15 / 5 heads of 128: 12.6, 22.4).
// A V row of the tree that is not finite is taken as 0 for the rows that do
// not see it, and makes the rows that do NaN.
// ---------------------------------------------------------------------------
// CTAs an SM is built to hold, by their registers.
__host__ __device__ constexpr int cc_ctas(int D, int BR) { return D > 128 || (D > 64 && BR > 32) ? 2 : 3; }

template <typename T, int DP, int BR>
__global__ void __launch_bounds__(kThreads, cc_ctas(DP, BR)) tree_cc_kernel(const TreeArgs a, bool vec) {
    constexpr int LD = DP + 4, LP = kBK + 4, RPT = BR / 16, W = 16 / sizeof(T);
    // S: KG groups of warps share the keys, the others the rows; a thread has SR rows and KT keys.
    // O: DG groups of warps share the elements, the others the rows; a thread has OR rows and DJ fours of elements.
    constexpr int KG = BR == 16 ? 4 : 2, SR = BR * KG / 16, KT = 4 / KG;
    constexpr int DG = DP >= 128 ? 4 : DP / 32, OR = BR * DG / 16, DJ = DP / 32 / DG;
    extern __shared__ float sm[];
    float *Qs = sm;                    // [BR][LD], scaled to base 2
    float *Ks = Qs + BR * LD;          // [kBK][LD]
    float *Vs = Ks + kBK * LD;         // [kBK][LD]
    float *Ps = Vs + kBK * LD;         // [BR][LP]: scores, then weights
    float *Cs = Ps + BR * LP;          // [BR]: what the tile's maxima scale O by
    __shared__ int64_t rowoff[2][kBK]; // element offset of each key's row, -1: not there; by tile parity
    __shared__ uint32_t live[2], poison[2];
    __shared__ int64_t warp_sums[kThreads / 32], first_s;
    __shared__ int32_t first_r;
    pdl_wait();
    pdl_trigger();
    const int q = blockIdx.x / a.H_kv, g = blockIdx.x - q * a.H_kv;
    const int nq = a.T * a.G, i0 = blockIdx.y * BR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ty = threadIdx.x >> 3, tx = threadIdx.x & 7;
    const int s_row = warp / KG * (4 * SR) + (ty & 3), s_key = warp % KG * (8 * KT) + tx;    // + 4 i, + 8 j
    const int o_row = warp / DG * (4 * OR) + (ty & 3), o_el = warp % DG * (32 * DJ) + 4 * tx;   // + 4 i, + 32 j
    const bool counts = a.err && g == 0 && blockIdx.y == 0;
    // the column's share [t0, t1) of the whole cost, and the request that it starts in (first_r, whose cost starts
    // at first_s): a run of requests a thread
    int64_t t0, t1, C, peff;
    {
        const int per = (a.num_reqs + kThreads - 1) / kThreads;
        const int lo = (int)min((int64_t)a.num_reqs, (int64_t)threadIdx.x * per);
        const int hi = (int)min((int64_t)a.num_reqs, (int64_t)lo + per);
        auto cost_of = [&](int r) {
            const int32_t L = tree_len(a, __ldg(a.ctx + r));
            return L > 0 ? (int64_t)((L + kBK - 1) / kBK + kCcEnd) : 0;
        };
        int64_t sum = 0;
        for (int r = lo; r < hi; ++r) {
            sum += cost_of(r);
            if (counts && q == 0 && __ldg(a.ctx + r) > a.max_ctx) atomicAdd(a.err, 1);
        }
        int64_t run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += y;
        }
        if (lane == 31) warp_sums[warp] = run;
        __syncthreads();
        C = 0;
        run -= sum;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) run += warp_sums[w];
            C += warp_sums[w];
        }
        peff = C < a.P ? C : a.P;
        t0 = t1 = C;
        if (q < peff) {
            const int64_t x0 = C * q, x1 = x0 + C;
            const bool small = x1 >> 32 == 0;   // (64-bit divisions take longer)
            t0 = small ? (int64_t)((uint32_t)x0 / (uint32_t)peff) : x0 / peff;
            t1 = small ? (int64_t)((uint32_t)x1 / (uint32_t)peff) : x1 / peff;
        }
        if (run <= t0 && t0 < run + sum) {
            int r = lo;
            for (int64_t c = cost_of(r); run + c <= t0; c = cost_of(++r)) run += c;
            first_r = r;
            first_s = run;
        }
    }
    // rows of requests without a position
    for (int64_t r = q + (int64_t)warp * a.P; r < a.num_reqs; r += (int64_t)(kThreads / 32) * a.P) {
        if (tree_len(a, __ldg(a.ctx + r)) > 0) continue;
        for (int row = i0; row < min(i0 + BR, nq); ++row)
            for (int d = lane; d < a.D; d += 32)
                store_out(static_cast<T *>(a.out) + ((r * a.T + row / a.G) * a.H_q + g * a.G + row % a.G) * a.D + d, 0.f);
    }
    __syncthreads();
    int2 split = make_int2(0, 0);
    int par = 0;
    int64_t s0 = first_s;   // the request's cost starts here
    for (int r = first_r; t0 < t1 && s0 < t1; ++r) {
        const int32_t L = tree_len(a, __ldg(a.ctx + r)), first = L - a.T;
        if (L == 0) continue;
        const int32_t tiles = (L + kBK - 1) / kBK;
        const int32_t lo = (int32_t)max(t0 - s0, (int64_t)0), hi = (int32_t)min(t1 - s0, (int64_t)tiles);
        const int64_t s_end = s0 + tiles;
        s0 = s_end + kCcEnd;
        if (lo >= hi) continue;
        const bool whole = lo == 0 && hi == tiles;
        if (lo == 0 && !whole) split = make_int2(r, (int)((s_end * peff - 1) / C) - q + 1);
        const int32_t start = lo * kBK, end = min(hi * kBK, L);
        if (a.err && blockIdx.y == 0) {   // a needed block counts once a KV head, where its first position is
            for (int32_t lb = (start + a.bs - 1) / a.bs + (int)threadIdx.x; lb <= (end - 1) / a.bs; lb += kThreads) {
                const bool bad = lb >= a.bt_cols || __ldg(a.bt + (int64_t)r * a.bt_stride + lb) >= a.total_blocks;
                if (bad) atomicAdd(a.err, 1);
            }
        }
        Pair o[OR][DJ][2];    // elements {0, 1}, {2, 3} of four
        float m[RPT], l[RPT]; // of rows ty + 16 i
#pragma unroll
        for (int i = 0; i < OR; ++i)
#pragma unroll
            for (int j = 0; j < DJ; ++j) o[i][j][0] = o[i][j][1] = Pair{0.f, 0.f};
        const uint32_t *mrow[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            const int row = min(i0 + ty + 16 * i, nq - 1);
            mrow[i] = a.mask + (int64_t)r * a.mask_stride + (int64_t)(row / a.G) * a.mask_words;
        }
        auto offset_of = [&](int32_t j) -> int64_t {
            if (j >= end) return -1;
            const int32_t lb = j / a.bs;
            const int64_t b = lb < a.bt_cols ? __ldg(a.bt + (int64_t)r * a.bt_stride + lb) : -1;
            return b > 0 && b < a.total_blocks ? ((b * a.bs + (j - lb * a.bs)) * a.H_kv + g) * a.D : -1;
        };
        auto publish = [&](int64_t off, int par) {   // by the first warp
            rowoff[par][threadIdx.x] = off;
            const uint32_t ok = __ballot_sync(0xffffffffu, off >= 0);
            if (threadIdx.x == 0) {
                live[par] = ok;
                poison[par] = 0u;
            }
        };
        // 16-byte loads of a tile, W elements each, NV a thread: all in flight before the first use, and (head_dim
        // up to 128) those of the next tile during this one's products
        constexpr int NV = kBK * DP / W / kThreads;
        static_assert(NV * W * kThreads == kBK * DP, "whole rounds of 16-byte loads");
        uint4 kw[NV], vw[NV];
        auto fetch = [&](int par) {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int e = (u * kThreads + (int)threadIdx.x) * W, i = e / DP, d = e - i * DP;
                const int64_t off = rowoff[par][i];
                const bool in = off >= 0 && d < a.D;
                kw[u] = vw[u] = make_uint4(0, 0, 0, 0);
                if (in) {
                    kw[u] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.k) + off + d));
                    vw[u] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.v) + off + d));
                }
            }
        };
        int64_t ahead = -1;   // the first warp's key of the next tile
        if (threadIdx.x < 32) {
            publish(offset_of(start + threadIdx.x), par);
            ahead = offset_of(start + kBK + threadIdx.x);
        }
        const T *Q = static_cast<const T *>(a.q);
        auto q_row = [&](int row) {
            const int t = row / a.G, h = g * a.G + (row - t * a.G);
            return Q + (((int64_t)r * a.T + t) * a.H_q + h) * a.D;
        };
        if (vec) {
#pragma unroll 8
            for (int e = threadIdx.x * W; e < BR * DP; e += kThreads * W) {
                const int i = e / DP, d = e - i * DP, row = i0 + i;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (row < nq && d < a.D) w = __ldg(reinterpret_cast<const uint4 *>(q_row(row) + d));
                float f[W];
                unpack(w, f);
#pragma unroll
                for (int z = 0; z < W; ++z) Qs[i * LD + d + z] = f[z] * a.scale_log2;
            }
        } else {
            for (int e = threadIdx.x; e < BR * DP; e += kThreads) {
                const int i = e / DP, d = e - i * DP, row = i0 + i;
                Qs[i * LD + d] = row < nq && d < a.D ? to_f(q_row(row)[d]) * a.scale_log2 : 0.f;
            }
        }
        __syncthreads();   // (the unit before is read out, too)
        if (vec) fetch(par);
        for (int32_t k0 = start; k0 < end; k0 += kBK, par ^= 1) {
            if (k0 > start) __syncthreads();   // the last tile is read out
            if (vec) {
#pragma unroll
                for (int u = 0; u < NV; ++u) {
                    const int e = (u * kThreads + (int)threadIdx.x) * W, i = e / DP, d = e - i * DP;
                    float f[W], h[W];
                    unpack(kw[u], f);
                    unpack(vw[u], h);
                    bool fine = true;
#pragma unroll
                    for (int z = 0; z < W; ++z) fine &= isfinite(h[z]);
#pragma unroll
                    for (int z = 0; z < W; z += 4) {
                        *reinterpret_cast<float4 *>(Ks + i * LD + d + z) = make_float4(f[z], f[z + 1], f[z + 2], f[z + 3]);
                        *reinterpret_cast<float4 *>(Vs + i * LD + d + z) = make_float4(h[z], h[z + 1], h[z + 2], h[z + 3]);
                    }
                    if (!fine && k0 + i >= first) atomicOr(&poison[par], 1u << i);
                }
            } else {
                for (int e = threadIdx.x; e < kBK * DP; e += kThreads) {
                    const int i = e / DP, d = e - i * DP;
                    const int64_t off = rowoff[par][i];
                    const bool in = off >= 0 && d < a.D;
                    const float kx = in ? to_f(static_cast<const T *>(a.k)[off + d]) : 0.f;
                    const float vx = in ? to_f(static_cast<const T *>(a.v)[off + d]) : 0.f;
                    Ks[i * LD + d] = kx;
                    Vs[i * LD + d] = vx;
                    if (k0 + i >= first && !isfinite(vx)) atomicOr(&poison[par], 1u << i);
                }
            }
            if (threadIdx.x < 32) {
                publish(ahead, par ^ 1);
                ahead = offset_of(k0 + 2 * kBK + threadIdx.x);
            }
            __syncthreads();
            const uint32_t bad = poison[par], there = live[par];
            if (vec && k0 + kBK < end) fetch(par ^ 1);
            if (bad) {
                for (int e = threadIdx.x; e < kBK * DP; e += kThreads) {
                    const int i = e / DP;
                    if ((bad >> i) & 1u) Vs[i * LD + (e - i * DP)] = 0.f;
                }
                __syncthreads();
            }
            Pair s2[SR][KT];   // sums over the even and the odd elements
#pragma unroll
            for (int i = 0; i < SR; ++i)
#pragma unroll
                for (int j = 0; j < KT; ++j) s2[i][j] = Pair{0.f, 0.f};
#pragma unroll 4
            for (int d = 0; d < DP; d += 4) {
                float4 kk[KT];
#pragma unroll
                for (int j = 0; j < KT; ++j) kk[j] = *reinterpret_cast<const float4 *>(Ks + (s_key + 8 * j) * LD + d);
#pragma unroll
                for (int i = 0; i < SR; ++i) {
                    const float4 qq = *reinterpret_cast<const float4 *>(Qs + (s_row + 4 * i) * LD + d);
#pragma unroll
                    for (int j = 0; j < KT; ++j) {
                        s2[i][j] = fma2(Pair{qq.x, qq.y}, Pair{kk[j].x, kk[j].y}, s2[i][j]);
                        s2[i][j] = fma2(Pair{qq.z, qq.w}, Pair{kk[j].z, kk[j].w}, s2[i][j]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < SR; ++i)
#pragma unroll
                for (int j = 0; j < KT; ++j) Ps[(s_row + 4 * i) * LP + s_key + 8 * j] = s2[i][j].x + s2[i][j].y;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                float *prow = Ps + (ty + 16 * i) * LP + tx;
                const uint32_t vis = there & (k0 + kBK <= first ? 0xffffffffu
                                                               : tree_vis32(mrow[i], a.mask_words, first, L, k0));
                float s[4], top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[j] = (vis >> (tx + 8 * j)) & 1u ? prow[8 * j] : -INFINITY;
                    top = fmaxf(top, s[j]);
                }
#pragma unroll
                for (int w = 4; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                const float mn = fmaxf(m[i], top);
                const float corr = mn == -INFINITY ? 1.f : exp2f(m[i] - mn);
                const float base = mn == -INFINITY ? 0.f : mn;   // nothing but scores of -inf so far: weights of 0
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // a seen NaN score stays NaN (fmaxf dropped it from the maximum)
                    const float p = (vis >> (tx + 8 * j)) & 1u ? exp2f(s[j] - base) : 0.f;
                    prow[8 * j] = p;
                    sum += p;
                }
#pragma unroll
                for (int w = 4; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                if (vis & bad) sum = NAN;
                l[i] = fmaf(l[i], corr, sum);
                m[i] = mn;
                if (tx == 0) Cs[ty + 16 * i] = corr;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < OR; ++i) {
                const float corr = Cs[o_row + 4 * i];
#pragma unroll
                for (int j = 0; j < DJ; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) o[i][j][e].x *= corr, o[i][j][e].y *= corr;
            }
#pragma unroll 2
            for (int k = 0; k < kBK; k += 4) {
                float4 vv[4][DJ];
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < DJ; ++j)
                        vv[e][j] = *reinterpret_cast<const float4 *>(Vs + (k + e) * LD + o_el + 32 * j);
#pragma unroll
                for (int i = 0; i < OR; ++i) {
                    const float4 p = *reinterpret_cast<const float4 *>(Ps + (o_row + 4 * i) * LP + k);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float w = e == 0 ? p.x : e == 1 ? p.y : e == 2 ? p.z : p.w;
#pragma unroll
                        for (int j = 0; j < DJ; ++j) {
                            o[i][j][0] = fma2(Pair{w, w}, Pair{vv[e][j].x, vv[e][j].y}, o[i][j][0]);
                            o[i][j][1] = fma2(Pair{w, w}, Pair{vv[e][j].z, vv[e][j].w}, o[i][j][1]);
                        }
                    }
                }
            }
        }
        if (whole) {   // the rows' 1 / l, for the threads that have their elements
            __syncthreads();
            if (tx == 0)
#pragma unroll
                for (int i = 0; i < RPT; ++i) Cs[ty + 16 * i] = l[i] == 0.f ? 0.f : 1.f / l[i];
            __syncthreads();
        }
        const int64_t slot = (int64_t)g * (2 * a.P) + (lo == 0 ? a.P + q : q);
#pragma unroll
        for (int i = 0; i < OR; ++i) {
            const int row = i0 + o_row + 4 * i;
            if (row >= nq) continue;
            const float inv = whole ? Cs[o_row + 4 * i] : 1.f;
            T *out = static_cast<T *>(a.out) + (((int64_t)r * a.T + row / a.G) * a.H_q + g * a.G + row % a.G) * a.D;
            float *po = a.ws_o + (slot * a.NR + row) * a.D;
#pragma unroll
            for (int j = 0; j < DJ; ++j) {
                const int d0 = o_el + 32 * j;
                const Pair x = o[i][j][0], y = o[i][j][1];
                if (!whole && a.D % 4 == 0) {
                    if (d0 < a.D) *reinterpret_cast<float4 *>(po + d0) = make_float4(x.x, x.y, y.x, y.y);
                } else {   // (head_dim is even)
                    if (d0 < a.D) {
                        if (whole) store_out(out + d0, x.x * inv), store_out(out + d0 + 1, x.y * inv);
                        else po[d0] = x.x, po[d0 + 1] = x.y;
                    }
                    if (d0 + 2 < a.D) {
                        if (whole) store_out(out + d0 + 2, y.x * inv), store_out(out + d0 + 3, y.y * inv);
                        else po[d0 + 2] = y.x, po[d0 + 3] = y.y;
                    }
                }
            }
        }
        if (!whole && tx == 0)
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int row = i0 + ty + 16 * i;
                if (row < nq) *reinterpret_cast<float2 *>(a.ws_ml + (slot * a.NR + row) * 2) = make_float2(m[i], l[i]);
            }
    }
    if (g == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.ws_split[q] = split;
}

// ---------------------------------------------------------------------------
// Merge of a stream's partials: out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M)
// l_c, 0 where nothing was seen.  A warp has one row: lane k keeps the weight of
// partial k, and the first partials are loaded beside the (m, l) pairs, so a
// stream of few partials costs one round of loads.  The kernels' table names
// the split stream that each column begins; a stream that one column finished
// is written already.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 8;

// MR rows of a warp at a time, MS of their partials in flight, for a head_dim of whole fours up to 128 (KD: 128, or 0
// for the others); MR 0: one row a warp by two elements a lane, any even head_dim.
template <typename T, int MR, int MS, int KD>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const TreeArgs a) {
    constexpr int kUnroll = 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int HP = a.H_kv * a.groups;
    const int q = (int)blockIdx.x / HP, hp = (int)blockIdx.x - q * HP;
    const int2 e = a.ws_split[q];   // the request that column q begins and does not end, and its columns
    const int r = e.x, nch = e.y;
    if (nch == 0) return;
    // partial c of the stream
    auto slot_of = [&](int c) { return (int64_t)hp * (2 * a.P) + (c == 0 ? a.P + q : q + c); };
    const int g = hp / a.groups, tok0 = (hp - g * a.groups) * a.TS;
    const int rows = min(a.NR, (a.T - tok0) * a.G);
    if constexpr (MR > 0) {
        // four elements a lane: a head_dim of whole fours up to 128
        const int D = KD ? KD : a.D;
        const bool act = 4 * lane < D;
        const int row0 = (blockIdx.y * kMergeWarps + warp) * MR;
#pragma unroll 1
        for (int rr = row0; rr < min(rows, row0 + MR); rr += MR) {
            float M[MR], sum[MR];
            float4 acc[MR];
#pragma unroll
            for (int i = 0; i < MR; ++i) {
                M[i] = -INFINITY;
                sum[i] = 0.f;
                acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            for (int base = 0; base < nch; base += 32) {   // lane k: slot base + k
                float2 ml[MR];
                float4 v[MR][MS];
                auto load = [&](int c) {
#pragma unroll
                    for (int i = 0; i < MR; ++i)
#pragma unroll
                        for (int k = 0; k < MS; ++k)
                            v[i][k] = act && rr + i < rows && c + k < nch
                                          ? *reinterpret_cast<const float4 *>(
                                                a.ws_o + (slot_of(c + k) * a.NR + rr + i) * D + 4 * lane)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                };
#pragma unroll
                for (int i = 0; i < MR; ++i)
                    ml[i] = rr + i < rows && base + lane < nch
                                ? *reinterpret_cast<const float2 *>(a.ws_ml + (slot_of(base + lane) * a.NR + rr + i) * 2)
                                : make_float2(-INFINITY, 0.f);
                load(base);
                float w[MR];
#pragma unroll
                for (int i = 0; i < MR; ++i) {
                    float top = ml[i].x;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const float mn = fmaxf(M[i], top);
                    const float corr = mn == -INFINITY ? 1.f : exp2f(M[i] - mn);   // of the slots before
                    w[i] = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - mn);
                    // a part that saw nothing but NaN scores has no maximum, and a NaN sum
                    float part = (ml[i].x == -INFINITY && ml[i].y != ml[i].y ? 1.f : w[i]) * ml[i].y;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
                    sum[i] = fmaf(sum[i], corr, part);
                    acc[i].x *= corr, acc[i].y *= corr, acc[i].z *= corr, acc[i].w *= corr;
                    M[i] = mn;
                }
                for (int c = base; c < min(nch, base + 32); c += MS) {
                    if (c > base) load(c);
#pragma unroll
                    for (int k = 0; k < MS; ++k)
#pragma unroll
                        for (int i = 0; i < MR; ++i) {
                            const float wk = __shfl_sync(0xffffffffu, w[i], (c + k) & 31);
                            acc[i].x = fmaf(wk, v[i][k].x, acc[i].x);
                            acc[i].y = fmaf(wk, v[i][k].y, acc[i].y);
                            acc[i].z = fmaf(wk, v[i][k].z, acc[i].z);
                            acc[i].w = fmaf(wk, v[i][k].w, acc[i].w);
                        }
                }
            }
#pragma unroll
            for (int i = 0; i < MR; ++i) {
                const int row = rr + i;
                if (row >= rows) break;
                const float inv = sum[i] == 0.f ? 0.f : 1.f / sum[i];
                T *out = static_cast<T *>(a.out) +
                         (((int64_t)r * a.T + tok0 + row / a.G) * a.H_q + g * a.G + row % a.G) * D + 4 * lane;
                if (!act) continue;
                store4(out, make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
            }
        }
        return;
    }
    const int row = blockIdx.y * kMergeWarps + warp;
    if (row >= rows) return;
    const int t = tok0 + row / a.G, h = g * a.G + row % a.G;
    T *out = static_cast<T *>(a.out) + (((int64_t)r * a.T + t) * a.H_q + h) * a.D;
    auto ml_of = [&](int c) {
        return c < nch ? *reinterpret_cast<const float2 *>(a.ws_ml + (slot_of(c) * a.NR + row) * 2)
                       : make_float2(-INFINITY, 0.f);
    };
    const float2 ml0 = ml_of(lane);
    for (int d0 = 0; d0 < a.D; d0 += 64) {   // two elements a lane
        const int d = d0 + 2 * lane;
        const bool act = d < a.D;
        auto part = [&](int c) {
            return act && c < nch ? *reinterpret_cast<const float2 *>(a.ws_o + (slot_of(c) * a.NR + row) * a.D + d)
                                  : make_float2(0.f, 0.f);
        };
        float2 v[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) v[k] = part(k);
        float M = ml0.x;
        for (int c = lane + 32; c < nch; c += 32) M = fmaxf(M, ml_of(c).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float sum = 0.f;
        float2 acc = make_float2(0.f, 0.f);
        for (int base = 0; base < nch; base += 32) {
            const float2 ml = base == 0 ? ml0 : ml_of(base + lane);
            const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
            // a part that saw nothing but NaN scores has no maximum, and a NaN sum
            sum = fmaf(ml.x == -INFINITY && ml.y != ml.y ? 1.f : w, ml.y, sum);
            for (int c = base; c < min(nch, base + 32); c += kUnroll) {
                if (c > 0)
#pragma unroll
                    for (int k = 0; k < kUnroll; ++k) v[k] = part(c + k);
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    const float wk = __shfl_sync(0xffffffffu, w, (c + k) & 31);
                    acc.x = fmaf(wk, v[k].x, acc.x);
                    acc.y = fmaf(wk, v[k].y, acc.y);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (act) {
            store_out(out + d, acc.x * inv);
            store_out(out + d + 1, acc.y * inv);
        }
    }
}

// ---------------------------------------------------------------------------
// Planner
// ---------------------------------------------------------------------------
struct Plan {
    int32_t P_cc;                 // the CUDA-core kernel's columns
    int64_t slots_cc, slots_tc;   // the kernels' partial slots (tensor-core: 0 where it cannot run)
    int64_t split_bytes;          // the table of split streams
    size_t ws_bytes;
};

// Tokens of a slot and CTA columns of the tensor-core kernel: a stream's T G
// rows are one query tile of 128 / G tokens, or pairs of them.
static void tc_split(int32_t T, int32_t G, int32_t H_kv, int32_t *TS, int32_t *groups, int32_t *P) {
    const int32_t tt = G <= 128 ? 128 / G : 1;
    *TS = T <= tt ? T : 2 * tt;
    *groups = (T + *TS - 1) / *TS;
    const int64_t cols = (int64_t)H_kv * *groups;
    const int64_t sms = current_sm_count();
    *P = (int32_t)(cols < sms ? sms / cols : 1);
}

// The query tile (16, 32, 48 or 64 rows; up to 32 with head_dim above 128, for
// its registers) that leaves the fewest rows idle, the larger of two.
static int query_tile(int32_t nq, int32_t D) {
    int best = 16;
    for (int br = 32; br <= (D > 128 ? 32 : 64); br += 16)
        if (ceil_div(nq, br) * br <= ceil_div(nq, best) * best) best = br;
    return best;
}

// Columns of the CUDA-core kernel: CTAs for one wave; where the heads and query tiles alone come near one, about four
// waves, so that the last one's idle part is small.
static int32_t cc_columns(int32_t nq, int32_t D, int32_t H_kv) {
    const int br = query_tile(nq, D);
    const int64_t resident = (int64_t)current_sm_count() * cc_ctas(D, br);
    const int64_t cols = (int64_t)H_kv * ceil_div(nq, br);
    return (int32_t)(cols <= resident / 4 ? resident / cols : ceil_div<int64_t>(4 * resident, cols));
}

static bool make_plan(int32_t num_reqs, int32_t T, int32_t H_q, int32_t H_kv, int32_t D, int32_t bs, int32_t max_ctx,
                      Plan *p) {
    if (num_reqs <= 0 || T <= 0 || T > kMaxT || H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0 || D <= 0 || D > 256 ||
        D % 2 != 0 || bs <= 0 || bs > 65536 || max_ctx < 0 || max_ctx > kMaxCtx)
        return false;
    const int32_t G = H_q / H_kv;
    const int64_t nq = (int64_t)T * G;
    p->P_cc = cc_columns((int32_t)nq, D, H_kv);
    p->slots_cc = (int64_t)H_kv * 2 * p->P_cc;
    // grids
    if ((int64_t)p->P_cc * H_kv >= ((int64_t)1 << 31) || ceil_div<int64_t>(nq, kMergeWarps) > 65535) return false;
    if ((int64_t)num_reqs * (max_ctx / kBK + 2 + kCcEnd) >= (int64_t)1 << 48) return false;   // costs
    int64_t rows = p->slots_cc * nq;
    p->slots_tc = 0;
    int32_t P = 1;
    if (D == 128 && G <= 128) {
        int32_t TS, groups;
        tc_split(T, G, H_kv, &TS, &groups, &P);
        p->slots_tc = (int64_t)H_kv * groups * 2 * P;
        const int64_t rt = p->slots_tc * TS * G;
        if (rt > rows) rows = rt;
    }
    p->split_bytes = ceil_div<int64_t>((p->P_cc > P ? p->P_cc : P) * (int64_t)sizeof(int2), 256) * 256;
    p->ws_bytes = (size_t)(p->split_bytes + ceil_div<int64_t>(rows * D * 4, 256) * 256 +
                           ceil_div<int64_t>(rows * 8, 256) * 256);
    return true;
}

template <typename T, int DP, int BR>
static cudaError_t launch_cc(const TreeArgs &a, cudaStream_t st) {
    constexpr int smem = ((BR + 2 * kBK) * (DP + 4) + BR * (kBK + 4) + BR) * 4;
    auto kern = tree_cc_kernel<T, DP, BR>;
    if (smem > 48 * 1024) {
        static bool set[64] = {};
        int dev = 0;
        cudaGetDevice(&dev);
        if (dev < 0 || dev >= 64 || !set[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) set[dev] = true;
        }
    }
    const dim3 grid((unsigned)(a.P * a.H_kv), (unsigned)ceil_div(a.T * a.G, BR));
    // rows of whole 16-byte pieces
    const bool vec = a.D * sizeof(T) % 16 == 0 && aligned(a.q, 16) && aligned(a.k, 16) && aligned(a.v, 16);
    return launch_pdl(kern, grid, dim3(kThreads), smem, st, a, vec);
}

template <typename T, int DP>
static cudaError_t launch_cc_rows(const TreeArgs &a, cudaStream_t st) {
    const int br = query_tile(a.T * a.G, a.D);
    if constexpr (DP <= 128) {
        if (br == 64) return launch_cc<T, DP, 64>(a, st);
        if (br == 48) return launch_cc<T, DP, 48>(a, st);
    }
    return br == 32 ? launch_cc<T, DP, 32>(a, st) : launch_cc<T, DP, 16>(a, st);
}

template <typename T>
static cudaError_t launch_cc_dims(const TreeArgs &a, cudaStream_t st) {
    if (a.D <= 32) return launch_cc_rows<T, 32>(a, st);
    if (a.D <= 64) return launch_cc_rows<T, 64>(a, st);
    if (a.D <= 128) return launch_cc_rows<T, 128>(a, st);
    return launch_cc_rows<T, 256>(a, st);
}

template <int MR, int MS, int KD>
static int launch_merge(const TreeArgs &a, cudaStream_t st) {
    const int64_t x = (int64_t)a.P * a.H_kv * a.groups;
    const dim3 grid((unsigned)x, (unsigned)ceil_div(a.NR, kMergeWarps * (MR ? MR : 1))), block(kMergeWarps * 32);
    cudaError_t e;
    if (a.dtype == BKV_BF16) e = launch_pdl(tree_merge_kernel<__nv_bfloat16, MR, MS, KD>, grid, block, 0, st, a);
    else e = launch_pdl(tree_merge_kernel<float, MR, MS, KD>, grid, block, 0, st, a);
    if (e != cudaSuccess) set_cuda_error(e);
    return launch_status();
}

// Few rows, or streams in many parts: one row a warp, eight of its parts at once (28 rows of 8 streams: 1.3 us a call
// less than by two rows; 3 requests of up to 13459 positions, 96 rows over 46 columns: 16.5 us, 18.3).  Else two rows a
// warp (32 requests of up to 4096, 64 rows over 19 columns: 51.4 us, 53.2 by one).
static int merge(const TreeArgs &a, cudaStream_t st) {
    const bool fours = a.D <= 128 && a.D % 4 == 0 && aligned(a.out, a.dtype == BKV_BF16 ? 8 : 16);
    if (!fours) return launch_merge<0, 0, 0>(a, st);
    const bool one = a.NR <= 32 || a.P > 2 * (int64_t)a.num_reqs;
    if (a.D == 128) return one ? launch_merge<1, 8, 128>(a, st) : launch_merge<2, 4, 128>(a, st);
    return one ? launch_merge<1, 8, 0>(a, st) : launch_merge<2, 4, 0>(a, st);
}

}  // namespace tree
}  // namespace bkv

extern "C" size_t bkv_paged_decode_tree_workspace_size(int32_t num_reqs, int32_t q_len, int32_t num_q_heads,
                                                       int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                                       int32_t max_context_len) {
    bkv::tree::Plan p;
    if (!bkv::tree::make_plan(num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, &p))
        return 0;
    return p.ws_bytes;
}

extern "C" int bkv_paged_decode_tree(const void *q, const void *k_cache, const void *v_cache,
                                     const int32_t *block_table, int64_t bt_stride, int32_t bt_cols,
                                     const int32_t *context_lens, int32_t max_context_len, int32_t num_reqs,
                                     int32_t q_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                     int32_t block_size, int64_t total_blocks, float softmax_scale,
                                     const uint32_t *tree_mask, int64_t mask_req_stride, int dtype, void *out,
                                     void *workspace, size_t workspace_bytes, int32_t *err_count,
                                     bkv_stream_t stream) {
    using namespace bkv;
    using namespace bkv::tree;
    if (dtype != BKV_BF16 && dtype != BKV_F32) return BKV_ERR_UNSUPPORTED;
    if (head_dim > 256 || head_dim % 2 != 0 || q_len > kMaxT) return BKV_ERR_UNSUPPORTED;
    if (bt_cols < 0 || bt_stride < bt_cols || total_blocks < 0) return BKV_ERR_INVALID_ARG;
    Plan plan;
    if (!make_plan(num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, &plan))
        return BKV_ERR_INVALID_ARG;
    const int32_t words = (q_len + 31) / 32;
    if (mask_req_stride != 0 && mask_req_stride < (int64_t)q_len * words) return BKV_ERR_INVALID_ARG;
    if (!q || !out || !context_lens || !tree_mask || (bt_cols > 0 && !block_table)) return BKV_ERR_INVALID_ARG;
    if (max_context_len > 0 && (!k_cache || !v_cache)) return BKV_ERR_INVALID_ARG;
    if (workspace_bytes < plan.ws_bytes || !workspace || !aligned(workspace, 32)) return BKV_ERR_INVALID_ARG;
    if (!(softmax_scale > 0.f)) softmax_scale = 1.0f / sqrtf((float)head_dim);
    TreeArgs a{};
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.bt = block_table;
    a.bt_stride = bt_stride;
    a.bt_cols = bt_cols;
    a.ctx = context_lens;
    a.max_ctx = max_context_len;
    a.num_reqs = num_reqs;
    a.T = q_len;
    a.H_q = num_q_heads;
    a.H_kv = num_kv_heads;
    a.D = head_dim;
    a.bs = block_size;
    a.G = num_q_heads / num_kv_heads;
    a.total_blocks = total_blocks;
    a.scale_log2 = softmax_scale * kLog2e;
    a.mask = tree_mask;
    a.mask_stride = mask_req_stride;
    a.mask_words = words;
    a.dtype = dtype;
    a.out = out;
    a.err = err_count;
    auto set_slots = [&](int64_t slots) {
        char *base = static_cast<char *>(workspace) + plan.split_bytes;
        a.ws_split = static_cast<int2 *>(workspace);
        a.ws_o = reinterpret_cast<float *>(base);
        a.ws_ml = reinterpret_cast<float *>(base + ceil_div<int64_t>(slots * a.NR * head_dim * 4, 256) * 256);
    };
    cudaStream_t st = (cudaStream_t)stream;
    TreeTc t;
    if (plan.slots_tc > 0) {
        tc_split(a.T, a.G, a.H_kv, &a.TS, &a.groups, &a.P);
        a.NR = a.TS * a.G;
        if (prepare_tree_tc(a, &t)) {
            set_slots(plan.slots_tc);
            const int rc = launch_tree_tc(a, t, st);
            if (rc != BKV_OK) return rc;
            return merge(a, st);
        }
    }
    // one query-row group for all tokens: the CUDA-core kernel's slots
    a.TS = q_len;
    a.NR = q_len * a.G;
    a.groups = 1;
    a.P = plan.P_cc;
    set_slots(plan.slots_cc);
    const cudaError_t e = dtype == BKV_BF16 ? launch_cc_dims<__nv_bfloat16>(a, st) : launch_cc_dims<float>(a, st);
    if (e != cudaSuccess) set_cuda_error(e);
    const int rc = launch_status();
    return rc != BKV_OK ? rc : merge(a, st);
}
