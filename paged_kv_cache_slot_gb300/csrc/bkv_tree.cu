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
constexpr int kBK = 32;          // keys a tile of the CUDA-core kernel
constexpr int kThreads = 128;

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
// CUDA-core kernel: any dtype, head_dim <= DP, any block size.  CTA = (stream
// (request, KV head), split of positions; BR query rows).  Keys come in tiles
// of 32 through shared memory as fp32; eight consecutive lanes own a query row:
// lane x of them the keys x, x + 8, .. of S and the elements 4 x + 32 j of O,
// so the row's max and sum are three shuffles and P only crosses its own warp.
// A V row of the tree that is not finite is taken as 0 for the rows that do
// not see it, and makes the rows that do NaN.
// ---------------------------------------------------------------------------
template <typename T, int DP, int BR>
__global__ void __launch_bounds__(kThreads) tree_cc_kernel(const TreeArgs a, bool vec) {
    constexpr int LD = DP + 4, RPT = BR / 16, DJ = DP / 32, W = 16 / sizeof(T);
    extern __shared__ float sm[];
    float *Qs = sm;                    // [BR][LD], scaled to base 2
    float *Ks = Qs + BR * LD;          // [kBK][LD]
    float *Vs = Ks + kBK * LD;         // [kBK][LD]
    float *Ps = Vs + kBK * LD;         // [BR][kBK + 4]
    __shared__ int64_t rowoff[2][kBK]; // element offset of each key's row, -1: not there; by tile parity
    __shared__ uint32_t live[2], poison[2];
    pdl_wait();
    pdl_trigger();
    const int rg = blockIdx.x / a.n_chunks, c = blockIdx.x - rg * a.n_chunks;
    const int r = rg / a.H_kv, g = rg - r * a.H_kv;
    const int nq = a.T * a.G, i0 = blockIdx.y * BR;
    const int ty = threadIdx.x >> 3, tx = threadIdx.x & 7;
    const int32_t ctx = __ldg(a.ctx + r);
    const int32_t L = tree_len(a, ctx), first = L - a.T;
    if (ctx > a.max_ctx && c == 0 && g == 0 && blockIdx.y == 0 && threadIdx.x == 0 && a.err) atomicAdd(a.err, 1);
    const int32_t start = c * a.chunk;
    if (start >= L) return;
    const int32_t end = min(start + a.chunk, L);
    if (a.err && blockIdx.y == 0) {   // splits hold whole blocks: each needed block counts once a KV head
        for (int32_t lb = start / a.bs + threadIdx.x; lb <= (end - 1) / a.bs; lb += kThreads) {
            const bool bad = lb >= a.bt_cols || __ldg(a.bt + (int64_t)r * a.bt_stride + lb) >= a.total_blocks;
            if (bad) atomicAdd(a.err, 1);
        }
    }
    Pair o[RPT][DJ][2];   // elements 4 tx + 32 j + {0, 1}, {2, 3}
    float m[RPT], l[RPT];
    const uint32_t *mrow[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        const int row = min(i0 + ty + 16 * i, nq - 1);
        mrow[i] = a.mask + (int64_t)r * a.mask_stride + (int64_t)(row / a.G) * a.mask_words;
#pragma unroll
        for (int j = 0; j < DJ; ++j) o[i][j][0] = o[i][j][1] = Pair{0.f, 0.f};
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
            kw[u] = in ? __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.k) + off + d)) : make_uint4(0, 0, 0, 0);
            vw[u] = in ? __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.v) + off + d)) : make_uint4(0, 0, 0, 0);
        }
    };
    int64_t ahead = -1;   // the first warp's key of the next tile
    if (threadIdx.x < 32) {
        publish(offset_of(start + threadIdx.x), 0);
        ahead = offset_of(start + kBK + threadIdx.x);
    }
    __syncthreads();
    if (vec) fetch(0);
    const T *Q = static_cast<const T *>(a.q);
    auto q_row = [&](int row) {
        const int t = row / a.G, h = g * a.G + (row - t * a.G);
        return Q + (((int64_t)r * a.T + t) * a.H_q + h) * a.D;
    };
    if (vec) {
#pragma unroll 8
        for (int e = threadIdx.x * W; e < BR * DP; e += kThreads * W) {
            const int i = e / DP, d = e - i * DP, row = i0 + i;
            const uint4 w = row < nq && d < a.D ? __ldg(reinterpret_cast<const uint4 *>(q_row(row) + d)) : make_uint4(0, 0, 0, 0);
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
    int par = 0;
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
        Pair s2[RPT][4];   // sums over the even and the odd elements
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s2[i][j] = Pair{0.f, 0.f};
#pragma unroll 4
        for (int d = 0; d < DP; d += 4) {
            float4 kk[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4 *>(Ks + (tx + 8 * j) * LD + d);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float4 qq = *reinterpret_cast<const float4 *>(Qs + (ty + 16 * i) * LD + d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s2[i][j] = fma2(Pair{qq.x, qq.y}, Pair{kk[j].x, kk[j].y}, s2[i][j]);
                    s2[i][j] = fma2(Pair{qq.z, qq.w}, Pair{kk[j].z, kk[j].w}, s2[i][j]);
                }
            }
        }
        float s[RPT][4];
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
        __syncwarp();   // this warp's P rows of the last tile are read
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const uint32_t vis = there & (k0 + kBK <= first ? 0xffffffffu
                                                           : tree_vis32(mrow[i], a.mask_words, first, L, k0));
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = (vis >> (tx + 8 * j)) & 1u ? s[i][j] : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int w = 4; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            const float mn = fmaxf(m[i], top);
            const float corr = mn == -INFINITY ? 1.f : exp2f(m[i] - mn);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // a seen NaN score stays NaN (fmaxf dropped it from the maximum)
                const float p = (vis >> (tx + 8 * j)) & 1u ? exp2f(s[i][j] - mn) : 0.f;
                Ps[(ty + 16 * i) * (kBK + 4) + tx + 8 * j] = p;
                sum += p;
            }
#pragma unroll
            for (int w = 4; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            if (vis & bad) sum = NAN;
            l[i] = fmaf(l[i], corr, sum);
            m[i] = mn;
#pragma unroll
            for (int j = 0; j < DJ; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) o[i][j][e].x *= corr, o[i][j][e].y *= corr;
        }
        __syncwarp();
#pragma unroll 2
        for (int k = 0; k < kBK; k += 4) {
            float4 p[RPT];
#pragma unroll
            for (int i = 0; i < RPT; ++i)
                p[i] = *reinterpret_cast<const float4 *>(Ps + (ty + 16 * i) * (kBK + 4) + k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int j = 0; j < DJ; ++j) {
                    const float4 vv = *reinterpret_cast<const float4 *>(Vs + (k + e) * LD + 4 * tx + 32 * j);
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const float w = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
                        o[i][j][0] = fma2(Pair{w, w}, Pair{vv.x, vv.y}, o[i][j][0]);
                        o[i][j][1] = fma2(Pair{w, w}, Pair{vv.z, vv.w}, o[i][j][1]);
                    }
                }
            }
        }
    }
    const int64_t slot = (int64_t)rg * a.n_chunks + c;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int row = i0 + ty + 16 * i;
        if (row >= nq) continue;
        const int64_t pr = slot * a.NR + row;
#pragma unroll
        for (int j = 0; j < DJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = 4 * tx + 32 * j + e;
                if (d < a.D) a.ws_o[pr * a.D + d] = e & 1 ? o[i][j][e >> 1].y : o[i][j][e >> 1].x;
            }
        if (tx == 0) {
            a.ws_ml[pr * 2] = m[i];
            a.ws_ml[pr * 2 + 1] = l[i];
        }
    }
}

// ---------------------------------------------------------------------------
// Merge of a stream's partials: out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M)
// l_c, 0 where nothing was seen.  A warp has one row: lane k keeps the weight of
// slot k, and the first eight slots' partials are loaded beside the (m, l)
// pairs, so a stream of few slots costs one round of loads.  The CUDA-core
// kernel's streams are all split by the host's plan; of the tensor-core
// kernel's, its table names the split one of each column, and those that one
// CTA finished are written already.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 8;

// MR rows of a warp at a time, MS of their slots in flight (tensor-core kernel's streams; MR 0: the others).
template <typename T, int MR, int MS>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const TreeArgs a) {
    constexpr bool kTc = MR > 0;
    constexpr int kUnroll = 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int HP = a.H_kv * a.groups;
    int r, hp, nch;
    int64_t slot0;
    if (kTc) {
        hp = (int)blockIdx.x % HP;
        const int4 e = a.ws_split[blockIdx.x / HP];   // request, its slots, the first
        r = e.x;
        nch = e.y;
        slot0 = (int64_t)hp * (a.P + a.num_reqs) + e.z;
        if (nch == 0) return;
    } else {
        r = (int)(blockIdx.x / HP);
        hp = (int)blockIdx.x - r * HP;
        const int32_t L = tree_len(a, __ldg(a.ctx + r));
        nch = L > 0 ? (L + a.chunk - 1) / a.chunk : 0;
        slot0 = (int64_t)blockIdx.x * a.n_chunks;
    }
    const int g = hp / a.groups, tok0 = (hp - g * a.groups) * a.TS;
    const int rows = min(a.NR, (a.T - tok0) * a.G);
    if constexpr (MR > 0) {
        // head_dim 128: four elements a lane
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
                            v[i][k] = rr + i < rows && c + k < nch
                                          ? *reinterpret_cast<const float4 *>(
                                                a.ws_o + ((slot0 + c + k) * a.NR + rr + i) * 128 + 4 * lane)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                };
#pragma unroll
                for (int i = 0; i < MR; ++i)
                    ml[i] = rr + i < rows && base + lane < nch
                                ? *reinterpret_cast<const float2 *>(a.ws_ml + ((slot0 + base + lane) * a.NR + rr + i) * 2)
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
                         (((int64_t)r * a.T + tok0 + row / a.G) * a.H_q + g * a.G + row % a.G) * 128 + 4 * lane;
                T o4[4];
                store_out(o4, acc[i].x * inv);
                store_out(o4 + 1, acc[i].y * inv);
                store_out(o4 + 2, acc[i].z * inv);
                store_out(o4 + 3, acc[i].w * inv);
                if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2 *>(out) = *reinterpret_cast<const uint2 *>(o4);
                else *reinterpret_cast<uint4 *>(out) = *reinterpret_cast<const uint4 *>(o4);
            }
        }
        return;
    }
    const int row = blockIdx.y * kMergeWarps + warp;
    if (row >= rows) return;
    const int t = tok0 + row / a.G, h = g * a.G + row % a.G;
    T *out = static_cast<T *>(a.out) + (((int64_t)r * a.T + t) * a.H_q + h) * a.D;
    auto ml_of = [&](int c) {
        return c < nch ? *reinterpret_cast<const float2 *>(a.ws_ml + ((slot0 + c) * a.NR + row) * 2)
                       : make_float2(-INFINITY, 0.f);
    };
    const float2 ml0 = ml_of(lane);
    for (int d0 = 0; d0 < a.D; d0 += 64) {   // two elements a lane
        const int d = d0 + 2 * lane;
        const bool act = d < a.D;
        auto part = [&](int c) {
            return act && c < nch ? *reinterpret_cast<const float2 *>(a.ws_o + ((slot0 + c) * a.NR + row) * a.D + d)
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
    int32_t chunk, n_chunks;
    int64_t slots_cc, slots_tc;   // the kernels' partial slots (tensor-core: 0 where it cannot run)
    int64_t split_bytes;          // the tensor-core kernel's table of split streams
    size_t ws_bytes;
};

static int64_t gcd64(int64_t x, int64_t y) {
    while (y) {
        const int64_t t = x % y;
        x = y;
        y = t;
    }
    return x;
}

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

static bool make_plan(int32_t num_reqs, int32_t T, int32_t H_q, int32_t H_kv, int32_t D, int32_t bs, int32_t max_ctx,
                      Plan *p) {
    if (num_reqs <= 0 || T <= 0 || T > kMaxT || H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0 || D <= 0 || D > 256 ||
        D % 2 != 0 || bs <= 0 || bs > 65536 || max_ctx < 0)
        return false;
    const int32_t G = H_q / H_kv;
    const int64_t nq = (int64_t)T * G;
    const int64_t units = (int64_t)num_reqs * H_kv;
    const int64_t sms = current_sm_count();
    // splits hold whole blocks, of 64 positions at least; about eight CTAs an SM where the batch alone has fewer
    const int64_t align = (int64_t)bs / gcd64(bs, 64) * 64;
    const int64_t row_tiles = ceil_div<int64_t>(nq, 64);
    int64_t chunk = ceil_div<int64_t>((int64_t)max_ctx * units * row_tiles, 8 * sms);
    chunk = ceil_div<int64_t>(chunk < 1 ? 1 : chunk, align) * align;
    if (chunk > (int64_t)1 << 30) return false;
    p->chunk = (int32_t)chunk;
    p->n_chunks = max_ctx > 0 ? (int32_t)ceil_div<int64_t>(max_ctx, chunk) : 1;
    p->slots_cc = units * p->n_chunks;
    if (p->slots_cc >= ((int64_t)1 << 31) || ceil_div<int64_t>(nq, kMergeWarps) > 65535) return false;   // grids
    int64_t rows = p->slots_cc * nq;
    p->slots_tc = 0;
    if (D == 128 && G <= 128) {
        int32_t TS, groups, P;
        tc_split(T, G, H_kv, &TS, &groups, &P);
        p->slots_tc = (int64_t)H_kv * groups * (P + (int64_t)num_reqs);
        const int64_t rt = p->slots_tc * TS * G;
        if (rt > rows) rows = rt;
    }
    p->split_bytes = p->slots_tc > 0 ? ceil_div<int64_t>(sms * 16, 256) * 256 : 0;   // at most a column an SM
    p->ws_bytes = (size_t)(p->split_bytes + ceil_div<int64_t>(rows * D * 4, 256) * 256 +
                           ceil_div<int64_t>(rows * 8, 256) * 256);
    return true;
}

template <typename T, int DP, int BR>
static cudaError_t launch_cc(const TreeArgs &a, cudaStream_t st) {
    constexpr int smem = ((BR + 2 * kBK) * (DP + 4) + BR * (kBK + 4)) * 4;
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
    const dim3 grid((unsigned)(a.num_reqs * a.H_kv * a.n_chunks), (unsigned)ceil_div(a.T * a.G, BR));
    // rows of whole 16-byte pieces
    const bool vec = a.D * sizeof(T) % 16 == 0 && aligned(a.q, 16) && aligned(a.k, 16) && aligned(a.v, 16);
    return launch_pdl(kern, grid, dim3(kThreads), smem, st, a, vec);
}

// The query tile (16, 32, 48 or 64 rows; up to 32 with head_dim above 128, for
// its registers) that leaves the fewest rows idle, the larger of two.
static int query_tile(int32_t nq, int32_t D) {
    int best = 16;
    for (int br = 32; br <= (D > 128 ? 32 : 64); br += 16)
        if (ceil_div(nq, br) * br <= ceil_div(nq, best) * best) best = br;
    return best;
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

template <int MR, int MS>
static int launch_merge(const TreeArgs &a, cudaStream_t st) {
    const int64_t x = (int64_t)(MR ? a.P : a.num_reqs) * a.H_kv * a.groups;
    const dim3 grid((unsigned)x, (unsigned)ceil_div(a.NR, kMergeWarps * (MR ? MR : 1))), block(kMergeWarps * 32);
    cudaError_t e;
    if (MR || a.dtype == BKV_BF16) e = launch_pdl(tree_merge_kernel<__nv_bfloat16, MR, MS>, grid, block, 0, st, a);
    else e = launch_pdl(tree_merge_kernel<float, 0, 0>, grid, block, 0, st, a);
    if (e != cudaSuccess) set_cuda_error(e);
    return launch_status();
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
    a.chunk = plan.chunk;
    a.n_chunks = plan.n_chunks;
    auto set_slots = [&](int64_t slots) {
        char *base = static_cast<char *>(workspace) + plan.split_bytes;
        a.ws_split = static_cast<int4 *>(workspace);
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
            // few rows: one a warp, all its loads at once (28 rows of 8 streams 11.8 us a call, 13.1 by two
            // rows); many: two a warp (244 rows of 128 streams 113 us a call, 117 by one)
            return a.NR <= 32 ? launch_merge<1, 8>(a, st) : launch_merge<2, 4>(a, st);
        }
    }
    // one query-row group for all tokens: the CUDA-core kernel's slots
    a.TS = q_len;
    a.NR = q_len * a.G;
    a.groups = 1;
    set_slots(plan.slots_cc);
    const cudaError_t e = dtype == BKV_BF16 ? launch_cc_dims<__nv_bfloat16>(a, st) : launch_cc_dims<float>(a, st);
    if (e != cudaSuccess) set_cuda_error(e);
    const int rc = launch_status();
    return rc != BKV_OK ? rc : launch_merge<0, 0>(a, st);
}
