// bkv_rope_write.cu -- norm of every query and key head, position rotation,
// slot mapping and cache write of a step's tokens, in one pass.
//
// For a head row x of D elements (queries and keys; fp32 arithmetic on the
// input's values, one rounding at the end):
//   y = x * rsqrt(mean(x^2) + eps) * w            (no weight given: y = x)
//   (y_a, y_b) -> (y_a c_i - y_b s_i, y_b c_i + y_a s_i),  i < rot / 2,
// with c_i = cos_sin[p][i], s_i = cos_sin[p][rot / 2 + i] of the token's
// rotation position p, (a, b) = (i, i + rot / 2), or (2i, 2i + 1) when
// interleaved.  Queries go to q_out, keys to their cache rows (rounded to the
// cache's type, or the E4M3 code of the binary32 quotient by k_scale), values
// are copied (or quantised) as bkv_cache_write(_fp8) does.  Slots are
// bkv_compute_slot_mapping's ("Padding and Batching with Block KV", The Core
// Formula; Slot ID -1: Padding Tokens; Block Structure); the norm and the
// rotation have no counterpart on the pages.
//
// Memory-bound: (Hq + 2 Hkv) D e bytes read and Hq D e + 2 Hkv D e_cache
// written a token, once each; for a few tokens the chain request / position
// -> table entry -> store and the launch are what counts, so the rows are
// loaded before the table's answer is needed.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "bkv_internal.cuh"
#include "bkv_slot.cuh"

namespace bkv {
namespace rope {

struct Args {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements between tokens
    const void *qw, *kw;                    // norm weights [D] or null
    float eps;
    const float *cos_sin;
    int64_t max_position;
    int32_t rot;
    const int32_t *bt;
    int32_t num_reqs;
    int64_t bt_stride;
    int32_t bt_cols;
    const int32_t *req;
    const int64_t *pos, *rpos;
    int64_t n, max_n;
    int64_t *slots;
    void *q_out, *kc, *vc;
    int64_t capacity;
    int32_t bs, hq, hkv, d;
    float k_scale, v_scale;
    int32_t *err;
};

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x, float) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(float *p, float x, float) { *p = x; }
__device__ __forceinline__ void put(uint8_t *p, float x, float scale) {
    *p = (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(x, scale), __NV_SATFINITE, __NV_E4M3);
}
// a value copied into a cache of its own type keeps its bits
__device__ __forceinline__ void copy(__nv_bfloat16 *p, __nv_bfloat16 x, float) { *p = x; }
__device__ __forceinline__ void copy(float *p, float x, float) { *p = x; }
template <typename T>
__device__ __forceinline__ void copy(uint8_t *p, T x, float scale) { put(p, to_f(x), scale); }

// What a token's row needs to know: whether it is a real token, its slot (-1:
// nothing is cached) and its rotation row.
struct Token {
    bool real;
    int64_t slot;
    const float *cs;
};

// A token's request and positions: what its slot and rotation row follow from.
struct Meta {
    int32_t r = -1;   // < 0: padding
    int64_t p = 0, rp = 0;
};
__device__ __forceinline__ Meta meta_at(const Args &a, int64_t i) {
    Meta m;
    if (i < a.n) {
        m.r = __ldg(a.req + i);
        m.p = __ldg(a.pos + i);
        m.rp = a.rpos ? __ldg(a.rpos + i) : m.p;
    }
    return m;
}

// Token i < max_n.  `lead`: this thread writes the slot and counts errors.
__device__ __forceinline__ Token token_of(const Args &a, int64_t i, const Meta &m, bool lead) {
    Token t{false, -1, nullptr};
    if (m.r >= 0) {
        bool bad = m.rp < 0 || m.rp >= a.max_position;
        if (!bad) {
            t.real = true;
            t.cs = a.cos_sin + m.rp * a.rot;
            t.slot = slot_of(a.bt, a.num_reqs, a.bt_stride, a.bt_cols, m.r, m.p, a.bs, 1, 0, 1, &bad);
        }
        if (lead && a.err && (bad || t.slot >= a.capacity)) atomicAdd(a.err, 1);
    }
    if (lead) a.slots[i] = t.slot;
    if (t.slot >= a.capacity) t.slot = -1;
    return t;
}

// Any head_dim up to 256, any strides and alignments: one warp per (token,
// head), lane l elements l, l + 32, ...; a rotated element reads its partner
// again rather than exchanging it.
template <typename T, typename C>
__global__ void __launch_bounds__(128) rope_write_any_kernel(const Args a, bool inter) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int heads = a.hq + 2 * a.hkv;
    const int64_t items = a.max_n * heads;
    const int64_t step = (int64_t)gridDim.x * 4;
    for (int64_t it = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); it < items; it += step) {
        const int64_t i = it / heads;
        const int h = (int)(it - i * heads);
        const Token t = token_of(a, i, meta_at(a, i), h == 0 && lane == 0);
        if (!t.real) continue;
        const int kind = h < a.hq ? 0 : (h < a.hq + a.hkv ? 1 : 2);
        if (kind > 0 && t.slot < 0) continue;
        if (kind == 2) {
            const int g = h - a.hq - a.hkv;
            const T *src = static_cast<const T *>(a.v) + i * a.v_stride + (int64_t)g * a.d;
            C *dst = static_cast<C *>(a.vc) + (t.slot * a.hkv + g) * a.d;
            for (int e = lane; e < a.d; e += 32) copy(dst + e, src[e], a.v_scale);
            continue;
        }
        const int g = kind == 0 ? h : h - a.hq;
        const T *src = kind == 0 ? static_cast<const T *>(a.q) + i * a.q_stride + (int64_t)g * a.d
                                 : static_cast<const T *>(a.k) + i * a.k_stride + (int64_t)g * a.d;
        const T *w = static_cast<const T *>(kind == 0 ? a.qw : a.kw);
        const int half = a.rot / 2;
        float x[8], y[8];   // own element and the one it rotates with
        float ss = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int e = lane + 32 * u;
            x[u] = y[u] = 0.f;
            if (e < a.d) {
                x[u] = to_f(src[e]);
                if (e < a.rot) y[u] = to_f(src[inter ? (e ^ 1) : (e < half ? e + half : e - half)]);
                ss = fmaf(x[u], x[u], ss);
            }
        }
        __syncwarp();   // q_out may be q: no lane stores before the others have read what turns with their elements
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = w ? rsqrtf(ss / (float)a.d + a.eps) : 1.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int e = lane + 32 * u;
            if (e >= a.d) break;
            float r = x[u] * inv * (w ? to_f(w[e]) : 1.f);
            if (e < a.rot) {
                const int pe = inter ? (e ^ 1) : (e < half ? e + half : e - half);
                const int ci = inter ? e >> 1 : (e < half ? e : e - half);
                const float m = y[u] * inv * (w ? to_f(w[pe]) : 1.f);
                const float c = __ldg(t.cs + ci), s = __ldg(t.cs + half + ci);
                const bool first = inter ? !(e & 1) : e < half;
                r = first ? r * c - m * s : r * c + m * s;
            }
            if (kind == 0)
                put(static_cast<T *>(a.q_out) + (i * a.hq + g) * a.d + e, r, 1.f);
            else
                put(static_cast<C *>(a.kc) + (t.slot * a.hkv + g) * a.d + e, r, a.k_scale);
        }
    }
}

// ---------------------------------------------------------------------------
// The common shapes: head_dim 32, 64, 128 or 256, a rotated part of whole
// 16-element pieces, 16-byte alignment everywhere.  LPH = head_dim / 16 lanes a
// head; a lane holds two pieces of 8 elements that rotate with one another:
// [8 l, ..) and [rot / 2 + 8 l, ..), or, interleaved and past the rotated part,
// 16 consecutive ones, so a pair never leaves its lane and both layouts use
// table entries 8 l .. 8 l + 7.  A CTA takes a token at a time, a head by LPH
// lanes a round, U rounds' loads in flight before the token's own answers (table
// entry, rotation row) are needed.
// ---------------------------------------------------------------------------
// CTAs of 128 threads an SM is built to hold: fewer leave too few loads in flight, more spill rows (8752 tokens of 32 +
// 2 x 8 heads of 128, bf16: 47.4, 45.6, 49.4 and 56.4 us with 4, 5, 6 and 8; 4.8 TB/s of the bytes that it has to move).
constexpr int kPerSm = 5;

template <typename T>
struct Piece {   // 8 elements as they are in memory
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = *(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(u[i] << 16);
                f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[4 * i] = __uint_as_float(w[i].x);
                f[4 * i + 1] = __uint_as_float(w[i].y);
                f[4 * i + 2] = __uint_as_float(w[i].z);
                f[4 * i + 3] = __uint_as_float(w[i].w);
            }
        }
    }
};

__device__ __forceinline__ void put8(__nv_bfloat16 *p, const float (&f)[8], float) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void put8(float *p, const float (&f)[8], float) {
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void put8(uint8_t *p, const float (&f)[8], float scale) {
    uint32_t u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            h[j] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f[4 * i + 2 * j], scale),
                                                        __fdiv_rn(f[4 * i + 2 * j + 1], scale)),
                                            __NV_SATFINITE, __NV_E4M3);
        u[i] = h[0] | (h[1] << 16);
    }
    *reinterpret_cast<uint2 *>(p) = make_uint2(u[0], u[1]);
}

// B: threads of the CTA, 0: any up to 160 (the registers of as many warps an SM).
template <typename T, typename C, int LPH, int U, int B>
__global__ void __launch_bounds__(B ? B : 160, B ? kPerSm : 4) rope_write_kernel(const Args a, bool inter) {
    constexpr int D = 16 * LPH;
    const int NG = (B ? B : blockDim.x) / LPH, l = threadIdx.x % LPH, grp = threadIdx.x / LPH;
    const int heads = a.hq + 2 * a.hkv, half = a.rot / 2;
    const bool turns = 16 * l < a.rot;
    const int ea = inter || !turns ? 16 * l : 8 * l;        // this lane's two pieces
    const int eb = inter || !turns ? ea + 8 : half + 8 * l;
    pdl_wait();
    pdl_trigger();
    Meta next = meta_at(a, blockIdx.x);   // a token ahead: its row loads wait for nothing
    for (int64_t i = blockIdx.x; i < a.max_n; i += gridDim.x) {
        const Meta meta = next;
        const bool lead = blockIdx.y == 0 && threadIdx.x == 0;
        if (i >= a.n) {
            if (lead) a.slots[i] = -1;
            continue;
        }
        bool known = false;
        Token t{};
        float cs[8], sn[8];
        for (int h0 = blockIdx.y * NG * U; h0 < heads; h0 += gridDim.y * NG * U) {
            Piece<T> pa[U], pb[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * NG + grp;
                if (h < heads) {
                    const T *src = h < a.hq ? static_cast<const T *>(a.q) + i * a.q_stride + (int64_t)h * D
                                   : h < a.hq + a.hkv
                                       ? static_cast<const T *>(a.k) + i * a.k_stride + (int64_t)(h - a.hq) * D
                                       : static_cast<const T *>(a.v) + i * a.v_stride + (int64_t)(h - a.hq - a.hkv) * D;
                    pa[u].load(src + ea);
                    pb[u].load(src + eb);
                }
            }
            if (!known) {
                known = true;
                next = meta_at(a, i + gridDim.x);
                t = token_of(a, i, meta, lead);
                if (t.real && turns) {
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 c4 = __ldg(reinterpret_cast<const float4 *>(t.cs + 8 * l + e));
                        const float4 s4 = __ldg(reinterpret_cast<const float4 *>(t.cs + half + 8 * l + e));
                        cs[e] = c4.x, cs[e + 1] = c4.y, cs[e + 2] = c4.z, cs[e + 3] = c4.w;
                        sn[e] = s4.x, sn[e + 1] = s4.y, sn[e + 2] = s4.z, sn[e + 3] = s4.w;
                    }
                }
            }
            if (!t.real) break;   // the same for the whole CTA
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * NG + grp;
                float x[8], y[8];
                float ss = 0.f;
                if (h < heads) {
                    pa[u].get(x);
                    pb[u].get(y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
                }
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (h >= heads) continue;
                const int kind = h < a.hq ? 0 : (h < a.hq + a.hkv ? 1 : 2);
                if (kind > 0 && t.slot < 0) continue;
                if (kind == 2) {
                    C *dst = static_cast<C *>(a.vc) + (t.slot * a.hkv + (h - a.hq - a.hkv)) * D;
                    if constexpr (sizeof(C) == 1) {
                        put8(dst + ea, x, a.v_scale);
                        put8(dst + eb, y, a.v_scale);
                    } else {
#pragma unroll
                        for (int w = 0; w < (int)sizeof(T) / 2; ++w) {
                            reinterpret_cast<uint4 *>(dst + ea)[w] = pa[u].w[w];
                            reinterpret_cast<uint4 *>(dst + eb)[w] = pb[u].w[w];
                        }
                    }
                    continue;
                }
                const T *w = static_cast<const T *>(kind == 0 ? a.qw : a.kw);
                if (w) {
                    const float inv = rsqrtf(ss / (float)D + a.eps);
                    Piece<T> wa, wb;
                    wa.load(w + ea);
                    wb.load(w + eb);
                    float fa[8], fb[8];
                    wa.get(fa);
                    wb.get(fb);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {   // (two fp32 roundings, as (x inv) w has)
                        x[e] *= inv * fa[e];
                        y[e] *= inv * fb[e];
                    }
                }
                if (turns) {
                    if (inter) {   // pairs (2 i, 2 i + 1): four in each piece
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float xa = x[2 * e], xb = x[2 * e + 1], ya = y[2 * e], yb = y[2 * e + 1];
                            x[2 * e] = xa * cs[e] - xb * sn[e];
                            x[2 * e + 1] = xb * cs[e] + xa * sn[e];
                            y[2 * e] = ya * cs[4 + e] - yb * sn[4 + e];
                            y[2 * e + 1] = yb * cs[4 + e] + ya * sn[4 + e];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float xa = x[e], xb = y[e];
                            x[e] = xa * cs[e] - xb * sn[e];
                            y[e] = xb * cs[e] + xa * sn[e];
                        }
                    }
                }
                if (kind == 0) {
                    T *dst = static_cast<T *>(a.q_out) + (i * a.hq + h) * D;
                    put8(dst + ea, x, 1.f);
                    put8(dst + eb, y, 1.f);
                } else {
                    C *dst = static_cast<C *>(a.kc) + (t.slot * a.hkv + (h - a.hq)) * D;
                    put8(dst + ea, x, a.k_scale);
                    put8(dst + eb, y, a.k_scale);
                }
            }
        }
    }
}

template <typename T, typename C, int LPH>
static cudaError_t launch_pieces(const Args &a, bool inter, cudaStream_t st) {
    // three rounds of 16-bit rows in flight (48 heads of 128 elements), two of 32-bit ones: registers
    constexpr int U = sizeof(T) == 2 ? 3 : 2;
    const int heads = a.hq + 2 * a.hkv, rounds = ceil_div(heads, 128 / LPH);
    const int64_t sms = current_sm_count();
    // fewer tokens than CTAs fit: a token's heads over several (1016 tokens, E4M3: 11.2 -> 10.5 us)
    const int64_t room = 16 * sms / (a.max_n < 1 ? 1 : a.max_n);
    if (room >= 2 && rounds > 1) {
        const unsigned y = (unsigned)(room < rounds ? room : rounds);
        return launch_pdl(rope_write_kernel<T, C, LPH, 1, 128>, dim3((unsigned)a.max_n, y), dim3(128), 0, st, a, inter);
    }
    // a CTA as wide as a token's heads, so that no round is left half empty (E4M3 caches, 128 threads against what this
    // gives: 15 + 2 x 5 heads of 256, bf16, 54.0 and 47.0 us; 4 + 2 x 1, fp32, 58.2 and 42.5)
    const int lanes = ceil_div(heads * LPH, U), steps = ceil_div(lanes, 160);
    const int threads = ceil_div(ceil_div(lanes, steps), 32) * 32;
    const int64_t ctas = sms * 2 * (kPerSm * 128 / threads);
    const dim3 grid((unsigned)(a.max_n < ctas ? a.max_n : ctas)), block(threads);
    if (threads == 128) return launch_pdl(rope_write_kernel<T, C, LPH, U, 128>, grid, block, 0, st, a, inter);
    return launch_pdl(rope_write_kernel<T, C, LPH, U, 0>, grid, block, 0, st, a, inter);
}

static bool in_pieces(const Args &a, int e, int ec) {
    return (a.d == 32 || a.d == 64 || a.d == 128 || a.d == 256) && a.rot % 16 == 0 && aligned(a.q, 16) &&
           aligned(a.k, 16) && aligned(a.v, 16) && aligned(a.q_out, 16) && aligned(a.kc, ec == 1 ? 8 : 16) &&
           aligned(a.vc, ec == 1 ? 8 : 16) && aligned(a.qw, 16) && aligned(a.kw, 16) && aligned(a.cos_sin, 16) &&
           a.q_stride * e % 16 == 0 && a.k_stride * e % 16 == 0 && a.v_stride * e % 16 == 0;
}

template <typename T, typename C>
static cudaError_t launch_rope(const Args &a, bool inter, cudaStream_t st) {
    if (in_pieces(a, sizeof(T), sizeof(C))) {
        if (a.d == 32) return launch_pieces<T, C, 2>(a, inter, st);
        if (a.d == 64) return launch_pieces<T, C, 4>(a, inter, st);
        if (a.d == 128) return launch_pieces<T, C, 8>(a, inter, st);
        return launch_pieces<T, C, 16>(a, inter, st);
    }
    const int64_t items = a.max_n * (a.hq + 2 * a.hkv);
    return launch_pdl(rope_write_any_kernel<T, C>, dim3(grid_for(items, 4, 64)), dim3(128), 0, st, a, inter);
}

static int run(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
               const void *q_weight, const void *k_weight, float norm_eps, const float *cos_sin, int64_t max_position,
               int32_t rot_dim, int interleaved, const int32_t *block_table, int32_t num_reqs, int64_t bt_stride,
               int32_t bt_cols, const int32_t *req_indices, const int64_t *positions, const int64_t *rope_positions,
               int64_t num_tokens, int64_t max_num_tokens, int64_t *slot_mapping, void *q_out, void *k_cache,
               void *v_cache, int64_t total_blocks, int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
               int32_t head_dim, int dtype, bool fp8, float k_scale, float v_scale, int32_t *err_count,
               bkv_stream_t stream) {
    if (dtype != BKV_BF16 && dtype != BKV_F32) return BKV_ERR_UNSUPPORTED;
    if (num_tokens < 0 || max_num_tokens < num_tokens || total_blocks < 0 || block_size <= 0 || num_q_heads <= 0 ||
        num_kv_heads <= 0 || head_dim <= 0 || num_reqs < 0 || bt_cols < 0 || bt_stride < bt_cols || max_position < 0)
        return BKV_ERR_INVALID_ARG;
    if (head_dim > 256 || head_dim % 2 != 0) return BKV_ERR_UNSUPPORTED;
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 != 0 || !(norm_eps >= 0.f) || !isfinite(norm_eps))
        return BKV_ERR_INVALID_ARG;
    if (fp8 && (!(k_scale > 0.f) || !(v_scale > 0.f) || !isfinite(k_scale) || !isfinite(v_scale)))
        return BKV_ERR_INVALID_ARG;
    if (q_stride < (int64_t)num_q_heads * head_dim || k_stride < (int64_t)num_kv_heads * head_dim ||
        v_stride < (int64_t)num_kv_heads * head_dim)
        return BKV_ERR_INVALID_ARG;
    if (max_num_tokens == 0) return BKV_OK;
    if (!slot_mapping) return BKV_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!q || !k || !v || !q_out || !req_indices || !positions || (bt_cols > 0 && !block_table) ||
                           (rot_dim > 0 && !cos_sin) || (total_blocks > 0 && (!k_cache || !v_cache))))
        return BKV_ERR_INVALID_ARG;
    Args a{q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, norm_eps, cos_sin, max_position, rot_dim,
           block_table, num_reqs, bt_stride, bt_cols, req_indices, positions, rope_positions, num_tokens,
           max_num_tokens, slot_mapping, q_out, k_cache, v_cache, total_blocks * (int64_t)block_size, block_size,
           num_q_heads, num_kv_heads, head_dim, k_scale, v_scale, err_count};
    cudaStream_t st = (cudaStream_t)stream;
    const bool inter = interleaved != 0;
    cudaError_t e;
    if (dtype == BKV_BF16)
        e = fp8 ? launch_rope<__nv_bfloat16, uint8_t>(a, inter, st) : launch_rope<__nv_bfloat16, __nv_bfloat16>(a, inter, st);
    else
        e = fp8 ? launch_rope<float, uint8_t>(a, inter, st) : launch_rope<float, float>(a, inter, st);
    if (e != cudaSuccess) set_cuda_error(e);
    return launch_status();
}

}  // namespace rope
}  // namespace bkv

#define BKV_ROPE_PARAMS                                                                                            \
    const void *q, const void *k, const void *v, int64_t q_token_stride, int64_t k_token_stride,                   \
        int64_t v_token_stride, const void *q_weight, const void *k_weight, float norm_eps, const float *cos_sin,  \
        int64_t max_position, int32_t rot_dim, int interleaved, const int32_t *block_table, int32_t num_reqs,      \
        int64_t bt_stride, int32_t bt_cols, const int32_t *req_indices, const int64_t *positions,                  \
        const int64_t *rope_positions, int64_t num_tokens, int64_t max_num_tokens, int64_t *slot_mapping,          \
        void *q_out
#define BKV_ROPE_ARGS                                                                                              \
    q, k, v, q_token_stride, k_token_stride, v_token_stride, q_weight, k_weight, norm_eps, cos_sin, max_position,  \
        rot_dim, interleaved, block_table, num_reqs, bt_stride, bt_cols, req_indices, positions, rope_positions,   \
        num_tokens, max_num_tokens, slot_mapping, q_out

extern "C" int bkv_qk_norm_rope_cache_write(BKV_ROPE_PARAMS, void *k_cache, void *v_cache, int64_t total_blocks,
                                            int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                                            int32_t head_dim, int dtype, int32_t *err_count, bkv_stream_t stream) {
    return bkv::rope::run(BKV_ROPE_ARGS, k_cache, v_cache, total_blocks, block_size, num_q_heads, num_kv_heads,
                          head_dim, dtype, false, 1.f, 1.f, err_count, stream);
}

extern "C" int bkv_qk_norm_rope_cache_write_fp8(BKV_ROPE_PARAMS, uint8_t *k_cache, uint8_t *v_cache,
                                                int64_t total_blocks, int32_t block_size, int32_t num_q_heads,
                                                int32_t num_kv_heads, int32_t head_dim, int dtype, float k_scale,
                                                float v_scale, int32_t *err_count, bkv_stream_t stream) {
    return bkv::rope::run(BKV_ROPE_ARGS, k_cache, v_cache, total_blocks, block_size, num_q_heads, num_kv_heads,
                          head_dim, dtype, true, k_scale, v_scale, err_count, stream);
}
