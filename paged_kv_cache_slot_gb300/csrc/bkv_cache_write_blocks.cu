// bkv_cache_write_blocks.cu -- writes a step's K and V rows into E4M3 caches
// with one scale for each block of tokens and KV head.
//
// A request's new tokens are its last cached positions ("Padding and Batching
// with Block KV", Batching with Block KV), so those that fall into one block
// are consecutive rows of it.  For a touched block b, KV head h, and K or V,
// with x the new rows of that head:
//   s' = 2^e, the smallest with max |x| <= 448 2^e (finite elements), e in [-40, 40];
//   s  = s' where the block's first row is among the new ones (what it held is void),
//        max(s', scale[b][h]) otherwise;
//   old rows where s grew: code = E4M3(value(code) scale[b][h] / s);
//   new rows: code = E4M3(x / s), nearest, ties to even, saturated at 448.
// A power of two costs E4M3 nothing (its precision is its mantissa's, whatever
// the scale), makes both quotients exact, and an old code only loses bits that
// leave the subnormal end.
//
// The work of one (touched block, KV head) is a group's: K and V rows are read
// once into registers, their maxima reduced, and the codes written.  The blocks
// a step touches are numbered floor(start_r / bs) + 2 r + j, j the request's
// own count: the numbers of different requests never meet (a request of n
// tokens touches at most n / bs + 2 blocks), gaps are skipped, and no scan over
// the requests has to come first.
//
// Memory-bound for prompts (e + 1 bytes an element); a decode step is the
// chain request -> table entry -> scale, with the row's loads beside it.
#include <math.h>

#include "bkv_eight.cuh"
#include "bkv_internal.cuh"

namespace bkv {
namespace wblk {

constexpr float kMaxFloat = 3.402823466e38f;

struct Args {
    const void *k, *v;
    int64_t stride;            // elements between tokens
    int64_t num_tokens;
    const int32_t *qsl, *ctx;
    int32_t num_reqs;
    const int32_t *bt;
    int64_t bt_stride;
    int32_t bt_cols;
    uint8_t *kc, *vc;
    float *ks, *vs;            // [total_blocks][hkv]
    int64_t total_blocks;
    int32_t bs, hkv, d, pieces;   // pieces of 8 elements a row
    int32_t *err;
    bool vec;
};

// Where the token rows of request r begin in the step, within [0, num_tokens].
__device__ __forceinline__ int64_t start_of(const Args &a, int r) {
    const int64_t t = __ldg(a.qsl + r);
    return t < 0 ? 0 : (t > a.num_tokens ? a.num_tokens : t);
}

// A touched block's rows: `cnt` tokens from `tok` on go to rows `first` on of
// block `id`; cnt 0: nothing.
struct Part {
    int64_t id, tok;
    int32_t first, cnt;
};

// Block number u of the step, by one warp.  count: this warp counts errors.
__device__ __forceinline__ Part part_of(const Args &a, int64_t u, bool count) {
    const int lane = threadIdx.x & 31;
    Part p{0, 0, 0, 0};
    // the last request whose numbers begin at or before u: 32 probes a round
    int lo = 0, n = a.num_reqs;
    while (n > 1) {
        const int step = (int)(((int64_t)n + 31) / 32);
        const bool in = (int64_t)lane * step < n && start_of(a, lo + lane * step) / a.bs + 2 * (int64_t)(lo + lane * step) <= u;
        const uint32_t m = __ballot_sync(0xffffffffu, in);
        const int last = m ? 31 - __clz(m) : 0;
        lo += last * step;
        n = min(step, n - last * step);
    }
    const int64_t t0 = start_of(a, lo), t1 = start_of(a, lo + 1);
    const int64_t L = __ldg(a.ctx + lo);
    const int64_t j = u - (t0 / a.bs + 2 * (int64_t)lo), start = L - (t1 - t0);
    if (t1 <= t0 || j < 0) return p;
    if (start < 0) {   // more new tokens than the request's length
        if (count && j == 0 && lane == 0 && a.err) atomicAdd(a.err, 1);
        return p;
    }
    const int64_t lb = start / a.bs + j;
    const int64_t p0 = max(start, lb * a.bs), p1 = min(L, (lb + 1) * a.bs);
    if (p0 >= p1) return p;
    const int64_t id = lb < a.bt_cols ? __ldg(a.bt + (int64_t)lo * a.bt_stride + lb) : a.total_blocks;
    if (id >= a.total_blocks) {
        if (count && lane == 0 && a.err) atomicAdd(a.err, 1);
        return p;
    }
    if (id <= 0) return p;
    p.id = id;
    p.tok = t0 + (p0 - start);
    p.first = (int32_t)(p0 - lb * a.bs);
    p.cnt = (int32_t)(p1 - p0);
    return p;
}

// The exponent of the smallest power of two s with top <= 448 s, held to [-40, 40].
__device__ __forceinline__ int exponent_of(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 127 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0) - 8;   // 448 = 1.75 x 2^8
    return min(max(e, -40), 40);
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ float finite_abs(float x) {
    const float y = fabsf(x);
    return y <= kMaxFloat ? y : 0.f;
}

template <typename T>
__device__ __forceinline__ float top_of(const Eight<T> &x) {
    float t = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float2 f = x.two(c);
        t = fmaxf(t, fmaxf(finite_abs(f.x), finite_abs(f.y)));
    }
    return t;
}

template <typename T>
__device__ __forceinline__ uint2 codes_of(const Eight<T> &x, float by) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = x.two(i);
        const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(f.x * by, f.y * by), __NV_SATFINITE, __NV_E4M3);
        w[i / 2] |= c << (16 * (i % 2));
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void put_codes(uint8_t *dst, uint2 w, int n, bool vec) {
    if (vec) {
        *reinterpret_cast<uint2 *>(dst) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= n) break;
        dst[i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i % 4)));
    }
}

// Groups of W warps, as many as fit into 128 threads a CTA; PT pieces of K and
// of V a thread in registers.  Rows that do not fit are read again for their codes.
template <int W>
constexpr int kThreadsOf = W < 4 ? 128 : 32 * W;

template <typename T, int W, int PT>
__global__ void __launch_bounds__(kThreadsOf<W>) write_blocks_kernel(const Args a, int64_t items) {
    constexpr int kGroups = kThreadsOf<W> / (32 * W);
    constexpr int kLanes = 32 * W;
    __shared__ float red[2][kGroups][W][2];
    const int group = threadIdx.x / kLanes, gl = threadIdx.x % kLanes, gw = gl >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    int turn = 0;
    for (int64_t it = (int64_t)blockIdx.x * kGroups + group; it < items; it += (int64_t)gridDim.x * kGroups) {
        const int64_t u = it / a.hkv;
        const int h = (int)(it - u * a.hkv);
        const Part p = part_of(a, u, h == 0 && gw == 0);
        if (p.cnt == 0) continue;
        const int np = p.cnt * a.pieces;
        const T *src[2] = {static_cast<const T *>(a.k), static_cast<const T *>(a.v)};
        uint8_t *dst[2] = {a.kc, a.vc};
        float *scales[2] = {a.ks, a.vs};
        const int64_t sc = p.id * a.hkv + h;
        float old[2] = {0.f, 0.f};
        if (p.first > 0) {
            old[0] = a.ks[sc];
            old[1] = a.vs[sc];
        }
        // piece x of the group's rows
        auto load = [&](Eight<T> &e, int kv, int x) {
            const int row = x / a.pieces, col = (x - row * a.pieces) * 8;
            e.load(src[kv] + (p.tok + row) * a.stride + (int64_t)h * a.d + col, min(a.d - col, 8), a.vec);
        };
        Eight<T> x[2][PT];
        float top[2] = {0.f, 0.f};
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                x[kv][i].zero();
                if (gl + i * kLanes < np) load(x[kv][i], kv, gl + i * kLanes);
            }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
            for (int i = 0; i < PT; ++i) top[kv] = fmaxf(top[kv], top_of(x[kv][i]));
            for (int y = gl + PT * kLanes; y < np; y += kLanes) {
                Eight<T> e;
                load(e, kv, y);
                top[kv] = fmaxf(top[kv], top_of(e));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top[kv] = fmaxf(top[kv], __shfl_xor_sync(0xffffffffu, top[kv], o));
        }
        if constexpr (W > 1) {
            // two sets in turn: a warp writes one again only behind the barrier that all passed after reading it.
            // Behind this barrier every warp has read the old scales, too.
            float(*r)[2] = red[turn][group];
            turn ^= 1;
            if (lane == 0) r[gw][0] = top[0], r[gw][1] = top[1];
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(kLanes) : "memory");
#pragma unroll
            for (int w = 0; w < W; ++w) top[0] = fmaxf(top[0], r[w][0]), top[1] = fmaxf(top[1], r[w][1]);
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            float s = two_to(exponent_of(top[kv]));
            if (old[kv] > 0.f && old[kv] <= kMaxFloat) {
                if (old[kv] >= s) {
                    s = old[kv];
                } else {
                    const float by = old[kv] / s;
                    for (int y = gl; y < p.first * a.pieces; y += kLanes) {
                        const int row = y / a.pieces, col = (y - row * a.pieces) * 8, n = min(a.d - col, 8);
                        uint8_t *at = dst[kv] + ((p.id * a.bs + row) * a.hkv + h) * a.d + col;
                        Eight<__nv_fp8_e4m3> e;
                        e.zero();
                        if (a.vec) {
                            const uint2 w = *reinterpret_cast<const uint2 *>(at);
                            e.w[0] = w.x, e.w[1] = w.y;
                        } else {
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                if (c < n) e.w[c / 4] |= (uint32_t)at[c] << (8 * (c % 4));
                        }
                        put_codes(at, codes_of(e, by), n, a.vec);
                    }
                }
            }
            if (gl == 0 && s != old[kv]) scales[kv][sc] = s;
            const float inv = 1.f / s;
            auto store = [&](const Eight<T> &e, int y) {
                const int row = y / a.pieces, col = (y - row * a.pieces) * 8;
                put_codes(dst[kv] + ((p.id * a.bs + p.first + row) * a.hkv + h) * a.d + col, codes_of(e, inv),
                          min(a.d - col, 8), a.vec);
            };
#pragma unroll
            for (int i = 0; i < PT; ++i)
                if (gl + i * kLanes < np) store(x[kv][i], gl + i * kLanes);
            for (int y = gl + PT * kLanes; y < np; y += kLanes) {
                Eight<T> e;
                load(e, kv, y);
                store(e, y);
            }
        }
    }
}

template <typename T, int W>
static int launch(const Args &a, int64_t items, cudaStream_t st) {
    constexpr int PT = sizeof(T) == 2 ? 8 : 4;
    constexpr int threads = kThreadsOf<W>;
    const int64_t blocks = ceil_div<int64_t>(items, threads / (32 * W));
    const int64_t most = (int64_t)current_sm_count() * 64;
    const cudaError_t e = launch_pdl(write_blocks_kernel<T, W, PT>, dim3((unsigned)(blocks < most ? blocks : most)),
                                     dim3(threads), 0, st, a, items);
    if (e != cudaSuccess) set_cuda_error(e);
    return launch_status();
}

template <typename T>
static int launch_warps(const Args &a, int64_t items, cudaStream_t st) {
    // the warps whose registers hold the rows that a block gets on average
    const int64_t mean = ceil_div<int64_t>(a.num_tokens, a.num_reqs);
    const int64_t pieces = (mean < a.bs ? mean : a.bs) * a.pieces;
    const int64_t each = 32 * (sizeof(T) == 2 ? 8 : 4);
    if (pieces <= each) return launch<T, 1>(a, items, st);
    if (pieces <= 2 * each) return launch<T, 2>(a, items, st);
    if (pieces <= 4 * each) return launch<T, 4>(a, items, st);
    return launch<T, 8>(a, items, st);
}

}  // namespace wblk
}  // namespace bkv

extern "C" int bkv_cache_write_fp8_blocks(const void *k_new, const void *v_new, int64_t num_tokens,
                                          int64_t new_token_stride, const int32_t *query_start_loc,
                                          const int32_t *context_lens, int32_t num_reqs, const int32_t *block_table,
                                          int64_t bt_stride, int32_t bt_cols, uint8_t *k_cache, uint8_t *v_cache,
                                          float *k_scales, float *v_scales, int64_t total_blocks, int32_t block_size,
                                          int32_t num_kv_heads, int32_t head_dim, int src_dtype, int32_t *err_count,
                                          bkv_stream_t stream) {
    using namespace bkv;
    if (src_dtype != BKV_BF16 && src_dtype != BKV_F32) return BKV_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_reqs < 0 || total_blocks < 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        bt_cols < 0 || bt_stride < bt_cols || new_token_stride < (int64_t)num_kv_heads * head_dim)
        return BKV_ERR_INVALID_ARG;
    // (rows times pieces of a block stay within int32)
    if (block_size > 65536 || head_dim > 65536 || num_tokens > INT32_MAX) return BKV_ERR_INVALID_ARG;
    if (num_tokens == 0 || num_reqs == 0) return BKV_OK;
    if (!k_new || !v_new || !query_start_loc || !context_lens || (bt_cols > 0 && !block_table)) return BKV_ERR_INVALID_ARG;
    if (total_blocks > 0 && (!k_cache || !v_cache || !k_scales || !v_scales)) return BKV_ERR_INVALID_ARG;
    const int e = src_dtype == BKV_BF16 ? 2 : 4;
    const bool vec = head_dim % 8 == 0 && (new_token_stride * e) % 16 == 0 && aligned(k_new, 16) && aligned(v_new, 16) &&
                     aligned(k_cache, 8) && aligned(v_cache, 8);
    const wblk::Args a{k_new, v_new, new_token_stride, num_tokens, query_start_loc, context_lens, num_reqs, block_table,
                       bt_stride, bt_cols, k_cache, v_cache, k_scales, v_scales, total_blocks, block_size, num_kv_heads,
                       head_dim, (head_dim + 7) / 8, err_count, vec};
    const int64_t items = (num_tokens / block_size + 2 * (int64_t)num_reqs) * num_kv_heads;
    return src_dtype == BKV_BF16 ? wblk::launch_warps<__nv_bfloat16>(a, items, (cudaStream_t)stream)
                                 : wblk::launch_warps<float>(a, items, (cudaStream_t)stream);
}
