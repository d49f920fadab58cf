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
// The work of one (touched block, KV head) is a group's: its K rows, then its V
// rows, are read once into registers, their maximum reduced, and the codes
// written; the next rows are loaded while these are worked on.  The blocks a step
// touches are numbered floor(start_r / bs) + 2 r + j, j the request's own count:
// the numbers of different requests never meet (a request of n tokens touches at
// most n / bs + 2 blocks), gaps are skipped, and no scan over the requests has to
// come first.  Where that is fewer numbers, they are start_r + j (a touched block
// has a token).
//
// Memory-bound for prompts (e + 1 bytes an element): 32 of 512 to 4096 tokens, 8
// heads of 128, bf16, blocks of 64: 85 us, 5.3 TB/s.  (One set of registers, no row
// loaded while others are worked on: 181.  128 registers a thread hold 16 warps an
// SM, whose two sets are 64 KB in flight; warps still wait on rows for 3.1 cycles an
// instruction.)  A decode step is the chain request -> row, table entry -> scale ->
// store behind a launch: 256 requests 4.6 us.
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
    int32_t shift;             // log2 of bs, or -1
    bool by_token;             // how touched blocks are numbered
    int32_t heads, runs;       // KV heads that a group takes one after the other, and runs of them a block
    int32_t *err;
    bool vec;
    __device__ __forceinline__ int32_t block_of(int32_t x) const {
        return (int32_t)(shift >= 0 ? (uint32_t)x >> shift : (uint32_t)x / (uint32_t)bs);
    }
};

// Where the token rows of request r begin in the step, within [0, num_tokens].
__device__ __forceinline__ int32_t start_of(const Args &a, int r) {
    return max(0, min(__ldg(a.qsl + r), (int32_t)a.num_tokens));
}
// The number of request r's first block.
__device__ __forceinline__ int32_t number_of(const Args &a, int r, int32_t start) {
    return a.by_token ? start : a.block_of(start) + 2 * r;
}

// A touched block's rows: `cnt` tokens from `tok` on go to rows `first` on of the
// block whose table entry is `entry`; first -1: the block lies past the table's
// columns; cnt 0: nothing.
struct Part {
    int32_t tok, first, cnt, entry;
};

// Block number u of the step, by one warp.  count: this warp counts errors.
// Nothing here looks at the entry, so that its load and the rows' overlap.
__device__ __forceinline__ Part part_of(const Args &a, int32_t u, bool count) {
    const int lane = threadIdx.x & 31;
    Part p{0, 0, 0, 0};
    // the last request whose numbers begin at or before u: 32 probes a round, and 256 in the last
    int lo = 0, n = a.num_reqs;
    while (n > 256) {
        const int step = (n + 31) / 32;
        const bool in = lane * step < n && number_of(a, lo + lane * step, start_of(a, lo + lane * step)) <= u;
        const uint32_t m = __ballot_sync(0xffffffffu, in);
        const int last = m ? 31 - __clz(m) : 0;
        lo += last * step;
        n = min(step, n - last * step);
    }
    int before = 0;
    if (n > 32) {
        int32_t at[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) at[i] = 32 * i + lane < n ? start_of(a, lo + 32 * i + lane) : -1;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            before += __popc(__ballot_sync(0xffffffffu, at[i] >= 0 && number_of(a, lo + 32 * i + lane, at[i]) <= u));
    } else {
        before = __popc(__ballot_sync(0xffffffffu, lane < n && number_of(a, lo + lane, start_of(a, lo + lane)) <= u));
    }
    lo += max(before - 1, 0);
    const int32_t t0 = start_of(a, lo), t1 = start_of(a, lo + 1);
    const int32_t L = __ldg(a.ctx + lo);
    const int32_t j = u - number_of(a, lo, t0);
    if (t1 <= t0 || j < 0) return p;
    if (L < t1 - t0) {   // more new tokens than the request's length
        if (count && j == 0 && lane == 0 && a.err) atomicAdd(a.err, 1);
        return p;
    }
    const int32_t start = L - (t1 - t0);
    // (64 bits: the numbers behind the last request's blocks are its own as well, however many they are)
    const int64_t b0 = ((int64_t)a.block_of(start) + j) * a.bs;
    if (b0 >= L) return p;
    const int32_t lb = a.block_of(start) + j;
    const int32_t p0 = max(start, (int32_t)b0), p1 = (int32_t)min((int64_t)L, b0 + a.bs);
    const bool past = lb >= a.bt_cols;
    p.entry = past ? 0 : __ldg(a.bt + (int64_t)lo * a.bt_stride + lb);
    p.tok = t0 + (p0 - start);
    p.first = past ? -1 : (int32_t)(p0 - b0);
    p.cnt = p1 - p0;
    return p;
}

// The exponent of the smallest power of two s with top <= 448 s, held to [-40, 40].
__device__ __forceinline__ int exponent_of(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 127 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0) - 8;   // 448 = 1.75 x 2^8
    return min(max(e, -40), 40);
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The largest magnitude of eight elements, as its bits (two bf16 side by side, or one fp32): infinities and NaN come
// out above every number.
__device__ __forceinline__ uint32_t top_of(uint32_t t, const Eight<__nv_bfloat16> &x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t = __vmaxu2(t, x.w[i] & 0x7fff7fffu);
    return t;
}
__device__ __forceinline__ uint32_t top_of(uint32_t t, const Eight<float> &x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, x.w[i] & 0x7fffffffu);
    return t;
}
// fp32 bits of a lane's largest; and, where that is no number, of its largest finite one
template <typename T>
__device__ __forceinline__ uint32_t top_bits(uint32_t t) {
    return sizeof(T) == 2 ? max(t & 0xffffu, t >> 16) << 16 : t;
}
template <typename T>
__device__ __forceinline__ uint32_t finite_top(uint32_t t, const Eight<T> &x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = x.two(i);
        const uint32_t a = __float_as_uint(f.x) & 0x7fffffffu, b = __float_as_uint(f.y) & 0x7fffffffu;
        t = max(t, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
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

// Groups of W warps, as many as fit into 128 threads a CTA; PT pieces a thread in
// registers, twice: one set is loaded while the other is worked on.  Rows that do
// not fit are read again for their codes.
template <int W>
constexpr int kThreadsOf = W < 4 ? 128 : 32 * W;

// kEven: whole aligned eights, and a group's pieces begin at one column, so that a thread's lie drow rows apart.
template <typename T, int W, int PT, bool kEven>
__global__ void __launch_bounds__(kThreadsOf<W>, 512 / kThreadsOf<W>) write_blocks_kernel(const Args a, int32_t items) {
    constexpr int kGroups = kThreadsOf<W> / (32 * W);
    constexpr int kLanes = 32 * W;
    __shared__ uint32_t red[2][kGroups][W];
    const int group = threadIdx.x / kLanes, gl = threadIdx.x % kLanes, gw = gl >> 5, lane = threadIdx.x & 31;
    // this thread's first piece of a group's rows, and how far apart its pieces are
    const int row0 = gl / a.pieces, col0 = gl - row0 * a.pieces, drow = kLanes / a.pieces, dcol = kEven ? 0 : kLanes - drow * a.pieces;
    const bool vec = kEven || a.vec;
    // f(i, row, first element) of this thread's pieces [from, to) of `rows` rows
    auto each_piece = [&](int rows, int from, int to, auto &&f) {
        int row = row0 + from * drow, col = col0 + from * dcol;
        if (!kEven) row += col / a.pieces, col %= a.pieces;
#pragma unroll 1
        for (int i = from; i < to && row < rows; ++i) {
            f(i, row, col * 8);
            row += drow, col += dcol;
            if (!kEven && col >= a.pieces) col -= a.pieces, ++row;
        }
    };
    auto each_held = [&](int rows, auto &&f) {   // the same of those in registers
        int row = row0, col = col0;
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            if (row < rows) f(i, row, col * 8);
            row += drow, col += dcol;
            if (!kEven && col >= a.pieces) col -= a.pieces, ++row;
        }
    };
    auto elems = [&](int col) { return kEven ? 8 : min(a.d - col, 8); };
    pdl_wait();
    pdl_trigger();
    int turn = 0;
    const int64_t pitch = (int64_t)a.hkv * a.d;
    auto src_of = [&](int kv, const Part &p, int h) {
        return static_cast<const T *>(kv ? a.v : a.k) + p.tok * a.stride + (int64_t)h * a.d;
    };
    auto load = [&](Eight<T> (&x)[PT], int kv, const Part &p, int h) {
        const T *src = src_of(kv, p, h);
#pragma unroll
        for (int i = 0; i < PT; ++i) x[i].zero();
        each_held(p.cnt, [&](int i, int row, int col) { x[i].load(src + row * a.stride + col, elems(col), vec); });
    };
    // maximum, scale, and codes of K's or V's rows of a part
    auto work = [&](const Eight<T> (&x)[PT], int kv, const Part &p, int h, int64_t id, float old) {
        const T *src = src_of(kv, p, h);
        auto again = [&](int row, int col) {
            Eight<T> e;
            e.load(src + row * a.stride + col, elems(col), vec);
            return e;
        };
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < PT; ++i) top = top_of(top, x[i]);
        each_piece(p.cnt, PT, INT32_MAX, [&](int, int row, int col) { top = top_of(top, again(row, col)); });
        top = top_bits<T>(top);
        if (top >= 0x7f800000u) {   // an infinity or a NaN: the finite elements alone
            top = 0u;
#pragma unroll
            for (int i = 0; i < PT; ++i) top = finite_top(top, x[i]);
            each_piece(p.cnt, PT, INT32_MAX, [&](int, int row, int col) { top = finite_top(top, again(row, col)); });
        }
        __syncwarp();
        top = __reduce_max_sync(0xffffffffu, top);
        if constexpr (W > 1) {
            // two sets in turn: a warp writes one again only behind the barrier that all passed after reading it.
            // Behind this barrier every warp has read the old scale, too.
            uint32_t *r = red[turn][group];
            turn ^= 1;
            if (lane == 0) r[gw] = top;
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(kLanes) : "memory");
#pragma unroll
            for (int w = 0; w < W; ++w) top = max(top, r[w]);
        }
        uint8_t *dst = (kv ? a.vc : a.kc) + (id * a.bs * a.hkv + h) * a.d;   // the block's first row
        float s = two_to(exponent_of(__uint_as_float(top)));
        if (old > 0.f && old <= kMaxFloat) {
            if (old >= s) {
                s = old;
            } else {
                const float by = old / s;
                each_piece(p.first, 0, INT32_MAX, [&](int, int row, int col) {
                    uint8_t *at = dst + row * pitch + col;
                    const int n = elems(col);
                    Eight<__nv_fp8_e4m3> e;
                    e.zero();
                    if (vec) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(at);
                        e.w[0] = w.x, e.w[1] = w.y;
                    } else {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            if (c < n) e.w[c / 4] |= (uint32_t)at[c] << (8 * (c % 4));
                    }
                    put_codes(at, codes_of(e, by), n, vec);
                });
            }
        }
        if (gl == 0 && s != old) (kv ? a.vs : a.ks)[id * a.hkv + h] = s;
        const float inv = 1.f / s;
        dst += p.first * pitch;
        each_held(p.cnt, [&](int i, int row, int col) { put_codes(dst + row * pitch + col, codes_of(x[i], inv), elems(col), vec); });
        each_piece(p.cnt, PT, INT32_MAX, [&](int, int row, int col) {
            put_codes(dst + row * pitch + col, codes_of(again(row, col), inv), elems(col), vec);
        });
    };

    // an item is a touched block's run of heads; `h` goes through it
    int32_t it = (int32_t)blockIdx.x * kGroups + group;
    const int32_t step = (int32_t)gridDim.x * kGroups;
    int h = 0, h_end = 0;
    auto find = [&](Part &p) -> bool {
        if (++h < h_end) return true;   // the same block's next head
        for (; it < items; it += step) {
            const int32_t u = it / a.runs;
            h = (it - u * a.runs) * a.heads;
            h_end = min(h + a.heads, a.hkv);
            p = part_of(a, u, h == 0 && gw == 0);
            if (p.cnt > 0) {
                it += step;
                return true;
            }
        }
        return false;
    };
    Eight<T> xk[PT], xv[PT];
    Part p{0, 0, 0, 0};
    bool have = find(p);
    if (have) load(xk, 0, p, h);
    while (have) {
        const int hp = h;
        const Part now = p;
        load(xv, 1, now, hp);
        // a real block, and its scales so far
        const bool real = now.entry > 0 && now.entry < a.total_blocks;
        if ((now.first < 0 || now.entry >= a.total_blocks) && hp == 0 && gl == 0 && a.err) atomicAdd(a.err, 1);
        float old_k = 0.f, old_v = 0.f;
        if (real && now.first > 0) {
            old_k = a.ks[(int64_t)now.entry * a.hkv + hp];
            old_v = a.vs[(int64_t)now.entry * a.hkv + hp];
        }
        have = find(p);
        if (real) work(xk, 0, now, hp, now.entry, old_k);
        if (have) load(xk, 0, p, h);
        if (real) work(xv, 1, now, hp, now.entry, old_v);
    }
}

template <typename T, int W>
static int launch(Args a, int32_t blocks, cudaStream_t st) {
    constexpr int PT = sizeof(T) == 2 ? 8 : 4;
    constexpr int threads = kThreadsOf<W>;
    constexpr int groups = threads / (32 * W);
    // as many CTAs as are resident at once: a group loads its next rows while it works
    const int64_t most = (int64_t)current_sm_count() * (512 / threads);
    // One search for a block serves a run of its heads, as long as every group has about four runs.
    a.heads = 1;
    while (a.heads < a.hkv && (int64_t)blocks * ceil_div(a.hkv, 2 * a.heads) >= 4 * most * groups) a.heads *= 2;
    a.runs = ceil_div(a.hkv, a.heads);
    const int32_t items = blocks * a.runs;
    const int64_t ctas = ceil_div<int64_t>(items, groups);
    const dim3 grid((unsigned)(ctas < most ? ctas : most));
    const bool even = a.vec && (32 * W) % a.pieces == 0;
    const cudaError_t e = even ? launch_pdl(write_blocks_kernel<T, W, PT, true>, grid, dim3(threads), 0, st, a, items)
                               : launch_pdl(write_blocks_kernel<T, W, PT, false>, grid, dim3(threads), 0, st, a, items);
    if (e != cudaSuccess) set_cuda_error(e);
    return launch_status();
}

template <typename T>
static int launch_warps(const Args &a, int32_t blocks, cudaStream_t st) {
    // the warps whose registers hold the rows that a block gets on average
    const int64_t mean = ceil_div<int64_t>(a.num_tokens, a.num_reqs);
    const int64_t pieces = (mean < a.bs ? mean : a.bs) * a.pieces;
    const int64_t each = 32 * (sizeof(T) == 2 ? 8 : 4);
    if (pieces <= each) return launch<T, 1>(a, blocks, st);
    if (pieces <= 2 * each) return launch<T, 2>(a, blocks, st);
    if (pieces <= 4 * each) return launch<T, 4>(a, blocks, st);
    return launch<T, 8>(a, blocks, st);
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
    // numbers of touched blocks
    const int64_t by_blocks = num_tokens / block_size + 2 * (int64_t)num_reqs;
    const int64_t blocks = num_tokens < by_blocks ? num_tokens : by_blocks;
    if (by_blocks * num_kv_heads >= ((int64_t)1 << 30)) return BKV_ERR_INVALID_ARG;
    const wblk::Args a{k_new, v_new, new_token_stride, num_tokens, query_start_loc, context_lens, num_reqs, block_table,
                       bt_stride, bt_cols, k_cache, v_cache, k_scales, v_scales, total_blocks, block_size, num_kv_heads,
                       head_dim, (head_dim + 7) / 8, (block_size & (block_size - 1)) == 0 ? __builtin_ctz((unsigned)block_size) : -1,
                       num_tokens < by_blocks, 1, num_kv_heads, err_count, vec};
    return src_dtype == BKV_BF16 ? wblk::launch_warps<__nv_bfloat16>(a, (int32_t)blocks, (cudaStream_t)stream)
                                 : wblk::launch_warps<float>(a, (int32_t)blocks, (cudaStream_t)stream);
}
