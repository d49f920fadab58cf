// bkv_step.cu -- a step's block tables, token list and slots from the
// requests' lengths.
//
// Request r holds c_r cached tokens and gets n_r new ones.  It has ceil(c_r /
// bs) blocks and needs ceil((c_r + n_r) / bs), at most the table's columns;
// those it lacks come from the free list, request after request, so that with
// f_r their number and F_r = sum_{r' < r} f_r'
//   table[r][have_r + j] = free[F_r + j],  j < f_r,
// and every entry behind them is -1.  Token i of request r (i < n_r) is number
// Q_r + i of the step, Q_r = sum_{r' < r} n_r', at position c_r + i, with the
// slot of that position ("Padding and Batching with Block KV", The Core
// Formula; Slot ID -1: Padding Tokens; "ブロック表" 設計動機: append_row, the
// padded tail of the slot buffer).
//
// One launch: every CTA sums all lengths itself (a run of requests a thread,
// then a scan over the threads), which costs less than a second launch, and
// keeps the sums before each run.  A warp takes a table row, a thread a token:
// it finds the run by bisection and walks the few requests in it.  Quotients by
// a block size that is a power of two are shifts (19.6 -> 11.7 us at 4096 rows:
// every CTA takes two a request).
//
// 32 requests: 3.8 us, the launch and the chain lengths -> sums -> table.  4096
// rows of up to 2048 blocks with 142984 tokens: 11.9 us, 3.0 TB/s of what it reads
// and stores.  That is this order of work, no bound: rows are stored behind the sums
// that only their taken blocks need (over 99% of the entries are -1 whatever the sums),
// every token searches the sums by itself, and warps wait on lengths and free ids for
// 4.9 cycles an instruction.
#include "bkv_internal.cuh"

namespace bkv {
namespace step {

struct Args {
    const int32_t *cached, *fresh;
    int32_t n;
    const int32_t *free_ids;
    int32_t num_free, bs;
    int32_t *bt;
    int64_t bt_stride;
    int32_t cols;
    int64_t max_tokens;
    int32_t *ctx, *qsl, *req;
    int64_t *pos, *slots;
    int32_t *used, *err;
    int32_t shift;   // log2 of bs, or -1
    bool vec;        // table rows begin at 16-byte boundaries
    __device__ __forceinline__ int32_t block_of(uint32_t x) const { return (int32_t)(shift >= 0 ? x >> shift : x / (uint32_t)bs); }
};

constexpr int kThreads = 512;

// A request's lengths, held to what an int32 can say: bad if they were not.
struct Len {
    int32_t c, n, have, all;   // blocks that it has, and with the new tokens'
    bool bad;
    __device__ __forceinline__ Len(const Args &a, int r) {
        c = __ldg(a.cached + r);
        n = __ldg(a.fresh + r);
        bad = c < 0 || n < 0 || n > INT32_MAX - (c > 0 ? c : 0);
        if (bad) {
            c = c > 0 ? c : 0;
            n = n < 0 ? 0 : (n > INT32_MAX - c ? INT32_MAX - c : n);
        }
        have = a.block_of((uint32_t)c + (uint32_t)(a.bs - 1));
        all = a.block_of((uint32_t)c + (uint32_t)n + (uint32_t)(a.bs - 1));
    }
    // blocks taken from the free list
    __device__ __forceinline__ int32_t take(const Args &a) const { return max(min(all, a.cols) - have, 0); }
};

__global__ void __launch_bounds__(kThreads) build_step_kernel(const Args a) {
    __shared__ int64_t tok[kThreads + 1], blk[kThreads + 1];   // sums before each thread's run of requests
    __shared__ int64_t wt[kThreads / 32], wb[kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int per = (int)(((int64_t)a.n + kThreads - 1) / kThreads);
    {
        const int lo = (int)min((int64_t)a.n, (int64_t)threadIdx.x * per), hi = (int)min((int64_t)a.n, (int64_t)lo + per);
        int64_t t = 0, b = 0;
        for (int r = lo; r < hi; ++r) {
            const Len x(a, r);
            t += x.n;
            b += x.take(a);
        }
        int64_t ti = t, bi = b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, ti, o), z = __shfl_up_sync(0xffffffffu, bi, o);
            if (lane >= o) ti += y, bi += z;
        }
        if (lane == 31) wt[warp] = ti, wb[warp] = bi;
        __syncthreads();
        int64_t t0 = ti - t, b0 = bi - b;
        for (int w = 0; w < warp; ++w) t0 += wt[w], b0 += wb[w];
        tok[threadIdx.x] = t0;
        blk[threadIdx.x] = b0;
        if (threadIdx.x == kThreads - 1) {
            tok[kThreads] = t0 + t;
            blk[kThreads] = b0 + b;
        }
        __syncthreads();
    }
    const int64_t total = tok[kThreads];
    auto fit = [](int64_t x) { return (int32_t)(x < INT32_MAX ? x : INT32_MAX); };
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.qsl[a.n] = fit(total);
        *a.used = (int32_t)(blk[kThreads] < a.num_free ? blk[kThreads] : a.num_free);
        if (total > a.max_tokens && a.err) atomicAdd(a.err, 1);
    }

    // ---- table rows: a warp each ----
    for (int64_t r64 = (int64_t)blockIdx.x * (kThreads / 32) + warp; r64 < a.n; r64 += (int64_t)gridDim.x * (kThreads / 32)) {
        const int r = (int)r64;
        const int run = r / per;
        int64_t t = 0, b = 0;   // of the requests before r in its run
        for (int x = run * per + lane; x < r; x += 32) {
            const Len y(a, x);
            t += y.n;
            b += y.take(a);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            t += __shfl_xor_sync(0xffffffffu, t, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        t += tok[run];
        b += blk[run];
        const Len x(a, r);
        const int32_t take = x.take(a);
        if (lane == 0) {
            a.ctx[r] = x.c + x.n;
            a.qsl[r] = fit(t);
            if (a.err) {
                // a bad length, blocks past the table's columns, blocks that the free list lacks
                const int64_t lack = min(max(b + take - a.num_free, (int64_t)0), (int64_t)take);
                const int bad = (x.bad ? 1 : 0) + (x.all > a.cols && x.n > 0 ? 1 : 0) + (int)lack;
                if (bad) atomicAdd(a.err, bad);
            }
        }
        int32_t *row = a.bt + r * a.bt_stride;
        const int64_t shift = b - x.have;
        auto entry = [&](int32_t j) {
            const int64_t at = shift + j;
            return j - x.have < take && at < a.num_free ? __ldg(a.free_ids + at) : -1;
        };
        int32_t j = min(x.have, a.cols);
        if (a.vec) {
            const int32_t j4 = min((j + 3) & ~3, a.cols);
            if (j + lane < j4) row[j + lane] = entry(j + lane);
            j = j4 + 4 * lane;
            for (; j + 4 <= a.cols; j += 128) {
                int4 v = make_int4(-1, -1, -1, -1);
                if (j - x.have < take) v = make_int4(entry(j), entry(j + 1), entry(j + 2), entry(j + 3));
                *reinterpret_cast<int4 *>(row + j) = v;
            }
            for (; j < a.cols; ++j) row[j] = entry(j);   // the one lane that the row's end falls to
        } else {
            for (j += lane; j < a.cols; j += 32) row[j] = entry(j);
        }
    }

    // ---- tokens: a thread each ----
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < a.max_tokens; i += (int64_t)gridDim.x * kThreads) {
        if (i >= total) {
            a.req[i] = -1;
            a.pos[i] = 0;
            a.slots[i] = -1;
            continue;
        }
        int lo = 0, hi = kThreads;   // the last run whose sum is not past i
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tok[mid] <= i) lo = mid;
            else hi = mid;
        }
        int64_t t = i - tok[lo], b = blk[lo];
        for (int r = lo * per;; ++r) {
            const Len x(a, r);
            if (t < x.n) {
                const int64_t p = x.c + t;
                const int32_t lb = a.block_of((uint32_t)p);
                int32_t id = -1;
                if (lb < a.cols) {
                    if (lb < x.have) {
                        id = a.bt[r * a.bt_stride + lb];
                    } else {
                        const int64_t at = b + lb - x.have;
                        if (at < a.num_free) id = __ldg(a.free_ids + at);
                    }
                }
                a.req[i] = r;
                a.pos[i] = p;
                a.slots[i] = id > 0 ? (int64_t)id * a.bs + (p - (int64_t)lb * a.bs) : -1;
                break;
            }
            t -= x.n;
            b += x.take(a);
        }
    }
}

}  // namespace step
}  // namespace bkv

extern "C" int bkv_build_step(const int32_t *cached_lens, const int32_t *new_lens, int32_t num_reqs,
                              const int32_t *free_blocks, int32_t num_free, int32_t block_size, int32_t *block_table,
                              int64_t bt_stride, int32_t bt_cols, int64_t max_num_tokens, int32_t *context_lens,
                              int32_t *query_start_loc, int32_t *req_indices, int64_t *positions, int64_t *slot_mapping,
                              int32_t *blocks_used, int32_t *err_count, bkv_stream_t stream) {
    using namespace bkv;
    if (num_reqs < 0 || num_free < 0 || block_size <= 0 || bt_cols < 0 || bt_stride < bt_cols || max_num_tokens < 0)
        return BKV_ERR_INVALID_ARG;
    if (num_reqs > 1 << 30 || bt_cols > 1 << 30) return BKV_ERR_INVALID_ARG;   // (walks over them stay within int32)
    if (!query_start_loc || !blocks_used) return BKV_ERR_INVALID_ARG;
    if (num_reqs > 0 && (!cached_lens || !new_lens || !context_lens || (bt_cols > 0 && !block_table)))
        return BKV_ERR_INVALID_ARG;
    if ((num_free > 0 && !free_blocks) || (max_num_tokens > 0 && (!req_indices || !positions || !slot_mapping)))
        return BKV_ERR_INVALID_ARG;
    if (num_reqs > 0 && (context_lens == cached_lens || context_lens == new_lens)) return BKV_ERR_INVALID_ARG;
    step::Args a{cached_lens, new_lens, num_reqs, free_blocks, num_free, block_size, block_table, bt_stride, bt_cols,
                 max_num_tokens, context_lens, query_start_loc, req_indices, positions, slot_mapping, blocks_used,
                 err_count, (block_size & (block_size - 1)) == 0 ? __builtin_ctz((unsigned)block_size) : -1,
                 aligned(block_table, 16) && bt_stride % 4 == 0};
    int64_t grid = ceil_div<int64_t>(num_reqs, step::kThreads / 32);
    const int64_t by_tokens = ceil_div<int64_t>(max_num_tokens, step::kThreads);
    if (by_tokens > grid) grid = by_tokens;
    const int64_t most = 2 * (int64_t)current_sm_count();
    if (grid > most) grid = most;
    if (grid < 1) grid = 1;
    const cudaError_t e = launch_pdl(step::build_step_kernel, dim3((unsigned)grid), dim3(step::kThreads), 0,
                                     (cudaStream_t)stream, a);
    if (e != cudaSuccess) set_cuda_error(e);
    return launch_status();
}
