// bkv_tree.cuh -- shared declarations of the attention of drafted trees over
// the paged cache.
#pragma once

#include <cuda.h>

#include "bkv_internal.cuh"

namespace bkv {

// Everything a tree attention launch needs; passed by value to its kernels.
// Request r's T tree tokens are the last T of its L_r cached positions; token
// t sees every position before L_r - T, and position L_r - T + i if bit i of
// its mask row is set.
struct TreeArgs {
    const void *q;           // [num_reqs][T][H_q][D]
    const void *k;
    const void *v;
    const int32_t *bt;
    int64_t bt_stride;
    int32_t bt_cols;
    const int32_t *ctx;
    int32_t max_ctx;
    int32_t num_reqs, T, H_q, H_kv, D, bs, G;
    int64_t total_blocks;
    float scale_log2;        // softmax_scale * log2(e): scores are kept in base 2
    const uint32_t *mask;    // [num_reqs][T][mask_words], or one tree for all (mask_stride 0)
    int64_t mask_stride;     // words between requests
    int32_t mask_words;
    int dtype;
    void *out;               // [num_reqs][T][H_q][D]
    int32_t *err;
    // The split: a stream is (request, KV head, token group of TS tokens, NR =
    // TS * G query rows); its partials are slots of NR rows in the workspace.
    int32_t TS, NR, groups;  // groups = ceil(T / TS)
    int32_t P;               // columns: each takes its share of the positions of all requests
    // A column may end one stream that it did not begin (its partial: slot q of 2 P a KV head and group) and begin
    // one that it does not end (slot P + q).
    int2 *ws_split;          // [P] the latter: (request, columns that share it), (0, 0) without one
    float *ws_o;             // [slots][NR][D] unnormalised partial outputs
    float *ws_ml;            // [slots][NR][2] (running max in base 2, sum of weights)
};

constexpr int kTreeTile = 128;   // positions a tile of the tensor-core kernel

__device__ __forceinline__ int32_t tree_len(const TreeArgs &a, int32_t ctx) {
    const int32_t L = ctx > a.max_ctx ? a.max_ctx : ctx;
    return L > 0 ? L : 0;
}

// Positions [lo, lo + 32) that token t of a request of length L sees by the
// tree's mask alone, as a bit mask: all before first = L - T, of the tree's
// own those of its mask row, none from L on.
__device__ __forceinline__ uint32_t tree_vis32(const uint32_t *row, int32_t words, int32_t first, int32_t L,
                                               int32_t lo) {
    const int32_t pre = first - lo, lim = L - lo;
    if (lim <= 0) return 0u;
    uint32_t v = pre >= 32 ? 0xffffffffu : (pre > 0 ? (1u << pre) - 1u : 0u);
    if (pre < 32) {
        const int32_t o = -pre;   // tree index of position lo
        if (o >= 0) {
            const int32_t w = o >> 5;
            const uint32_t a = w < words ? __ldg(row + w) : 0u;
            const uint32_t b = w + 1 < words ? __ldg(row + w + 1) : 0u;
            v |= __funnelshift_r(a, b, o & 31);
        } else {
            v |= __ldg(row) << pre;
        }
    }
    return lim >= 32 ? v : v & ((1u << lim) - 1u);
}

// A launch of the tensor-core kernel: its boxes and its shared memory.
struct TreeShape {
    int seg_rows;       // cache rows of a load: min(block size, 128)
    int tok_per_tile;   // tree tokens a 128-row query tile holds: 128 / G
    int box_tok;        // tokens a load of q brings
    int q_half;         // bytes of a query tile's head_dim half
    int q_buffers;      // query tiles kept: two units' one, a unit's two, or one
    int q_bytes;
    int k_stages, v_stages;
    int smem;
};

struct TreeTc {
    CUtensorMap mk, mv, mq;
    TreeShape sh;
};
bool prepare_tree_tc(const TreeArgs &a, TreeTc *t);
int launch_tree_tc(const TreeArgs &a, const TreeTc &t, cudaStream_t stream);

}  // namespace bkv
