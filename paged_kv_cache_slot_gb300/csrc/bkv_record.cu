// bkv_record.cu -- entry points whose arguments come as one record, for the
// Python binding.
//
// ctypes converts a call's arguments one by one, which takes longer than some of
// these calls run on the GPU (8 us for the 27 of a decode on the host, where
// packing them into a record takes 1).  A record is the C struct below in native
// alignment; each call does what the entry point of bkv.h does that it names.
#include <string.h>

#include "bkv_internal.cuh"

namespace {

struct Step {
    const int32_t *cached_lens, *new_lens;
    int32_t num_reqs;
    const int32_t *free_blocks;
    int32_t num_free, block_size;
    int32_t *block_table;
    int64_t bt_stride;
    int32_t bt_cols;
    int64_t max_num_tokens;
    int32_t *context_lens, *query_start_loc, *req_indices;
    int64_t *positions, *slot_mapping;
    int32_t *blocks_used, *err_count;
    bkv_stream_t stream;
};

struct Write {
    const void *k_new, *v_new;
    int64_t num_tokens, new_token_stride;
    const int32_t *query_start_loc, *context_lens;
    int32_t num_reqs;
    const int32_t *block_table;
    int64_t bt_stride;
    int32_t bt_cols;
    uint8_t *k_cache, *v_cache;
    float *k_scales, *v_scales;
    int64_t total_blocks;
    int32_t block_size, num_kv_heads, head_dim, src_dtype;
    int32_t *err_count;
    bkv_stream_t stream;
};

struct Attend {
    const void *q, *k_cache, *v_cache;
    const float *k_scales, *v_scales;   // null: bkv_paged_decode_sink
    const int32_t *block_table;
    int64_t bt_stride;
    int32_t bt_cols;
    const int32_t *context_lens;
    int32_t max_context_len, num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size;
    int64_t total_blocks;
    float softmax_scale;
    int32_t mask_mode, sliding_window, num_sinks, dtype;
    void *out, *workspace;
    size_t workspace_bytes;
    int32_t *err_count;
    bkv_stream_t stream;
};

template <typename T>
T read(const char *record) {
    T a;
    memcpy(&a, record, sizeof a);
    return a;
}

}  // namespace

extern "C" int bkv_build_step_record(const char *record) {
    const Step a = read<Step>(record);
    return bkv_build_step(a.cached_lens, a.new_lens, a.num_reqs, a.free_blocks, a.num_free, a.block_size, a.block_table,
                          a.bt_stride, a.bt_cols, a.max_num_tokens, a.context_lens, a.query_start_loc, a.req_indices,
                          a.positions, a.slot_mapping, a.blocks_used, a.err_count, a.stream);
}

extern "C" int bkv_cache_write_fp8_blocks_record(const char *record) {
    const Write a = read<Write>(record);
    return bkv_cache_write_fp8_blocks(a.k_new, a.v_new, a.num_tokens, a.new_token_stride, a.query_start_loc, a.context_lens,
                                      a.num_reqs, a.block_table, a.bt_stride, a.bt_cols, a.k_cache, a.v_cache, a.k_scales,
                                      a.v_scales, a.total_blocks, a.block_size, a.num_kv_heads, a.head_dim, a.src_dtype,
                                      a.err_count, a.stream);
}

extern "C" int bkv_paged_decode_sink_record(const char *record) {
    const Attend a = read<Attend>(record);
    return bkv_paged_decode_sink(a.q, a.k_cache, a.v_cache, a.block_table, a.bt_stride, a.bt_cols, a.context_lens,
                                 a.max_context_len, a.num_reqs, a.q_len, a.num_q_heads, a.num_kv_heads, a.head_dim,
                                 a.block_size, a.total_blocks, a.softmax_scale, a.mask_mode, a.sliding_window, a.num_sinks,
                                 a.dtype, a.out, a.workspace, a.workspace_bytes, a.err_count, a.stream);
}

extern "C" int bkv_paged_decode_fp8_blocks_record(const char *record) {
    const Attend a = read<Attend>(record);
    return bkv_paged_decode_fp8_blocks(a.q, static_cast<const uint8_t *>(a.k_cache), static_cast<const uint8_t *>(a.v_cache),
                                       a.k_scales, a.v_scales, a.block_table, a.bt_stride, a.bt_cols, a.context_lens,
                                       a.max_context_len, a.num_reqs, a.q_len, a.num_q_heads, a.num_kv_heads, a.head_dim,
                                       a.block_size, a.total_blocks, a.softmax_scale, a.mask_mode, a.sliding_window,
                                       a.num_sinks, a.dtype, a.out, a.workspace, a.workspace_bytes, a.err_count, a.stream);
}
