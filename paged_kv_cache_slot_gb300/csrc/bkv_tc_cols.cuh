// bkv_tc_cols.cuh -- what the tcgen05 decode kernels share whose accumulators
// hold query rows in columns: column loads, row reductions over a warp's lanes,
// ring slots, and the encoding of 3-D tensor maps on the host.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "bkv_internal.cuh"
#include "bkv_tc_ptx.cuh"

namespace bkv {
namespace tc {

// The first NQ accumulator columns of this thread's TMEM lane.
template <int NQ>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[NQ]) {
    if constexpr (NQ == 16) tmem_ld16(taddr, v);
    else if constexpr (NQ == 8) tmem_ld8(taddr, v);
    else tmem_ld4(taddr, v);
}

// FP8 caches: an S or O tile holds the products with the hi part in columns
// [0, 16) and with the lo part in [16, 32); the sum of the first NQ of each.
template <int NQ>
__device__ __forceinline__ void tmem_ld_sum2(uint32_t taddr, float (&v)[NQ]) {
    uint32_t h[NQ], l[NQ];
    if constexpr (NQ == 16) {
        tmem_ld16_nw(taddr, h);
        tmem_ld16_nw(taddr + 16u, l);
    } else if constexpr (NQ == 8) {
        tmem_ld8_nw(taddr, h);
        tmem_ld8_nw(taddr + 16u, l);
    } else {
        tmem_ld4_nw(taddr, h);
        tmem_ld4_nw(taddr + 16u, l);
    }
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < NQ; ++i) v[i] = __uint_as_float(h[i]) + __uint_as_float(l[i]);
}

// A ring slot and its phase parity, advanced one tile at a time (no division
// by the ring size on the per-tile path).
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void advance(int n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// Transposed butterfly over a warp: NQ values per lane in, one value out.
// Each halving step exchanges half of the remaining values with the partner
// lane, so after log2(NQ) steps lane l holds query row (l >> (5 - log2 NQ)) &
// (NQ - 1), reduced over the lanes that differ in the high bits; the last
// steps reduce over the low lane bits.  NQ + 5 - log2(NQ) - ... shuffles in
// all (16 for NQ = 16, 6 for NQ = 4).
template <bool kMax, int NQ>
__device__ __forceinline__ float warp_reduce_rows(const float (&v)[NQ], int lane) {
    auto op = [](float x, float y) { return kMax ? fmaxf(x, y) : x + y; };
    float cur[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) cur[i] = v[i];
    int width = NQ;
    int shift = 16;
#pragma unroll
    for (int step = 0; step < 4; ++step) {
        if (width > 1) {
            const bool hi = lane & shift;
            const int h = width / 2;
#pragma unroll
            for (int i = 0; i < NQ / 2; ++i) {
                if (i < h) {
                    const float send = hi ? cur[i] : cur[i + h];
                    const float keep = hi ? cur[i + h] : cur[i];
                    cur[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, shift));
                }
            }
            width = h;
            shift >>= 1;
        }
    }
    float x = cur[0];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o <= shift) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

template <int NQ>
__device__ __forceinline__ int reduced_row(int lane) {
    constexpr int k = NQ == 16 ? 4 : (NQ == 8 ? 3 : 2);
    return (lane >> (5 - k)) & (NQ - 1);
}

template <int NQ>
__device__ __forceinline__ bool reduced_writer(int lane) {
    constexpr int k = NQ == 16 ? 4 : (NQ == 8 ? 3 : 2);
    return (lane & ((1 << (5 - k)) - 1)) == 0;
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

inline bool encode_3d(CUtensorMap *m, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1_bytes,
                      uint64_t s2_bytes, uint32_t b0, uint32_t b1, uint32_t b2,
                      CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {d0, d1, d2};
    const cuuint64_t strides[2] = {s1_bytes, s2_bytes};
    const cuuint32_t box[3] = {b0, b1, b2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, type, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace bkv
