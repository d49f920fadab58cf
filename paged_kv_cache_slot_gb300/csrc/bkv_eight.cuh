// bkv_eight.cuh -- eight consecutive elements of a cache or projection row in
// registers: bf16, fp32 or E4M3 codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace bkv {

template <typename T>
struct Eight {
    uint32_t w[2 * sizeof(T)];   // as they are in memory
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 2 * (int)sizeof(T); ++i) w[i] = 0u;
    }
    // n of the eight exist (the others 0); vec: aligned whole eights
    __device__ __forceinline__ void load(const T *p, int n, bool vec) {
        if (vec) {
            if constexpr (sizeof(T) == 1) {
                const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p));
                w[0] = x.x, w[1] = x.y;
            } else {
#pragma unroll
                for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p) + i);
                    w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
                }
            }
            return;
        }
        zero();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= n) break;
            if constexpr (sizeof(T) == 1) w[i / 4] |= (uint32_t)reinterpret_cast<const uint8_t *>(p)[i] << (8 * (i % 4));
            else if constexpr (sizeof(T) == 2)
                w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << (16 * (i % 2));
            else w[i] = reinterpret_cast<const uint32_t *>(p)[i];
        }
    }
    __device__ __forceinline__ float2 two(int i) const {   // elements 2 i, 2 i + 1
        if constexpr (sizeof(T) == 1) {
            const __nv_fp8x2_storage_t c = (__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i % 2)));
            return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
        } else if constexpr (sizeof(T) == 2) {
            return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        }
    }
};

}  // namespace bkv
