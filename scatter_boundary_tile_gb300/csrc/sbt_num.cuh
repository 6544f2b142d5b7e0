// Number types of the operators that compute in fp32: conversions of single
// elements and of 16-byte vectors.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sbt_internal.cuh"

namespace sbt_num {

enum Kind { kF32 = 0, kBF16 = 1, kF16 = 2 };

template <int KIND> struct Num;
template <> struct Num<kF32> {
    typedef uint32_t T;
    static constexpr int V = 4;
    static __device__ __forceinline__ float get(uint32_t x) { return __uint_as_float(x); }
    static __device__ __forceinline__ uint32_t put(float x) { return __float_as_uint(x); }
};
template <> struct Num<kBF16> {
    typedef uint16_t T;
    static constexpr int V = 8;
    static __device__ __forceinline__ float get(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
    static __device__ __forceinline__ uint16_t put(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};
template <> struct Num<kF16> {
    typedef uint16_t T;
    static constexpr int V = 8;
    static __device__ __forceinline__ float get(uint16_t x) { return __half2float(__ushort_as_half(x)); }
    static __device__ __forceinline__ uint16_t put(float x) { return __half_as_ushort(__float2half_rn(x)); }
};

template <int KIND>
__device__ __forceinline__ void unpack(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (KIND == kF32) {
            x[i] = __uint_as_float(w[i]);
        } else if (KIND == kBF16) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}

template <int KIND>
__device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (KIND == kF32) {
            w[i] = __float_as_uint(x[i]);
        } else if (KIND == kBF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

inline int kind_of(sbt_dtype t) { return t == SBT_F32 ? kF32 : t == SBT_BF16 ? kBF16 : kF16; }

}  // namespace sbt_num
