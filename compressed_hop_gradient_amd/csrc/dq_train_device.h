// dq_train_device.h -- element types and 8-element loads and stores of the
// training-step kernels (device code).
#pragma once

#include "dq_train.h"

namespace dq {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
    return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

// fp32 -> bf16 bits, round to nearest even (NaN stays NaN)
__device__ __forceinline__ uint32_t bf16_bits(float x) {
    const __bf16 h = (__bf16)x;
    return __builtin_bit_cast(unsigned short, h);
}

template <bool F32>
struct Elem;
template <>
struct Elem<false> {
    typedef uint16_t type;
    static __device__ __forceinline__ float up(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t down(float v) { return (uint16_t)bf16_bits(v); }
};
template <>
struct Elem<true> {
    typedef float type;
    static __device__ __forceinline__ float up(float v) { return v; }
    static __device__ __forceinline__ float down(float v) { return v; }
};

template <bool F32>
__device__ __forceinline__ void load8(const void *p, int64_t at, float v[8]) {
    if (F32) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
        const float4 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const u32x4 a = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + at);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            v[2 * j] = __uint_as_float(a[j] << 16);
            v[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
        }
    }
}

template <bool F32>
__device__ __forceinline__ void store8(void *p, int64_t at, const float v[8]) {
    if (F32) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        u32x4 a;
#pragma unroll
        for (int j = 0; j < 4; j++) a[j] = bf16_bits(v[2 * j]) | bf16_bits(v[2 * j + 1]) << 16;
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + at) = a;
    }
}

}  // namespace
}  // namespace dq
