// dq_train_device.h -- element types and 8-element loads and stores of the
// training-step kernels (device code).
#pragma once

#include <type_traits>

#include "dq_train.h"

namespace dq {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
    return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

// Philox4x32-10 (Salmon et al., SC'11) of counter (x0, x1, x2, x3).  A product is one
// 64-bit multiply, a three-way xor one instruction.
__device__ __forceinline__ void philox_words(uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3, uint32_t k0,
                                             uint32_t k1, uint32_t w[4]) {
#pragma unroll
    for (int r = 0; r < 10; r++) {
        if (r > 0) {
            k0 += 0x9E3779B9u;
            k1 += 0xBB67AE85u;
        }
        const uint64_t pa = (uint64_t)0xD2511F53u * x0;
        const uint64_t pb = (uint64_t)0xCD9E8D57u * x2;
        x0 = xor3((uint32_t)(pb >> 32), x1, k0);
        x1 = (uint32_t)pb;
        x2 = xor3((uint32_t)(pa >> 32), x3, k1);
        x3 = (uint32_t)pa;
    }
    w[0] = x0;
    w[1] = x1;
    w[2] = x2;
    w[3] = x3;
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

// The same at any alignment of the elements (the hardware splits such accesses); FULL:
// all eight are there, else `have` of them, the others read as 0 and are not written.  A
// branch on it stands around all accesses of an eight, not at each: where branches join,
// loads are waited for.
template <bool F32, bool FULL>
__device__ __forceinline__ void load_eight(const void *p, int64_t at, int have, float v[8]) {
    typedef typename Elem<F32>::type T;
    const T *q = static_cast<const T *>(p) + at;
    if constexpr (FULL) {
        T w[8];
        __builtin_memcpy(w, q, sizeof(w));
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = Elem<F32>::up(w[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = j < have ? Elem<F32>::up(q[j]) : 0.0f;
    }
}
template <bool F32, bool FULL>
__device__ __forceinline__ void store_eight(void *p, int64_t at, int have, const float v[8]) {
    typedef typename Elem<F32>::type T;
    T *q = static_cast<T *>(p) + at;
    if constexpr (FULL) {
        T w[8];
#pragma unroll
        for (int j = 0; j < 8; j++) w[j] = Elem<F32>::down(v[j]);
        __builtin_memcpy(q, w, sizeof(w));
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < have) q[j] = Elem<F32>::down(v[j]);
    }
}

// body(full, c) for the eights from column `first`, `step` columns apart, of rows of
// `width`; EVEN: of whole eights.
template <bool EVEN, class Body>
__device__ __forceinline__ void by_eights(int first, int step, int width, Body body) {
    for (int c = first; c < width; c += step) {
        if (EVEN || c + 8 <= width)
            body(std::true_type(), c);
        else
            body(std::false_type(), c);
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
