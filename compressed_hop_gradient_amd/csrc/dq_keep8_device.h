// dq_keep8_device.h -- activations kept in 8 bits: a block's scale, the dithers, the
// codes and back (device code).
#pragma once

#include "dq_experts.h"
#include "dq_train_device.h"

namespace dq {
namespace {

// 32 elements of a row share 2^s, s the smallest (from -110) with max|x| <= 127 2^s;
// the byte is s + 127, and 255 where an element is not finite or beyond 127 2^121, whose
// code's value could pass the largest number.  With max|x| = f 2^e, f in [1, 2), s is
// e - 6, or one more where 64 f > 127.
__device__ __forceinline__ uint32_t keep_exponent(uint32_t max_bits) {
    if (max_bits > 0x7F7E0000u) return 255;
    const int e = (int)(max_bits >> 23) - 6 + ((max_bits & 0x7FFFFFu) > 0x7E0000u);
    return (uint32_t)(e < 17 ? 17 : e);
}

// 2^(16 - s): what makes an element a fixed-point number with 16 fractional bits;
// 0 for a block that is not finite, whose codes are 0.
__device__ __forceinline__ float keep_scale(uint32_t exponent) {
    return exponent == 255 ? 0.0f : __uint_as_float((270 - exponent) << 23);
}

// sign(x) floor((floor(|x| 2^(16 - s)) + d) / 2^16), in the low byte: the product is
// exact and at most 127 2^16, the sum an integer, so that the code is the same in
// any precision.
__device__ __forceinline__ uint32_t keep_code(float x, float scale, uint32_t d) {
    const int q = (int)(((uint32_t)(__builtin_fabsf(x) * scale) + d) >> 16);
    return (uint32_t)(x < 0.0f ? -q : q) & 0xFFu;
}

// 0 times the infinity of exponent 255 is NaN
__device__ __forceinline__ float kept_scale(uint32_t exponent) { return __uint_as_float(exponent << 23); }
__device__ __forceinline__ float kept_value(uint32_t codes, int j, float scale) {
    return (float)(int8_t)(codes >> 8 * j) * scale;
}

// The dithers of elements 8b .. 8b + 7: dropout's counter with bit 15 of the second
// word set, which no element of dropout's that memory can hold reaches.
__device__ __forceinline__ void keep_words(uint64_t b, const KeepKey &k, uint32_t round, uint32_t w[4]) {
    philox_words((uint32_t)b, (uint32_t)(b >> 32) | 0x8000u | k.worker << 16, round, 0x80000000u | k.site, k.key0,
                 k.key1, w);
}

// The dithers of elements at .. at + 7 as words, low half first.
template <bool ON8>
__device__ __forceinline__ void keep_dithers(int64_t at, const KeepKey &k, uint32_t round, uint32_t w[4]) {
    if (!k.dither) {
#pragma unroll
        for (int j = 0; j < 4; j++) w[j] = 0x80008000u;
        return;
    }
    keep_words((uint64_t)(at >> 3), k, round, w);
    if (ON8) return;
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = w[j];
    keep_words((uint64_t)(at >> 3) + 1, k, round, v + 4);
    // eight of the sixteen halves, from at & 7
#pragma unroll
    for (int j = 0; j < 6; j++) v[j] = at & 4 ? v[j + 2 < 8 ? j + 2 : 7] : v[j];
#pragma unroll
    for (int j = 0; j < 5; j++) v[j] = at & 2 ? v[j + 1] : v[j];
#pragma unroll
    for (int j = 0; j < 4; j++) w[j] = at & 1 ? v[j] >> 16 | v[j + 1] << 16 : v[j];
}

// The largest of four neighbouring lanes.
__device__ __forceinline__ uint32_t max_of_four(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));   // lanes 1 0 3 2
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// `have` of eight codes, to or from any address.
template <bool FULL>
__device__ __forceinline__ void store_codes(int8_t *p, int have, uint2 c) {
    if constexpr (FULL) {
        __builtin_memcpy(p, &c, 8);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < have) p[j] = (int8_t)((j < 4 ? c.x : c.y) >> 8 * (j & 3));
    }
}
template <bool FULL>
__device__ __forceinline__ uint2 load_codes(const int8_t *p, int have) {
    uint2 c = make_uint2(0, 0);
    if constexpr (FULL) {
        __builtin_memcpy(&c, p, 8);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < have) (j < 4 ? c.x : c.y) |= (uint32_t)(uint8_t)p[j] << 8 * (j & 3);
    }
    return c;
}

// Eight neighbouring elements of a block that four neighbouring lanes hold together:
// their codes as two words, and the block's exponent.
__device__ __forceinline__ uint2 keep_eight(const float x[8], const uint32_t w[4], uint32_t &exponent) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, abs_bits(x[j]));
    exponent = keep_exponent(max_of_four(m));
    const float scale = keep_scale(exponent);
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; j++)
        c[j / 4] |= keep_code(exponent == 255 ? 0.0f : x[j], scale, j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xFFFFu)
                    << 8 * (j & 3);
    return make_uint2(c[0], c[1]);
}

}  // namespace
}  // namespace dq
