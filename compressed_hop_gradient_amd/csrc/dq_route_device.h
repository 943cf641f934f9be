// dq_route_device.h -- how the router's kernels hold a token's logits, and the
// softmax that the forward pass and the gradient share (device code).
#pragma once

#include <type_traits>

#include "dq_train_device.h"

namespace dq {
namespace {

// A token's logits lie in G lanes (a power of two), 8 CH of them in each, in
// chunks of W: chunk i of lane g holds experts W (i G + g) .. + W - 1.  A wave
// takes 64 / G tokens.  Chunks are 16 bytes where every row is 16-byte aligned and
// E a multiple of W, else single logits, so that lanes side by side read and
// write logits side by side.

constexpr float kLog2e = 1.44269504088896340736f;

// One chunk as loaded; what does not exist is set to -inf by clear().
template <bool F32, bool VEC>
struct Chunk;
template <>
struct Chunk<false, true> {
    static constexpr int W = 8;
    u32x4 w;
    __device__ __forceinline__ void clear() { w = u32x4{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u}; }
    __device__ __forceinline__ void load(const uint16_t *p) { w = *reinterpret_cast<const u32x4 *>(p); }
    __device__ __forceinline__ float at(int j) const {
        return __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
    }
    __device__ __forceinline__ void arrived() { asm volatile("" : "+v"(w)); }
    static __device__ __forceinline__ void store(uint16_t *p, const float d[8]) { store8<false>(p, 0, d); }
};
template <>
struct Chunk<true, true> {
    static constexpr int W = 4;
    float v[4];
    __device__ __forceinline__ void clear() { v[0] = v[1] = v[2] = v[3] = -INFINITY; }
    __device__ __forceinline__ void load(const float *p) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    }
    __device__ __forceinline__ float at(int j) const { return v[j]; }
    __device__ __forceinline__ void arrived() { asm volatile("" : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3])); }
    static __device__ __forceinline__ void store(float *p, const float d[4]) {
        *reinterpret_cast<float4 *>(p) = make_float4(d[0], d[1], d[2], d[3]);
    }
};
template <bool F32>
struct Chunk<F32, false> {
    typedef typename Elem<F32>::type T;
    static constexpr int W = 1;
    T v;
    __device__ __forceinline__ void clear() { v = Elem<F32>::down(-INFINITY); }
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ float at(int) const { return Elem<F32>::up(v); }
    __device__ __forceinline__ void arrived() { asm volatile("" : "+v"(v)); }
    static __device__ __forceinline__ void store(T *p, const float d[1]) { *p = Elem<F32>::down(d[0]); }
};

// The logits of a row that one lane holds
template <bool F32, int G, int CH, bool VEC>
struct Slice {
    typedef Chunk<F32, VEC> C;
    static constexpr int W = C::W, V = 8 * CH, N = V / W;
    C c[N];
    // expert of element v in lane g
    static __device__ __forceinline__ constexpr int expert(int v, int g) { return W * ((v / W) * G + g) + v % W; }
    __device__ __forceinline__ float at(int v) const { return c[v / W].at(v % W); }
    // Loads that nothing waits for: no branch, every address inside the row;
    // keep() then leaves -inf where no logit belongs.
    __device__ __forceinline__ void load(const typename Elem<F32>::type *row, int g, int E) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int at = W * (i * G + g);
            c[i].load(row + (at < E ? at : 0));
        }
    }
    __device__ __forceinline__ void arrived() {
#pragma unroll
        for (int i = 0; i < N; i++) c[i].arrived();
    }
    __device__ __forceinline__ void keep(bool there, int g, int E) {
#pragma unroll
        for (int i = 0; i < N; i++)
            if (!there || W * (i * G + g) >= E) c[i].clear();
    }
};

// op(x, the value of the other half of a group of 2 D lanes), the same in both
// halves: lane ^ 1 and ^ 2, the mirrored lane of the half row and of the row (where
// a half's lanes hold one value), then rows and halves of the wave swapped.
template <int D, class Op>
__device__ __forceinline__ uint32_t with_other_half(uint32_t x, Op op) {
    if constexpr (D <= 8) {
        constexpr int kControl = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;
        return op(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kControl, 0xF, 0xF, false));
    } else {
        const auto both = D == 16 ? __builtin_amdgcn_permlane16_swap(x, x, false, false)
                                  : __builtin_amdgcn_permlane32_swap(x, x, false, false);
        return op(both[0], both[1]);
    }
}
template <int G, int D = 1>
__device__ __forceinline__ float group_max(float x) {
    if constexpr (D < G)
        return group_max<G, 2 * D>(__uint_as_float(with_other_half<D>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
            return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
        })));
    return x;
}
template <int G, int D = 1>
__device__ __forceinline__ float group_sum(float x) {
    if constexpr (D < G)
        return group_sum<G, 2 * D>(__uint_as_float(with_other_half<D>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
            return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
        })));
    return x;
}
// 1 / x to an ulp for 2^-1 <= x < 2^126; NaN stays NaN
__device__ __forceinline__ float reciprocal(float x) {
    const float r = __builtin_amdgcn_rcpf(x);
    return __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r);
}

// exp(l - m) where m is the row's largest logit, or 0.  The exponent takes one
// fma, whose rounding of m log2 e is the same factor for all of the row and
// cancels in quotients.  Up to |m| = 2^20 that factor is within 2^(1/16) of 1;
// far from zero it would pass every bound, and the difference comes first.  Beside
// that factor a value is off by at most (1.25 |l - m| + 2) 2^-24 of itself: half a step
// of the exponent, log2 e's own rounding and the instruction's last place.
// (One token of 64 experts is off by 8e-8 in its outputs, where a library's exp
// leaves 2e-8.)  A longer exponent would cost instructions, which are the bound.
constexpr float kFar = 1048576.0f;
__device__ __forceinline__ float exponential(float l, float m) {
    const float x = __builtin_fmaf(l, kLog2e, -m * kLog2e), y = (l - m) * kLog2e;
    return __builtin_amdgcn_exp2f(fabsf(m) < kFar ? x : y);
}

// e = exp(l - m) of a row and Z = sum e.  Z = 0 only where every logit is -inf;
// NaN or +inf makes Z NaN, and with it all that is divided by it.
template <bool F32, int G, int CH, bool VEC>
__device__ __forceinline__ void exponentials(const Slice<F32, G, CH, VEC> &l, float m, float e[8 * CH], float &Z) {
    float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (__any(!(fabsf(m) < kFar))) {
        asm volatile("; logits far from zero");        // a branch, not selects
#pragma unroll
        for (int v = 0; v < 8 * CH; v++) e[v] = exponential(l.at(v), m);
    } else {
        const float by = -m * kLog2e;
#pragma unroll
        for (int v = 0; v < 8 * CH; v++) e[v] = __builtin_amdgcn_exp2f(__builtin_fmaf(l.at(v), kLog2e, by));
    }
#pragma unroll
    for (int v = 0; v < 8 * CH; v++) z[v % 4] += e[v];
    Z = group_sum<G>((z[0] + z[1]) + (z[2] + z[3]));
}

// Lanes and chunks of a token of E experts: f(G, CH).  Measured at E = 256 with
// 131072 bf16 and 65536 fp32 tokens, k = 8: forward (32, 1) 39.0 and 30.9 us, (16, 2)
// 30.0 and 22.1, (8, 4) 26.2 and 23.6; gradient 37.4 and 26.4, 28.8 and 26.0, 29.2 and
// 28.0.  Forward at E = 64 and 8192 tokens (8, 1) 3.7 and 3.9, (4, 2) 4.5 and 5.1; at
// 131072 bf16 12.0 and 11.8.
template <int G, int CH, class F>
auto shape(F f) {
    return f(std::integral_constant<int, G>(), std::integral_constant<int, CH>());
}
template <class F>
auto by_experts(int E, F f) {
    if (E <= 8) return shape<1, 1>(f);
    if (E <= 16) return shape<2, 1>(f);
    if (E <= 32) return shape<4, 1>(f);
    if (E <= 64) return shape<8, 1>(f);
    if (E <= 128) return shape<8, 2>(f);
    if (E <= 256) return shape<16, 2>(f);
    if (E <= 512) return shape<32, 2>(f);
    return shape<64, 2>(f);
}
inline bool rows_on_16(const void *p, int64_t stride, int E, bool f32) {
    return E % (f32 ? 4 : 8) == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * (f32 ? 4 : 2) % 16 == 0;
}

}  // namespace
}  // namespace dq
