// dq_train.hip -- HIP kernels of the training-step operators for gfx950: dropout
// from the counter-based generator, and the expert router with its balance
// statistics and gradients.  fp32 arithmetic, no contraction.
#include "dq_train.h"

#include <type_traits>

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

// ---------------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------------

// The eight 16-bit dithers of elements 8b .. 8b + 7 as four words, low half
// first: Philox4x32-10 (Salmon et al., SC'11) on (b, worker, round, site).
__device__ __forceinline__ void dropout_words(uint64_t b, const DropoutArgs &a, uint32_t round, uint32_t w[4]) {
    uint32_t x0 = (uint32_t)b, x1 = (uint32_t)(b >> 32) | a.worker << 16, x2 = round, x3 = 0x80000000u | a.site;
    uint32_t k0 = a.key0, k1 = a.key1;
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

__device__ __forceinline__ uint32_t dither(const uint32_t w[4], int j) {
    return j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu;
}

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

template <bool F32, bool RES>
__device__ __forceinline__ float dropout_one(float x, float r, bool keep, float scale) {
    const float y = keep ? x * scale : 0.0f;
    return RES ? r + y : y;
}

// Rows of a multiple of 8 elements, all 16-byte aligned, or one row of any
// length (ROWS false): a thread takes the eight elements of one Philox block.
template <bool F32, bool RES, bool ROWS>
__global__ __launch_bounds__(256) void k_dropout(DropoutArgs a, int64_t blocks) {
    typedef Elem<F32> El;
    typedef typename El::type T;
    const uint32_t round = a.round + (a.d_round ? *a.d_round : 0);
    const int64_t n = a.rows * a.cols;
    for (int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x; b < blocks; b += (int64_t)gridDim.x * 256) {
        uint32_t w[4] = {0, 0, 0, 0};
        if (a.threshold) dropout_words((uint64_t)b, a, round, w);   // T = 0 keeps everything
        int64_t row = 0, col = 8 * b;
        if (ROWS) {
            row = col / a.cols;
            col -= row * a.cols;
        }
        if (ROWS || 8 * b + 8 <= n) {
            float x[8], r[8];
            load8<F32>(a.x, row * a.xs + col, x);
            if (RES) load8<F32>(a.residual, row * a.rs + col, r);
#pragma unroll
            for (int j = 0; j < 8; j++)
                x[j] = dropout_one<F32, RES>(x[j], r[j], dither(w, j) >= a.threshold, a.scale);
            store8<F32>(a.y, row * a.ys + col, x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (col + j >= n) break;
                const float r = RES ? El::up(static_cast<const T *>(a.residual)[col + j]) : 0.0f;
                static_cast<T *>(a.y)[col + j] = El::down(dropout_one<F32, RES>(
                    El::up(static_cast<const T *>(a.x)[col + j]), r, dither(w, j) >= a.threshold, a.scale));
            }
        }
    }
}

// Any alignment and row length: a wave draws 64 Philox blocks and then takes
// their 512 elements 64 at a time, side by side in its lanes.
template <bool F32, bool RES>
__global__ __launch_bounds__(256) void k_dropout_any(DropoutArgs a, int64_t tiles) {
    typedef Elem<F32> El;
    typedef typename El::type T;
    const uint32_t round = a.round + (a.d_round ? *a.d_round : 0);
    const int64_t n = a.rows * a.cols;
    const int lane = threadIdx.x & 63;
    // cols < 64: the rows that 64 elements go down, and what is left of them
    const int skip = a.cols < 64 ? 64 / (int)a.cols : 1;
    const int64_t left = a.cols < 64 ? 64 % (int)a.cols : 64 - a.cols;
    for (int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); tile < tiles; tile += (int64_t)gridDim.x * 4) {
        uint32_t keep = 0xFF;
        if (a.threshold) {
            uint32_t w[4];
            dropout_words((uint64_t)(64 * tile + lane), a, round, w);
            keep = 0;
#pragma unroll
            for (int j = 0; j < 8; j++) keep |= (uint32_t)(dither(w, j) >= a.threshold) << j;
        }
        int64_t at = 512 * tile + lane, row = at / a.cols, col = at - row * a.cols;
        T x[8], r[8];
        int64_t y[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const bool there = at + 64 * i < n;
            x[i] = static_cast<const T *>(a.x)[there ? row * a.xs + col : 0];
            if (RES) r[i] = static_cast<const T *>(a.residual)[there ? row * a.rs + col : 0];
            y[i] = there ? row * a.ys + col : -1;
            // 64 elements on
            if (a.cols < 64) {
                row += skip;
                col += left;
                if (col >= a.cols) {
                    col -= a.cols;
                    row++;
                }
            } else {
                const bool next = col + 64 >= a.cols;
                col += next ? left : 64;
                row += next;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const bool kept = (uint32_t)__shfl((int)keep, 8 * i + lane / 8, 64) >> (lane & 7) & 1;
            if (y[i] >= 0)
                static_cast<T *>(a.y)[y[i]] =
                    El::down(dropout_one<F32, RES>(El::up(x[i]), RES ? El::up(r[i]) : 0.0f, kept, a.scale));
        }
    }
}

template <bool F32, bool RES>
hipError_t dropout_access(const DropoutArgs &a, hipStream_t s) {
    const int64_t es = F32 ? 4 : 2;
    const int64_t blocks = (a.rows * a.cols + 7) / 8, tiles = (blocks + 63) / 64;
    const auto grid = [](int64_t want) { return dim3((unsigned)(want < (1 << 20) ? want : (1 << 20))); };
    const dim3 block(256);
    const auto on16 = [&](const void *p, int64_t stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.rows == 1 || stride * es % 16 == 0);
    };
    const bool vec = on16(a.x, a.xs) && on16(a.y, a.ys) && (!RES || on16(a.residual, a.rs));
    if (vec && a.rows == 1)
        hipLaunchKernelGGL((k_dropout<F32, RES, false>), grid((blocks + 255) / 256), block, 0, s, a, blocks);
    else if (vec && a.cols % 8 == 0)
        hipLaunchKernelGGL((k_dropout<F32, RES, true>), grid((blocks + 255) / 256), block, 0, s, a, blocks);
    else
        hipLaunchKernelGGL((k_dropout_any<F32, RES>), grid((tiles + 3) / 4), block, 0, s, a, tiles);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// router
// ---------------------------------------------------------------------------

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

// Order key of a logit and its expert: keys are distinct, a larger logit has
// the larger key and of equal ones the lower index.  bf16: the bits in signed
// order, then 16 bits of ~index.  fp32: the bits in unsigned order and 20 bits of
// ~index as the mantissa of a double in [1, 2), which has a one-instruction
// maximum.  chunk is for rows without NaN and ranks -0 below +0; make takes
// anything (-0 = +0, NaN above +inf).  inv: ~index, of a chunk's first expert.
template <bool F32>
struct Key;
template <>
struct Key<false> {
    typedef int32_t type;
    static constexpr int32_t kNone = INT32_MIN;
    static __device__ __forceinline__ uint32_t ordered(uint32_t w) {     // both halves; its own inverse
        typedef short s16x2 __attribute__((ext_vector_type(2)));
        const s16x2 sign = __builtin_bit_cast(s16x2, w) >> 15;
        return __builtin_amdgcn_bitop3_b32(__builtin_bit_cast(uint32_t, sign), 0x7FFF7FFFu, w, 0x6A);   // (a & b) ^ c
    }
    static __device__ __forceinline__ void chunk(const Chunk<false, false> &c, uint32_t inv, int32_t key[1]) {
        key[0] = (int32_t)(ordered(c.v) << 16 | inv);
    }
    static __device__ __forceinline__ void chunk(const Chunk<false, true> &c, uint32_t inv, int32_t key[8]) {
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const uint32_t o = ordered(c.w[q]);
            key[2 * q] = (int32_t)(o << 16 | (inv ^ (2 * q)));
            key[2 * q + 1] = (int32_t)((o & 0xFFFF0000u) | (inv ^ (2 * q + 1)));
        }
    }
    static __device__ __forceinline__ int32_t make(float x, uint32_t inv) {
        x += 0.0f;
        const uint32_t o = x != x ? 0x7FFF0000u : ordered(__float_as_uint(x)) & 0xFFFF0000u;
        return (int32_t)(o | inv);
    }
    static __device__ __forceinline__ int32_t hi(int32_t a, int32_t b) { return max(a, b); }
    static __device__ __forceinline__ int32_t lo(int32_t a, int32_t b) { return min(a, b); }
    static __device__ __forceinline__ int32_t flip(int32_t k, uint32_t x) { return (int32_t)((uint32_t)k ^ x); }
    static __device__ __forceinline__ bool open(int32_t k) { return k >= (int32_t)0x80800000u; }   // above -inf
    static __device__ __forceinline__ bool zero(int32_t k) { return (uint32_t)(k + 0x10000) < 0x20000u; }
    static __device__ __forceinline__ int index(int32_t k) { return (int)(~(uint32_t)k & 0xFFFFu); }
    static __device__ __forceinline__ float value(int32_t k) {
        return __uint_as_float(ordered((uint32_t)k) & 0xFFFF0000u);
    }
};
template <>
struct Key<true> {
    typedef double type;
    static constexpr double kNone = 1.0;
    static __device__ __forceinline__ double pack(uint32_t o, uint32_t inv) {
        const uint32_t h = __builtin_amdgcn_alignbit(0x3FFu, o, 12), l = o << 20 | inv;
        return __builtin_bit_cast(double, (uint64_t)h << 32 | l);
    }
    static __device__ __forceinline__ uint32_t ordered(uint32_t u) {
        return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    }
    static __device__ __forceinline__ void chunk(const Chunk<true, false> &c, uint32_t inv, double key[1]) {
        key[0] = pack(ordered(__float_as_uint(c.v)), inv);
    }
    static __device__ __forceinline__ void chunk(const Chunk<true, true> &c, uint32_t inv, double key[4]) {
#pragma unroll
        for (int j = 0; j < 4; j++) key[j] = pack(ordered(__float_as_uint(c.v[j])), inv ^ j);
    }
    static __device__ __forceinline__ double make(float x, uint32_t inv) {
        x += 0.0f;
        return pack(x != x ? 0xFFFFFFFFu : ordered(__float_as_uint(x)), inv);
    }
    // (fmax and fmin would first quiet every operand that they cannot prove to
    // be no signalling NaN)
    static __device__ __forceinline__ double hi(double a, double b) {
        double r;
        asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
        return r;
    }
    static __device__ __forceinline__ double lo(double a, double b) {
        double r;
        asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
        return r;
    }
    static __device__ __forceinline__ double flip(double k, uint32_t x) {
        return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) ^ x);
    }
    static __device__ __forceinline__ uint32_t order(double k) {
        return (uint32_t)(__builtin_bit_cast(uint64_t, k) >> 20);
    }
    static __device__ __forceinline__ bool open(double k) { return order(k) > 0x007FFFFFu; }       // above -inf
    static __device__ __forceinline__ bool zero(double k) { return order(k) - 0x7FFFFFFFu < 2u; }
    static __device__ __forceinline__ int index(double k) {
        return (int)(~(uint32_t)__builtin_bit_cast(uint64_t, k) & 0xFFFFu);
    }
    static __device__ __forceinline__ float value(double k) {
        const uint32_t o = order(k);
        return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
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
template <int G, int D = 1>
__device__ __forceinline__ int32_t group_most(int32_t x) {
    if constexpr (D < G)
        return group_most<G, 2 * D>((int32_t)with_other_half<D>(
            (uint32_t)x, [](uint32_t a, uint32_t b) { return (uint32_t)max((int32_t)a, (int32_t)b); }));
    return x;
}
// of both words of a double, then the larger
template <int G, int D = 1>
__device__ __forceinline__ double group_most(double x) {
    if constexpr (D < G) {
        const uint64_t b = __builtin_bit_cast(uint64_t, x);
        uint32_t own[2] = {(uint32_t)b, (uint32_t)(b >> 32)}, other[2];
#pragma unroll
        for (int i = 0; i < 2; i++)
            with_other_half<D>(own[i], [&](uint32_t p, uint32_t q) {
                own[i] = p;
                other[i] = q;
                return p;
            });
        return group_most<G, 2 * D>(
            Key<true>::hi(__builtin_bit_cast(double, (uint64_t)own[1] << 32 | own[0]),
                          __builtin_bit_cast(double, (uint64_t)other[1] << 32 | other[0])));
    }
    return x;
}

// Falling lists of the KP largest keys.  Sorting: Batcher's odd-even merge
// network; two lists: the larger of a_i and b_(KP-1-i) are the KP largest, a
// bitonic sequence that log2 KP stages sort.
template <bool F32, int KP>
struct Best {
    typedef Key<F32> K;
    typedef typename K::type T;
    static __device__ __forceinline__ void order(T &a, T &b) {
        const T h = K::hi(a, b);
        b = K::lo(a, b);
        a = h;
    }
    static __device__ __forceinline__ void sort(T *v) {
#pragma unroll
        for (int p = 1; p < KP; p *= 2)
#pragma unroll
            for (int q = p; q >= 1; q /= 2)
#pragma unroll
                for (int j = q % p; j + q < KP; j += 2 * q)
#pragma unroll
                    for (int i = 0; i < q; i++)
                        if (i + j + q < KP && (i + j) / (2 * p) == (i + j + q) / (2 * p)) order(v[i + j], v[i + j + q]);
    }
    static __device__ __forceinline__ void settle(T *v) {
#pragma unroll
        for (int d = KP / 2; d >= 1; d /= 2)
#pragma unroll
            for (int i = 0; i < KP; i++)
                if (!(i & d)) order(v[i], v[i | d]);
    }
    // v takes the KP largest of v and w
    static __device__ __forceinline__ void merge(T *v, const T *w) {
#pragma unroll
        for (int i = 0; i < KP; i++) v[i] = K::hi(v[i], w[KP - 1 - i]);
        settle(v);
    }
};

// 1 / x to an ulp for 1 <= x < 2^126; NaN stays NaN
__device__ __forceinline__ float reciprocal(float x) {
    const float r = __builtin_amdgcn_rcpf(x);
    return __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r);
}

// exp(l - m) where m is the row's largest logit, or 0.  The exponent takes one
// fma, whose rounding of m log2 e is the same factor for all of the row and
// cancels in quotients; near the ends of the range m log2 e overflows, and the
// difference comes first.
constexpr float kNearTheEnds = 1e37f;
__device__ __forceinline__ float exponential(float l, float m) {
    const float x = __builtin_fmaf(l, kLog2e, -m * kLog2e), y = (l - m) * kLog2e;
    return __builtin_amdgcn_exp2f(fabsf(m) < kNearTheEnds ? x : y);
}

// e = exp(l - m) of a row and Z = sum e.  Z = 0 only where every logit is -inf;
// NaN or +inf makes Z NaN, and with it all that is divided by it.
template <bool F32, int G, int CH, bool VEC>
__device__ __forceinline__ void exponentials(const Slice<F32, G, CH, VEC> &l, float m, float e[8 * CH], float &Z) {
    float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (__any(!(fabsf(m) < kNearTheEnds))) {
        asm volatile("; extreme logits");        // a branch, not selects
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

// The KP largest keys of a row in falling order: lane g has the ones at g, g + G,
// .. in mine, all lanes the first in most.  Each lane sorts its own KP largest; then
// KP times the largest head of the G lists is taken off its list.  inv: ~index of
// the lane's first expert
template <int KP, bool F32, int G, int CH, bool VEC>
__device__ __forceinline__ void pick(const Slice<F32, G, CH, VEC> &l, uint32_t inv, int g,
                                     typename Key<F32>::type mine[(KP + G - 1) / G], typename Key<F32>::type &most) {
    typedef Key<F32> K;
    typename K::type best[KP];
    typedef Best<F32, KP> B;
    constexpr int W = Slice<F32, G, CH, VEC>::W, U = KP < 8 ? 8 : KP, N = U / W;   // elements and chunks sorted together
#pragma unroll
    for (int i = 0; i < Slice<F32, G, CH, VEC>::N; i += N) {
        typename K::type key[U];
#pragma unroll
        for (int n = 0; n < N; n++) {
            if (i + n < Slice<F32, G, CH, VEC>::N) {
                K::chunk(l.c[i + n], inv, key + W * n);
                if (n > 0)
#pragma unroll
                    for (int j = 0; j < W; j++) key[W * n + j] = K::flip(key[W * n + j], W * G * n);
            } else {
#pragma unroll
                for (int j = 0; j < W; j++) key[W * n + j] = K::kNone;
            }
        }
        B::sort(key);
#pragma unroll
        for (int v = KP; v < U; v += KP) {
            B::sort(key + v);
            B::merge(key, key + v);
        }
        if (i == 0) {
#pragma unroll
            for (int j = 0; j < KP; j++) best[j] = key[j];
        } else {
            // chunk i's indices
#pragma unroll
            for (int j = 0; j < KP; j++) key[j] = K::flip(key[j], W * G * i);
            B::merge(best, key);
        }
    }
    if constexpr (G == 1) {
#pragma unroll
        for (int i = 0; i < KP; i++) mine[i] = best[i];
        most = best[0];
    } else {
#pragma unroll
        for (int s = 0; s < KP; s++) {
            const typename K::type head = group_most<G>(best[0]);
            if (s == 0) most = head;
            if (g == s % G) mine[s / G] = head;
            const bool taken = best[0] == head;
            typename K::type own = best[0];
#pragma unroll
            for (int i = 0; i + 1 < KP - s; i++) {
                typename K::type next = best[i + 1];
                asm("" : "+v"(next));         // a select of values, not of their places in the list
                best[i] = taken ? next : own;
                own = next;
            }
        }
    }
}

// The same one key at a time, for rows with NaN or with zeros of both signs
// among the choices; the largest key is not needed again
template <int KP, bool F32, int G, int CH, bool VEC>
__device__ __forceinline__ void pick_any(const Slice<F32, G, CH, VEC> &l, uint32_t inv, int g, int k,
                                         typename Key<F32>::type mine[(KP + G - 1) / G]) {
    typedef Key<F32> K;
    typename K::type last = K::kNone;
#pragma nounroll
    for (int s = 0; s < k; s++) {
        typename K::type most = K::kNone;
#pragma unroll
        for (int v = 0; v < 8 * CH; v++) {
            const typename K::type key = K::make(l.at(v), inv ^ Slice<F32, G, CH, VEC>::expert(v, 0));
            if (s == 0 || key < last) most = K::hi(most, key);
        }
        last = group_most<G>(most);
#pragma unroll
        for (int i = 0; i < (KP + G - 1) / G; i++)
            if (s == i * G + g) mine[i] = last;
    }
}

template <bool F32, int G, int CH, int KP, bool VEC>
__global__ __launch_bounds__(256, KP == 16 || CH == 4 || !VEC ? 3 : 4) void k_route(RouteArgs a) {
    typedef typename Elem<F32>::type T;
    typedef Key<F32> K;
    typedef typename K::type KT;
    typedef Slice<F32, G, CH, VEC> L;
    constexpr int V = L::V, C = V * G, R = 256 / G;       // per lane; columns; tokens of a block's pass
    constexpr int S = (KP + G - 1) / G;                   // choices of a lane: g, g + G, ..
    __shared__ uint32_t hist[C];
    __shared__ float sums[R * C];
    __shared__ uint32_t routed_of[4];
    const int g = threadIdx.x % G, r = threadIdx.x / G;
    for (int j = threadIdx.x; j < C; j += 256) hist[j] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; v++) acc[v] = 0.0f;
    uint32_t routed = 0;
    const uint32_t inv = 0xFFFFu ^ (uint32_t)L::expert(0, g);
    const int64_t step = (int64_t)gridDim.x * R;
    int64_t t = (int64_t)blockIdx.x * R + r;
    for (int64_t base = (int64_t)blockIdx.x * R; base < a.tokens; base += step, t += step) {
        L l;
        const int64_t at = t < a.tokens ? t : 0;
        l.load(static_cast<const T *>(a.logits) + at * a.stride, g, a.E);
        const bool there = t < a.tokens && (!a.mask || a.mask[at]);
        if (!__all(there) || a.E < C) {
            asm volatile("; logits that do not exist");
            l.keep(there, g, a.E);
        }
        KT mine[S], most;
        pick<KP>(l, inv, g, mine, most);
        const float m = K::open(most) ? K::value(most) : 0.0f;
        float e[V], Z;
        exponentials(l, m, e, Z);
        bool odd = Z != Z;
#pragma unroll
        for (int s = 0; s < S; s++) odd = odd || (s * G + g < KP && K::zero(mine[s]));
        if (__any(odd)) {
            uint32_t start = inv;
            asm volatile("; NaN, or zeros that may tie" : "+v"(start));   // (opaque: no constants of it are kept)
            pick_any<KP>(l, start, g, a.k, mine);
        }
        const float by_z = Z == 0.0f ? 0.0f : reciprocal(Z);
        if (g == 0) routed += Z != 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++) acc[v] = __builtin_fmaf(e[v], by_z, acc[v]);

        float ge[S], top = 0.0f;
        int id[S];
#pragma unroll
        for (int s = 0; s < S; s++) {
            const bool open = s * G + g < a.k && K::open(mine[s]);
            id[s] = open ? K::index(mine[s]) : -1;
            ge[s] = open ? exponential(K::value(mine[s]), m) : 0.0f;
            top += ge[s];
        }
        // a choice is the row's largest logit, so that the sum is 1 or more
        const float by = Z != Z ? Z : Z == 0.0f ? 0.0f : a.renorm ? reciprocal(group_sum<G>(top)) : by_z;
#pragma unroll
        for (int s = 0; s < S; s++) {
            if (s * G + g < a.k && t < a.tokens) {
                a.ids[t * a.k + s * G + g] = id[s];
                a.gates[t * a.k + s * G + g] = id[s] < 0 ? 0.0f : ge[s] * by;
                if (id[s] >= 0) atomicAdd(&hist[id[s]], 1u);
            }
        }
    }
    // the block's sums: token rows side by side in LDS, then over the rows
#pragma unroll
    for (int v = 0; v < V; v++) sums[r * C + L::expert(v, g)] = acc[v];
    for (int d = 32; d; d >>= 1) routed += __shfl_xor((int)routed, d, 64);
    if ((threadIdx.x & 63) == 0) routed_of[threadIdx.x >> 6] = routed;
    __syncthreads();
    constexpr int P = C < 256 ? 256 / C : 1;            // threads per column
    for (int j = threadIdx.x; j < C * P; j += 256) {
        const int col = j % C, part = j / C;
        float sum = 0.0f;
        for (int i = part; i < R; i += P) sum += sums[i * C + col];
        if (P > 1) {
            __syncthreads();
            sums[part * C + col] = sum;
            __syncthreads();
            if (part != 0) break;
            for (int i = 1; i < P; i++) sum += sums[i * C + col];
        }
        if (col < a.E) {
            a.part.psum[(int)blockIdx.x * a.E + col] = sum;
            a.part.count[(int)blockIdx.x * a.E + col] = hist[col];
        }
    }
    if (threadIdx.x == 0) {
        a.part.routed[blockIdx.x] = routed_of[0] + routed_of[1] + routed_of[2] + routed_of[3];
        if (blockIdx.x == 0) *a.part.done = 0;
    }
}

__device__ __forceinline__ double wave_sum(double v, int from = 32) {
    for (int d = from; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// Folds the parts and computes the loss, every sum in a fixed order.  A block
// of 16 waves takes 16 experts, 64 threads for each over the rows; where there
// are few rows one block takes all experts, a thread each.  The last of several
// blocks to finish adds up their shares of the loss.
template <bool ONE>
__global__ __launch_bounds__(1024) void k_balance(BalanceArgs a) {
    constexpr int COLUMNS = ONE ? kRouteMaxExperts : kBalanceColumns;
    __shared__ double ps[16][16], cs[16][16], ts[16];
    const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
    const int j = ONE ? i : (int)blockIdx.x * COLUMNS + i % COLUMNS;
    const double sum_n = a.sums ? a.sums[2 * a.E] : 0.0;
    double p = 0.0, n = 0.0, t = 0.0;
    // rows in groups of U whose loads are all in flight before the first is added
    constexpr int STEP = ONE ? 1 : 1024 / COLUMNS, U = 12;
    const int col = j < a.E ? j : 0;
    for (int q = 0; q < a.parts; q++) {
        const RoutePart &part = a.part[q];
        const int rows = part.nblk;
        for (int b0 = ONE ? 0 : i / COLUMNS; b0 < rows; b0 += U * STEP) {
            float x[U];
            uint32_t m[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int at = min(b0 + u * STEP, rows - 1) * a.E + col;
                x[u] = part.psum[at];
                m[u] = part.count[at];
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                const bool there = b0 + u * STEP < rows;
                p += there ? x[u] : 0.0f;
                n += there ? m[u] : 0u;
            }
        }
        for (int b = i; b < rows; b += 1024) t += part.routed[b];
    }
    t = wave_sum(t);
    if (!ONE) {
        p += __shfl_xor(p, 32, 64);
        p += __shfl_xor(p, 16, 64);
        n += __shfl_xor(n, 32, 64);
        n += __shfl_xor(n, 16, 64);
        if (lane < 16) {
            ps[wave][lane] = p;
            cs[wave][lane] = n;
        }
    }
    if (lane == 0) ts[wave] = t;
    __syncthreads();
    if (!ONE && wave != 0) return;
    double N = sum_n;
    for (int w = 0; w < 16; w++) N += ts[w];
    if (!ONE) {
        // lane c adds up the waves w, w + 4, .. with w = c / 16
        p = n = 0.0;
        for (int w = lane / 16; w < 16; w += 4) {
            p += ps[w][lane % 16];
            n += cs[w][lane % 16];
        }
        p += __shfl_xor(p, 32, 64);
        p += __shfl_xor(p, 16, 64);
        n += __shfl_xor(n, 32, 64);
        n += __shfl_xor(n, 16, 64);
    }
    const double f = N > 0.0 ? (double)a.E / ((double)a.k * N * N) : 0.0;
    double share = 0.0;
    if ((ONE || lane < 16) && j < a.E) {
        if (a.sums) {
            n += a.sums[j];
            p += a.sums[a.E + j];
        }
        if (a.stats) {
            a.stats[j] = n;
            a.stats[a.E + j] = p;
        }
        const double w = f * n;
        if (a.coef) a.coef[j] = (float)w;
        if (a.counts) a.counts[j] = (int64_t)n;
        share = w * p;
    }
    share = wave_sum(share, ONE ? 32 : 8);
    if (ONE) {
        if (lane == 0) ps[0][wave] = share;
        __syncthreads();
        share = 0.0;
        for (int w = 0; w < 16; w++) share += ps[0][w];
    } else if (gridDim.x > 1) {
        const RoutePart &first = a.part[0];
        uint32_t before = 0;
        if (lane == 0) {
            __hip_atomic_store(first.share + blockIdx.x, share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            before = __hip_atomic_fetch_add(first.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        }
        if (__builtin_amdgcn_readfirstlane(before) != gridDim.x - 1) return;
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        share = lane < (int)gridDim.x ? __hip_atomic_load(first.share + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                                      : 0.0;
        share = wave_sum(share);
        if (lane == 0) *first.done = 0;
    }
    // a.stats may be a.sums, whose last element every block reads
    if (i == 0) {
        if (a.loss) *a.loss = (float)share;
        if (a.stats) a.stats[2 * a.E] = N;
    }
}

// LDS traffic between the lanes of one wave: orders it for the compiler too
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The gradient of a row is p_j (a_j - D) + h_j, where h is 0 but for the chosen
// experts: the lanes that hold the choices scatter it into a row of LDS, which is 0
// between rows.  A row is read and written once; its choices are read a row
// ahead, so that their logits are on the way while the softmax is computed.
template <bool F32, int G, int CH, int S, bool VEC>
__global__ __launch_bounds__(256) void k_route_backward(RouteBackwardArgs a) {
    typedef Elem<F32> El;
    typedef typename El::type T;
    typedef Slice<F32, G, CH, VEC> L;
    constexpr int V = L::V, W = L::W, C = V * G, R = 256 / G;
    __shared__ alignas(16) float rows[R * C];
    const int g = threadIdx.x % G, r = threadIdx.x / G;
    float *h = rows + r * C;
    const T *logits = static_cast<const T *>(a.logits);
    struct Row {
        L l;
        int id[S];
        float dg[S];
        uint8_t mask;
    };
    // lane g holds choices g, g + G, ..; nothing waits for these loads
    const auto load = [&](Row &row, int64_t t) {
        if (t >= a.tokens) t = 0;
        row.l.load(logits + t * a.stride, g, a.E);
        row.mask = 1;
        if (a.mask) row.mask = a.mask[t];
#pragma unroll
        for (int s = 0; s < S; s++) {
            const int64_t at = t * a.k + (s * G + g < a.k ? s * G + g : 0);
            row.id[s] = -1;
            row.dg[s] = 0.0f;
            if (a.dgates) {
                row.id[s] = a.ids[at];
                row.dg[s] = a.dgates[at];
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * R;
    int64_t t = (int64_t)blockIdx.x * R + r;
    Row next;
    load(next, t);
    // dloss coef of the lane's experts; loads of all of them in flight at once
    float up[V];
    const float w = a.coef ? (a.dloss ? *a.dloss : 1.0f) : 0.0f;
    if (VEC && a.coef && reinterpret_cast<uintptr_t>(a.coef) % 16 == 0) {
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const int at = L::expert(v, g);
            const float4 x = *reinterpret_cast<const float4 *>(a.coef + (at < a.E ? at : 0));
            up[v] = x.x;
            up[v + 1] = x.y;
            up[v + 2] = x.z;
            up[v + 3] = x.w;
        }
    } else if (a.coef) {
#pragma unroll
        for (int v = 0; v < V; v++) up[v] = a.coef[min(L::expert(v, g), a.E - 1)];
    } else {
#pragma unroll
        for (int v = 0; v < V; v++) up[v] = 0.0f;
    }
#pragma unroll
    for (int v = 0; v < V; v++) up[v] *= w;
#pragma unroll
    for (int v = 0; v < V; v += 4)
        *reinterpret_cast<float4 *>(__builtin_assume_aligned(h + 4 * g + v * G, 16)) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    wave_lds_sync();
    for (int64_t base = (int64_t)blockIdx.x * R; base < a.tokens; base += step, t += step) {
        Row row = next;
        const bool there = t < a.tokens && row.mask;
        typename El::type ls[S];
#pragma unroll
        for (int s = 0; s < S; s++) {
            if (!there || s * G + g >= a.k || (uint32_t)row.id[s] >= (uint32_t)a.E) row.id[s] = -1;
            ls[s] = logits[(there ? t : 0) * a.stride + (row.id[s] < 0 ? 0 : row.id[s])];
        }
        load(next, t + step);
        row.l.keep(there, g, a.E);
        float m = -INFINITY, e[V], Z;
#pragma unroll
        for (int v = 0; v < V; v++) m = fmaxf(m, row.l.at(v));
        m = group_max<G>(m);
        if (m == -INFINITY) m = 0.0f;
        exponentials(row.l, m, e, Z);
        const float inv = Z == 0.0f ? 0.0f : reciprocal(Z);
        float dots[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; v++) dots[v % 4] = __builtin_fmaf(e[v], up[v], dots[v % 4]);
        float gs[S], top = 0.0f, gd = 0.0f;
#pragma unroll
        for (int s = 0; s < S; s++) {
            gs[s] = row.id[s] >= 0 ? exponential(El::up(ls[s]), m) : 0.0f;
            top += gs[s];
        }
        float by = inv;
        if (a.renorm) {
            top = group_sum<G>(top);
            by = top == 0.0f ? 0.0f : 1.0f / top;      // no choice
        }
#pragma unroll
        for (int s = 0; s < S; s++) {
            gs[s] *= by;
            if (row.id[s] >= 0) gd = __builtin_fmaf(gs[s], row.dg[s], gd);
        }
        gd = group_sum<G>(gd);
        // p (a - D) = e (a / Z - D / Z)
        float dot = inv * group_sum<G>((dots[0] + dots[1]) + (dots[2] + dots[3]));
        dot = -inv * (dot + (a.renorm ? 0.0f : gd));
#pragma unroll
        for (int s = 0; s < S; s++)
            if (row.id[s] >= 0) h[row.id[s]] = gs[s] * (a.renorm ? row.dg[s] - gd : row.dg[s]);
        wave_lds_sync();
        // the next row is waited for here: after the stores below it would be
        // waited for together with them
        next.l.arrived();
#pragma unroll
        for (int s = 0; s < S; s++) asm volatile("" : "+v"(next.id[s]), "+v"(next.dg[s]));
        if (t < a.tokens) {
            T *out = static_cast<T *>(a.dlogits) + t * a.dstride;
#pragma unroll
            for (int i = 0; i < L::N; i++) {
                const int at = L::expert(W * i, g);
                float d[W];
                __builtin_memcpy(d, __builtin_assume_aligned(h + at, W < 4 ? 4 : 16), sizeof d);
#pragma unroll
                for (int j = 0; j < W; j++)
                    d[j] = __builtin_fmaf(e[W * i + j], __builtin_fmaf(up[W * i + j], inv, dot), d[j]);
                if (at < a.E) L::C::store(out + at, d);
            }
        }
        wave_lds_sync();
#pragma unroll
        for (int s = 0; s < S; s++)
            if (row.id[s] >= 0) h[row.id[s]] = 0.0f;
    }
}

template <bool F32, int G, int CH, bool VEC>
hipError_t route_choices(const RouteArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.part.nblk), block(256);
    if (a.k <= 2) hipLaunchKernelGGL((k_route<F32, G, CH, 2, VEC>), grid, block, 0, s, a);
    else if (a.k <= 4) hipLaunchKernelGGL((k_route<F32, G, CH, 4, VEC>), grid, block, 0, s, a);
    else if (a.k <= 8 || G * CH == 1) hipLaunchKernelGGL((k_route<F32, G, CH, 8, VEC>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_route<F32, G, CH, G * CH == 1 ? 8 : 16, VEC>), grid, block, 0, s, a);
    return hipGetLastError();
}

// Lanes and chunks of a token of E experts: f(G, CH)
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
constexpr int64_t kManyTokens = 32768;
// The same with longer lists in fewer lanes, for E > 128: fewer steps across
// lanes per token, but half as many waves
template <class F>
auto by_experts_long(int E, F f) {
    if (E <= 256) return shape<8, 4>(f);
    if (E <= 512) return shape<16, 4>(f);
    return shape<32, 4>(f);
}

bool rows_on_16(const void *p, int64_t stride, int E, bool f32) {
    return E % (f32 ? 4 : 8) == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * (f32 ? 4 : 2) % 16 == 0;
}

template <bool F32>
hipError_t route_experts(const RouteArgs &a, hipStream_t s) {
    const bool vec = rows_on_16(a.logits, a.stride, a.E, F32);
    if constexpr (!F32)
        if (vec && a.E > 128 && a.tokens >= kManyTokens)
            return by_experts_long(a.E, [&](auto G, auto CH) { return route_choices<F32, G.value, CH.value, true>(a, s); });
    return by_experts(a.E, [&](auto G, auto CH) {
        return vec ? route_choices<F32, G.value, CH.value, true>(a, s)
                   : route_choices<F32, G.value, CH.value, false>(a, s);
    });
}

template <bool F32, int G, int CH, bool VEC>
hipError_t backward_choices(const RouteBackwardArgs &a, hipStream_t s) {
    // choices of a lane: at most all of 8 experts in one lane
    constexpr int R = 256 / G, most = G == 1 ? 8 : G < kRouteMaxTopK ? kRouteMaxTopK / G : 1;
    static_assert(G > 1 || CH == 1, "");
    const int64_t want = (a.tokens + R - 1) / R;
    const dim3 grid((unsigned)(want < 1024 ? want : 1024)), block(256);
    const int each = (a.k + G - 1) / G;
    if (each <= 1 || most == 1) hipLaunchKernelGGL((k_route_backward<F32, G, CH, 1, VEC>), grid, block, 0, s, a);
    else if (each <= 2 || most == 2)
        hipLaunchKernelGGL((k_route_backward<F32, G, CH, most < 2 ? most : 2, VEC>), grid, block, 0, s, a);
    else if (each <= 4 || most == 4)
        hipLaunchKernelGGL((k_route_backward<F32, G, CH, most < 4 ? most : 4, VEC>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_route_backward<F32, G, CH, most, VEC>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <bool F32>
hipError_t backward_experts(const RouteBackwardArgs &a, hipStream_t s) {
    const bool vec = rows_on_16(a.logits, a.stride, a.E, F32) && rows_on_16(a.dlogits, a.dstride, a.E, F32);
    return by_experts(a.E, [&](auto G, auto CH) {
        return vec ? backward_choices<F32, G.value, CH.value, true>(a, s)
                   : backward_choices<F32, G.value, CH.value, false>(a, s);
    });
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs &a, int f32, hipStream_t s) {
    if (f32) return a.residual ? dropout_access<true, true>(a, s) : dropout_access<true, false>(a, s);
    return a.residual ? dropout_access<false, true>(a, s) : dropout_access<false, false>(a, s);
}

int route_blocks(int64_t tokens, int E) {
    // at most what the chip holds at once
    const int64_t rows = by_experts(E, [](auto G, auto) { return 256 / G.value; });
    const int64_t most = by_experts(E, [](auto, auto CH) { return 256 * (CH.value == 1 ? 6 : 4); });
    const int64_t want = (tokens + rows - 1) / rows;
    return (int)(want < 1 ? 1 : want < most ? want : most);
}

hipError_t launch_route(const RouteArgs &a, int f32, hipStream_t s) {
    return f32 ? route_experts<true>(a, s) : route_experts<false>(a, s);
}

hipError_t launch_balance(const BalanceArgs &a, hipStream_t s) {
    static_assert(kRouteMaxExperts / kBalanceColumns <= 64, "a wave adds up the blocks' shares");
    int64_t rows = 0;
    for (int q = 0; q < a.parts; q++) rows += a.part[q].nblk;
    if (rows <= kBalanceFewRows)
        hipLaunchKernelGGL(k_balance<true>, dim3(1), dim3(1024), 0, s, a);
    else
        hipLaunchKernelGGL(k_balance<false>, dim3((unsigned)((a.E + kBalanceColumns - 1) / kBalanceColumns)), dim3(1024),
                           0, s, a);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs &a, int f32, hipStream_t s) {
    return f32 ? backward_experts<true>(a, s) : backward_experts<false>(a, s);
}

}  // namespace dq
