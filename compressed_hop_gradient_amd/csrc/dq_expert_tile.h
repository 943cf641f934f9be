// dq_expert_tile.h -- tiles of the products grouped by expert (device code): how an
// operand comes into LDS, the inner loop, and the accumulators' way out.
#pragma once

#include <type_traits>

#include "dq_experts.h"
#include "dq_train_device.h"

namespace dq {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

#define DQ_LDS(p) ((__attribute__((address_space(3))) void *)(p))
#define DQ_GLOBAL(p) ((const __attribute__((address_space(1))) void *)(p))

// What is read in the place of what is not there.
__device__ const __align__(16) uint32_t kZeros[4] = {0, 0, 0, 0};

// A block's tile is BM x BN, its inner step BK elements (128 bytes); its waves are
// WM x WN, each with (BM / WM) x (BN / WN) in accumulators of 16 x 16.
template <typename Element, int BM_, int BN_, int WM_, int WN_>
struct Tiling {
    typedef Element T;
    static constexpr bool kF32 = sizeof(T) == 4;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = 128 / (int)sizeof(T);
    static constexpr int kThreads = 64 * WM * WN, kChunk = 16 / (int)sizeof(T);
    static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    static constexpr int kBytesA = BM * 128, kBytesB = BN * 128;
    static constexpr int kStages = 2, kLds = kStages * (kBytesA + kBytesB);
};
typedef Tiling<uint16_t, 128, 128, 2, 2> TileMid;
typedef Tiling<float, 128, 128, 2, 2> TileF32;

// How an operand is loaded: 16 bytes at a time straight into LDS; element by
// element through registers; from 8-bit codes, 16 at a time or one by one.
constexpr int kAsync = 0, kAny = 1, kKept = 2, kKeptAny = 3;

// First row of expert e: the offsets, held to the rows there are and in order (an
// offset below the one before it makes that expert empty).
__device__ __forceinline__ int expert_first(const ExpertLists &l, int e) { return clampi(l.offsets[e], 0, l.slots); }

// The token of a row; -1 where the lists hold none.
__device__ __forceinline__ int64_t token_of(const ExpertLists &l, int row) {
    const uint32_t slot = (uint32_t)l.source[row];
    return slot < (uint32_t)l.slots ? (int64_t)(slot / (uint32_t)l.k) : -1;
}

// Where an operand's row starts: the row itself or, gathered, its token; below 0: nowhere.
__device__ __forceinline__ int64_t row_at(const ExpertLists &l, int row, int gather, int64_t stride) {
    if (!gather) return (int64_t)row * stride;
    const int64_t t = token_of(l, row);
    return t < 0 ? -1 : t * stride;
}

// Blocks come to the eight XCDs in turn; each XCD gets a run of neighbouring tiles,
// which share operands in its L2.
__device__ __forceinline__ int64_t own_tile(int64_t block, int64_t total) {
    const int64_t run = (total + 7) / 8, at = block / 8;
    return at < run ? block % 8 * run + at : total;
}

struct RowTile {
    int e, first, rows, n;
};

// The block's tile among the experts' ragged rows: expert by expert, column of
// tiles by column.  All threads call it; false: nothing left for this block.
template <int THREADS>
__device__ __forceinline__ bool find_tile(const ExpertLists &l, int bm, int nt, RowTile &t, int *sh) {
    constexpr int kWaves = THREADS / 64, kPer = (kExpertsMost + THREADS - 1) / THREADS;
    const int tid = threadIdx.x, per = (l.E + THREADS - 1) / THREADS;
    int first[kPer], rows[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int e = tid * per + i;
        rows[i] = 0;
        if (i < per && e < l.E) {
            first[i] = expert_first(l, e);
            rows[i] = expert_first(l, e + 1) - first[i];
            if (rows[i] > 0) sum += (rows[i] + bm - 1) / bm;
        }
    }
    int upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(upto, d, 64);
        if ((tid & 63) >= d) upto += o;
    }
    if ((tid & 63) == 63) sh[tid >> 6] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        if (w < tid >> 6) upto += sh[w];
        total += sh[w];
    }
    const int64_t tiles = (int64_t)total * nt, id = own_tile(blockIdx.x, tiles);
    if (id >= tiles) return false;
    int64_t at = (int64_t)(upto - sum) * nt;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        if (rows[i] <= 0) continue;
        const int mt = (rows[i] + bm - 1) / bm;
        const int64_t in = id - at;
        if (in >= 0 && in < (int64_t)mt * nt) {
            const int n = (int)(in / mt), m = (int)in - n * mt;
            sh[kWaves] = tid * per + i;
            sh[kWaves + 1] = first[i] + m * bm;
            sh[kWaves + 2] = rows[i] - m * bm;
            sh[kWaves + 3] = n;
        }
        at += (int64_t)mt * nt;
    }
    __syncthreads();
    t.e = __builtin_amdgcn_readfirstlane(sh[kWaves]);
    t.first = __builtin_amdgcn_readfirstlane(sh[kWaves + 1]);
    t.rows = __builtin_amdgcn_readfirstlane(sh[kWaves + 2]);
    t.n = __builtin_amdgcn_readfirstlane(sh[kWaves + 3]);
    __syncthreads();
    return true;
}

// kChunk elements from p, those below `have` (of which there may be none).
template <typename T>
__device__ __forceinline__ u32x4 load_some(const T *p, int have) {
    u32x4 v = {0, 0, 0, 0};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < have) v[j / 2] |= (uint32_t)p[j] << 16 * (j & 1);
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (j < have) v[j] = __float_as_uint(p[j]);
    }
    return v;
}

__device__ __forceinline__ void to_lds(const void *from, char *wave_base) {
    __builtin_amdgcn_global_load_lds(DQ_GLOBAL(from), DQ_LDS(wave_base), 16, 0, 0);
}

// An operand whose rows (the tile's M or N) are contiguous along the inner index.
// In LDS a row is 128 bytes, its chunk c at place c ^ (row & 7), so that the
// 16 rows of a matrix operand are read without bank conflicts.
template <class C, int ROWS, int L>
struct Along {
    typedef typename C::T T;
    static constexpr int kBytes = ROWS * 128, kPer = ROWS * 8 / C::kThreads;
    static_assert(ROWS * 8 % C::kThreads == 0 && C::kThreads % 64 == 0, "whole chunks");
    const T *p[kPer];
    int K, kc;
    u32x4 v[L == kAsync ? 1 : kPer];

    template <class Row>
    __device__ __forceinline__ void start(const T *base, int inner, Row row) {
        K = inner;
        const int r0 = threadIdx.x >> 3;
        kc = ((threadIdx.x & 7) ^ (r0 & 7)) * C::kChunk;
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const int64_t at = row(r0 + i * (C::kThreads / 8));
            p[i] = at < 0 ? nullptr : base + at + kc;
        }
    }
    template <class Row>
    __device__ __forceinline__ void ahead(int, Row) {}
    __device__ __forceinline__ void issue(char *buf, int k0) {
        const int have = K - k0 - kc;
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const bool there = p[i] != nullptr && have > 0;
            if constexpr (L == kAsync) {
                const void *from = there ? static_cast<const void *>(p[i] + k0) : kZeros;
                to_lds(from, buf + ((threadIdx.x & ~63) + i * C::kThreads) * 16);
            } else {
                v[i] = load_some(p[i] + k0, there ? have : 0);
            }
        }
    }
    __device__ __forceinline__ void commit(char *buf) {
        if constexpr (L != kAsync)
#pragma unroll
            for (int i = 0; i < kPer; i++)
                *reinterpret_cast<u32x4 *>(buf + (threadIdx.x + i * C::kThreads) * 16) = v[i];
    }
    // rows row0 .. row0 + 15, half h of the step: lane l has row l & 15, chunk (l >> 4) + 4 h
    static __device__ __forceinline__ u32x4 frag(const char *buf, int row0, int h) {
        const int lane = threadIdx.x & 63, row = row0 + (lane & 15);
        return *reinterpret_cast<const u32x4 *>(buf + row * 128 + (((lane >> 4) + 4 * h) ^ (lane & 7)) * 16);
    }
};

// An operand whose inner index runs down its rows, each contiguous along M or N.  In
// LDS as it lies in memory, BK rows of COLS elements, with units of 16 elements
// exchanged within a row: bf16 is turned by the transposing LDS read, where 16 lanes
// take 4 rows of 32 bytes, fp32 read by elements, where the wave takes 4 rows.
template <class C, int COLS, int L>
struct Across {
    typedef typename C::T T;
    static constexpr int kRow = COLS * (int)sizeof(T), kBytes = C::BK * kRow, kUnits = COLS / 16;
    static constexpr bool kFromKept = L == kKept || L == kKeptAny;
    static constexpr int kPieces = kFromKept ? C::BK * kUnits : kBytes / 16;
    static constexpr int kPer = kPieces / C::kThreads, kPerRow = kPieces / C::BK;
    static_assert(kPieces % C::kThreads == 0 && kUnits % 4 == 0, "whole pieces");
    const T *base;
    const int8_t *codes;
    const uint8_t *exponents;
    int64_t off[kPer];
    int K, N, col0;
    u32x4 v[L == kAsync ? 1 : kPer];
    uint8_t ex[kFromKept ? kPer : 1];

    static __device__ __forceinline__ int swap(int k) {
        if constexpr (C::kF32) return k >> 2 & 3;
        if constexpr (kUnits % 8 == 0) return (k & 3) | (k >> 1 & 4);
        return k & 3;
    }
    __device__ __forceinline__ void start(const T *b, int c0, int cols, int inner) {
        base = b;
        col0 = c0;
        N = cols;
        K = inner;
    }
    __device__ __forceinline__ void start(const int8_t *c, const uint8_t *e, int c0, int cols, int inner) {
        codes = c;
        exponents = e;
        col0 = c0;
        N = cols;
        K = inner;
    }
    static __device__ __forceinline__ int piece_row(int i) { return (threadIdx.x + i * C::kThreads) / kPerRow; }
    __device__ __forceinline__ int piece_col(int i) const {
        const int at = (threadIdx.x + i * C::kThreads) % kPerRow;
        if (kFromKept) return col0 + 16 * at;
        constexpr int kUnit = 16 / C::kChunk;
        return col0 + ((at / kUnit ^ swap(piece_row(i))) * kUnit + at % kUnit) * C::kChunk;
    }
    // where the rows of the step at k0 lie (its lists are read a step ahead)
    template <class Row>
    __device__ __forceinline__ void ahead(int k0, Row row) {
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const int k = k0 + piece_row(i);
            off[i] = k < K ? row(k) : -1;
        }
    }
    __device__ __forceinline__ void issue(char *buf, int) {
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const int col = piece_col(i);
            const bool there = off[i] >= 0 && col < N;
            if constexpr (L == kAsync) {
                const void *from = there ? static_cast<const void *>(base + off[i] + col) : kZeros;
                to_lds(from, buf + ((threadIdx.x & ~63) + i * C::kThreads) * 16);
            } else if constexpr (L == kAny) {
                v[i] = load_some(base + off[i] + col, there ? N - col : 0);
            } else {
                v[i] = u32x4{0, 0, 0, 0};
                ex[i] = 127;
                if (there) {
                    ex[i] = exponents[off[i] * ((N + 31) / 32) + col / 32];
                    const int8_t *c = codes + off[i] * N + col;
                    if constexpr (L == kKept) {
                        v[i] = *reinterpret_cast<const u32x4 *>(c);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; j++)
                            if (col + j < N) v[i][j / 4] |= (uint32_t)(uint8_t)c[j] << 8 * (j & 3);
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void commit(char *buf) {
        if constexpr (L == kAny) {
#pragma unroll
            for (int i = 0; i < kPer; i++)
                *reinterpret_cast<u32x4 *>(buf + (threadIdx.x + i * C::kThreads) * 16) = v[i];
        } else if constexpr (kFromKept) {
#pragma unroll
            for (int i = 0; i < kPer; i++) {
                const int k = piece_row(i), unit = (threadIdx.x + i * C::kThreads) % kPerRow;
                u32x4 *to = reinterpret_cast<u32x4 *>(buf + k * kRow + (unit ^ swap(k)) * 16 * sizeof(T));
                const float scale = __uint_as_float((uint32_t)ex[i] << 23);
                float f[16];
#pragma unroll
                for (int j = 0; j < 16; j++) f[j] = (float)(int8_t)(v[i][j / 4] >> 8 * (j & 3)) * scale;
                if constexpr (C::kF32) {
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        to[j] = u32x4{__float_as_uint(f[4 * j]), __float_as_uint(f[4 * j + 1]),
                                      __float_as_uint(f[4 * j + 2]), __float_as_uint(f[4 * j + 3])};
                } else {
                    // 7 bits and a power of two: exact in bf16
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        u32x4 o;
#pragma unroll
                        for (int q = 0; q < 4; q++)
                            o[q] = bf16_bits(f[8 * j + 2 * q]) | bf16_bits(f[8 * j + 2 * q + 1]) << 16;
                        to[j] = o;
                    }
                }
            }
        }
    }
    // columns col .. col + 15, half h of the step, as Along::frag
    static __device__ __forceinline__ u32x4 frag(const char *buf, int col, int h) {
        const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
        u32x4 o;
        if constexpr (C::kF32) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int k = 4 * (g + 4 * h) + j;
                o[j] = *reinterpret_cast<const uint32_t *>(buf + k * kRow + ((col >> 4 ^ swap(k)) * 16 + i) * 4);
            }
        } else {
            // lane i of 16 names row i >> 2, elements 4 (i & 3) .., and gets column i
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int k = 32 * h + 8 * g + 4 * j + (i >> 2);
                const char *p = buf + k * kRow + (col >> 4 ^ swap(k)) * 32 + (i & 3) * 8;
                const s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4 *)DQ_LDS(const_cast<char *>(p)));
                const uint64_t q = __builtin_bit_cast(uint64_t, r);
                o[2 * j] = (uint32_t)q;
                o[2 * j + 1] = (uint32_t)(q >> 32);
            }
        }
        return o;
    }
};

__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_one(uint16_t *p, float v) { *p = (uint16_t)bf16_bits(v); }
__device__ __forceinline__ void store_four(float *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }
__device__ __forceinline__ void store_four(uint16_t *p, f32x4 v) {
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(bf16_bits(v[0]) | bf16_bits(v[1]) << 16, bf16_bits(v[2]) | bf16_bits(v[3]) << 16);
}

// Whether four neighbouring outputs can be stored together.
template <typename Out>
__device__ __forceinline__ bool vec_out(const void *p, int64_t stride, int n) {
    return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(Out)) == 0 && stride % 4 == 0 && n % 4 == 0;
}

// fp32 accumulators of a wave.  The products are taken turned (B first), so that a
// lane holds four neighbouring columns of one row.
template <class C>
struct Acc {
    f32x4 v[C::TM][C::TN];
    __device__ __forceinline__ Acc() {
#pragma unroll
        for (int i = 0; i < C::TM; i++)
#pragma unroll
            for (int j = 0; j < C::TN; j++) v[i][j] = f32x4{0, 0, 0, 0};
    }
    static __device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
    static __device__ __forceinline__ int m0() { return wave() / C::WN * (C::BM / C::WM); }
    static __device__ __forceinline__ int n0() { return wave() % C::WN * (C::BN / C::WN); }

    template <class A, class B>
    __device__ __forceinline__ void step(const char *a, const char *b) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            u32x4 fa[C::TM], fb[C::TN];
#pragma unroll
            for (int j = 0; j < C::TN; j++) fb[j] = B::frag(b, n0() + 16 * j, h);
#pragma unroll
            for (int i = 0; i < C::TM; i++) fa[i] = A::frag(a, m0() + 16 * i, h);
#pragma unroll
            for (int i = 0; i < C::TM; i++)
#pragma unroll
                for (int j = 0; j < C::TN; j++) {
                    if constexpr (C::kF32) {
#pragma unroll
                        for (int q = 0; q < 4; q++)
                            v[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                __uint_as_float(fb[j][q]), __uint_as_float(fa[i][q]), v[i][j], 0, 0, 0);
                    } else {
                        v[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb[j]),
                                                                         __builtin_bit_cast(bf16x8, fa[i]), v[i][j],
                                                                         0, 0, 0);
                    }
                }
        }
    }
    // row(m): where the tile's row m goes, NULL: nowhere
    template <class Row>
    __device__ __forceinline__ void store(Row row, int col0, int N, bool four) const {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < C::TM; i++) {
            auto *p = row(m0() + 16 * i + (lane & 15));
            if (!p) continue;
#pragma unroll
            for (int j = 0; j < C::TN; j++) {
                const int n = col0 + n0() + 16 * j + (lane >> 4) * 4;
                if (four && n < N) {
                    store_four(p + n, v[i][j]);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        if (n + q < N) store_one(p + n + q, v[i][j][q]);
                }
            }
        }
    }
};

// LDS filled by every wave, its old contents read by every wave.
__device__ __forceinline__ void step_done() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// acc += A B over `inner`, two steps in LDS: one is loaded while the other is used.
template <class C, class A, class B, class RowA, class RowB>
__device__ __forceinline__ void multiply(char *lds, A &a, B &b, int inner, RowA row_a, RowB row_b, Acc<C> &acc) {
    constexpr int kStep = C::kBytesA + C::kBytesB;
    if (inner <= 0) return;
    const int steps = (inner + C::BK - 1) / C::BK;
    a.ahead(0, row_a);
    b.ahead(0, row_b);
    a.issue(lds, 0);
    b.issue(lds + C::kBytesA, 0);
    a.ahead(C::BK, row_a);
    b.ahead(C::BK, row_b);
    a.commit(lds);
    b.commit(lds + C::kBytesA);
    step_done();
    for (int t = 0; t < steps; t++) {
        char *now = lds + (t & 1) * kStep, *next = lds + (~t & 1) * kStep;
        const bool more = t + 1 < steps;
        if (more) {
            a.issue(next, (t + 1) * C::BK);
            b.issue(next + C::kBytesA, (t + 1) * C::BK);
            a.ahead((t + 2) * C::BK, row_a);
            b.ahead((t + 2) * C::BK, row_b);
        }
        acc.template step<A, B>(now, now + C::kBytesA);
        if (more) {
            a.commit(next);
            b.commit(next + C::kBytesA);
        }
        step_done();
    }
}

template <class K>
hipError_t room_for(K kernel, int lds) {
    if (lds <= 65536) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
}

bool on16(const void *p, int64_t stride_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0;
}

}  // namespace
}  // namespace dq
