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

// A block's tile is BM x BN, its inner step BK elements (64 bytes or 128 of a row);
// its waves are WM x WN, each with (BM / WM) x (BN / WN) in accumulators of 16 x 16.
// kStages steps lie in LDS.
template <typename Element, int BM_, int BN_, int WM_, int WN_, int ROW_, int STAGES_>
struct Tiling {
    typedef Element T;
    static constexpr bool kF32 = sizeof(T) == 4;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, kRow = ROW_, BK = kRow / (int)sizeof(T);
    static constexpr int kThreads = 64 * WM * WN, kChunk = 16 / (int)sizeof(T);
    static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    static constexpr int kBytesA = BM * kRow, kBytesB = BN * kRow;
    static constexpr int kStages = STAGES_, kLds = kStages * (kBytesA + kBytesB);
    // the thread within the tile's threads: all of a block's, or one wave's
    static __device__ __forceinline__ int tid() { return kThreads == 64 ? threadIdx.x & 63 : threadIdx.x; }
    // the tile's wave, the same in all lanes
    static __device__ __forceinline__ int wave() {
        return kThreads == 64 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    }
};
// Steps of 64 bytes with four in LDS where loads go straight there; of 128 with two where an
// operand comes through registers.
typedef Tiling<uint16_t, 256, 256, 2, 4, 64, 4> TileBig;
typedef Tiling<uint16_t, 128, 128, 2, 2, 64, 4> TileMid;
typedef Tiling<uint16_t, 64, 128, 2, 2, 64, 4> TileSmall;
typedef Tiling<uint16_t, 16, 64, 1, 1, 64, 4> TileFew;      // a wave's
typedef Tiling<uint16_t, 128, 128, 2, 2, 128, 2> TileAny;
typedef Tiling<float, 128, 128, 2, 2, 64, 4> TileMidF32;
typedef Tiling<float, 64, 64, 2, 2, 64, 4> TileSmallF32;
typedef Tiling<float, 16, 64, 1, 1, 64, 4> TileFewF32;
typedef Tiling<float, 64, 64, 2, 2, 128, 2> TileAnyF32;
typedef Tiling<uint16_t, 16, 64, 1, 1, 128, 2> TileFewAny;
typedef Tiling<float, 16, 64, 1, 1, 128, 2> TileFewAnyF32;
typedef Tiling<uint16_t, 64, 64, 2, 2, 64, 4> TileNarrow;

// How an operand is loaded: straight into LDS, where everything lies on 16 bytes; at any
// alignment through registers; from 8-bit codes, decoded in registers.
constexpr int kAsync = 0, kAny = 1, kKept = 2;

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

// The rows down which an operand's inner index runs: `first` + k, or GATHERed the token
// of that row.  In two halves, so that a list's entry is in flight while a step is
// computed: entry() is one load, always made (a load under a condition would be waited
// for where the branches join, and with it every load into LDS before it).
template <bool GATHER>
struct RowsDown {
    int64_t stride;
    const int32_t *source;
    uint32_t slots, k;
    int first;
    __device__ __forceinline__ explicit RowsDown(int64_t s, int f = 0)
        : stride(s), source(nullptr), slots(0), k(1), first(f) {}
    __device__ __forceinline__ RowsDown(const ExpertLists &l, int f, int64_t s)
        : stride(s), source(l.source), slots((uint32_t)l.slots), k((uint32_t)l.k), first(f) {}
    __device__ __forceinline__ uint32_t entry(int at) const {
        if constexpr (GATHER) return (uint32_t)source[min((uint32_t)(first + at), slots - 1)];
        return (uint32_t)(first + at);
    }
    // of an `at` that all lanes share
    __device__ __forceinline__ uint32_t shared_entry(int at) const {
        const uint32_t i = __builtin_amdgcn_readfirstlane(min((uint32_t)(first + at), slots - 1));
        return (uint32_t)((const __attribute__((address_space(4))) int32_t *)(uintptr_t)source)[i];
    }
    // slot / k: (slot + 1/2) / k is 1/32 or more from any whole number, the product off
    // by less than 2^-20
    __device__ __forceinline__ uint32_t token(uint32_t slot) const {
        return (uint32_t)__builtin_fma((double)slot, 1.0 / k, 0.5 / k);
    }
    // elements; below 0: nowhere
    __device__ __forceinline__ int64_t offset(uint32_t entry) const {
        if constexpr (!GATHER) return (int64_t)entry * stride;
        return entry < slots ? (int64_t)token(entry) * stride : -1;
    }
    // bytes, of a tensor that has fewer than kNowhere
    __device__ __forceinline__ uint32_t near_offset(uint32_t entry, uint32_t es) const {
        const uint32_t at = token(entry) * ((uint32_t)stride * es);
        return entry < slots ? at : 0xFFFFFFFFu;
    }
};

// Blocks come to the eight XCDs in turn; each XCD gets a run of neighbouring tiles,
// which share operands in its L2.
__device__ __forceinline__ int64_t own_tile(int64_t block, int64_t total) {
    const int64_t run = (total + 7) / 8, at = block / 8;
    return at < run ? block % 8 * run + at : total;
}
// The same in runs of `run` tiles, for tiles of unequal work.
__device__ __forceinline__ int64_t own_tile_in_runs(int64_t block, int run) {
    const int64_t at = block / 8;
    return at / run * (8 * run) + block % 8 * run + at % run;
}

struct RowTile {
    int e, first, rows, n;
};

// The block's tile among the experts' ragged rows: expert by expert, column of
// tiles by column.  All threads call it; false: nothing left for this block.  Counted in
// 64 bits: offsets out of order may name every row for each other expert.
template <int THREADS>
__device__ __forceinline__ bool find_tile(const ExpertLists &l, int bm, int nt, RowTile &t, void *lds) {
    constexpr int kWaves = THREADS / 64, kPer = (kExpertsMost + THREADS - 1) / THREADS;
    int64_t *const sums = static_cast<int64_t *>(lds);
    int *const sh = reinterpret_cast<int *>(sums + kWaves);
    const int tid = threadIdx.x, per = (l.E + THREADS - 1) / THREADS;
    int first[kPer], rows[kPer];
    int64_t sum = 0;
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
    int64_t upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t o = __shfl_up(upto, d, 64);
        if ((tid & 63) >= d) upto += o;
    }
    if ((tid & 63) == 63) sums[tid >> 6] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        if (w < tid >> 6) upto += sums[w];
        total += sums[w];
    }
    const int64_t tiles = total * nt, id = own_tile(blockIdx.x, tiles);
    if (id >= tiles) return false;
    int64_t at = (upto - sum) * nt;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        if (rows[i] <= 0) continue;
        const int mt = (rows[i] + bm - 1) / bm;
        const int64_t in = id - at;
        if (in >= 0 && in < (int64_t)mt * nt) {
            const int n = (int)(in / mt), m = (int)(in - (int64_t)n * mt);
            sh[0] = tid * per + i;
            sh[1] = first[i] + m * bm;
            sh[2] = rows[i] - m * bm;
            sh[3] = n;
        }
        at += (int64_t)mt * nt;
    }
    __syncthreads();
    t.e = __builtin_amdgcn_readfirstlane(sh[0]);
    t.first = __builtin_amdgcn_readfirstlane(sh[1]);
    t.rows = __builtin_amdgcn_readfirstlane(sh[2]);
    t.n = __builtin_amdgcn_readfirstlane(sh[3]);
    __syncthreads();
    return true;
}

// 16 bytes of elements from p (at any alignment: the hardware splits such loads), of
// which `have` are before the row's end, perhaps none, and none if not `there`; the others
// are 0.  kWhole: all are before it.  kEdge: one load without a branch, of the row's last
// 16 bytes where that is less, moved down (a load under a condition is waited for where
// the branches join).  kTiny: rows shorter than 16 bytes.
constexpr int kWhole = 0, kEdge = 1, kTiny = 2;
template <int HOW, typename T>
__device__ __forceinline__ u32x4 load_some(const T *p, int have, bool there) {
    constexpr int kMost = 16 / (int)sizeof(T), kWord = 4 / (int)sizeof(T);
    u32x4 v = {0, 0, 0, 0};
    if constexpr (HOW == kTiny) {
#pragma unroll
        for (int j = 0; j < kMost; j++) {
            if (!there || j >= have) continue;
            if constexpr (sizeof(T) == 4)
                v[j] = __builtin_bit_cast(uint32_t, p[j]);
            else
                v[j / kWord] |= (uint32_t)(typename std::make_unsigned<T>::type)p[j] << 32 / kWord * (j % kWord);
        }
    } else if constexpr (HOW == kWhole) {
        u32x4 w;
        __builtin_memcpy(&w, p, 16);
        v = there ? w : v;
    } else {
        uint64_t q[2];
        __builtin_memcpy(q, p + (have < kMost ? have - kMost : 0), 16);
        const uint32_t bytes = have < kMost ? (uint32_t)(kMost - have) * sizeof(T) : 0, bits = bytes % 8 * 8;
        const uint64_t lo = bytes & 8 ? q[1] : q[0], hi = bytes & 8 ? 0 : q[1];
        const bool some = there && have > 0;
        q[0] = some ? lo >> bits | (hi << 1) << (63 - bits) : 0;
        q[1] = some ? hi >> bits : 0;
        v = u32x4{(uint32_t)q[0], (uint32_t)(q[0] >> 32), (uint32_t)q[1], (uint32_t)(q[1] >> 32)};
    }
    return v;
}

// Loads of 16 bytes a lane from a moving base (the same in all lanes) and 32-bit
// offsets straight into LDS, 1 KB for a wave.  At kNowhere and beyond, the range
// check of the buffer gives zeros.  The load is written out because the compiler, told
// of it, holds every transposing LDS read back until all such loads have landed; it has
// no result in registers, and all_waves() waits for it.  M0, where in LDS it goes, is an
// operand, which the compiler sets; the load follows a cycle later, as it has to.
struct Stream {
    uint32_t lo, hi;
    __device__ __forceinline__ void at(const void *p) {
        const uint64_t q = reinterpret_cast<uint64_t>(p);
        lo = __builtin_amdgcn_readfirstlane((uint32_t)q);
        hi = __builtin_amdgcn_readfirstlane((uint32_t)(q >> 32));
    }
    __device__ __forceinline__ void to_lds(int64_t ahead, uint32_t offset, const char *wave_base) const {
        const uint64_t q = ((uint64_t)hi << 32 | lo) + (uint64_t)ahead;
        const u32x4 buffer = {(uint32_t)q, (uint32_t)(q >> 32) & 0xFFFFu, kNowhere, 0x00020000u};
        const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)DQ_LDS(const_cast<char *>(wave_base)));
        asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(m0), "v"(offset), "s"(buffer)
                     : "memory");
    }
};

// An operand whose rows (the tile's M or N) are contiguous along the inner index.
// In LDS a row's chunks of 16 bytes are exchanged, by c ^ (row & 7) in rows of 128
// bytes, by c ^ (row / 2 & 3) in rows of 64, so that eight neighbouring rows of a matrix
// operand meet all banks.
template <class C, int ROWS, int L>
struct Along {
    typedef typename C::T T;
    static constexpr int kRowChunks = C::kRow / 16, kPer = ROWS * kRowChunks / C::kThreads, BK = C::BK;
    static constexpr bool kAsyncLoad = L == kAsync;
    static_assert(ROWS * kRowChunks % C::kThreads == 0 && C::kThreads % (8 * kRowChunks) == 0, "whole chunks");
    struct Entries {};
    Stream from;                       // kAsync
    uint32_t off[kAsyncLoad ? kPer : 1];
    const T *p[kAsyncLoad ? 1 : kPer];  // else
    uint32_t none;                     // a bit for every chunk of a row that starts nowhere
    bool tiny;
    struct Regs {
        u32x4 v[kAsyncLoad ? 1 : kPer];
    };
    int K, kc;

    static __device__ __forceinline__ int swap(int chunk, int row) {
        return kRowChunks == 8 ? chunk ^ (row & 7) : chunk ^ (row >> 1 & 3);
    }
    // row(i): where the tile's row i starts, from base (below 0: nowhere); of rows of
    // `whole` elements the next `inner`
    template <class Row>
    __device__ __forceinline__ void start(const T *base, int whole, int inner, Row row) {
        K = inner;
        tiny = whole < C::kChunk;
        none = 0;
        const int r0 = C::tid() / kRowChunks;
        kc = swap(C::tid() % kRowChunks, r0) * C::kChunk;
        if constexpr (kAsyncLoad) from.at(base);
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const int64_t at = row(r0 + i * (C::kThreads / kRowChunks));
            if constexpr (kAsyncLoad) {
                off[i] = at < 0 ? kNowhere : (uint32_t)((at + kc) * sizeof(T));
            } else {
                p[i] = base + (at < 0 ? 0 : at) + kc;
                none |= (uint32_t)(at < 0) << i;
            }
        }
    }
    template <int HOW>
    __device__ __forceinline__ void to_regs(int k0, Regs &r) {
#pragma unroll
        for (int i = 0; i < kPer; i++) r.v[i] = load_some<HOW>(p[i] + k0, K - k0 - kc, !(none >> i & 1));
    }
    __device__ __forceinline__ void ahead(int, Entries &) const {}
    __device__ __forceinline__ void issue(char *buf, int k0, const Entries &, Regs &r) {
        if constexpr (kAsyncLoad) {
#pragma unroll
            for (int i = 0; i < kPer; i++)
                from.to_lds((int64_t)k0 * sizeof(T), K - k0 > kc ? off[i] : kNowhere,
                            buf + (64 * C::wave() + i * C::kThreads) * 16);
        } else if (K - k0 >= C::BK) {
            to_regs<kWhole>(k0, r);
        } else if (!tiny) {
            to_regs<kEdge>(k0, r);
        } else {
            to_regs<kTiny>(k0, r);
        }
    }
    __device__ __forceinline__ void commit(char *buf, const Regs &r) {
        if constexpr (!kAsyncLoad)
#pragma unroll
            for (int i = 0; i < kPer; i++)
                *reinterpret_cast<u32x4 *>(buf + (C::tid() + i * C::kThreads) * 16) = r.v[i];
    }
    // rows row0 .. row0 + 15, half h of the step: lane l has row l & 15, chunk (l >> 4) + 4 h
    static __device__ __forceinline__ u32x4 frag(const char *buf, int row0, int h) {
        const int lane = threadIdx.x & 63, row = row0 + (lane & 15);
        return *reinterpret_cast<const u32x4 *>(buf + row * C::kRow + swap((lane >> 4) + 4 * h, lane) * 16);
    }
};

// An operand whose inner index runs down its rows, each contiguous along M or N.  In
// LDS as it lies in memory, BK rows of COLS elements, with units of 16 elements
// exchanged within a row: bf16 is turned by the transposing LDS read, where 16 lanes
// take 4 rows of 32 bytes, fp32 read by elements, where the wave takes 4 rows.
template <class C, int COLS, int L, bool GATHER>
struct Across {
    typedef typename C::T T;
    static constexpr int kRow = COLS * (int)sizeof(T), kBytes = C::BK * kRow, kUnits = COLS / 16;
    static constexpr bool kFromKept = L == kKept;
    static constexpr int kPieces = kFromKept ? C::BK * kUnits : kBytes / 16;
    static constexpr bool kSome = kPieces < C::kThreads;     // the last waves have none
    static constexpr int kPer = kSome ? 1 : kPieces / C::kThreads, kPerRow = kPieces / C::BK, BK = C::BK;
    static constexpr bool kAsyncLoad = L == kAsync;
    static_assert(kPieces % C::kThreads == 0 || (kSome && !kAsyncLoad && kPieces % 64 == 0), "whole pieces");
    static_assert(kUnits % 4 == 0, "units are exchanged by fours");
    Stream from;                       // kAsync
    const T *base;                     // kAny
    const int8_t *codes;               // kKept
    const uint8_t *exponents;
    RowsDown<GATHER> rows;
    // through the scalar cache: a wave's load of 1 KB meets kShared rows
    static constexpr bool kScalar = kAsyncLoad && GATHER && C::kRow == 64;
    static constexpr int kShared = kScalar ? 64 / kPerRow : 1;
    struct Entries {
        uint32_t at[GATHER || !kAsyncLoad ? kPer : 1][kShared];
    };
    int K, N, col0;
    struct Regs {
        u32x4 v[L == kAsync ? 1 : kPer];
        uint8_t ex[kFromKept ? kPer : 1];
    };

    static __device__ __forceinline__ int swap(int k) {
        if constexpr (C::kF32) return k >> 2 & 3;
        if constexpr (kUnits % 8 == 0) return (k & 3) | (k >> 1 & 4);
        return k & 3;
    }
    __device__ __forceinline__ explicit Across(const RowsDown<GATHER> &r) : rows(r) {}
    __device__ __forceinline__ void start(const T *b, int c0, int cols, int inner) {
        base = b;
        if constexpr (kAsyncLoad) from.at(b);
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
    static __device__ __forceinline__ int piece_row(int i) { return (C::tid() + i * C::kThreads) / kPerRow; }
    __device__ __forceinline__ int piece_col(int i) const {
        const int at = (C::tid() + i * C::kThreads) % kPerRow;
        if (kFromKept) return col0 + 16 * at;
        constexpr int kUnit = 16 / C::kChunk;
        return col0 + ((at / kUnit ^ swap(piece_row(i))) * kUnit + at % kUnit) * C::kChunk;
    }
    // the lists' entries for the step at k0
    __device__ __forceinline__ void ahead(int k0, Entries &e) const {
        if constexpr (kScalar) {
            const int row = C::wave() * kShared;
#pragma unroll
            for (int i = 0; i < kPer; i++)
#pragma unroll
                for (int j = 0; j < kShared; j++)
                    e.at[i][j] = rows.shared_entry(k0 + row + j + i * (C::kThreads / kPerRow));
        } else if constexpr (GATHER || !kAsyncLoad) {
#pragma unroll
            for (int i = 0; i < kPer; i++) e.at[i][0] = rows.entry(min(k0 + piece_row(i), K - 1));
        }
    }
    static __device__ __forceinline__ uint32_t entry_of(const Entries &e, int i) {
        uint32_t v = e.at[i][0];
#pragma unroll
        for (int j = 1; j < kShared; j++)
            // by a mask: a select would become an indexed read of the list, from scratch memory
            v ^= (e.at[i][j - 1] ^ e.at[i][j]) & -(uint32_t)((threadIdx.x & 63) / kPerRow >= j);
        return v;
    }
    template <int HOW>
    __device__ __forceinline__ void to_regs(int k0, const Entries &e, Regs &r) {
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            if (kSome && C::tid() >= kPieces) continue;
            const int col = piece_col(i);
            int64_t off = rows.offset(e.at[i][0]);
            const bool there = off >= 0 && k0 + piece_row(i) < K;
            off = off < 0 ? 0 : off;
            if constexpr (kFromKept) {
                // zeros of a row past the end are not to meet another block's infinity
                const uint8_t ex = exponents[off * ((N + 31) / 32) + min(col, N - 1) / 32];
                r.ex[i] = there ? ex : 127;
                r.v[i] = load_some<HOW>(codes + off * N + col, N - col, there);
            } else {
                r.v[i] = load_some<HOW>(base + off + col, N - col, there);
            }
        }
    }
    __device__ __forceinline__ void issue(char *buf, int k0, const Entries &e, Regs &r) {
        if constexpr (kAsyncLoad) {
#pragma unroll
            for (int i = 0; i < kPer; i++) {
                const int col = piece_col(i);
                // rows that are not gathered: the base moves, the offsets stay
                const int64_t moved = GATHER ? 0 : (int64_t)(rows.first + k0) * rows.stride * (int64_t)sizeof(T);
                const uint32_t off = GATHER ? rows.near_offset(entry_of(e, GATHER ? i : 0), sizeof(T))
                                            : (uint32_t)piece_row(i) * (uint32_t)(rows.stride * (int64_t)sizeof(T));
                const bool there = off < kNowhere && col < N && k0 + piece_row(i) < K;
                from.to_lds(moved, there ? off + (uint32_t)(col * sizeof(T)) : kNowhere,
                            buf + (64 * C::wave() + i * C::kThreads) * 16);
            }
        } else if (N - col0 >= COLS) {
            to_regs<kWhole>(k0, e, r);
        } else if (N >= (kFromKept ? 16 : C::kChunk)) {
            to_regs<kEdge>(k0, e, r);
        } else {
            to_regs<kTiny>(k0, e, r);
        }
    }
    __device__ __forceinline__ void commit(char *buf, const Regs &r) {
        if constexpr (L == kAny) {
#pragma unroll
            for (int i = 0; i < kPer; i++)
                *reinterpret_cast<u32x4 *>(buf + (C::tid() + i * C::kThreads) * 16) = r.v[i];
        } else if constexpr (kFromKept) {
#pragma unroll
            for (int i = 0; i < kPer; i++) {
                if (kSome && C::tid() >= kPieces) continue;
                const int k = piece_row(i), unit = (C::tid() + i * C::kThreads) % kPerRow;
                u32x4 *to = reinterpret_cast<u32x4 *>(buf + k * kRow + (unit ^ swap(k)) * 16 * sizeof(T));
                const float scale = __uint_as_float((uint32_t)r.ex[i] << 23);
                float f[16];
#pragma unroll
                for (int j = 0; j < 16; j++) f[j] = (float)(int8_t)(r.v[i][j / 4] >> 8 * (j & 3)) * scale;
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

__device__ __forceinline__ void put_one(float *p, float v) { *p = v; }
__device__ __forceinline__ void put_one(uint16_t *p, float v) { *p = (uint16_t)bf16_bits(v); }

// Whether results of rows this far apart are stored past the caches (they are read by
// another kernel, if at all).  Rows on 32 bytes of bf16 operands gain: dW of 2048 x 2816
// over 128 rows an expert 325 us instead of 391 in fp32 and 256 instead of 300 in bf16, 2784
// columns 251 instead of 304, over 512 rows 507 instead of 544.  Rows off 32 bytes lose,
// since the caches no longer put neighbouring pieces together: 3880 bf16 columns 256 instead
// of 226, 4072 columns 380 instead of 250.  Of fp32 operands rows on 128 bytes alone gain,
// and that little: 1024 columns 66 instead of 75, but 1000 columns 91 instead of 81.  A
// product's results are read next by the activation, which shows where the last-level cache
// would have held them; both calls together, 369 MB of bf16 861 us instead of 869, 92 MB 313
// instead of 316, but 67 MB 115 instead of 112, and of fp32 311 instead of 309.
template <class C, typename Out>
__device__ __forceinline__ bool past_caches(const Out *base, int64_t stride) {
    constexpr int kLine = C::kF32 ? 128 : 32;
    return ((reinterpret_cast<uintptr_t>(base) | (uintptr_t)stride * sizeof(Out)) & (kLine - 1)) == 0;
}

// columns n .. n + COUNT - 1 of a row of N, from as many elements; past: 16 aligned bytes
// go past the caches
template <int COUNT, typename Out>
__device__ __forceinline__ void store_columns(Out *row, int n, int N, const Out *v, bool past = false) {
    if (n + COUNT <= N) {
        if constexpr (COUNT * sizeof(Out) == 16) {
            if (past) {
                u32x4 w;
                __builtin_memcpy(&w, v, 16);
                __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(row + n));
                return;
            }
        }
        __builtin_memcpy(row + n, v, COUNT * sizeof(Out));
    } else {
#pragma unroll
        for (int q = 0; q < COUNT - 1; q++)
            if (n + q < N) row[n + q] = v[q];
    }
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
    static __device__ __forceinline__ int m0() { return C::wave() / C::WN * (C::BM / C::WM); }
    static __device__ __forceinline__ int n0() { return C::wave() % C::WN * (C::BN / C::WN); }

    // half a step's matrix operands
    struct Half {
        u32x4 a[C::TM], b[C::TN];
        template <class A, class B>
        __device__ __forceinline__ void read(const char *lds, int h) {
#pragma unroll
            for (int j = 0; j < C::TN; j++) b[j] = B::frag(lds + C::kBytesA, n0() + 16 * j, h);
#pragma unroll
            for (int i = 0; i < C::TM; i++) a[i] = A::frag(lds, m0() + 16 * i, h);
        }
    };
    __device__ __forceinline__ void add(const Half &f) {
#pragma unroll
        for (int i = 0; i < C::TM; i++)
#pragma unroll
            for (int j = 0; j < C::TN; j++) {
                if constexpr (C::kF32) {
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        v[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(f.b[j][q]),
                                                                       __uint_as_float(f.a[i][q]), v[i][j], 0, 0, 0);
                } else {
                    v[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.b[j]),
                                                                     __builtin_bit_cast(bf16x8, f.a[i]), v[i][j], 0, 0,
                                                                     0);
                }
            }
    }
    // into LDS, [BM][BN] floats
    __device__ __forceinline__ void put(float *to) const {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < C::TM; i++)
#pragma unroll
            for (int j = 0; j < C::TN; j++)
                *reinterpret_cast<f32x4 *>(to + (m0() + 16 * i + (lane & 15)) * C::BN + n0() + 16 * j +
                                           (lane >> 4) * 4) = v[i][j];
    }
    // row(m): where the tile's row m goes, NULL: nowhere.  By way of LDS (of the wave's own
    // share of the block's, which no wave reads any more), so that neighbouring lanes
    // store the whole of a row's piece: straight from the accumulators a row gets 32
    // bytes at a time, and 369 MB take 160 us instead of 80.
    template <typename Out, class Row>
    __device__ __forceinline__ void store(char *lds, Row row, int col0, int N, bool past) const {
        constexpr int kRowBytes = 16 * C::TN * (int)sizeof(Out), kChunks = kRowBytes / 16;
        constexpr int kEach = 16 / (int)sizeof(Out);
        constexpr int kShare = C::kLds / (C::WM * C::WN) / kRowBytes / 16 * 16;
        constexpr int kRows = kShare < 16 * C::TM ? kShare : 16 * C::TM, kPass = kRows / 16;
        static_assert(kRows >= 16 && C::TM % kPass == 0, "whole passes");
        char *own = lds + C::wave() * (C::kLds / (C::WM * C::WN));
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i0 = 0; i0 < C::TM; i0 += kPass) {
            asm volatile("" ::: "memory");
#pragma unroll
            for (int i = 0; i < kPass; i++)
#pragma unroll
                for (int j = 0; j < C::TN; j++) {
                    const int m = 16 * i + (lane & 15), at = (16 * j + (lane >> 4) * 4) * (int)sizeof(Out);
                    Out e[4];
#pragma unroll
                    for (int q = 0; q < 4; q++) put_one(e + q, v[i0 + i][j][q]);
                    __builtin_memcpy(__builtin_assume_aligned(own + m * kRowBytes +
                                                                  ((at / 16 ^ (m & (kChunks - 1))) * 16 + at % 16),
                                                              sizeof(e)),
                                     e, sizeof(e));
                }
            // other lanes' elements: a wave's LDS accesses are in order
            asm volatile("" ::: "memory");
#pragma unroll
            for (int r = 0; r < kRows; r += 64 / kChunks) {
                const int m = r + lane / kChunks, c = lane % kChunks;
                Out e[kEach];
                const char *at = own + m * kRowBytes + (c ^ (m & (kChunks - 1))) * 16;
                __builtin_memcpy(e, __builtin_assume_aligned(at, 16), 16);
                Out *p = row(m0() + 16 * i0 + m);
                if (p) store_columns<kEach>(p, col0 + n0() + c * kEach, N, e, past);
            }
        }
    }
};

// All but the last LEFT loads of this wave have landed, its LDS reads and writes are
// done, and so for every wave of the tile.
template <class C, int LEFT>
__device__ __forceinline__ void all_waves() {
    static_assert(LEFT < 64, "six bits");
    // by the builtin, so that the compiler counts no LDS read as open behind it: beside a
    // scalar load it could only wait for all of them
    __builtin_amdgcn_s_waitcnt(0xC07F);                  // lgkmcnt(0)
    if constexpr (C::kThreads == 64)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
    else
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// Step k0 into LDS: by loads that land there, or from registers, which then take the step
// two after it.  Past the end zeros are stored.
template <class Op>
__device__ __forceinline__ void fill(Op &op, char *buf, int k0, typename Op::Entries &e, typename Op::Regs &r) {
    if constexpr (Op::kAsyncLoad) {
        op.issue(buf, k0, e, r);
        op.ahead(k0 + Op::BK, e);
    } else {
        op.commit(buf, r);
        op.issue(nullptr, k0 + 2 * Op::BK, e, r);
        op.ahead(k0 + 3 * Op::BK, e);
    }
}

// acc += A B over `inner`, an operand at least through registers, where two steps are on
// their way; two more are in LDS.  The barrier stands in the middle of a step's products,
// when the step after it is in LDS and the second half's operands are in registers: LDS
// reads run beside the other half's products, loads beside two steps'.
template <class C, class A, class B>
__device__ __forceinline__ void multiply_halves(char *lds, A &a, B &b, int inner, Acc<C> &acc) {
    constexpr int kStep = C::kBytesA + C::kBytesB;
    // loads into registers are waited for where they are used; beside an operand that lands in
    // LDS all are waited for at every barrier, those two steps ahead too
    constexpr int kLeft = A::kAsyncLoad || B::kAsyncLoad ? 0 : 63;
    if (inner <= 0) return;
    const int steps = (inner + C::BK - 1) / C::BK;
    typename A::Entries ea[2];
    typename B::Entries eb[2];
    typename A::Regs ra[2];
    typename B::Regs rb[2];
    const auto entries = [&](int i, int t) {
        a.ahead(t * C::BK, ea[i]);
        b.ahead(t * C::BK, eb[i]);
    };
    entries(0, 0);
    entries(1, 1);
#pragma unroll
    for (int i = 0; i < 2; i++) {
        a.issue(lds + i * kStep, i * C::BK, ea[i], ra[i]);
        b.issue(lds + i * kStep + C::kBytesA, i * C::BK, eb[i], rb[i]);
    }
    entries(0, 2);
    entries(1, 3);
#pragma unroll
    for (int i = 0; i < 2; i++) {
        a.commit(lds + i * kStep, ra[i]);
        b.commit(lds + i * kStep + C::kBytesA, rb[i]);
        if constexpr (!A::kAsyncLoad) a.issue(nullptr, (2 + i) * C::BK, ea[i], ra[i]);
        if constexpr (!B::kAsyncLoad) b.issue(nullptr, (2 + i) * C::BK, eb[i], rb[i]);
    }
    // from here: entries of the staged operands' next step, of the others' step t + 2
    if constexpr (!A::kAsyncLoad) a.ahead(4 * C::BK, ea[0]);
    if constexpr (!B::kAsyncLoad) b.ahead(4 * C::BK, eb[0]);
    all_waves<C, kLeft>();
    typename Acc<C>::Half first, second;
    first.template read<A, B>(lds, 0);
    const auto step = [&](int t, typename A::Regs &va, typename B::Regs &vb) {
        char *now = lds + (t & 1) * kStep, *next = lds + (~t & 1) * kStep;
        second.template read<A, B>(now, 1);
        acc.add(first);
        __builtin_amdgcn_sched_barrier(0);
        all_waves<C, kLeft>();
        __builtin_amdgcn_sched_barrier(0);
        if (t + 1 < steps) {
            first.template read<A, B>(next, 0);
            const int k = (t + 2) * C::BK;
            fill(a, now, k, ea[0], va);
            fill(b, now + C::kBytesA, k, eb[0], vb);
        }
        acc.add(second);
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int t = 0; t < steps; t += 2) {
        step(t, ra[0], rb[0]);
        if (t + 1 < steps) step(t + 1, ra[1], rb[1]);
    }
}

// acc += A B over `inner`, all operands by loads into LDS: a step's products run beside
// the LDS reads of the next and the loads of the kStages - 1 after it.  One barrier a step:
// behind it the next step has landed, and the operands of this one are in registers, so
// that its place in LDS is free.  Loads past the end are made, of zeros, to keep count.
// `mine`: whether any of the wave's part of the tile is wanted; a wave without loads and
// waits with the others, and leaves its SIMD to them.
template <class C, class A, class B>
__device__ __forceinline__ void multiply_stages(char *lds, A &a, B &b, int inner, bool mine, Acc<C> &acc) {
    constexpr int kStep = C::kBytesA + C::kBytesB, S = C::kStages;
    static_assert(C::kRow == 64 && S >= 3, "a step is one matrix instruction deep");
    if (inner <= 0) return;
    const int steps = (inner + C::BK - 1) / C::BK;
    typename A::Regs ra;                                 // unused
    typename B::Regs rb;
    {
        typename A::Entries ea[S];
        typename B::Entries eb[S];
#pragma unroll
        for (int i = 0; i < S; i++) {
            a.ahead(i * C::BK, ea[i]);
            b.ahead(i * C::BK, eb[i]);
        }
#pragma unroll
        for (int i = 0; i < S; i++) {
            a.issue(lds + i * kStep, i * C::BK, ea[i], ra);
            b.issue(lds + i * kStep + C::kBytesA, i * C::BK, eb[i], rb);
        }
    }
    constexpr int kLoads = A::kPer + B::kPer;
    typename Acc<C>::Half half[2];
    all_waves<C, (S - 1) * kLoads>();
    if (mine) half[0].template read<A, B>(lds, 0);
    all_waves<C, (S - 2) * kLoads>();
    int at = 0;                                          // the stage of step t
    typename A::Entries ea;
    typename B::Entries eb;
    a.ahead(S * C::BK, ea);
    b.ahead(S * C::BK, eb);
    const auto load = [&](int t) {
        const int k = (t + S) * C::BK;
        a.issue(lds + at, k, ea, ra);
        b.issue(lds + at + C::kBytesA, k, eb, rb);
        a.ahead(k + C::BK, ea);
        b.ahead(k + C::BK, eb);
        at = at + kStep == S * kStep ? 0 : at + kStep;
    };
    const auto wait = [&] {
        __builtin_amdgcn_sched_barrier(0);
        all_waves<C, (S - 2) * kLoads>();
        __builtin_amdgcn_sched_barrier(0);
    };
    if (mine) {
        const auto step = [&](int t, typename Acc<C>::Half &now, typename Acc<C>::Half &next) {
            load(t);
            next.template read<A, B>(lds + at, 0);
            acc.add(now);
            wait();
        };
        int t = 0;
        for (; t + 1 < steps; t += 2) {
            step(t, half[0], half[1]);
            step(t + 1, half[1], half[0]);
        }
        if (t < steps) acc.add(half[0]);
    } else {
        for (int t = 0; t < steps / 2 * 2; t++) {
            load(t);
            wait();
        }
    }
    all_waves<C, 0>();                                   // nothing may land in LDS after the block
}

template <class C, class A, class B>
__device__ __forceinline__ void multiply(char *lds, A &a, B &b, int inner, bool mine, Acc<C> &acc) {
    if constexpr (C::kRow == 64)
        multiply_stages<C>(lds, a, b, inner, mine, acc);
    else
        multiply_halves<C>(lds, a, b, inner, acc);
}

template <class K>
hipError_t room_for(K kernel, int lds) {
    if (lds <= 65536) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
}

}  // namespace
}  // namespace dq
