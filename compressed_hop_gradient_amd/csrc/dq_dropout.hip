// dq_dropout.hip -- dropout from the counter-based generator for gfx950: the mask
// is drawn where it is used, in the forward and in the backward pass.  fp32
// arithmetic, no contraction.
#include "dq_train_device.h"

namespace dq {

namespace {

// y = r + m x s with m the mask and s the inverse of the probability that it
// keeps an element; the gradient by x is the same m s on dy.  Every operand is
// touched once, and what is left to do is the mask: one generator call for 8
// elements (16 random bits each), so that its 20 64-bit products are shared and
// memory stays the bound, with the VALUs busy 62% of the time (bf16, no residual).
//
// 16384 x 8192 bf16 with a residual (805 MB): 136 us, 5.9 TB/s; 8192 x 8192 bf16
// without one (268 MB): 45 us, 6.0 TB/s; 8192 x 2048 fp32 (134 MB): 25 us, 5.3 TB/s.
// A copy of 256 MB reaches 5.5 TB/s on the same card.

// The eight 16-bit dithers of elements 8b .. 8b + 7 as four words, low half
// first: Philox4x32-10 (Salmon et al., SC'11) on (b, worker, round, site).  A
// product is one 64-bit multiply, a three-way xor one instruction.  The compiler may
// hold all round keys (the codec's kernels may not): 57 to 106 SGPRs, none spilled.
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

template <bool RES>
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
                x[j] = dropout_one<RES>(x[j], RES ? r[j] : 0.0f, dither(w, j) >= a.threshold, a.scale);
            store8<F32>(a.y, row * a.ys + col, x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (col + j >= n) break;
                const float r = RES ? El::up(static_cast<const T *>(a.residual)[col + j]) : 0.0f;
                static_cast<T *>(a.y)[col + j] = El::down(dropout_one<RES>(
                    El::up(static_cast<const T *>(a.x)[col + j]), r, dither(w, j) >= a.threshold, a.scale));
            }
        }
    }
}

// Any alignment and row length: a wave draws 64 Philox blocks and then takes
// their 512 elements 64 at a time, side by side in its lanes, each with its bit
// of the mask from the lane that drew it.  8192 x 2047 of rows 4094 wide: fp32 27 us
// (4.9 TB/s), bf16 23 us (2.9 TB/s); with a thread on the 8 elements of its own
// block, which spreads a load over 16 lines, 93 and 29 us.
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
                    El::down(dropout_one<RES>(El::up(x[i]), RES ? El::up(r[i]) : 0.0f, kept, a.scale));
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

}  // namespace

hipError_t launch_dropout(const DropoutArgs &a, int f32, hipStream_t s) {
    if (f32) return a.residual ? dropout_access<true, true>(a, s) : dropout_access<true, false>(a, s);
    return a.residual ? dropout_access<false, true>(a, s) : dropout_access<false, false>(a, s);
}

}  // namespace dq
