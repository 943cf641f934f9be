// dq_keep8.hip -- activations kept in 8 bits for the backward pass, for gfx950.
#include "dq_keep8_device.h"

namespace dq {

namespace {

// A thread takes eight elements of a row, four neighbouring threads a block of 32 (a
// row's last block may be short: its missing elements are zeros).  EIGHTS: rows of
// whole eights, whose dithers come from one generator call.  8192 x 4096 bf16 (102 MB): 27 us,
// 3.7 TB/s; the generator's products, the codes' arithmetic and the 64-bit division that finds
// a thread's row come to as much time as the bytes.  Restored: 18 us, 5.6 TB/s.
template <bool F32, bool EIGHTS>
__global__ __launch_bounds__(256) void k_keep8(KeepArgs a, int32_t blocks, int64_t total) {
    const uint32_t round = a.key.round + (a.key.d_round ? *a.key.d_round : 0);
    const int64_t rows = a.d_rows ? min(a.rows, (int64_t)max(0, *a.d_rows)) : a.rows;
    const uint32_t per_row = 4 * (uint32_t)blocks;
    // whole groups of four go on together
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 256) {
        const int64_t row = id / per_row;
        if (row >= rows) return;
        const int64_t col = (id - row * per_row) * 8;
        const int have = (int)(a.cols - col < 8 ? a.cols - col : 8);
        const bool full = have == 8;
        float x[8];
        if (full)
            load_eight<F32, true>(a.x, row * a.xs + col, have, x);
        else
            load_eight<F32, false>(a.x, row * a.xs + col, have, x);
        uint32_t w[4], exponent;
        keep_dithers<EIGHTS>(row * a.cols + col, a.key, round, w);
        const uint2 c = keep_eight(x, w, exponent);
        int8_t *to = a.codes + row * a.cols + col;
        if (full)
            store_codes<true>(to, have, c);
        else if (!EIGHTS)
            store_codes<false>(to, have, c);
        if ((threadIdx.x & 3) == 0) a.exponents[row * blocks + col / 32] = (uint8_t)exponent;
    }
}

template <bool F32>
__global__ __launch_bounds__(256) void k_restore8(RestoreArgs a, int32_t blocks, int64_t total) {
    const int64_t per_row = (a.cols + 7) / 8, rows = a.d_rows ? min(a.rows, (int64_t)max(0, *a.d_rows)) : a.rows;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 256) {
        const int64_t row = id / per_row, col = (id - row * per_row) * 8;
        if (row >= rows) return;
        const float scale = kept_scale(a.exponents[row * blocks + col / 32]);
        const auto eight = [&](auto full) {
            constexpr bool kFull = decltype(full)::value;
            const int have = (int)(a.cols - col);
            const uint2 c = load_codes<kFull>(a.codes + row * a.cols + col, have);
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = kept_value(j < 4 ? c.x : c.y, j & 3, scale);
            store_eight<F32, kFull>(a.y, row * a.ys + col, have, x);
        };
        if (col + 8 <= a.cols)
            eight(std::true_type());
        else
            eight(std::false_type());
    }
}

dim3 grid_of(int64_t threads) {
    const int64_t want = (threads + 255) / 256;
    return dim3((unsigned)(want < (1 << 20) ? want : (1 << 20)));
}

}  // namespace

hipError_t launch_keep8(const KeepArgs &a, int f32, hipStream_t s) {
    const int32_t blocks = (int32_t)((a.cols + 31) / 32);
    const int64_t total = a.rows * blocks * 4;
    const bool e = a.cols % 8 == 0;
    const dim3 grid = grid_of(total), block(256);
    if (f32 && e)
        hipLaunchKernelGGL((k_keep8<true, true>), grid, block, 0, s, a, blocks, total);
    else if (f32)
        hipLaunchKernelGGL((k_keep8<true, false>), grid, block, 0, s, a, blocks, total);
    else if (e)
        hipLaunchKernelGGL((k_keep8<false, true>), grid, block, 0, s, a, blocks, total);
    else
        hipLaunchKernelGGL((k_keep8<false, false>), grid, block, 0, s, a, blocks, total);
    return hipGetLastError();
}

hipError_t launch_restore8(const RestoreArgs &a, int f32, hipStream_t s) {
    const int32_t blocks = (int32_t)((a.cols + 31) / 32);
    const int64_t total = a.rows * ((a.cols + 7) / 8);
    const dim3 grid = grid_of(total), block(256);
    if (f32)
        hipLaunchKernelGGL((k_restore8<true>), grid, block, 0, s, a, blocks, total);
    else
        hipLaunchKernelGGL((k_restore8<false>), grid, block, 0, s, a, blocks, total);
    return hipGetLastError();
}

}  // namespace dq
