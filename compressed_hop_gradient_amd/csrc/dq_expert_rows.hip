// dq_expert_rows.hip -- the order of the experts' rows and the way back, and the
// activation between the experts' products, for gfx950.
#include "dq_keep8_device.h"

namespace dq {

namespace {

// ---- order --------------------------------------------------------------------

constexpr int kRowsThreads = 512, kRowsWaves = kRowsThreads / 64;
constexpr int kRowsAlone = 8192;         // slots that one block sorts
constexpr int kRowsMostBlocks = 256;

// Slots of a wave: a run of whole 64s of its block's run.
struct Run {
    int first, end;
};
__device__ __forceinline__ Run run_of(int slots, int blocks, int block, int wave) {
    const int waves = blocks * kRowsWaves, per = ((slots + waves - 1) / waves + 63) / 64 * 64;
    const int64_t at = (int64_t)(block * kRowsWaves + wave) * per;
    const int64_t end = at + per;
    return Run{(int)(at < slots ? at : slots), (int)(end < slots ? end : slots)};
}

__device__ __forceinline__ int bucket(const ExpertRowsArgs &a, int slot) {
    const uint32_t e = (uint32_t)a.ids[slot];
    return e < (uint32_t)a.E ? (int)e : a.E;
}

// Slots of every bucket (the last: without an expert) in a block's run.
__global__ __launch_bounds__(kRowsThreads) void k_rows_count(ExpertRowsArgs a) {
    extern __shared__ uint32_t count[];
    for (int e = threadIdx.x; e <= a.E; e += kRowsThreads) count[e] = 0;
    __syncthreads();
    const Run r = run_of(a.slots, a.blocks, blockIdx.x, threadIdx.x >> 6);
    for (int i = r.first + (threadIdx.x & 63); i < r.end; i += 64) atomicAdd(&count[bucket(a, i)], 1u);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += kRowsThreads) a.counts[(size_t)blockIdx.x * (a.E + 1) + e] = count[e];
}

// What bounds it is latency: 32 slots take 3.4 us, 8192 15 (three passes over a few KB by one
// block), 262144 slots of 256 experts 4.8 + 13.8 us for 3 MB in and out.
//
// A stable counting sort: every wave counts its run, learns where its buckets start
// from all counts before it, and places 64 slots at a time, those of one bucket in
// their order (found by a ballot for each bit of the bucket).  One block of it does
// short lists alone; else each block adds up the other blocks' counts itself.
// Integer sums throughout: the same lists on every run.
__global__ __launch_bounds__(kRowsThreads) void k_rows_place(ExpertRowsArgs a) {
    extern __shared__ uint32_t lds[];
    const int n = a.E + 1, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t *start = lds, *before = lds + kRowsWaves * n, *all = before + n;      // start[wave][bucket]
    __shared__ uint32_t upto[kRowsWaves];
    for (int i = tid; i < (kRowsWaves + 2) * n; i += kRowsThreads) lds[i] = 0;
    __syncthreads();
    const Run r = run_of(a.slots, a.blocks, blockIdx.x, wave);
    for (int i = r.first + lane; i < r.end; i += 64) atomicAdd(&start[wave * n + bucket(a, i)], 1u);
    if (a.blocks > 1) {
        const int groups = n < kRowsThreads ? kRowsThreads / n : 1;
        for (int e = tid % n; e < n && tid / n < groups; e += n < kRowsThreads ? n : kRowsThreads) {
            uint32_t pre = 0, sum = 0;
#pragma unroll 8
            for (int b = n < kRowsThreads ? tid / n : 0; b < a.blocks; b += groups) {
                const uint32_t c = a.counts[(size_t)b * n + e];
                sum += c;
                pre += b < (int)blockIdx.x ? c : 0;
            }
            atomicAdd(&before[e], pre);
            atomicAdd(&all[e], sum);
        }
    }
    __syncthreads();
    if (a.blocks == 1) {
        for (int e = tid; e < n; e += kRowsThreads)
            for (int w = 0; w < kRowsWaves; w++) all[e] += start[w * n + e];
        __syncthreads();
    }
    // the buckets' first rows: thread t has buckets 3 t .. 3 t + 2
    constexpr int kPer = (kExpertsMost + 1 + kRowsThreads - 1) / kRowsThreads;
    uint32_t own = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++)
        if (tid * kPer + i < n) own += all[tid * kPer + i];
    uint32_t scan = own;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_up(scan, d, 64);
        if (lane >= d) scan += o;
    }
    if (lane == 63) upto[wave] = scan;
    __syncthreads();
    for (int w = 0; w < wave; w++) scan += upto[w];
    uint32_t first = scan - own;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int e = tid * kPer + i;
        if (e < n) {
            if (blockIdx.x == 0) a.offsets[e] = (int32_t)first;
            uint32_t at = first + before[e];
            for (int w = 0; w < kRowsWaves; w++) {
                const uint32_t c = start[w * n + e];
                start[w * n + e] = at;
                at += c;
            }
            first += all[e];
        }
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz((unsigned)a.E);
    for (int i0 = r.first; i0 < r.end; i0 += 64) {
        const int slot = i0 + lane;
        const bool there = slot < r.end;
        const int e = there ? bucket(a, slot) : 0;
        uint64_t same = __ballot(there);
        for (int b = 0; b < bits; b++) {
            const uint64_t set = __ballot(e >> b & 1);
            same &= e >> b & 1 ? set : ~set;
        }
        if (there) {
            const int rank = __popcll(same & ((1ull << lane) - 1));
            const uint32_t at = start[wave * n + e] + (uint32_t)rank;
            a.source[at] = slot;
            a.row[slot] = e < a.E ? (int32_t)at : -1;
            if (rank == 0) start[wave * n + e] += (uint32_t)__popcll(same);
        }
    }
}

// ---- way back -----------------------------------------------------------------

// out[t] = residual[t] + the token's rows in the order of its choices, fp32, rounded
// once; a choice without a row adds nothing.  A thread takes eight elements, four of a
// token's rows in flight.  Bound by memory: 32768 tokens of 8 rows, 2048 bf16 (1.24 GB):
// 230 us, 5.4 TB/s.
template <bool F32, bool RES, bool EVEN>
__global__ __launch_bounds__(256) void k_expert_sum(ExpertSumArgs a, int lanes) {
    const int each = 256 / lanes;
    for (int64_t token = (int64_t)blockIdx.x * each + threadIdx.x / lanes; token < a.l.tokens;
         token += (int64_t)gridDim.x * each) {
        const int32_t *rows = a.l.row + token * a.l.k;
        by_eights<EVEN>((threadIdx.x % lanes) * 8, lanes * 8, a.width, [&](auto full, int c) {
            constexpr bool kFull = decltype(full)::value;
            const int have = a.width - c;
            float s[8];
            if constexpr (RES) {
                load_eight<F32, kFull>(a.residual, token * a.rs + c, have, s);
            } else {
#pragma unroll
                for (int q = 0; q < 8; q++) s[q] = 0.0f;
            }
            for (int j0 = 0; j0 < a.l.k; j0 += 4) {
                float v[4][8];
                bool there[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const uint32_t r = j0 + j < a.l.k ? (uint32_t)rows[j0 + j] : 0xFFFFFFFFu;
                    there[j] = r < (uint32_t)a.l.slots;
                    load_eight<F32, kFull>(a.y, (there[j] ? (int64_t)r : 0) * a.ys + c, have, v[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int q = 0; q < 8; q++) s[q] += there[j] ? v[j][q] : 0.0f;
            }
            store_eight<F32, kFull>(a.out, token * a.os + c, have, s);
        });
    }
}

// ---- activation ---------------------------------------------------------------

// 1 / (1 + exp(-x)), off by a few units of the last place: the exponent's product is
// carried with its error (2^p (1 + r ln 2)).  0 below -87, where the sum's reciprocal is
// no normal number: x of fp32's lowest end times the least normal one would be -4, and is 0.
// Above 126 the exponential is 0 and the result 1; held there, since of x beyond 2.36e38 the
// product is infinite and its error NaN.
__device__ __forceinline__ float sigmoid(float x) {
    const float t = __builtin_fmaxf(__builtin_fminf(-x, 87.0f), -126.0f);
    const float p = t * 1.44269502f;
    const float r = __builtin_fmaf(t, 1.92596303e-08f, __builtin_fmaf(t, 1.44269502f, -p));
    const float e = __builtin_amdgcn_exp2f(p);
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e, r * 0.693147182f, e));
    return x < -87.0f ? 0.0f : s;
}

// max(x, 0) and its gradient; a NaN stays one
__device__ __forceinline__ float relu(float x) { return x <= 0.0f ? 0.0f : x; }
__device__ __forceinline__ float relu_back(float x, float d) { return x <= 0.0f ? 0.0f : x > 0.0f ? d : x; }

// `lanes` threads to a row (64 or a power of two below), eight columns each: no
// division, and the gate's gradient, a sum over the row, stays in a wave.  EVEN: widths of
// whole eights; KEEP: of whole blocks of 32, which four neighbouring threads hold.
template <bool F32, bool GATED, bool EVEN, bool KEEP>
__global__ __launch_bounds__(256) void k_act(ExpertActArgs a, int lanes) {
    const int rows = clampi(a.l.offsets[a.l.E], 0, a.l.slots), U = GATED ? 2 * a.width : a.width;
    const uint32_t round = KEEP ? a.key.round + (a.key.d_round ? *a.key.d_round : 0) : 0;
    const int each = 256 / lanes;
    for (int64_t row = (int64_t)blockIdx.x * each + threadIdx.x / lanes; row < rows; row += (int64_t)gridDim.x * each) {
        const uint32_t slot = (uint32_t)a.l.source[row];
        const float gate = slot < (uint32_t)a.l.slots ? a.gates[slot] : 0.0f;
        by_eights<EVEN>((threadIdx.x % lanes) * 8, lanes * 8, a.width, [&](auto full, int c) {
            constexpr bool kFull = decltype(full)::value;
            const int have = a.width - c;
            float g[8], v[8], o[8];
            load_eight<F32, kFull>(a.u, row * a.us + c, have, g);
            if (GATED) load_eight<F32, kFull>(a.u, row * a.us + a.width + c, have, v);
#pragma unroll
            for (int q = 0; q < 8; q++) o[q] = gate * (GATED ? g[q] * sigmoid(g[q]) * v[q] : relu(g[q]));
            store_eight<F32, kFull>(a.a, row * a.as + c, have, o);
            if constexpr (KEEP && kFull) {
                const int64_t blocks = U / 32;
#pragma unroll
                for (int half = 0; half < (GATED ? 2 : 1); half++) {
                    const int col = half * a.width + c;
                    uint32_t w[4], exponent;
                    keep_dithers<true>(row * U + col, a.key, round, w);
                    store_codes<true>(a.codes + row * U + col, 8, keep_eight(half ? v : g, w, exponent));
                    if ((threadIdx.x & 3) == 0) a.exponents[row * blocks + col / 32] = (uint8_t)exponent;
                }
            }
        });
    }
}

// From the kept codes or from u itself: du, the activation again, and the gates'
// gradient (0 for a slot without an expert).  16384 rows of 2 x 2048 bf16 from codes: 48 us
// for 320 MB, 6 TB/s or more, part of it from the last-level cache.
template <bool F32, bool GATED, bool EVEN, bool KEPT>
__global__ __launch_bounds__(256) void k_act_backward(ExpertActArgs a, int lanes) {
    const int rows = clampi(a.l.offsets[a.l.E], 0, a.l.slots), U = GATED ? 2 * a.width : a.width;
    const int each = 256 / lanes;
    for (int64_t row = (int64_t)blockIdx.x * each + threadIdx.x / lanes; row < a.l.slots;
         row += (int64_t)gridDim.x * each) {
        const uint32_t slot = (uint32_t)a.l.source[row];
        const bool known = slot < (uint32_t)a.l.slots;
        const int lane = threadIdx.x % lanes;
        if (row >= rows) {
            if (a.dgates && known && lane == 0) a.dgates[slot] = 0.0f;
            continue;
        }
        const float gate = known ? a.gates[slot] : 0.0f;
        const int64_t blocks = (U + 31) / 32;
        float sum = 0.0f;
        by_eights<EVEN>(lane * 8, lanes * 8, a.width, [&](auto full, int c) {
            constexpr bool kFull = decltype(full)::value;
            const int have = a.width - c;
            const auto columns = [&](int col, float *v) {
                if constexpr (!KEPT) {
                    load_eight<F32, kFull>(a.u, row * a.us + col, have, v);
                } else {
                    // of one block, or (the value half of an odd width) of two
                    const uint8_t *e = a.exponents + row * blocks;
                    const float s0 = kept_scale(e[col / 32]);
                    const float s1 = EVEN ? s0 : kept_scale(e[(col + (have < 8 ? have : 8) - 1) / 32]);
                    const uint2 w = load_codes<kFull>(a.codes + row * U + col, have);
#pragma unroll
                    for (int q = 0; q < 8; q++)
                        v[q] = kept_value(q < 4 ? w.x : w.y, q & 3, EVEN || col % 32 + q < 32 ? s0 : s1);
                }
            };
            float g[8], v[8], d[8], dg[8], dv[8], o[8];
            columns(c, g);
            if (GATED) columns(a.width + c, v);
            load_eight<F32, kFull>(a.da, row * a.das + c, have, d);
#pragma unroll
            for (int q = 0; q < 8; q++) {
                float h;
                if (GATED) {
                    const float s = sigmoid(g[q]), silu = g[q] * s, t = gate * d[q];
                    h = silu * v[q];
                    dv[q] = t * silu;
                    dg[q] = t * v[q] * s * (1.0f + g[q] * (1.0f - s));
                } else {
                    h = relu(g[q]);
                    dg[q] = relu_back(g[q], gate * d[q]);
                }
                o[q] = gate * h;
                sum += kFull || q < have ? d[q] * h : 0.0f;
            }
            store_eight<F32, kFull>(a.du, row * a.dus + c, have, dg);
            if (GATED) store_eight<F32, kFull>(a.du, row * a.dus + a.width + c, have, dv);
            if (a.a) store_eight<F32, kFull>(a.a, row * a.as + c, have, o);
        });
        for (int d = lanes / 2; d > 0; d /= 2) sum += __shfl_xor(sum, d, 64);
        if (a.dgates && known && lane == 0) a.dgates[slot] = sum;
    }
}

// Threads to a row of so many columns.
int lanes_for(int width, int least) {
    int lanes = least;
    while (8 * lanes < width && lanes < 64) lanes *= 2;
    return lanes;
}

// Blocks that go over so many rows once, up to 2^22 (a launch has below 2^32 threads).
dim3 row_grid(int64_t rows, int lanes) {
    const int64_t want = (rows + 256 / lanes - 1) / (256 / lanes);
    return dim3((unsigned)(want < (1 << 22) ? want : (1 << 22)));
}

template <bool F32, bool GATED>
hipError_t act_as(const ExpertActArgs &a, hipStream_t s) {
    const bool fused = a.codes && a.width % 32 == 0;
    const int lanes = lanes_for(a.width, 4);
    const dim3 grid = row_grid(a.l.slots, lanes), block(256);
    if (fused)
        hipLaunchKernelGGL((k_act<F32, GATED, true, true>), grid, block, 0, s, a, lanes);
    else if (a.width % 8 == 0)
        hipLaunchKernelGGL((k_act<F32, GATED, true, false>), grid, block, 0, s, a, lanes);
    else
        hipLaunchKernelGGL((k_act<F32, GATED, false, false>), grid, block, 0, s, a, lanes);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.codes || fused) return e;
    // blocks of 32 that cross the halves, or are short
    const int64_t U = GATED ? 2 * (int64_t)a.width : a.width;
    const KeepArgs k{a.u, a.l.slots, U, a.us, a.l.offsets + a.l.E, a.codes, a.exponents, a.key};
    return launch_keep8(k, F32, s);
}

template <bool F32, bool GATED, bool EVEN>
hipError_t act_backward_as(const ExpertActArgs &a, hipStream_t s) {
    const int lanes = lanes_for(a.width, 4);
    const dim3 grid = row_grid(a.l.slots, lanes), block(256);
    if (a.codes)
        hipLaunchKernelGGL((k_act_backward<F32, GATED, EVEN, true>), grid, block, 0, s, a, lanes);
    else
        hipLaunchKernelGGL((k_act_backward<F32, GATED, EVEN, false>), grid, block, 0, s, a, lanes);
    return hipGetLastError();
}
template <bool F32>
hipError_t act_backward_of(const ExpertActArgs &a, hipStream_t s) {
    const bool even = a.width % 8 == 0;
    if (a.gated) return even ? act_backward_as<F32, true, true>(a, s) : act_backward_as<F32, true, false>(a, s);
    return even ? act_backward_as<F32, false, true>(a, s) : act_backward_as<F32, false, false>(a, s);
}

template <bool F32, bool EVEN>
hipError_t sum_as(const ExpertSumArgs &a, hipStream_t s) {
    const int lanes = a.width > 1024 ? 256 : lanes_for(a.width, 1);
    const dim3 grid = row_grid(a.l.tokens, lanes), block(256);
    if (a.residual)
        hipLaunchKernelGGL((k_expert_sum<F32, true, EVEN>), grid, block, 0, s, a, lanes);
    else
        hipLaunchKernelGGL((k_expert_sum<F32, false, EVEN>), grid, block, 0, s, a, lanes);
    return hipGetLastError();
}

}  // namespace

int expert_rows_blocks(int64_t slots) {
    if (slots <= kRowsAlone) return 1;
    const int64_t want = (slots + 2047) / 2048;
    return (int)(want < kRowsMostBlocks ? want : kRowsMostBlocks);
}

hipError_t launch_expert_rows(const ExpertRowsArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.blocks), block(kRowsThreads);
    if (a.blocks > 1) {
        hipLaunchKernelGGL(k_rows_count, grid, block, 4 * (a.E + 1), s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k_rows_place, grid, block, 4 * (kRowsWaves + 2) * (a.E + 1), s, a);
    return hipGetLastError();
}

hipError_t launch_expert_sum(const ExpertSumArgs &a, int f32, hipStream_t s) {
    if (a.l.tokens == 0) return hipSuccess;
    if (a.width % 8 == 0) return f32 ? sum_as<true, true>(a, s) : sum_as<false, true>(a, s);
    return f32 ? sum_as<true, false>(a, s) : sum_as<false, false>(a, s);
}

hipError_t launch_expert_act(const ExpertActArgs &a, int f32, hipStream_t s) {
    if (a.l.slots == 0) return hipSuccess;
    if (f32) return a.gated ? act_as<true, true>(a, s) : act_as<true, false>(a, s);
    return a.gated ? act_as<false, true>(a, s) : act_as<false, false>(a, s);
}

hipError_t launch_expert_act_backward(const ExpertActArgs &a, int f32, hipStream_t s) {
    if (a.l.slots == 0) return hipSuccess;
    return f32 ? act_backward_of<true>(a, s) : act_backward_of<false>(a, s);
}

}  // namespace dq
