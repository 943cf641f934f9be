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
// once; a choice without a row adds nothing.  VEC: eight elements a thread.
template <bool F32, bool RES, bool VEC>
__global__ __launch_bounds__(256) void k_expert_sum(ExpertSumArgs a, int lanes) {
    typedef Elem<F32> El;
    typedef typename El::type T;
    constexpr int kEach = VEC ? 8 : 1;
    const int64_t token = (int64_t)blockIdx.x * (256 / lanes) + threadIdx.x / lanes;
    if (token >= a.l.tokens) return;
    const int32_t *rows = a.l.row + token * a.l.k;
    const T *y = static_cast<const T *>(a.y);
    for (int c = (threadIdx.x % lanes) * kEach; c < a.width; c += lanes * kEach) {
        float s[kEach];
        if constexpr (!RES) {
#pragma unroll
            for (int q = 0; q < kEach; q++) s[q] = 0.0f;
        } else if constexpr (VEC) {
            load8<F32>(a.residual, token * a.rs + c, s);
        } else {
            s[0] = El::up(static_cast<const T *>(a.residual)[token * a.rs + c]);
        }
        for (int j0 = 0; j0 < a.l.k; j0 += 4) {
            float v[4][kEach];
            bool there[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t r = j0 + j < a.l.k ? (uint32_t)rows[j0 + j] : 0xFFFFFFFFu;
                there[j] = r < (uint32_t)a.l.slots;
                const int64_t at = (there[j] ? (int64_t)r : 0) * a.ys + c;
                if constexpr (VEC)
                    load8<F32>(y, at, v[j]);
                else
                    v[j][0] = El::up(y[at]);
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int q = 0; q < kEach; q++) s[q] += there[j] ? v[j][q] : 0.0f;
        }
        if constexpr (VEC)
            store8<F32>(a.out, token * a.os + c, s);
        else
            static_cast<T *>(a.out)[token * a.os + c] = El::down(s[0]);
    }
}

// ---- activation ---------------------------------------------------------------

// 1 / (1 + exp(-x)), off by a few units of the last place: the exponent's product is
// carried with its error (2^p (1 + r ln 2)), and held below 2^126, where the sum's
// reciprocal is still a normal number.
__device__ __forceinline__ float sigmoid(float x) {
    const float t = __builtin_fminf(-x, 87.0f);
    const float p = t * 1.44269502f;
    const float r = __builtin_fmaf(t, 1.92596303e-08f, __builtin_fmaf(t, 1.44269502f, -p));
    const float e = __builtin_amdgcn_exp2f(p);
    return __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e, r * 0.693147182f, e));
}

// max(x, 0) and its gradient; a NaN stays one
__device__ __forceinline__ float relu(float x) { return x <= 0.0f ? 0.0f : x; }
__device__ __forceinline__ float relu_back(float x, float d) { return x <= 0.0f ? 0.0f : x > 0.0f ? d : x; }

template <bool F32, bool VEC>
__device__ __forceinline__ void read(const void *p, int64_t at, float *v) {
    if constexpr (VEC)
        load8<F32>(p, at, v);
    else
        v[0] = Elem<F32>::up(static_cast<const typename Elem<F32>::type *>(p)[at]);
}
template <bool F32, bool VEC>
__device__ __forceinline__ void write(void *p, int64_t at, const float *v) {
    if constexpr (VEC)
        store8<F32>(p, at, v);
    else
        static_cast<typename Elem<F32>::type *>(p)[at] = Elem<F32>::down(v[0]);
}

// `lanes` threads to a row (64 or a power of two below): no division, and the gate's
// gradient, a sum over the row, stays in a wave.
template <bool F32, bool GATED, bool VEC, bool KEEP>
__global__ __launch_bounds__(256) void k_act(ExpertActArgs a, int lanes) {
    constexpr int kEach = VEC ? 8 : 1;
    const int rows = clampi(a.l.offsets[a.l.E], 0, a.l.slots), U = GATED ? 2 * a.width : a.width;
    const uint32_t round = KEEP ? a.key.round + (a.key.d_round ? *a.key.d_round : 0) : 0;
    const int64_t row = (int64_t)blockIdx.x * (256 / lanes) + threadIdx.x / lanes;
    if (row >= rows) return;
    const uint32_t slot = (uint32_t)a.l.source[row];
    const float gate = slot < (uint32_t)a.l.slots ? a.gates[slot] : 0.0f;
    for (int c = (threadIdx.x % lanes) * kEach; c < a.width; c += lanes * kEach) {
        float g[kEach], v[kEach], o[kEach];
        read<F32, VEC>(a.u, row * a.us + c, g);
        if (GATED) read<F32, VEC>(a.u, row * a.us + a.width + c, v);
#pragma unroll
        for (int q = 0; q < kEach; q++)
            o[q] = gate * (GATED ? g[q] * sigmoid(g[q]) * v[q] : relu(g[q]));
        write<F32, VEC>(a.a, row * a.as + c, o);
        if constexpr (KEEP) {
            const int64_t blocks = U / 32;
#pragma unroll
            for (int half = 0; half < (GATED ? 2 : 1); half++) {
                const int col = half * a.width + c;
                uint32_t w[4], exponent;
                keep_dithers<true>(row * U + col, a.key, round, w);
                *reinterpret_cast<uint2 *>(a.codes + row * U + col) = keep_eight(half ? v : g, w, exponent);
                if ((threadIdx.x & 3) == 0) a.exponents[row * blocks + col / 32] = (uint8_t)exponent;
            }
        }
    }
}

// From the kept codes or from u itself: du, the activation again, and the gates'
// gradient (0 for a slot without an expert).
template <bool F32, bool GATED, bool VEC, bool KEPT>
__global__ __launch_bounds__(256) void k_act_backward(ExpertActArgs a, int lanes) {
    constexpr int kEach = VEC ? 8 : 1;
    const int rows = clampi(a.l.offsets[a.l.E], 0, a.l.slots), U = GATED ? 2 * a.width : a.width;
    const int64_t row = (int64_t)blockIdx.x * (256 / lanes) + threadIdx.x / lanes;
    if (row >= a.l.slots) return;
    const uint32_t slot = (uint32_t)a.l.source[row];
    const bool known = slot < (uint32_t)a.l.slots;
    const int lane = threadIdx.x % lanes;
    if (row >= rows) {
        if (a.dgates && known && lane == 0) a.dgates[slot] = 0.0f;
        return;
    }
    const float gate = known ? a.gates[slot] : 0.0f;
    const int64_t blocks = (U + 31) / 32;
    const auto half = [&](int col, float *v) {
        if constexpr (!KEPT) {
            read<F32, VEC>(a.u, row * a.us + col, v);
        } else {
            const float scale = kept_scale(a.exponents[row * blocks + col / 32]);
            if constexpr (VEC) {
                const uint2 c = *reinterpret_cast<const uint2 *>(a.codes + row * U + col);
#pragma unroll
                for (int q = 0; q < 8; q++) v[q] = kept_value(q < 4 ? c.x : c.y, q & 3, scale);
            } else {
                v[0] = (float)a.codes[row * U + col] * scale;
            }
        }
    };
    float sum = 0.0f;
    for (int c = lane * kEach; c < a.width; c += lanes * kEach) {
        float g[kEach], v[kEach], d[kEach], dg[kEach], dv[kEach], o[kEach];
        half(c, g);
        if (GATED) half(a.width + c, v);
        read<F32, VEC>(a.da, row * a.das + c, d);
#pragma unroll
        for (int q = 0; q < kEach; q++) {
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
            sum += d[q] * h;
        }
        write<F32, VEC>(a.du, row * a.dus + c, dg);
        if (GATED) write<F32, VEC>(a.du, row * a.dus + a.width + c, dv);
        if (a.a) write<F32, VEC>(a.a, row * a.as + c, o);
    }
    for (int d = lanes / 2; d > 0; d /= 2) sum += __shfl_xor(sum, d, 64);
    if (a.dgates && known && lane == 0) a.dgates[slot] = sum;
}

int lanes_for(int chunks, int least) {
    int lanes = least;
    while (lanes < chunks && lanes < 64) lanes *= 2;
    return lanes;
}

bool vec8(const void *p, int64_t stride, int64_t es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * es % 16 == 0;
}

dim3 row_grid(int64_t rows, int lanes) { return dim3((unsigned)((rows + 256 / lanes - 1) / (256 / lanes))); }

template <bool F32, bool GATED>
hipError_t act_as(const ExpertActArgs &a, hipStream_t s) {
    const int64_t es = F32 ? 4 : 2, U = GATED ? 2 * a.width : a.width;
    const bool vec = a.width % 8 == 0 && vec8(a.u, a.us, es) && vec8(a.a, a.as, es);
    const bool fused = a.codes && vec && a.width % 32 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
    const int lanes = vec ? lanes_for(a.width / 8, 4) : lanes_for(a.width, 4);
    const dim3 grid = row_grid(a.l.slots, lanes), block(256);
    if (fused)
        hipLaunchKernelGGL((k_act<F32, GATED, true, true>), grid, block, 0, s, a, lanes);
    else if (vec)
        hipLaunchKernelGGL((k_act<F32, GATED, true, false>), grid, block, 0, s, a, lanes);
    else
        hipLaunchKernelGGL((k_act<F32, GATED, false, false>), grid, block, 0, s, a, lanes);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.codes || fused) return e;
    // blocks of 32 that cross the halves, or rows off their alignment
    const KeepArgs k{a.u, a.l.slots, U, a.us, a.l.offsets + a.l.E, a.codes, a.exponents, a.key};
    return launch_keep8(k, F32, s);
}

template <bool F32, bool GATED>
hipError_t act_backward_as(const ExpertActArgs &a, hipStream_t s) {
    const int64_t es = F32 ? 4 : 2;
    const bool vec = a.width % 8 == 0 && vec8(a.du, a.dus, es) && vec8(a.da, a.das, es) &&
                     (!a.a || vec8(a.a, a.as, es)) &&
                     (a.codes ? reinterpret_cast<uintptr_t>(a.codes) % 8 == 0 : vec8(a.u, a.us, es));
    const int lanes = vec ? lanes_for(a.width / 8, 4) : lanes_for(a.width, 4);
    const dim3 grid = row_grid(a.l.slots, lanes), block(256);
    if (a.codes && vec)
        hipLaunchKernelGGL((k_act_backward<F32, GATED, true, true>), grid, block, 0, s, a, lanes);
    else if (a.codes)
        hipLaunchKernelGGL((k_act_backward<F32, GATED, false, true>), grid, block, 0, s, a, lanes);
    else if (vec)
        hipLaunchKernelGGL((k_act_backward<F32, GATED, true, false>), grid, block, 0, s, a, lanes);
    else
        hipLaunchKernelGGL((k_act_backward<F32, GATED, false, false>), grid, block, 0, s, a, lanes);
    return hipGetLastError();
}

template <bool F32>
hipError_t sum_as(const ExpertSumArgs &a, hipStream_t s) {
    const int64_t es = F32 ? 4 : 2;
    const bool vec = a.width % 8 == 0 && vec8(a.y, a.ys, es) && vec8(a.out, a.os, es) &&
                     (!a.residual || vec8(a.residual, a.rs, es));
    int lanes = vec ? lanes_for(a.width / 8, 1) : lanes_for(a.width, 1);
    if (lanes == 64 && a.width > (vec ? 1024 : 128)) lanes = 256;
    const dim3 grid = row_grid(a.l.tokens, lanes), block(256);
    if (a.residual && vec)
        hipLaunchKernelGGL((k_expert_sum<F32, true, true>), grid, block, 0, s, a, lanes);
    else if (a.residual)
        hipLaunchKernelGGL((k_expert_sum<F32, true, false>), grid, block, 0, s, a, lanes);
    else if (vec)
        hipLaunchKernelGGL((k_expert_sum<F32, false, true>), grid, block, 0, s, a, lanes);
    else
        hipLaunchKernelGGL((k_expert_sum<F32, false, false>), grid, block, 0, s, a, lanes);
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
    return f32 ? sum_as<true>(a, s) : sum_as<false>(a, s);
}

hipError_t launch_expert_act(const ExpertActArgs &a, int f32, hipStream_t s) {
    if (a.l.slots == 0) return hipSuccess;
    if (f32) return a.gated ? act_as<true, true>(a, s) : act_as<true, false>(a, s);
    return a.gated ? act_as<false, true>(a, s) : act_as<false, false>(a, s);
}

hipError_t launch_expert_act_backward(const ExpertActArgs &a, int f32, hipStream_t s) {
    if (a.l.slots == 0) return hipSuccess;
    if (f32) return a.gated ? act_backward_as<true, true>(a, s) : act_backward_as<true, false>(a, s);
    return a.gated ? act_backward_as<false, true>(a, s) : act_backward_as<false, false>(a, s);
}

}  // namespace dq
