// dq_train.hip -- HIP kernels of the training-step operators for gfx950: dropout
// from the counter-based generator, and the expert router with its balance
// statistics and gradients.  fp32 arithmetic, no contraction.
#include "dq_train.h"

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

// kFlat: one row, 16-byte aligned; kRows: rows of a multiple of 8 elements,
// every row 16-byte aligned; kAny: element by element, any alignment
enum Access { kFlat, kRows, kAny };

// A thread takes the eight elements of one Philox block.
template <bool F32, bool RES, int ACCESS>
__global__ __launch_bounds__(256) void k_dropout(DropoutArgs a, int64_t blocks) {
    typedef Elem<F32> El;
    typedef typename El::type T;
    const uint32_t round = a.round + (a.d_round ? *a.d_round : 0);
    const int64_t n = a.rows * a.cols;
    for (int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x; b < blocks; b += (int64_t)gridDim.x * 256) {
        uint32_t w[4] = {0, 0, 0, 0};
        if (a.threshold) dropout_words((uint64_t)b, a, round, w);   // T = 0 keeps everything
        int64_t row = 0, col = 8 * b;
        if (ACCESS != kFlat) {
            row = col / a.cols;
            col -= row * a.cols;
        }
        if (ACCESS != kAny && 8 * b + 8 <= n) {
            float x[8], r[8];
            load8<F32>(a.x, row * a.xs + col, x);
            if (RES) load8<F32>(a.residual, row * a.rs + col, r);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                x[j] = dither(w, j) >= a.threshold ? x[j] * a.scale : 0.0f;
                if (RES) x[j] = r[j] + x[j];
            }
            store8<F32>(a.y, row * a.ys + col, x);
        } else {
            const int m = (int)(n - 8 * b < 8 ? n - 8 * b : 8);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (j >= m) break;
                float v = El::up(static_cast<const T *>(a.x)[row * a.xs + col]);
                v = dither(w, j) >= a.threshold ? v * a.scale : 0.0f;
                if (RES) v = El::up(static_cast<const T *>(a.residual)[row * a.rs + col]) + v;
                static_cast<T *>(a.y)[row * a.ys + col] = El::down(v);
                if (++col == a.cols) {
                    col = 0;
                    row++;
                }
            }
        }
    }
}

template <bool F32, bool RES>
hipError_t dropout_access(const DropoutArgs &a, hipStream_t s) {
    const int64_t es = F32 ? 4 : 2;
    const int64_t blocks = (a.rows * a.cols + 7) / 8;
    const int64_t want = (blocks + 255) / 256;
    const dim3 grid((unsigned)(want < (1 << 20) ? want : (1 << 20))), block(256);
    const auto on16 = [&](const void *p, int64_t stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.rows == 1 || stride * es % 16 == 0);
    };
    const bool vec = on16(a.x, a.xs) && on16(a.y, a.ys) && (!RES || on16(a.residual, a.rs));
    if (vec && a.rows == 1)
        hipLaunchKernelGGL((k_dropout<F32, RES, kFlat>), grid, block, 0, s, a, blocks);
    else if (vec && a.cols % 8 == 0)
        hipLaunchKernelGGL((k_dropout<F32, RES, kRows>), grid, block, 0, s, a, blocks);
    else
        hipLaunchKernelGGL((k_dropout<F32, RES, kAny>), grid, block, 0, s, a, blocks);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// router
// ---------------------------------------------------------------------------

// Order key of a logit: the unsigned order of keys is the order of the values,
// -0 = +0, NaN above +inf.  The key of -inf, 0x007FFFFF, is the smallest.
__device__ __forceinline__ uint32_t order_key(float x) {
    x += 0.0f;
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
constexpr uint32_t kKeyMinusInf = 0x007FFFFFu;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, d, 64);
        v = o > v ? o : v;
    }
    return v;
}

// One wave per token, V experts per lane (lane, lane + 64, ..).  With m the
// largest logit, e = exp(l - m) and Z = sum e; Z = 0 only where every logit is
// -inf, and NaN or +inf makes Z NaN and with it the row's gates and sums.
template <bool F32, int V>
__device__ __forceinline__ void softmax_row(const typename Elem<F32>::type *row, int E, int lane, float l[V],
                                            float e[V], float &m, float &Z) {
    m = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int j = lane + 64 * v;
        l[v] = j < E ? Elem<F32>::up(row[j]) : -INFINITY;
        m = fmaxf(m, l[v]);
    }
    m = wave_max(m);
    if (m == -INFINITY) m = 0.0f;
    Z = 0.0f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        e[v] = expf(l[v] - m);
        Z += e[v];
    }
    Z = wave_sum(Z);
}

template <bool F32, int V>
__global__ __launch_bounds__(256) void k_route(RouteArgs a) {
    typedef typename Elem<F32>::type T;
    __shared__ uint32_t hist[64 * V];
    __shared__ float sums[4][64 * V];
    __shared__ uint32_t routed_of[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j = threadIdx.x; j < a.E; j += 256) hist[j] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; v++) acc[v] = 0.0f;
    uint32_t routed = 0;
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.tokens; t += 4 * (int64_t)gridDim.x) {
        float l[V], e[V], m = 0.0f, Z = 0.0f;
        if (!a.mask || a.mask[t])
            softmax_row<F32, V>(static_cast<const T *>(a.logits) + t * a.stride, a.E, lane, l, e, m, Z);
        if (Z == 0.0f) {   // left out, or no expert open
            if (lane < a.k) {
                a.ids[t * a.k + lane] = -1;
                a.gates[t * a.k + lane] = 0.0f;
            }
            continue;
        }
        routed++;
        const float inv = 1.0f / Z;
        uint64_t key[V];
#pragma unroll
        for (int v = 0; v < V; v++) {
            acc[v] += e[v] * inv;
            key[v] = (uint64_t)order_key(l[v]) << 32 | (uint32_t)~(lane + 64 * v);
        }
        // k times the largest key (value, then lowest index); lane s keeps choice s
        int id = -1;
        float g = 0.0f, top = 0.0f;
        for (int s = 0; s < a.k; s++) {
            uint64_t best = 0;
#pragma unroll
            for (int v = 0; v < V; v++) best = key[v] > best ? key[v] : best;
            best = wave_max(best);
            if ((uint32_t)(best >> 32) <= kKeyMinusInf) break;
            const int j = (int)~(uint32_t)best;
            float es = 0.0f;
#pragma unroll
            for (int v = 0; v < V; v++) {
                if (key[v] == best) {
                    key[v] = 0;
                    es = e[v];
                }
            }
            es = __shfl(es, j & 63, 64);
            top += es;
            if (lane == s) {
                id = j;
                g = es;
            }
        }
        if (lane < a.k) {
            a.ids[t * a.k + lane] = id;
            a.gates[t * a.k + lane] = id < 0 ? 0.0f : g / (a.renorm ? top : Z);
            if (id >= 0) atomicAdd(&hist[id], 1u);
        }
    }
#pragma unroll
    for (int v = 0; v < V; v++) sums[wave][lane + 64 * v] = acc[v];
    if (lane == 0) routed_of[wave] = routed;
    __syncthreads();
    for (int j = threadIdx.x; j < a.E; j += 256) {
        a.psum[(int64_t)blockIdx.x * a.E + j] = ((sums[0][j] + sums[1][j]) + sums[2][j]) + sums[3][j];
        a.count[(int64_t)blockIdx.x * a.E + j] = hist[j];
    }
    if (threadIdx.x == 0)
        a.routed[blockIdx.x] = routed_of[0] + routed_of[1] + routed_of[2] + routed_of[3];
}

// Folds the blocks' partial statistics in a fixed order: a block per 64
// experts, 16 threads per expert over the rows, then a tree; the extra block
// sums the routed tokens.
__global__ __launch_bounds__(1024) void k_route_fold(RouteArgs a, double *stats, int accumulate) {
    __shared__ double ps[16][64];
    __shared__ double cs[16][64];
    const int c = threadIdx.x & 63, r = threadIdx.x >> 6;
    const bool tokens = blockIdx.x == gridDim.x - 1;
    const int j = tokens ? 0 : (int)blockIdx.x * 64 + c;
    double p = 0.0, n = 0.0;
    if (tokens) {
        for (int b = threadIdx.x; b < a.nblk; b += 1024) n += a.routed[b];
    } else if (j < a.E) {
        for (int b = r; b < a.nblk; b += 16) {
            p += a.psum[(int64_t)b * a.E + j];
            n += a.count[(int64_t)b * a.E + j];
        }
    }
    ps[r][c] = p;
    cs[r][c] = n;
    __syncthreads();
    if (r != 0) return;
    for (int i = 1; i < 16; i++) {
        p += ps[i][c];
        n += cs[i][c];
    }
    if (tokens) {
        for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d, 64);
        if (c == 0) stats[2 * a.E] = accumulate ? stats[2 * a.E] + n : n;
    } else if (j < a.E) {
        stats[j] = accumulate ? stats[j] + n : n;
        stats[a.E + j] = accumulate ? stats[a.E + j] + p : p;
    }
}

__global__ __launch_bounds__(256) void k_balance(const double *stats, int E, int k, float *loss, float *coef,
                                                 int64_t *counts) {
    __shared__ double part[4];
    const double N = stats[2 * E];
    const double f = N > 0.0 ? (double)E / ((double)k * N * N) : 0.0;
    double sum = 0.0;
    for (int j = threadIdx.x; j < E; j += 256) {
        const double c = stats[j], w = f * c;
        if (coef) coef[j] = (float)w;
        if (counts) counts[j] = (int64_t)c;
        sum += w * stats[E + j];
    }
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (loss && threadIdx.x == 0) *loss = (float)(((part[0] + part[1]) + part[2]) + part[3]);
}

// LDS traffic between the lanes of one wave: orders it for the compiler too
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// One wave per token.  The chosen experts' own term goes through a row of LDS,
// scattered by the lanes that hold the choices.
template <bool F32, int V>
__global__ __launch_bounds__(256) void k_route_backward(RouteBackwardArgs a) {
    typedef typename Elem<F32>::type T;
    __shared__ float chosen[4][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float *own = chosen[wave];
    float up[V];
    const float w = a.dloss ? *a.dloss : 1.0f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int j = lane + 64 * v;
        up[v] = a.coef && j < a.E ? w * a.coef[j] : 0.0f;
        own[j] = 0.0f;
    }
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.tokens; t += 4 * (int64_t)gridDim.x) {
        float l[V], e[V], m = 0.0f, Z = 0.0f;
        if (!a.mask || a.mask[t])
            softmax_row<F32, V>(static_cast<const T *>(a.logits) + t * a.stride, a.E, lane, l, e, m, Z);
        T *out = static_cast<T *>(a.dlogits) + t * a.dstride;
        if (Z == 0.0f) {
#pragma unroll
            for (int v = 0; v < V; v++)
                if (lane + 64 * v < a.E) out[lane + 64 * v] = Elem<F32>::down(0.0f);
            continue;
        }
        const float inv = 1.0f / Z;
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++) {
            e[v] *= inv;
            dot += e[v] * up[v];
        }
        int id = -1;
        float dg = 0.0f, g = 0.0f;
        if (a.dgates && lane < a.k) {
            id = a.ids[t * a.k + lane];
            if ((uint32_t)id >= (uint32_t)a.E) id = -1;
            if (id >= 0) {
                dg = a.dgates[t * a.k + lane];
                g = expf(Elem<F32>::up(static_cast<const T *>(a.logits)[t * a.stride + id]) - m);
            }
        }
        float top = 0.0f;
        if (a.renorm) {
            top = wave_sum(g);
            g = top != 0.0f ? g / top : 0.0f;   // top = 0 without a choice
        } else {
            g *= inv;
        }
        const float gd = wave_sum(g * dg);
        if (id >= 0) own[id] = g * (a.renorm ? dg - gd : dg);
        dot = wave_sum(dot) + (a.renorm ? 0.0f : gd);
        wave_lds_sync();
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int j = lane + 64 * v;
            if (j < a.E) out[j] = Elem<F32>::down(e[v] * (up[v] - dot) + own[j]);
        }
        wave_lds_sync();
        if (id >= 0) own[id] = 0.0f;
    }
}

template <template <bool, int> class Launch, class... Args>
hipError_t by_width(int E, int f32, Args... args) {
    const int v = (E + 63) / 64;
    if (f32) {
        if (v <= 1) return Launch<true, 1>::go(args...);
        if (v <= 2) return Launch<true, 2>::go(args...);
        if (v <= 4) return Launch<true, 4>::go(args...);
        if (v <= 8) return Launch<true, 8>::go(args...);
        return Launch<true, 16>::go(args...);
    }
    if (v <= 1) return Launch<false, 1>::go(args...);
    if (v <= 2) return Launch<false, 2>::go(args...);
    if (v <= 4) return Launch<false, 4>::go(args...);
    if (v <= 8) return Launch<false, 8>::go(args...);
    return Launch<false, 16>::go(args...);
}

template <bool F32, int V>
struct Forward {
    static hipError_t go(const RouteArgs *a, hipStream_t s) {
        hipLaunchKernelGGL((k_route<F32, V>), dim3((unsigned)a->nblk), dim3(256), 0, s, *a);
        return hipGetLastError();
    }
};
template <bool F32, int V>
struct Backward {
    static hipError_t go(const RouteBackwardArgs *a, hipStream_t s) {
        const int64_t want = (a->tokens + 3) / 4;
        hipLaunchKernelGGL((k_route_backward<F32, V>), dim3((unsigned)(want < 8192 ? want : 8192)), dim3(256), 0, s,
                           *a);
        return hipGetLastError();
    }
};

}  // namespace

hipError_t launch_dropout(const DropoutArgs &a, int f32, hipStream_t s) {
    if (f32) return a.residual ? dropout_access<true, true>(a, s) : dropout_access<true, false>(a, s);
    return a.residual ? dropout_access<false, true>(a, s) : dropout_access<false, false>(a, s);
}

int route_blocks(int64_t tokens, int) {
    const int64_t want = (tokens + 3) / 4;
    return (int)(want < 1 ? 1 : want < 2048 ? want : 2048);
}

hipError_t launch_route(const RouteArgs &a, int f32, hipStream_t s) { return by_width<Forward>(a.E, f32, &a, s); }

hipError_t launch_route_fold(const RouteArgs &a, double *stats, int accumulate, hipStream_t s) {
    hipLaunchKernelGGL(k_route_fold, dim3((unsigned)(a.E + 63) / 64 + 1), dim3(1024), 0, s, a, stats, accumulate);
    return hipGetLastError();
}

hipError_t launch_balance(const double *stats, int E, int k, float *loss, float *coef, int64_t *counts,
                          hipStream_t s) {
    hipLaunchKernelGGL(k_balance, dim3(1), dim3(256), 0, s, stats, E, k, loss, coef, counts);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs &a, int f32, hipStream_t s) {
    return by_width<Backward>(a.E, f32, &a, s);
}

}  // namespace dq
