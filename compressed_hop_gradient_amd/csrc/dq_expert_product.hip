// dq_expert_product.hip -- products grouped by expert for gfx950: rows by the
// experts' weights, and the weights' gradient.
#include "dq_expert_tile.h"

namespace dq {

namespace {

// y[r] = x[r] w[e(r)] over the experts' rows: A is x, contiguous along the inner
// index; B is w, contiguous along the outer one, or along the inner one (TURNED).
template <class C, int LA, int LB, bool TURNED>
__global__ __launch_bounds__(C::kThreads) void k_product(ExpertProductArgs a, int nt) {
    typedef typename C::T T;
    extern __shared__ __align__(1024) char lds[];
    RowTile t;
    if (!find_tile<C::kThreads>(a.l, C::BM, nt, t, reinterpret_cast<int *>(lds))) return;
    const int n0 = t.n * C::BN;
    Acc<C> acc;
    typename std::conditional<TURNED, Along<C, C::BN, LB>, Across<C, C::BN, LB>>::type b;
    Along<C, C::BM, LA> x;
    x.start(static_cast<const T *>(a.x), a.K, [&](int i) {
        const int r = t.first + (i < t.rows ? i : t.rows - 1);
        return row_at(a.l, r, a.gather, a.xs);
    });
    const T *w = static_cast<const T *>(a.w) + t.e * a.we;
    if constexpr (TURNED)
        b.start(w, a.K, [&](int i) { return (int64_t)min(n0 + i, a.N - 1) * a.ws; });
    else
        b.start(w, n0, a.N, a.K);
    const auto row_b = [&](int k) { return (int64_t)k * a.ws; };
    multiply<C>(lds, x, b, a.K, [](int) { return (int64_t)0; }, row_b, acc);
    acc.store([&](int m) { return m < t.rows ? static_cast<T *>(a.y) + (t.first + m) * a.ys : nullptr; }, n0, a.N,
              vec_out<T>(a.y, a.ys, a.N));
}

// dw[e] = the sum of x[r]^T dy[r] over e's rows (or over a part of them, into fp32).
template <class C, int LA, int LB, typename Out>
__global__ __launch_bounds__(C::kThreads) void k_weights(ExpertWeightsArgs a, int mt, int nt, int64_t total) {
    typedef typename C::T T;
    extern __shared__ __align__(1024) char lds[];
    int64_t id = own_tile(blockIdx.x, total);
    if (id >= total) return;
    const int part = (int)(id % a.parts);
    id /= a.parts;
    const int m0 = (int)(id % mt) * C::BM;
    id /= mt;
    const int n0 = (int)(id % nt) * C::BN, e = (int)(id / nt);
    int first = expert_first(a.l, e), rows = max(0, expert_first(a.l, e + 1) - first);
    if (a.parts > 1) {
        // whole steps of the inner loop
        const int per = ((rows + a.parts - 1) / a.parts + C::BK - 1) / C::BK * C::BK;
        const int at = min(part * per, rows);
        rows = min(per, rows - at);
        first += at;
    }
    Acc<C> acc;
    Across<C, C::BM, LA> x;
    Across<C, C::BN, LB> dy;
    if constexpr (LA == kKept || LA == kKeptAny)
        x.start(a.codes, a.exponents, m0, a.K, rows);
    else
        x.start(static_cast<const T *>(a.x), m0, a.K, rows);
    dy.start(static_cast<const T *>(a.dy), n0, a.N, rows);
    // of codes, the row's number
    const int64_t xs = LA == kKept || LA == kKeptAny ? 1 : a.xs;
    multiply<C>(lds, x, dy, rows, [&](int k) { return row_at(a.l, first + k, a.gather_x, xs); },
                [&](int k) { return row_at(a.l, first + k, a.gather_dy, a.dys); }, acc);
    Out *dw = static_cast<Out *>(a.parts > 1 ? (void *)a.partial : a.dw) +
              ((int64_t)part * a.l.E + e) * a.K * a.N;
    acc.store([&](int m) { return m0 + m < a.K ? dw + (int64_t)(m0 + m) * a.N : nullptr; }, n0, a.N,
              vec_out<Out>(dw, a.N, a.N));
}

// The parts' sums, in their order.
template <typename Out>
__global__ __launch_bounds__(256) void k_weights_join(const float *partial, int parts, int64_t n, Out *dw) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float s = partial[i];
        for (int p = 1; p < parts; p++) s += partial[p * n + i];
        store_one(dw + i, s);
    }
}

template <class C>
int64_t most_row_tiles(const ExpertLists &l) {
    const int64_t most = ((int64_t)l.slots + (int64_t)l.E * (C::BM - 1)) / C::BM;
    return most < l.slots ? most : l.slots;
}

dim3 whole_rounds(int64_t tiles) { return dim3((unsigned)((tiles + 7) / 8 * 8)); }

template <class C, int LA, int LB, bool TURNED>
hipError_t product_as(const ExpertProductArgs &a, hipStream_t s) {
    const int nt = (a.N + C::BN - 1) / C::BN;
    const int64_t tiles = most_row_tiles<C>(a.l) * nt;
    if (tiles > (1 << 30)) return hipErrorInvalidValue;
    const auto kernel = k_product<C, LA, LB, TURNED>;
    const hipError_t e = room_for(kernel, C::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, whole_rounds(tiles), dim3(C::kThreads), C::kLds, s, a, nt);
    return hipGetLastError();
}

template <class C>
hipError_t product_loads(const ExpertProductArgs &a, hipStream_t s) {
    constexpr int64_t es = sizeof(typename C::T);
    const bool va = on16(a.x, a.xs * es) && a.K % C::kChunk == 0;
    const bool vb = on16(a.w, a.ws * es) && (a.l.E == 1 || a.we * es % 16 == 0) &&
                    (a.turned ? a.K : a.N) % C::kChunk == 0;
    if (a.turned) {
        if (va && vb) return product_as<C, kAsync, kAsync, true>(a, s);
        return product_as<C, kAny, kAny, true>(a, s);
    }
    if (va && vb) return product_as<C, kAsync, kAsync, false>(a, s);
    return product_as<C, kAny, kAny, false>(a, s);
}

template <class C, int LA, int LB, typename Out>
hipError_t weights_as(const ExpertWeightsArgs &a, hipStream_t s) {
    const int mt = (a.K + C::BM - 1) / C::BM, nt = (a.N + C::BN - 1) / C::BN;
    const int64_t tiles = (int64_t)mt * nt * a.l.E * a.parts;
    if (tiles > (1 << 30)) return hipErrorInvalidValue;
    const auto kernel = k_weights<C, LA, LB, Out>;
    const hipError_t e = room_for(kernel, C::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, whole_rounds(tiles), dim3(C::kThreads), C::kLds, s, a, mt, nt, tiles);
    return hipGetLastError();
}

template <class C, typename Out>
hipError_t weights_loads(const ExpertWeightsArgs &a, hipStream_t s) {
    constexpr int64_t es = sizeof(typename C::T);
    const bool vb = on16(a.dy, a.dys * es) && a.N % C::kChunk == 0;
    if (a.codes) {
        const bool va = on16(a.codes, 16) && a.K % 16 == 0;
        if (va && vb) return weights_as<C, kKept, kAsync, Out>(a, s);
        return weights_as<C, kKeptAny, kAny, Out>(a, s);
    }
    const bool va = on16(a.x, a.xs * es) && a.K % C::kChunk == 0;
    if (va && vb) return weights_as<C, kAsync, kAsync, Out>(a, s);
    return weights_as<C, kAny, kAny, Out>(a, s);
}

template <class C>
hipError_t weights_out(const ExpertWeightsArgs &a, hipStream_t s) {
    if (a.out_f32 || a.parts > 1) return weights_loads<C, float>(a, s);
    if constexpr (sizeof(typename C::T) == 2) return weights_loads<C, uint16_t>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_expert_product(const ExpertProductArgs &a, int f32, hipStream_t s) {
    if (a.l.slots == 0 || a.N == 0) return hipSuccess;
    if (f32) return product_loads<TileF32>(a, s);
    return product_loads<TileMid>(a, s);
}

int expert_weights_parts(int64_t, int, int64_t, int64_t, int) { return 1; }

hipError_t launch_expert_weights(const ExpertWeightsArgs &a, int f32, hipStream_t s) {
    if (a.K == 0 || a.N == 0) return hipSuccess;
    hipError_t e = f32 ? weights_out<TileF32>(a, s) : weights_out<TileMid>(a, s);
    if (e != hipSuccess || a.parts == 1) return e;
    const int64_t n = (int64_t)a.l.E * a.K * a.N, blocks = (n + 1023) / 1024;
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
    if (a.out_f32)
        hipLaunchKernelGGL((k_weights_join<float>), grid, dim3(256), 0, s, a.partial, a.parts, n, static_cast<float *>(a.dw));
    else
        hipLaunchKernelGGL((k_weights_join<uint16_t>), grid, dim3(256), 0, s, a.partial, a.parts, n,
                           static_cast<uint16_t *>(a.dw));
    return hipGetLastError();
}

}  // namespace dq
