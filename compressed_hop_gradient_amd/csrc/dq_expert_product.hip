// dq_expert_product.hip -- products grouped by expert for gfx950: rows by the
// experts' weights, and the weights' gradient.
#include "dq.h"
#include "dq_expert_tile.h"

namespace dq {

namespace {

// y[r] = x[r] w[e(r)] over the experts' rows: A is x, contiguous along the inner
// index; B is w, contiguous along the outer one (turned by the LDS read), or along the
// inner one (TURNED).  Gathered rows cost nothing: a lane's loads carry their own
// addresses.  The products of inner indexes from `from`, `inner` of them.
template <class C, int LA, int LB, bool TURNED>
__device__ __forceinline__ void product_tile(const ExpertProductArgs &a, const RowTile &t, int n0, int from, int inner,
                                             char *lds, Acc<C> &acc) {
    typedef typename C::T T;
    const bool mine = acc.m0() < t.rows && n0 + acc.n0() < a.N;
    Along<C, C::BM, LA> x;
    x.start(static_cast<const T *>(a.x) + (a.gather ? 0 : t.first * a.xs) + from, a.K, inner, [&](int i) {
        i = min(i, t.rows - 1);
        return a.gather ? row_at(a.l, t.first + i, 1, a.xs) : i * a.xs;
    });
    const T *w = static_cast<const T *>(a.w) + t.e * a.we;
    if constexpr (TURNED) {
        Along<C, C::BN, LB> b;
        b.start(w + n0 * a.ws + from, a.K, inner, [&](int i) { return min(i, a.N - 1 - n0) * a.ws; });
        multiply<C>(lds, x, b, inner, mine, acc);
    } else {
        Across<C, C::BN, LB, false> b(RowsDown<false>(a.ws, from));
        b.start(w, n0, a.N, inner);
        multiply<C>(lds, x, b, inner, mine, acc);
    }
}

// Many rows: matrix instructions bound it.  65536 rows of 64 experts, 2048 x 2816 bf16
// (756 GFLOP): 700 to 740 us with equal experts, 768 to 784 with a router's, 970 TFLOP/s, where
// one library product of all rows by one weight takes 625 to 640 (1200 TFLOP/s).  By way of
// registers (TileAny), 2049 x 2817: 1855 us; fp32, 65536 rows of 8 experts, 1024 x 1024 (137
// GFLOP): 1128 us, 122 TFLOP/s.  A step of 256 x 256 x
// 32 takes 0.92 us, 0.75 on zeros: the products' power brings the clock down to 1.75 GHz.
// The matrix units are busy 54% of the cycles; LDS moves 96 KB out and 32 in for a step, as
// many cycles as its products.  What is left per tile, 9 us, is its first loads (no other block on
// the CU runs meanwhile) and its store.  Tried and slower: steps of 64 with two in LDS (979
// us), one block of 256 x 128 with two to a CU (1031), 4 waves of 128 x 128, which read a third
// less from LDS (905; without spills, a row's operand replaced behind its last use, 947, and
// TURNED 790 instead of 737: one wave on a SIMD waits for nobody's products), 32 x 32 products
// (820), a higher wave priority for the products (850), blocks that go on to a next tile whose
// first loads run beside the store (818).
template <class C, int LA, int LB, bool TURNED>
__global__ __launch_bounds__(C::kThreads) void k_product(ExpertProductArgs a, int nt) {
    typedef typename C::T T;
    extern __shared__ __align__(1024) char lds[];
    RowTile t;
    if (!find_tile<C::kThreads>(a.l, C::BM, nt, t, lds)) return;
    const int n0 = t.n * C::BN;
    Acc<C> acc;
    product_tile<C, LA, LB, TURNED>(a, t, n0, 0, a.K, lds, acc);
    const auto row = [&](int m) { return m < t.rows ? static_cast<T *>(a.y) + (t.first + m) * a.ys : nullptr; };
    acc.template store<T>(lds, row, n0, a.N, past_caches<C>(static_cast<const T *>(a.y), a.ys));
}

// The same for few rows, which the weights' bytes bound: a tile is one wave's, four of
// them take a quarter of the inner index each, wait for their own loads alone, and add up
// in the waves' order.  One token of 8 experts, 2048 x 2816 bf16 (92 MB): 20 us, 4.6 TB/s.
template <class C, int L, bool TURNED>
__global__ __launch_bounds__(64 * kFewWaves) void k_product_few(ExpertProductArgs a, int nt) {
    typedef typename C::T T;
    extern __shared__ __align__(1024) char lds[];
    RowTile t;
    if (!find_tile<64 * kFewWaves>(a.l, C::BM, nt, t, lds)) return;
    const int n0 = t.n * C::BN, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per = ((a.K + kFewWaves - 1) / kFewWaves + C::BK - 1) / C::BK * C::BK, from = min(wave * per, a.K);
    char *own = lds + wave * C::kLds;
    Acc<C> acc;
    product_tile<C, L, L, TURNED>(a, t, n0, from, min(per, a.K - from), own, acc);
    acc.put(reinterpret_cast<float *>(own));
    __syncthreads();
    static_assert(C::BM * C::BN == 4 * 64 * kFewWaves && C::kLds >= 4 * C::BM * C::BN, "four sums a thread");
    const int m = threadIdx.x * 4 / C::BN, n = threadIdx.x * 4 % C::BN;
    if (m >= t.rows) return;
    f32x4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kFewWaves; w++)
        sum += *reinterpret_cast<const f32x4 *>(lds + w * C::kLds + 16 * threadIdx.x);
    T out[4];
#pragma unroll
    for (int q = 0; q < 4; q++) put_one(out + q, sum[q]);
    store_columns<4>(static_cast<T *>(a.y) + (t.first + m) * a.ys, n0 + n, a.N, out);
}

// dw[e] = the sum of x[r]^T dy[r] over e's rows (or over a part of them, into fp32): both
// operands lie across the inner index and are turned by the LDS read.  64 experts of 1024
// rows, 2048 x 2816 bf16 (756 GFLOP, 738 MB out): 835 to 850 us, with a router's experts,
// gathered, 857 to 880 (870 TFLOP/s); 32 steps a tile, so that a tile's start and end weigh more
// than above, and 2.7 GB are read where the operands are 0.64: a run is a column of all row
// tiles, the next column another XCD's, so that every XCD reads all of an expert's x.  With 32 rows
// an expert 187 us, 4.0 TB/s out.  By way of registers, 2049 x 2817: 2150 us; fp32, 16 experts of
// 512 rows, 1024 x 1024 (17 GFLOP): 200 us, 274 at 1025 x 1025.
template <class C, int LA, int LB, int GATHER, typename Out>
__global__ __launch_bounds__(C::kThreads) void k_weights(ExpertWeightsArgs a, int mt, int nt, int64_t total) {
    typedef typename C::T T;
    extern __shared__ __align__(1024) char lds[];
    int64_t id = own_tile_in_runs(blockIdx.x, kWeightsRun);
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
    // of codes, the row's number
    constexpr bool kGatherX = GATHER == DQ_GATHER_X, kGatherDy = GATHER == DQ_GATHER_DOUT;
    Across<C, C::BM, LA, kGatherX> x(RowsDown<kGatherX>(a.l, first, LA == kKept ? 1 : a.xs));
    Across<C, C::BN, LB, kGatherDy> dy(RowsDown<kGatherDy>(a.l, first, a.dys));
    if constexpr (LA == kKept)
        x.start(a.codes, a.exponents, m0, a.K, rows);
    else
        x.start(static_cast<const T *>(a.x), m0, a.K, rows);
    dy.start(static_cast<const T *>(a.dy), n0, a.N, rows);
    multiply<C>(lds, x, dy, rows, m0 + acc.m0() < a.K && n0 + acc.n0() < a.N, acc);
    Out *dw = static_cast<Out *>(a.parts > 1 ? (void *)a.partial : a.dw) +
              ((int64_t)part * a.l.E + e) * a.K * a.N;
    acc.template store<Out>(lds, [&](int m) { return m0 + m < a.K ? dw + (int64_t)(m0 + m) * a.N : nullptr; }, n0, a.N,
                            a.parts == 1 && past_caches<C>(dw, a.N));   // k_weights_join reads parts at once
}

// The parts' sums, in their order.
template <typename Out>
__global__ __launch_bounds__(256) void k_weights_join(const float *partial, int parts, int64_t n, Out *dw) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float s = partial[i];
        for (int p = 1; p < parts; p++) s += partial[p * n + i];
        put_one(dw + i, s);
    }
}

template <class C, bool FEW = false>
constexpr bool shaped(ExpertTile t) {
    constexpr int kThreads = FEW ? 64 * kFewWaves : C::kThreads;
    const TileShape s = expert_tile_shape(t, C::kF32);
    return s.bm == C::BM && s.bn == C::BN && s.threads == kThreads;
}
static_assert(shaped<TileBig>(ExpertTile::Big) && shaped<TileMid>(ExpertTile::Mid) &&
                  shaped<TileSmall>(ExpertTile::Small) && shaped<TileNarrow>(ExpertTile::Narrow) &&
                  shaped<TileAny>(ExpertTile::Any) && shaped<TileFew, true>(ExpertTile::Few) &&
                  shaped<TileFewAny, true>(ExpertTile::FewAny),
              "the blocks were counted for these");
static_assert(shaped<TileMidF32>(ExpertTile::Mid) && shaped<TileSmallF32>(ExpertTile::Small) &&
                  shaped<TileAnyF32>(ExpertTile::Any) && shaped<TileFewF32, true>(ExpertTile::Few) &&
                  shaped<TileFewAnyF32, true>(ExpertTile::FewAny),
              "and for these");

template <class C, class K>
hipError_t product_launch(K kernel, int threads, int lds, const ExpertProductArgs &a, const ExpertPick &p,
                          hipStream_t s) {
    const hipError_t e = room_for(kernel, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)p.blocks), dim3(threads), lds, s, a, (a.N + C::BN - 1) / C::BN);
    return hipGetLastError();
}
template <class C, int LA, int LB>
hipError_t product_as(const ExpertProductArgs &a, const ExpertPick &p, hipStream_t s) {
    if (a.turned) return product_launch<C>(k_product<C, LA, LB, true>, C::kThreads, C::kLds, a, p, s);
    return product_launch<C>(k_product<C, LA, LB, false>, C::kThreads, C::kLds, a, p, s);
}
template <class C, int L>
hipError_t product_few(const ExpertProductArgs &a, const ExpertPick &p, hipStream_t s) {
    if (a.turned) return product_launch<C>(k_product_few<C, L, true>, 64 * kFewWaves, kFewWaves * C::kLds, a, p, s);
    return product_launch<C>(k_product_few<C, L, false>, 64 * kFewWaves, kFewWaves * C::kLds, a, p, s);
}

template <class C, int LA, int LB, int GATHER, typename Out>
hipError_t weights_gathered(const ExpertWeightsArgs &a, const ExpertPick &p, hipStream_t s) {
    const int mt = (a.K + C::BM - 1) / C::BM, nt = (a.N + C::BN - 1) / C::BN;
    const auto kernel = k_weights<C, LA, LB, GATHER, Out>;
    const hipError_t e = room_for(kernel, C::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)p.blocks), dim3(C::kThreads), C::kLds, s, a, mt, nt, p.tiles);
    return hipGetLastError();
}

template <class C, int LA, int LB, typename Out>
hipError_t weights_as(const ExpertWeightsArgs &a, const ExpertPick &p, hipStream_t s) {
    if (a.gather == DQ_GATHER_X) return weights_gathered<C, LA, LB, DQ_GATHER_X, Out>(a, p, s);
    if (a.gather == DQ_GATHER_DOUT) return weights_gathered<C, LA, LB, DQ_GATHER_DOUT, Out>(a, p, s);
    return weights_gathered<C, LA, LB, DQ_GATHER_NONE, Out>(a, p, s);
}

template <typename Out>
hipError_t weights_bf16(const ExpertWeightsArgs &a, const ExpertPick &p, hipStream_t s) {
    if (a.codes && p.dy_async) return weights_as<TileAny, kKept, kAsync, Out>(a, p, s);
    if (a.codes) return weights_as<TileAny, kKept, kAny, Out>(a, p, s);
    if (p.tile == ExpertTile::Any) return weights_as<TileAny, kAny, kAny, Out>(a, p, s);
    if (p.tile == ExpertTile::Big) return weights_as<TileBig, kAsync, kAsync, Out>(a, p, s);
    if (p.tile == ExpertTile::Mid) return weights_as<TileMid, kAsync, kAsync, Out>(a, p, s);
    return weights_as<TileNarrow, kAsync, kAsync, Out>(a, p, s);
}
hipError_t weights_f32(const ExpertWeightsArgs &a, const ExpertPick &p, hipStream_t s) {
    if (a.codes && p.dy_async) return weights_as<TileAnyF32, kKept, kAsync, float>(a, p, s);
    if (a.codes) return weights_as<TileAnyF32, kKept, kAny, float>(a, p, s);
    if (p.tile == ExpertTile::Any) return weights_as<TileAnyF32, kAny, kAny, float>(a, p, s);
    if (p.tile == ExpertTile::Mid) return weights_as<TileMidF32, kAsync, kAsync, float>(a, p, s);
    return weights_as<TileSmallF32, kAsync, kAsync, float>(a, p, s);
}

}  // namespace

hipError_t launch_expert_product(const ExpertProductArgs &a, const ExpertPick &p, int f32, hipStream_t s) {
    if (a.l.slots == 0) return hipSuccess;
    if (f32) {
        if (p.tile == ExpertTile::FewAny) return product_few<TileFewAnyF32, kAny>(a, p, s);
        if (p.tile == ExpertTile::Any) return product_as<TileAnyF32, kAny, kAny>(a, p, s);
        if (p.tile == ExpertTile::Small) return product_as<TileSmallF32, kAsync, kAsync>(a, p, s);
        if (p.tile == ExpertTile::Mid) return product_as<TileMidF32, kAsync, kAsync>(a, p, s);
        return product_few<TileFewF32, kAsync>(a, p, s);
    }
    if (p.tile == ExpertTile::FewAny) return product_few<TileFewAny, kAny>(a, p, s);
    if (p.tile == ExpertTile::Any) return product_as<TileAny, kAny, kAny>(a, p, s);
    if (p.tile == ExpertTile::Small) return product_as<TileSmall, kAsync, kAsync>(a, p, s);
    if (p.tile == ExpertTile::Mid) return product_as<TileMid, kAsync, kAsync>(a, p, s);
    if (p.tile == ExpertTile::Big) return product_as<TileBig, kAsync, kAsync>(a, p, s);
    return product_few<TileFew, kAsync>(a, p, s);
}

hipError_t launch_expert_weights(const ExpertWeightsArgs &a, const ExpertPick &p, int f32, hipStream_t s) {
    const hipError_t e = f32                          ? weights_f32(a, p, s)
                         : a.out_f32 || a.parts > 1 ? weights_bf16<float>(a, p, s)
                                                    : weights_bf16<uint16_t>(a, p, s);
    if (e != hipSuccess || a.parts == 1) return e;
    const int64_t n = (int64_t)a.l.E * a.K * a.N, blocks = (n + 255) / 256;
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
    if (a.out_f32)
        hipLaunchKernelGGL((k_weights_join<float>), grid, dim3(256), 0, s, a.partial, a.parts, n,
                           static_cast<float *>(a.dw));
    else
        hipLaunchKernelGGL((k_weights_join<uint16_t>), grid, dim3(256), 0, s, a.partial, a.parts, n,
                           static_cast<uint16_t *>(a.dw));
    return hipGetLastError();
}

}  // namespace dq
