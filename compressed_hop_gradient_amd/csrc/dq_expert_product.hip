// dq_expert_product.hip -- products grouped by expert for gfx950: rows by the
// experts' weights, and the weights' gradient.
#include <algorithm>

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
// (756 GFLOP): 735 us with equal experts, 776 with a router's, 970 TFLOP/s, where one library
// product of all rows by one weight takes 625 to 640 (1210 TFLOP/s).  A step of 256 x 256 x
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
    if (!find_tile<C::kThreads>(a.l, C::BM, nt, t, reinterpret_cast<int *>(lds))) return;
    const int n0 = t.n * C::BN;
    Acc<C> acc;
    product_tile<C, LA, LB, TURNED>(a, t, n0, 0, a.K, lds, acc);
    const auto row = [&](int m) { return m < t.rows ? static_cast<T *>(a.y) + (t.first + m) * a.ys : nullptr; };
    acc.template store<T>(lds, row, n0, a.N, past_caches<C>(static_cast<const T *>(a.y), a.ys));
}

// The same for few rows, which the weights' bytes bound: a tile is one wave's, four of
// them take a quarter of the inner index each, wait for their own loads alone, and add up
// in the waves' order.  One token of 8 experts, 2048 x 2816 bf16 (92 MB): 20 us, 4.6 TB/s; 8
// tokens (about 460 MB of weights met) 84 us, 5.5 TB/s.
constexpr int kFewWaves = 4;
template <class C, int L, bool TURNED>
__global__ __launch_bounds__(64 * kFewWaves) void k_product_few(ExpertProductArgs a, int nt) {
    typedef typename C::T T;
    extern __shared__ __align__(1024) char lds[];
    RowTile t;
    if (!find_tile<64 * kFewWaves>(a.l, C::BM, nt, t, reinterpret_cast<int *>(lds))) return;
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

// Tiles of an XCD's run: 2000 us where 32 took 2260 and an eighth of all at once 2830 (a
// router's uneven experts, before the loads went ahead).
constexpr int kWeightsRun = 8;

// dw[e] = the sum of x[r]^T dy[r] over e's rows (or over a part of them, into fp32): both
// operands lie across the inner index and are turned by the LDS read.  64 experts of 1024
// rows, 2048 x 2816 bf16 (756 GFLOP, 738 MB out): 790 us, with a router's experts, gathered,
// 877 (860 TFLOP/s); 32 steps a tile, so that a tile's start and end weigh more than above.
// With 32 rows an expert 192 us, 3.9 TB/s out.
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

template <class C>
int64_t most_row_tiles(const ExpertLists &l) {
    const int64_t most = ((int64_t)l.slots + (int64_t)l.E * (C::BM - 1)) / C::BM;
    return most < l.slots ? most : l.slots;
}

int64_t whole_rounds(int64_t tiles, int run = 1) { return (tiles + 8 * run - 1) / (8 * run) * (8 * run); }
// A launch has below 2^32 threads.
bool too_many(int64_t blocks, int threads) { return blocks > ((int64_t)1 << 32) / threads - 1; }

template <class C, class K>
hipError_t product_launch(K kernel, int threads, int lds, const ExpertProductArgs &a, hipStream_t s) {
    const int nt = (a.N + C::BN - 1) / C::BN;
    const int64_t tiles = most_row_tiles<C>(a.l) * nt;
    const int64_t blocks = whole_rounds(tiles);
    if (too_many(blocks, threads)) return hipErrorInvalidConfiguration;
    const hipError_t e = room_for(kernel, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), lds, s, a, nt);
    return hipGetLastError();
}
template <class C, int LA, int LB>
hipError_t product_as(const ExpertProductArgs &a, hipStream_t s) {
    if (a.turned) return product_launch<C>(k_product<C, LA, LB, true>, C::kThreads, C::kLds, a, s);
    return product_launch<C>(k_product<C, LA, LB, false>, C::kThreads, C::kLds, a, s);
}
template <class C, int L>
hipError_t product_few(const ExpertProductArgs &a, hipStream_t s) {
    if (a.turned) return product_launch<C>(k_product_few<C, L, true>, 64 * kFewWaves, kFewWaves * C::kLds, a, s);
    return product_launch<C>(k_product_few<C, L, false>, 64 * kFewWaves, kFewWaves * C::kLds, a, s);
}

// Whether offsets into so many rows fit the 32 bits of the loads into LDS.
bool near(int64_t rows, int64_t stride, int64_t cols, int64_t es) {
    return ((rows - 1) * stride + cols) * es < (int64_t)kNowhere;
}

template <typename T>
bool product_async(const ExpertProductArgs &a) {
    constexpr int64_t es = sizeof(T), chunk = 16 / es;
    return on16(a.x, a.xs * es) && a.K % chunk == 0 && on16(a.w, a.ws * es) && (a.l.E == 1 || a.we * es % 16 == 0) &&
           (a.turned ? a.K : a.N) % chunk == 0 && near(a.gather ? a.l.tokens : 256, a.xs, a.K, es) &&
           near(a.turned ? 256 : 64, a.ws, a.turned ? a.K : a.N, es);
}

template <class C, int LA, int LB, int GATHER, typename Out>
hipError_t weights_gathered(const ExpertWeightsArgs &a, hipStream_t s) {
    const int mt = (a.K + C::BM - 1) / C::BM, nt = (a.N + C::BN - 1) / C::BN;
    const int64_t tiles = (int64_t)mt * nt * a.l.E * a.parts;
    const int64_t blocks = whole_rounds(tiles, kWeightsRun);
    if (too_many(blocks, C::kThreads)) return hipErrorInvalidConfiguration;
    const auto kernel = k_weights<C, LA, LB, GATHER, Out>;
    const hipError_t e = room_for(kernel, C::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(C::kThreads), C::kLds, s, a, mt, nt, tiles);
    return hipGetLastError();
}

template <class C, int LA, int LB, typename Out>
hipError_t weights_as(const ExpertWeightsArgs &a, hipStream_t s) {
    if (a.gather == DQ_GATHER_X) return weights_gathered<C, LA, LB, DQ_GATHER_X, Out>(a, s);
    if (a.gather == DQ_GATHER_DOUT) return weights_gathered<C, LA, LB, DQ_GATHER_DOUT, Out>(a, s);
    return weights_gathered<C, LA, LB, DQ_GATHER_NONE, Out>(a, s);
}

template <typename T>
struct WeightsLoads {
    static constexpr int64_t es = sizeof(T), chunk = 16 / es;
    bool x, dy;
    explicit WeightsLoads(const ExpertWeightsArgs &a) {
        dy = on16(a.dy, a.dys * es) && a.N % chunk == 0 &&
             near(a.gather == DQ_GATHER_DOUT ? a.l.tokens : 64, a.dys, a.N, es);
        x = a.x && on16(a.x, a.xs * es) && a.K % chunk == 0 &&
            near(a.gather == DQ_GATHER_X ? a.l.tokens : 64, a.xs, a.K, es);
    }
};

// Which tile: the one whose blocks are done first, by how many of them a CU gets.
// Measured: a block's start and end take about 4 us, a step s1 where it has the CU to
// itself and sN where the CU is full of them; a wave of the few-row form takes a quarter
// of the steps.  bf16, 64 experts, 2048 x 2816, us of few / small / mid / big: 0.125 rows
// an expert 20 / 24 / 29 / 52, 16: 163 / 142 / 146 / 191, 64: 328 / 185 / 190 / 200, 512:
// 1909 / 673 / 559 / 457; 8 experts of 1024 x 1024 and 64 rows 14 / 15 / 18 / 29, 512 rows
// 60 / 24 / 25 / 36.  fp32, 8 experts of 1024 x 1024, few / small / mid: 2 rows 13 / 29 /
// 76, 64: 28 / 30 / 78, 1024: 238 / 170 / 209.
struct TileCost {
    int bm, bn, step, full;              // step: inner elements; full: blocks a CU holds
    float s1, sn;                        // us
};
constexpr TileCost kCostBf16[] = {
    {64, 128, 32, 3, 0.30f, 0.68f}, {128, 128, 32, 2, 0.39f, 0.70f}, {256, 256, 32, 1, 0.80f, 0.80f},
    {16, 64, 32 * kFewWaves, 2, 0.40f, 0.67f}};
constexpr TileCost kCostF32[] = {
    {64, 64, 16, 5, 0.39f, 1.45f}, {128, 128, 16, 2, 1.12f, 2.10f}, {16, 64, 16 * kFewWaves, 2, 0.40f, 0.90f}};

template <int N>
int pick_tile(const TileCost (&costs)[N], const ExpertProductArgs &a, double es) {
    const double slots = a.l.slots, E = a.l.E, met = slots < E ? slots : E;
    const double memory = met * a.K * a.N * es / 5.5e6;
    int best = 0;
    double least = 0;
    for (int i = 0; i < N; i++) {
        const TileCost &c = costs[i];
        const double mt = std::max(met, std::min(slots, slots / c.bm + E / 2));
        const int64_t per_cu = ((int64_t)mt * ((a.N + c.bn - 1) / c.bn) + 255) / 256, rest = per_cu % c.full;
        const double rounds = (double)(per_cu / c.full) * c.sn +
                              (rest ? c.s1 + (c.sn - c.s1) * (rest - 1) / std::max(1, c.full - 1) : 0.0);
        const double us = std::max(memory, 4 + rounds * ((a.K + c.step - 1) / c.step));
        if (i == 0 || us < 0.97 * least) {
            best = i;
            least = us;
        }
    }
    return best;
}

// As above, for tiles of dw whose inner index is an expert's rows.  bf16, us of big / mid /
// narrow: 60 experts, 218 rows, 1000 x 1416 into fp32 155 / 194 / 264; 8 experts, 1024 rows,
// 1024 x 1024 58 / 50 / 79; 4096 rows, 256 x 512 64 / 52 / 55; 128 rows, 512 x 512 15 / 13 / 12.
// fp32, mid / small: 16 experts, 512 rows, 1024 x 1024 226 / 193; 8 of 2048 rows, 1024 x 2048 694 /
// 653; 64 of 8 rows, 1024 x 1024 76 / 83.
template <int N>
int pick_weights_tile(const TileCost (&costs)[N], const ExpertWeightsArgs &a) {
    int best = 0;
    double least = 0;
    for (int i = 0; i < N; i++) {
        const TileCost &c = costs[i];
        const int64_t blocks = (int64_t)((a.K + c.bm - 1) / c.bm) * ((a.N + c.bn - 1) / c.bn) * a.l.E * a.parts;
        const int64_t per_cu = (blocks + 255) / 256, rest = per_cu % c.full;
        const double steps = (double)a.l.slots / a.l.E / a.parts / c.step + 8;       // 8: a tile's start and end
        const double us = steps * ((double)(per_cu / c.full) * c.sn +
                                   (rest ? c.s1 + (c.sn - c.s1) * (rest - 1) / std::max(1, c.full - 1) : 0.0));
        if (i == 0 || us < 0.97 * least) {
            best = i;
            least = us;
        }
    }
    return best;
}
constexpr TileCost kWeightsBf16[] = {
    {256, 256, 32, 1, 0.80f, 0.80f}, {128, 128, 32, 2, 0.39f, 0.70f}, {64, 64, 32, 4, 0.25f, 0.55f}};
constexpr TileCost kWeightsF32[] = {{128, 128, 16, 2, 1.12f, 2.10f}, {64, 64, 16, 5, 0.39f, 1.45f}};

template <typename Out>
hipError_t weights_bf16(const ExpertWeightsArgs &a, hipStream_t s) {
    const WeightsLoads<uint16_t> on(a);
    if (a.codes && on.dy) return weights_as<TileAny, kKept, kAsync, Out>(a, s);
    if (a.codes) return weights_as<TileAny, kKept, kAny, Out>(a, s);
    if (!on.x || !on.dy) return weights_as<TileAny, kAny, kAny, Out>(a, s);
    const int pick = pick_weights_tile(kWeightsBf16, a);
    if (pick == 0) return weights_as<TileBig, kAsync, kAsync, Out>(a, s);
    if (pick == 1) return weights_as<TileMid, kAsync, kAsync, Out>(a, s);
    return weights_as<TileNarrow, kAsync, kAsync, Out>(a, s);
}
hipError_t weights_f32(const ExpertWeightsArgs &a, hipStream_t s) {
    const WeightsLoads<float> on(a);
    if (a.codes && on.dy) return weights_as<TileAnyF32, kKept, kAsync, float>(a, s);
    if (a.codes) return weights_as<TileAnyF32, kKept, kAny, float>(a, s);
    if (!on.x || !on.dy) return weights_as<TileAnyF32, kAny, kAny, float>(a, s);
    const int pick = pick_weights_tile(kWeightsF32, a);
    if (pick == 0) return weights_as<TileMidF32, kAsync, kAsync, float>(a, s);
    return weights_as<TileSmallF32, kAsync, kAsync, float>(a, s);
}

}  // namespace

hipError_t launch_expert_product(const ExpertProductArgs &a, int f32, hipStream_t s) {
    if (a.l.slots == 0) return hipSuccess;
    if (f32) {
        const int pick = pick_tile(kCostF32, a, 4);
        if (!product_async<float>(a))
            return pick == 2 ? product_few<TileFewAnyF32, kAny>(a, s) : product_as<TileAnyF32, kAny, kAny>(a, s);
        if (pick == 0) return product_as<TileSmallF32, kAsync, kAsync>(a, s);
        if (pick == 1) return product_as<TileMidF32, kAsync, kAsync>(a, s);
        return product_few<TileFewF32, kAsync>(a, s);
    }
    const int pick = pick_tile(kCostBf16, a, 2);
    if (!product_async<uint16_t>(a))
        return pick == 3 ? product_few<TileFewAny, kAny>(a, s) : product_as<TileAny, kAny, kAny>(a, s);
    if (pick == 0) return product_as<TileSmall, kAsync, kAsync>(a, s);
    if (pick == 1) return product_as<TileMid, kAsync, kAsync>(a, s);
    if (pick == 2) return product_as<TileBig, kAsync, kAsync>(a, s);
    return product_few<TileFew, kAsync>(a, s);
}

// Enough parts that tiles of 128 x 128 give every CU a block, of 128 rows of an average
// expert at least: 3 experts of 3300 rows, 8 x 24 13 us, in one part 106.
int expert_weights_parts(int64_t slots, int E, int64_t K, int64_t N) {
    const int64_t tiles = (K + 127) / 128 * ((N + 127) / 128) * E, most = slots / E / 128;
    const int64_t parts = tiles >= 256 ? 1 : (255 + tiles) / tiles;
    return (int)std::max((int64_t)1, std::min(parts, most));
}

hipError_t launch_expert_weights(const ExpertWeightsArgs &a, int f32, hipStream_t s) {
    const hipError_t e = f32 ? weights_f32(a, s)
                             : a.out_f32 || a.parts > 1 ? weights_bf16<float>(a, s) : weights_bf16<uint16_t>(a, s);
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
