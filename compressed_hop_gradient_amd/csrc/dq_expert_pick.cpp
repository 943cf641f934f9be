// dq_expert_pick.cpp -- which kernel a product grouped by expert is computed by, and in
// how many blocks (host code, no HIP calls): all that a call has to know before it launches
// anything.
#include <algorithm>

#include "dq.h"
#include "dq_experts.h"

namespace dq {

namespace {

// Whether offsets into so many rows fit the 32 bits of the loads into LDS.
bool near(int64_t rows, int64_t stride, int64_t cols, int64_t es) {
    return ((__int128)(rows - 1) * stride + cols) * es < (__int128)kNowhere;
}

bool on16(const void *p, int64_t stride_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0;
}

bool product_async(const ExpertProductArgs &a, int64_t es) {
    const int64_t chunk = 16 / es;
    return on16(a.x, a.xs * es) && a.K % chunk == 0 && on16(a.w, a.ws * es) && (a.l.E == 1 || a.we * es % 16 == 0) &&
           (a.turned ? a.K : a.N) % chunk == 0 && near(a.gather ? a.l.tokens : 256, a.xs, a.K, es) &&
           near(a.turned ? 256 : 64, a.ws, a.turned ? a.K : a.N, es);
}

// Row tiles that so many slots may take: every expert's last one may be short.
int64_t most_row_tiles(const ExpertLists &l, int bm) {
    const int64_t most = ((int64_t)l.slots + (int64_t)l.E * (bm - 1)) / bm;
    return most < l.slots ? most : l.slots;
}
int64_t weights_tiles(const ExpertWeightsArgs &a, const TileShape &t) {
    return (int64_t)((a.K + t.bm - 1) / t.bm) * ((a.N + t.bn - 1) / t.bn) * a.l.E * a.parts;
}

int64_t whole_rounds(int64_t tiles, int run = 1) { return (tiles + 8 * run - 1) / (8 * run) * (8 * run); }
// A launch has below 2^32 threads.
bool fits(int64_t blocks, int threads) { return blocks <= ((int64_t)1 << 32) / threads - 1; }

// Which tile: the one whose blocks are done first, by how many of them a CU gets.
// Measured: a block's start and end take about 4 us, a step s1 where it has the CU to
// itself and sN where the CU is full of them; a wave of the few-row form takes a quarter
// of the steps.  bf16, 64 experts, 2048 x 2816, us of few / small / mid / big: 0.125 rows
// an expert 20 / 25 / 32 / 38, 16: 163 / 141 / 146 / 142, 64: 328 / 182 / 188 / 168 (the costs
// say small), 512: 1924 / 672 / 570 / 428; 8 experts of 1024 x 1024 and 64 rows 15 / 16 / 20 /
// 23, 512 rows 65 / 25 / 27 / 31.  fp32, 8 experts of 1024 x 1024, few / small / mid: 2 rows 12 /
// 25 / 77, 64: 28 / 28 / 78, 1024: 243 / 158 / 208, 8192: 1784 / 1130 / 1127.
//
// Operands off 16 bytes go by the same costs, few or not, and what is not is one tile, Any.  Its
// steps through registers cost more than these, so that few would do for longer than it is
// taken: bf16, 64 experts, 2049 x 2817, us of few / any: 0.125 rows 30 / 61, 1: 138 / 184 and 2:
// 169 / 256 (any is taken), 8: 214 / 276 (any), 16: 290 / 274, 64: 696 / 349, 512: 4276 / 990; 8
// experts of 1025 x 1025, 2 rows 16 / 32, 64: 30 / 33 (any), 512: 135 / 44.  fp32, the same 8:
// 21 / 45, 45 / 52, 1024 rows 424 / 228; 16 of 257 x 515, 8 rows 11 / 16, 125: 32 / 21.
struct TileCost {
    ExpertTile tile;
    int step, full;                      // step: inner elements; full: blocks a CU holds
    float s1, sn;                        // us
};
constexpr TileCost kCostBf16[] = {{ExpertTile::Small, 32, 3, 0.30f, 0.68f},
                                  {ExpertTile::Mid, 32, 2, 0.39f, 0.70f},
                                  {ExpertTile::Big, 32, 1, 0.80f, 0.80f},
                                  {ExpertTile::Few, 32 * kFewWaves, 2, 0.40f, 0.67f}};
constexpr TileCost kCostF32[] = {{ExpertTile::Small, 16, 5, 0.39f, 1.45f},
                                 {ExpertTile::Mid, 16, 2, 1.12f, 2.10f},
                                 {ExpertTile::Few, 16 * kFewWaves, 2, 0.40f, 0.90f}};

template <int N>
ExpertTile pick_tile(const TileCost (&costs)[N], const ExpertProductArgs &a, bool f32) {
    const double slots = a.l.slots, E = a.l.E, met = slots < E ? slots : E;
    const double memory = met * a.K * a.N * (f32 ? 4 : 2) / 5.5e6;
    int best = 0;
    double least = 0;
    for (int i = 0; i < N; i++) {
        const TileCost &c = costs[i];
        const TileShape t = expert_tile_shape(c.tile, f32);
        const double mt = std::max(met, std::min(slots, slots / t.bm + E / 2));
        const int64_t per_cu = ((int64_t)mt * ((a.N + t.bn - 1) / t.bn) + 255) / 256, rest = per_cu % c.full;
        const double rounds = (double)(per_cu / c.full) * c.sn +
                              (rest ? c.s1 + (c.sn - c.s1) * (rest - 1) / std::max(1, c.full - 1) : 0.0);
        const double us = std::max(memory, 4 + rounds * ((a.K + c.step - 1) / c.step));
        if (i == 0 || us < 0.97 * least) {
            best = i;
            least = us;
        }
    }
    return costs[best].tile;
}

// As above, for tiles of dw whose inner index is an expert's rows; operands off 16 bytes, or
// in codes, have the tile Any alone.  bf16, us of big / mid / narrow: 60 experts, 218 rows, 1000 x
// 1416 into fp32 117 / 145 / 215; 8 experts, 1024 rows, 1024 x 1024 55 / 49 / 77; 4096 rows, 256 x
// 512 64 / 52 / 55; 128 rows, 512 x 512 15 / 11 / 10; 64 of 32 rows, 2048 x 2816 187 / 253 / 466.
// fp32, mid / small: 16 experts, 512 rows, 1024 x 1024 199 / 175 and 8 of 2048 rows, 1024 x 2048
// 666 / 616 (the costs say mid for both); 64 of 8 rows, 1024 x 1024 66 / 81.
template <int N>
ExpertTile pick_weights_tile(const TileCost (&costs)[N], const ExpertWeightsArgs &a, bool f32) {
    int best = 0;
    double least = 0;
    for (int i = 0; i < N; i++) {
        const TileCost &c = costs[i];
        const int64_t blocks = weights_tiles(a, expert_tile_shape(c.tile, f32));
        const int64_t per_cu = (blocks + 255) / 256, rest = per_cu % c.full;
        const double steps = (double)a.l.slots / a.l.E / a.parts / c.step + 8;       // 8: a tile's start and end
        const double us = steps * ((double)(per_cu / c.full) * c.sn +
                                   (rest ? c.s1 + (c.sn - c.s1) * (rest - 1) / std::max(1, c.full - 1) : 0.0));
        if (i == 0 || us < 0.97 * least) {
            best = i;
            least = us;
        }
    }
    return costs[best].tile;
}
constexpr TileCost kWeightsBf16[] = {{ExpertTile::Big, 32, 1, 0.80f, 0.80f},
                                     {ExpertTile::Mid, 32, 2, 0.39f, 0.70f},
                                     {ExpertTile::Narrow, 32, 4, 0.25f, 0.55f}};
constexpr TileCost kWeightsF32[] = {{ExpertTile::Mid, 16, 2, 1.12f, 2.10f}, {ExpertTile::Small, 16, 5, 0.39f, 1.45f}};

}  // namespace

ExpertPick pick_expert_product(const ExpertProductArgs &a, bool f32) {
    ExpertPick p{};
    p.x_async = product_async(a, f32 ? 4 : 2);
    p.tile = f32 ? pick_tile(kCostF32, a, f32) : pick_tile(kCostBf16, a, f32);
    if (!p.x_async) p.tile = p.tile == ExpertTile::Few ? ExpertTile::FewAny : ExpertTile::Any;
    const TileShape t = expert_tile_shape(p.tile, f32);
    p.tiles = most_row_tiles(a.l, t.bm) * ((a.N + t.bn - 1) / t.bn);
    p.blocks = whole_rounds(p.tiles);
    p.fits = fits(p.blocks, t.threads);
    return p;
}

ExpertPick pick_expert_weights(const ExpertWeightsArgs &a, bool f32) {
    const int64_t es = f32 ? 4 : 2, chunk = 16 / es;
    ExpertPick p{};
    p.dy_async = on16(a.dy, a.dys * es) && a.N % chunk == 0 &&
                 near(a.gather == DQ_GATHER_DOUT ? a.l.tokens : 64, a.dys, a.N, es);
    p.x_async = a.x && on16(a.x, a.xs * es) && a.K % chunk == 0 &&
                near(a.gather == DQ_GATHER_X ? a.l.tokens : 64, a.xs, a.K, es);
    if (a.codes || !p.x_async || !p.dy_async)
        p.tile = ExpertTile::Any;
    else
        p.tile = f32 ? pick_weights_tile(kWeightsF32, a, f32) : pick_weights_tile(kWeightsBf16, a, f32);
    const TileShape t = expert_tile_shape(p.tile, f32);
    p.tiles = weights_tiles(a, t);
    p.blocks = whole_rounds(p.tiles, kWeightsRun);
    p.fits = fits(p.blocks, t.threads);
    return p;
}

// Enough parts that tiles of 128 x 128 give every CU a block, of 128 rows of an average
// expert at least: 3 experts of 3300 rows, 8 x 24 13 us, in one part 106.
int expert_weights_parts(int64_t slots, int E, int64_t K, int64_t N) {
    const int64_t tiles = (K + 127) / 128 * ((N + 127) / 128) * E, most = slots / E / 128;
    const int64_t parts = tiles >= 256 ? 1 : (255 + tiles) / tiles;
    return (int)std::max((int64_t)1, std::min(parts, most));
}

}  // namespace dq
