// dq_experts.h -- declarations shared by the experts' entry points
// (dq_experts_api.cpp), their kernels (dq_expert_rows.hip, dq_expert_product.hip,
// dq_keep8.hip) and the choice among the products' (dq_expert_pick.cpp).  Not part of
// the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dq {

constexpr int kExpertsMost = 1024;
constexpr int kExpertsMostTopK = 16;
// the offset of a load into LDS that reads zeros, and all beyond it
constexpr uint32_t kNowhere = 0xFFFFFFF0u;

// Rows of every expert.  A kernel takes nothing in the lists on trust: offsets are
// held to 0 .. slots and in order, a slot outside of them has no token.
struct ExpertLists {
    const int32_t *offsets, *source, *row;
    int64_t tokens;
    int32_t slots, k, E;
};

struct ExpertRowsArgs {
    const int32_t *ids;
    int32_t *offsets, *source, *row;
    uint32_t *counts;                   // [blocks][E + 1]
    int32_t slots, E, blocks;
};
// blocks of the two-launch form, 1 where one block does it all
int expert_rows_blocks(int64_t slots);
hipError_t launch_expert_rows(const ExpertRowsArgs &a, hipStream_t s);

struct ExpertSumArgs {
    ExpertLists l;
    const void *y, *residual;
    void *out;
    int64_t ys, rs, os;
    int32_t width;
};
hipError_t launch_expert_sum(const ExpertSumArgs &a, int f32, hipStream_t s);

// The generator's numbers of a keep call.
struct KeepKey {
    uint32_t key0, key1, round, worker, site;
    const uint32_t *d_round;
    int32_t dither;                     // 0: to the nearest
};
struct KeepArgs {
    const void *x;
    int64_t rows, cols, xs;
    const int32_t *d_rows;              // rows there are, at most `rows`; NULL: all
    int8_t *codes;
    uint8_t *exponents;
    KeepKey key;
};
hipError_t launch_keep8(const KeepArgs &a, int f32, hipStream_t s);
struct RestoreArgs {
    const int8_t *codes;
    const uint8_t *exponents;
    void *y;
    int64_t rows, cols, ys;
    const int32_t *d_rows;              // as above
};
hipError_t launch_restore8(const RestoreArgs &a, int f32, hipStream_t s);

struct ExpertActArgs {
    ExpertLists l;
    int32_t gated;                      // u = (g, v): silu(g) v; else max(u, 0)
    int32_t width;
    const void *u;                      // backward: may be NULL, then from the codes
    int64_t us;
    const float *gates;
    void *a;
    int64_t as;
    int8_t *codes;                      // forward: written if given
    uint8_t *exponents;
    KeepKey key;
    const void *da;                     // backward
    int64_t das;
    void *du;
    int64_t dus;
    float *dgates;
};
hipError_t launch_expert_act(const ExpertActArgs &a, int f32, hipStream_t s);
hipError_t launch_expert_act_backward(const ExpertActArgs &a, int f32, hipStream_t s);

struct ExpertProductArgs {
    ExpertLists l;
    const void *x;
    int64_t xs;
    int32_t gather;
    const void *w;
    int64_t we, ws;
    int32_t turned;                     // w[e] stored as [outer][inner]
    void *y;
    int64_t ys;
    int32_t K, N;
};

struct ExpertWeightsArgs {
    ExpertLists l;
    const void *x;                      // NULL: from the codes
    int64_t xs;
    const int8_t *codes;
    const uint8_t *exponents;
    const void *dy;
    int64_t dys;
    int32_t gather;                     // dq_expert_gather
    void *dw;                           // [E][K][N]
    int32_t out_f32;
    int32_t K, N;
    float *partial;                     // [parts][E][K][N] where parts > 1
    int32_t parts;
};
// parts into which the rows are split, whose sums meet in a second launch
int expert_weights_parts(int64_t slots, int E, int64_t K, int64_t N);

// Tiles of a product, rows by columns.  Any: operands through registers or from codes; Few: one
// wave's, whose block's waves share the inner index.
enum class ExpertTile { Big, Mid, Small, Narrow, Few, Any, FewAny };
struct TileShape {
    int bm, bn, threads;
};
constexpr int kFewWaves = 4;
constexpr TileShape expert_tile_shape(ExpertTile t, bool f32) {
    switch (t) {
    case ExpertTile::Big: return TileShape{256, 256, 512};
    case ExpertTile::Mid: return TileShape{128, 128, 256};
    case ExpertTile::Small: return TileShape{64, f32 ? 64 : 128, 256};
    case ExpertTile::Any: return f32 ? TileShape{64, 64, 256} : TileShape{128, 128, 256};
    case ExpertTile::Narrow: return TileShape{64, 64, 256};
    default: return TileShape{16, 64, 64 * kFewWaves};
    }
}
// Tiles of an XCD's run, us of runs of 4 / 8 / 32 / an eighth of all tiles, with a router's
// uneven experts: 64 experts, 1024 rows, 2048 x 2816 bf16 846 / 865 / 919 / 1062; 60 experts, 273
// rows, 1000 x 1416 into fp32 130 / 127 / 131 / 368.
constexpr int kWeightsRun = 8;

// The kernel of a call.
struct ExpertPick {
    ExpertTile tile;
    bool x_async, dy_async;             // loads straight into LDS (of a product: of both operands)
    int64_t tiles, blocks;
    bool fits;                          // a launch has so many blocks
};
ExpertPick pick_expert_product(const ExpertProductArgs &a, bool f32);
ExpertPick pick_expert_weights(const ExpertWeightsArgs &a, bool f32);
hipError_t launch_expert_product(const ExpertProductArgs &a, const ExpertPick &p, int f32, hipStream_t s);
hipError_t launch_expert_weights(const ExpertWeightsArgs &a, const ExpertPick &p, int f32, hipStream_t s);

}  // namespace dq
