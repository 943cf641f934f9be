// dq_train.h -- declarations shared by the training-step entry points
// (dq_train_api.cpp) and their kernels (dq_train.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dq {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 16;

struct DropoutArgs {
    const void *x, *residual;
    void *y;
    int64_t rows, cols;
    int64_t xs, rs, ys;                 // row strides, elements
    uint32_t threshold;                 // T: dropped iff dither < T
    float scale;                        // fl(65536 / (65536 - T)); 0 for T = 65536
    uint32_t key0, key1, round, worker, site;
    const uint32_t *d_round;
};

// Statistics of one router call: a row per block of its kernel.
struct RoutePart {
    float *psum;            // [nblk][E] summed probabilities
    uint32_t *count;        // [nblk][E] choices
    uint32_t *routed;       // [nblk] routed tokens
    int32_t nblk;
    // scratch of a balance call: blocks that are done (of the first part's call; 0
    // between calls), and this part's folded statistics, double[2 E + 1]
    uint32_t *done;
    double *fold;
};
constexpr int kRouteMaxParts = 16;
constexpr int kBalanceColumns = 16;     // experts of a balance block

struct RouteArgs {
    const void *logits;
    int64_t tokens, stride;
    int32_t E, k;
    const uint8_t *mask;
    int32_t renorm;
    int32_t *ids;
    float *gates;
    RoutePart part;              // out: nblk rows of partial statistics
};

struct BalanceArgs {
    RoutePart part[kRouteMaxParts];
    int32_t parts;
    const double *sums;
    int32_t E, k;
    double *stats;
    float *loss, *coef;
    int64_t *counts;
};

struct RouteBackwardArgs {
    const void *logits;
    int64_t tokens, stride, dstride;
    int32_t E, k;
    const uint8_t *mask;
    int32_t renorm;
    const int32_t *ids;
    const float *dgates, *coef, *dloss;
    void *dlogits;
};

hipError_t launch_dropout(const DropoutArgs &a, int f32, hipStream_t s);
// blocks of the router's forward kernel for this many tokens (its partials' rows)
int route_blocks(int64_t tokens, int E);
hipError_t launch_route(const RouteArgs &a, int f32, hipStream_t s);
hipError_t launch_balance(const BalanceArgs &a, hipStream_t s);
hipError_t launch_route_backward(const RouteBackwardArgs &a, int f32, hipStream_t s);

}  // namespace dq
