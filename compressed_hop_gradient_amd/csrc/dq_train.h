// dq_train.h -- declarations shared by the training-step entry points
// (dq_train_api.cpp) and their kernels (dq_dropout.hip, dq_route.hip,
// dq_route_backward.hip).  Not part of the public ABI.
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

// Statistics of one worker's tokens, in the caller's buffer: a row per block of
// the router's kernel, then the scratch of a balance call.
struct RoutePart {
    uint8_t *base;
    int32_t nblk;
    static __host__ __device__ size_t up(size_t x) { return (x + 255) / 256 * 256; }
    __host__ __device__ size_t table(int E) const { return up(4 * (size_t)nblk * (size_t)E); }
    // [nblk][E] summed probabilities, [nblk][E] choices, [nblk] routed tokens
    __host__ __device__ float *psum() const { return reinterpret_cast<float *>(base); }
    __host__ __device__ uint32_t *count(int E) const { return reinterpret_cast<uint32_t *>(base + table(E)); }
    __host__ __device__ uint32_t *routed(int E) const { return reinterpret_cast<uint32_t *>(base + 2 * table(E)); }
    // the part folded, double[2 E + 1], and blocks that are done (of the call
    // whose first part this is; 0 between calls)
    __host__ __device__ size_t fold_at(int E) const { return 2 * table(E) + up(4 * (size_t)nblk); }
    __host__ __device__ size_t done_at(int E) const { return fold_at(E) + up(8 * (2 * (size_t)E + 1)); }
    __host__ __device__ double *fold(int E) const { return reinterpret_cast<double *>(base + fold_at(E)); }
    __host__ __device__ uint32_t *done(int E) const { return reinterpret_cast<uint32_t *>(base + done_at(E)); }
    size_t bytes(int E) const { return done_at(E) + 256; }
};
constexpr int kRouteMaxParts = 16;
constexpr int kBalanceColumns = 16;     // experts of a balance block

// One worker's tokens in a router launch; the launch's workers are the second
// dimension of the grid.  Four of them: arguments of 2 KB for sixteen would make
// every launch, of one worker too, 1.2 us longer on the host.
constexpr int kRouteGroup = 4;
struct RouteWorker {
    const void *logits;
    int64_t tokens, stride;
    const uint8_t *mask;
    int32_t *ids;
    float *gates;
    RoutePart part;              // out: nblk rows of partial statistics
};
struct RouteArgs {
    RouteWorker worker[kRouteGroup];
    int32_t workers;
    int32_t E, k, renorm;
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

struct RouteBackwardWorker {
    const void *logits;
    int64_t tokens, stride, dstride;
    const uint8_t *mask;
    const int32_t *ids;
    const float *dgates;
    void *dlogits;
};
struct RouteBackwardArgs {
    RouteBackwardWorker worker[kRouteGroup];
    int32_t workers;
    int32_t E, k, renorm;
    const float *coef, *dloss;
};

hipError_t launch_dropout(const DropoutArgs &a, int f32, hipStream_t s);
// blocks of the router's forward kernel for this many tokens (its partials' rows)
int route_blocks(int64_t tokens, int E);
hipError_t launch_route(const RouteArgs &a, int f32, hipStream_t s);
hipError_t launch_balance(const BalanceArgs &a, hipStream_t s);
hipError_t launch_route_backward(const RouteBackwardArgs &a, int f32, hipStream_t s);

}  // namespace dq
