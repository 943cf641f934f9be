// dq_train_api.cpp -- the training-step entry points of include/dq.h: argument
// checks and launches.  Stateless; all device work is enqueued on the caller's
// stream and nothing synchronises.
#include "dq.h"

#include <cmath>

#include "dq_train.h"

using namespace dq;

namespace {

constexpr size_t kAlign = 256;

bool is_kind(int32_t kind) { return kind == DQ_BF16 || kind == DQ_F32; }
uintptr_t elem_bytes(int32_t kind) { return kind == DQ_F32 ? 4 : 2; }
bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

dq_status hip_status(hipError_t e) { return e == hipSuccess ? DQ_OK : DQ_EHIP; }

// Whether an output (rows x cols, row stride os) meets an operand (row stride
// is) other than element on element.  Row windows of equal stride may
// interleave (two halves of one wide tensor).
bool clash(const void *out, int64_t os, const void *in, int64_t is, int64_t rows, int64_t cols, int64_t es) {
    if (!in || rows == 0 || cols == 0) return false;
    if (rows == 1) os = is = cols;
    if (out == in && os == is) return false;
    const __int128 o = (__int128) reinterpret_cast<uintptr_t>(out), i = (__int128) reinterpret_cast<uintptr_t>(in);
    const __int128 olen = ((__int128)(rows - 1) * os + cols) * es, ilen = ((__int128)(rows - 1) * is + cols) * es;
    if (o + olen <= i || i + ilen <= o) return false;
    if (os == is && (o - i) % es == 0) {
        const int64_t at = (int64_t)((((o - i) / es) % os + os) % os);
        if (at >= cols && at <= os - cols) return false;
    }
    return true;
}

constexpr int64_t kMostTokens = (int64_t)1 << 40;

RoutePart part_at(void *d_part, int64_t tokens, int32_t E) {
    return RoutePart{static_cast<uint8_t *>(d_part), route_blocks(tokens, E)};
}

bool bad_router(int32_t kind, int64_t tokens, int32_t E, int64_t stride, int32_t k) {
    return !is_kind(kind) || tokens < 0 || tokens > kMostTokens || E < 1 || E > kRouteMaxExperts || k < 1 ||
           k > E || k > kRouteMaxTopK || stride < 0 || stride > ((int64_t)1 << 40);
}

}  // namespace

extern "C" {

dq_status dq_dropout(const void *x, const void *residual, void *y, int32_t kind, int64_t rows, int64_t cols,
                     int64_t xs, int64_t rs, int64_t ys, double p, uint64_t seed, uint32_t round,
                     const uint32_t *d_round, int32_t worker, uint32_t site, void *stream) {
    constexpr int64_t kMost = (int64_t)1 << 51;
    if (!is_kind(kind) || rows < 0 || cols < 0 || !(p >= 0.0 && p <= 1.0)) return DQ_EINVAL;
    if (cols > 0 && rows >= kMost / cols + 1) return DQ_EINVAL;
    if (rows * cols >= kMost || worker < 0 || worker > 65535 || site >= 0x80000000u) return DQ_EINVAL;
    if (xs < 0 || rs < 0 || xs >= kMost || rs >= kMost || ys >= kMost) return DQ_EINVAL;
    if (rows > 1 && ys < cols) return DQ_EINVAL;
    if (rows == 0 || cols == 0) return DQ_OK;
    if (!x || !y) return DQ_ENULL;
    const uintptr_t es = elem_bytes(kind);
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(y, es) || !aligned(d_round, 4)) return DQ_EINVAL;
    if (clash(y, ys, x, xs, rows, cols, (int64_t)es) || clash(y, ys, residual, rs, rows, cols, (int64_t)es))
        return DQ_EINVAL;
    DropoutArgs a{};
    a.x = x;
    a.residual = residual;
    a.y = y;
    // contiguous operands are one row, whatever their shape
    if (rows == 1 || (xs == cols && ys == cols && (!residual || rs == cols))) {
        cols *= rows;
        rows = 1;
        xs = rs = ys = cols;
    }
    a.rows = rows;
    a.cols = cols;
    a.xs = xs;
    a.rs = rs;
    a.ys = ys;
    a.threshold = (uint32_t)std::floor(65536.0 * p + 0.5);
    a.scale = a.threshold == 65536 ? 0.0f : (float)(65536.0 / (65536 - (int)a.threshold));
    a.key0 = (uint32_t)seed;
    a.key1 = (uint32_t)(seed >> 32);
    a.round = round;
    a.d_round = d_round;
    a.worker = (uint32_t)worker;
    a.site = site;
    return hip_status(launch_dropout(a, kind == DQ_F32, static_cast<hipStream_t>(stream)));
}

size_t dq_route_part_bytes(int64_t tokens, int32_t E) {
    if (tokens < 0 || tokens > kMostTokens || E < 1 || E > kRouteMaxExperts) return 0;
    return part_at(nullptr, tokens, E).bytes(E);
}

dq_status dq_route(const dq_route_worker *workers, int32_t n, int32_t kind, int32_t E, int32_t k, int32_t flags,
                   void *stream) {
    if (n < 0 || (flags & ~DQ_ROUTE_RENORM) || bad_router(kind, 0, E, 0, k)) return DQ_EINVAL;
    if (n > 0 && !workers) return DQ_ENULL;
    for (int32_t w = 0; w < n; w++) {
        const dq_route_worker &in = workers[w];
        if (bad_router(kind, in.tokens, E, in.stride, k)) return DQ_EINVAL;
        if (in.tokens > 0 && (!in.d_logits || !in.d_ids || !in.d_gates)) return DQ_ENULL;
        if (!aligned(in.d_logits, elem_bytes(kind)) || !aligned(in.d_ids, 4) || !aligned(in.d_gates, 4))
            return DQ_EINVAL;
        if (!in.d_part || !aligned(in.d_part, kAlign) || in.part_bytes < dq_route_part_bytes(in.tokens, E))
            return DQ_EWORKSPACE;
    }
    RouteArgs a{};
    a.E = E;
    a.k = k;
    a.renorm = (flags & DQ_ROUTE_RENORM) != 0;
    for (int32_t w = 0; w < n; w++) {
        const dq_route_worker &in = workers[w];
        a.worker[a.workers++] = RouteWorker{in.d_logits, in.tokens, in.stride, in.d_mask, in.d_ids, in.d_gates,
                                            part_at(in.d_part, in.tokens, E)};
        if (a.workers == kRouteGroup || w == n - 1) {
            const hipError_t e = launch_route(a, kind == DQ_F32, static_cast<hipStream_t>(stream));
            if (e != hipSuccess) return hip_status(e);
            a.workers = 0;
        }
    }
    return DQ_OK;
}

dq_status dq_balance(const dq_route_part *parts, int32_t n_parts, const double *sums, int32_t E, int32_t k,
                     double *stats, float *loss, float *coef, int64_t *counts, void *stream) {
    if (E < 1 || E > kRouteMaxExperts || k < 1 || k > E || k > kRouteMaxTopK) return DQ_EINVAL;
    if (n_parts < 0 || n_parts > kRouteMaxParts) return DQ_EINVAL;
    if ((n_parts > 0 && !parts) || (n_parts == 0 && !sums)) return DQ_ENULL;
    if (!aligned(sums, 8) || !aligned(stats, 8) || !aligned(loss, 4) || !aligned(coef, 4) || !aligned(counts, 8))
        return DQ_EINVAL;
    BalanceArgs a{};
    a.parts = n_parts;
    for (int32_t q = 0; q < n_parts; q++) {
        if (parts[q].tokens < 0 || parts[q].tokens > kMostTokens) return DQ_EINVAL;
        if (!parts[q].d_part) return DQ_ENULL;
        if (!aligned(parts[q].d_part, kAlign)) return DQ_EINVAL;
        a.part[q] = part_at(parts[q].d_part, parts[q].tokens, E);
    }
    a.sums = sums;
    a.E = E;
    a.k = k;
    a.stats = stats;
    a.loss = loss;
    a.coef = coef;
    a.counts = counts;
    return hip_status(launch_balance(a, static_cast<hipStream_t>(stream)));
}

dq_status dq_route_backward(const dq_route_grad *workers, int32_t n, int32_t kind, int32_t E, int32_t k,
                            int32_t flags, const float *coef, const float *dloss, void *stream) {
    if (n < 0 || (flags & ~DQ_ROUTE_RENORM) || bad_router(kind, 0, E, 0, k)) return DQ_EINVAL;
    if (!aligned(coef, 4) || !aligned(dloss, 4)) return DQ_EINVAL;
    if (n > 0 && !workers) return DQ_ENULL;
    const uintptr_t es = elem_bytes(kind);
    for (int32_t w = 0; w < n; w++) {
        const dq_route_grad &in = workers[w];
        if (bad_router(kind, in.tokens, E, in.stride, k)) return DQ_EINVAL;
        if (in.dstride > kMostTokens || (in.tokens > 1 && in.dstride < E)) return DQ_EINVAL;
        if (in.tokens == 0) continue;
        if (!in.d_logits || !in.d_ids || !in.d_dlogits) return DQ_ENULL;
        if (!aligned(in.d_logits, es) || !aligned(in.d_dlogits, es) || !aligned(in.d_ids, 4) ||
            !aligned(in.d_dgates, 4))
            return DQ_EINVAL;
        if (clash(in.d_dlogits, in.dstride, in.d_logits, in.stride, in.tokens, E, (int64_t)es)) return DQ_EINVAL;
    }
    RouteBackwardArgs a{};
    a.E = E;
    a.k = k;
    a.renorm = (flags & DQ_ROUTE_RENORM) != 0;
    a.coef = coef;
    a.dloss = dloss;
    for (int32_t w = 0; w < n; w++) {
        const dq_route_grad &in = workers[w];
        if (in.tokens > 0)
            a.worker[a.workers++] = RouteBackwardWorker{in.d_logits, in.tokens, in.stride, in.dstride,
                                                        in.d_mask, in.d_ids, in.d_dgates, in.d_dlogits};
        if (a.workers == kRouteGroup || (w == n - 1 && a.workers > 0)) {
            const hipError_t e = launch_route_backward(a, kind == DQ_F32, static_cast<hipStream_t>(stream));
            if (e != hipSuccess) return hip_status(e);
            a.workers = 0;
        }
    }
    return DQ_OK;
}

}  // extern "C"
