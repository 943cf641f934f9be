// dq_train_api.cpp -- the training-step entry points of include/dq.h: argument
// checks and launches.  Stateless; all device work is enqueued on the caller's
// stream and nothing synchronises.
#include "dq.h"

#include <cmath>

#include "dq_checks.h"
#include "dq_train.h"

using namespace dq;

namespace {

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
    const Span into = span(y, rows, ys, cols, (int64_t)es, true);
    // element on element is as well
    const auto clash = [&](const void *p, int64_t stride) {
        return !(p == y && (rows == 1 || stride == ys)) && meet(into, span(p, rows, stride, cols, (int64_t)es, false));
    };
    if (clash(x, xs) || clash(residual, rs) || meet(into, bytes(d_round, 4, false))) return DQ_EINVAL;
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
    Spans spans;
    if (!spans.reserve(5 * (size_t)n)) return DQ_EINVAL;
    for (int32_t w = 0; w < n; w++) {
        const dq_route_worker &in = workers[w];
        spans.add(span(in.d_logits, in.tokens, in.stride, E, (int64_t)elem_bytes(kind), false));
        spans.add(bytes(in.d_mask, (size_t)in.tokens, false));
        spans.add(bytes(in.d_ids, 4 * (size_t)in.tokens * k, true));
        spans.add(bytes(in.d_gates, 4 * (size_t)in.tokens * k, true));
        spans.add(bytes(in.d_part, dq_route_part_bytes(in.tokens, E), true));
    }
    if (spans.clash()) return DQ_EINVAL;
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
    Spans spans;
    if (!spans.reserve(kRouteMaxParts + 5)) return DQ_EINVAL;
    a.parts = n_parts;
    for (int32_t q = 0; q < n_parts; q++) {
        if (parts[q].tokens < 0 || parts[q].tokens > kMostTokens) return DQ_EINVAL;
        if (!parts[q].d_part) return DQ_ENULL;
        if (!aligned(parts[q].d_part, kAlign)) return DQ_EINVAL;
        a.part[q] = part_at(parts[q].d_part, parts[q].tokens, E);
        bool again = false;                  // a part may be counted twice
        for (int32_t o = 0; o < q; o++)
            again = again || (parts[o].d_part == parts[q].d_part && parts[o].tokens == parts[q].tokens);
        if (!again) spans.add(bytes(parts[q].d_part, a.part[q].bytes(E), true));
    }
    if (sums != stats) spans.add(bytes(sums, 8 * (2 * (size_t)E + 1), false));
    spans.add(bytes(stats, 8 * (2 * (size_t)E + 1), true));
    spans.add(bytes(loss, 4, true));
    spans.add(bytes(coef, 4 * (size_t)E, true));
    spans.add(bytes(counts, 8 * (size_t)E, true));
    if (spans.clash()) return DQ_EINVAL;
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
    }
    Spans spans;
    if (!spans.reserve(5 * (size_t)n + 2)) return DQ_EINVAL;
    for (int32_t w = 0; w < n; w++) {
        const dq_route_grad &in = workers[w];
        // in place, the gradient's span stands for the logits' too
        if (in.d_dlogits != in.d_logits || (in.tokens > 1 && in.dstride != in.stride))
            spans.add(span(in.d_logits, in.tokens, in.stride, E, (int64_t)es, false));
        spans.add(bytes(in.d_mask, (size_t)in.tokens, false));
        spans.add(bytes(in.d_ids, 4 * (size_t)in.tokens * k, false));
        spans.add(bytes(in.d_dgates, 4 * (size_t)in.tokens * k, false));
        spans.add(span(in.d_dlogits, in.tokens, in.dstride, E, (int64_t)es, true));
    }
    spans.add(bytes(coef, 4 * (size_t)E, false));
    spans.add(bytes(dloss, 4, false));
    if (spans.clash()) return DQ_EINVAL;
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
