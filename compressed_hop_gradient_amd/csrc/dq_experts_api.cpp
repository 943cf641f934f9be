// dq_experts_api.cpp -- the experts' entry points of include/dq.h: argument checks
// and launches.  Stateless; all device work is enqueued on the caller's stream and
// nothing synchronises.
#include "dq.h"

#include "dq_checks.h"
#include "dq_experts.h"

using namespace dq;

namespace {

constexpr int64_t kMostSlots = (int64_t)1 << 30;
constexpr int64_t kMostWidth = (int64_t)1 << 24;
constexpr int64_t kMostStride = (int64_t)1 << 40;

bool bad_counts(int64_t tokens, int32_t k, int32_t E) {
    return E < 1 || E > kExpertsMost || k < 1 || k > kExpertsMostTopK || tokens < 0 || tokens > kMostSlots / k;
}
bool bad_width(int64_t w) { return w < 1 || w > kMostWidth; }
// rows of an operand at one stride; of an output they may not overlap
bool bad_rows(int64_t rows, int64_t stride, int64_t cols, bool out) {
    return stride < 0 || stride > kMostStride || (out && rows > 1 && stride < cols);
}

dq_status check_lists(const dq_expert_lists *l) {
    if (!l) return DQ_ENULL;
    if (bad_counts(l->tokens, l->top_k, l->n_experts)) return DQ_EINVAL;
    if (!l->d_offsets || (l->tokens > 0 && (!l->d_source || !l->d_row))) return DQ_ENULL;
    return aligned(l->d_offsets, 4) && aligned(l->d_source, 4) && aligned(l->d_row, 4) ? DQ_OK : DQ_EINVAL;
}
ExpertLists lists_of(const dq_expert_lists *l) {
    return ExpertLists{l->d_offsets, l->d_source, l->d_row, l->tokens, (int32_t)(l->tokens * l->top_k), l->top_k,
                       l->n_experts};
}
void add_lists(Spans &s, const dq_expert_lists *l) {
    const size_t slots = (size_t)(l->tokens * l->top_k);
    s.add(bytes(l->d_offsets, 4 * ((size_t)l->n_experts + 1), false));
    s.add(bytes(l->d_source, 4 * slots, false));
    s.add(bytes(l->d_row, 4 * slots, false));
}

bool bad_key(const dq_keep_key *k) {
    return (k->flags & ~DQ_KEEP_DITHER) || k->worker < 0 || k->worker > 65535 || k->site >= 0x80000000u ||
           !aligned(k->d_round, 4);
}
KeepKey key_of(const dq_keep_key *k) {
    return KeepKey{(uint32_t)k->seed, (uint32_t)(k->seed >> 32), k->round, (uint32_t)k->worker, k->site, k->d_round,
                   k->flags & DQ_KEEP_DITHER};
}

// The workspace of a weights' gradient: parts' sums, then x restored from its codes.
size_t weights_partial_bytes(int64_t slots, int32_t E, int64_t inner, int64_t outer) {
    const int parts = expert_weights_parts(slots, E, inner, outer);
    return parts > 1 ? (4 * (size_t)parts * E * inner * outer + kAlign - 1) / kAlign * kAlign : 0;
}
// 0 where the codes are decoded as they are read.  Where the product is long, x restored
// once and read 16 bytes at a time is faster.  bf16, us from the codes / restored, with that
// launch: 60 experts, 273 rows, 1000 x 1416 into fp32 178 / 130; 64 of 1024 rows, 2048 x 2816 1474 /
// 863; 64 of 8 rows, 1024 x 1024 58 / 40, of 64 rows 68 / 46.  Short ones save the launch: 8 of
// 16 rows, 512 x 512 10 / 13.
size_t weights_restored_bytes(int64_t rows_x, int64_t slots, int32_t E, int64_t inner, int64_t outer, int f32) {
    const double weights = (double)E * inner * outer, work = (double)slots * inner * outer;
    if (inner % 8 != 0 || (weights < (double)(1 << 25) && work < 4.0 * (1 << 30))) return 0;
    return (size_t)rows_x * inner * (f32 ? 4 : 2);
}

}  // namespace

extern "C" {

size_t dq_expert_rows_bytes(int64_t tokens, int32_t k, int32_t E) {
    if (bad_counts(tokens, k, E)) return 0;
    const int blocks = expert_rows_blocks(tokens * k);
    return kAlign + (blocks > 1 ? 4 * (size_t)blocks * ((size_t)E + 1) : 0);
}

dq_status dq_expert_rows(const int32_t *ids, int64_t tokens, int32_t k, int32_t E, int32_t *offsets, int32_t *source,
                         int32_t *row, void *work, size_t work_bytes, void *stream) {
    if (bad_counts(tokens, k, E)) return DQ_EINVAL;
    const int64_t slots = tokens * k;
    if (!offsets || (slots > 0 && (!ids || !source || !row))) return DQ_ENULL;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(source, 4) || !aligned(row, 4)) return DQ_EINVAL;
    const size_t need = dq_expert_rows_bytes(tokens, k, E);
    if ((!work && need > kAlign) || !aligned(work, kAlign) || work_bytes < need) return DQ_EWORKSPACE;
    Spans spans;
    spans.add(bytes(ids, 4 * (size_t)slots, false));
    spans.add(bytes(offsets, 4 * ((size_t)E + 1), true));
    spans.add(bytes(source, 4 * (size_t)slots, true));
    spans.add(bytes(row, 4 * (size_t)slots, true));
    spans.add(bytes(work, need, true));
    if (spans.clash()) return DQ_EINVAL;
    const ExpertRowsArgs a{ids, offsets, source, row, static_cast<uint32_t *>(work), (int32_t)slots, E,
                           expert_rows_blocks(slots)};
    return hip_status(launch_expert_rows(a, static_cast<hipStream_t>(stream)));
}

dq_status dq_expert_sum(const dq_expert_lists *l, const void *y, int64_t ys, const void *residual, int64_t rs,
                        void *out, int64_t os, int32_t kind, int64_t width, void *stream) {
    const dq_status bad = check_lists(l);
    if (bad != DQ_OK) return bad;
    const int64_t slots = l->tokens * l->top_k;
    if (!is_kind(kind) || bad_width(width) || bad_rows(slots, ys, width, false) ||
        bad_rows(l->tokens, rs, width, false) || bad_rows(l->tokens, os, width, true))
        return DQ_EINVAL;
    if (l->tokens == 0) return DQ_OK;
    if (!y || !out) return DQ_ENULL;
    const int64_t es = (int64_t)elem_bytes(kind);
    if (!aligned(y, es) || !aligned(residual, es) || !aligned(out, es)) return DQ_EINVAL;
    Spans spans;
    add_lists(spans, l);
    spans.add(span(y, slots, ys, width, es, false));
    // the residual's own elements may be replaced by the sums
    if (!(residual == out && (l->tokens == 1 || rs == os)))
        spans.add(span(residual, l->tokens, rs, width, es, false));
    spans.add(span(out, l->tokens, os, width, es, true));
    if (spans.clash()) return DQ_EINVAL;
    const ExpertSumArgs a{lists_of(l), y, residual, out, ys, rs, os, (int32_t)width};
    return hip_status(launch_expert_sum(a, kind == DQ_F32, static_cast<hipStream_t>(stream)));
}

dq_status dq_keep8(const void *x, int32_t kind, int64_t rows, int64_t cols, int64_t xs, int8_t *codes,
                   uint8_t *exponents, const dq_keep_key *key, void *stream) {
    if (!key) return DQ_ENULL;
    if (!is_kind(kind) || rows < 0 || cols < 0 || cols > ((int64_t)1 << 31) || bad_rows(rows, xs, cols, false) ||
        bad_key(key))
        return DQ_EINVAL;
    if (cols > 0 && rows > kMostStride * 1024 / cols) return DQ_EINVAL;          // below 2^50 elements
    if (rows == 0 || cols == 0) return DQ_OK;
    if (!x || !codes || !exponents) return DQ_ENULL;
    const int64_t es = (int64_t)elem_bytes(kind);
    if (!aligned(x, es)) return DQ_EINVAL;
    Spans spans;
    spans.add(span(x, rows, xs, cols, es, false));
    spans.add(bytes(key->d_round, 4, false));
    spans.add(bytes(codes, (size_t)(rows * cols), true));
    spans.add(bytes(exponents, (size_t)(rows * ((cols + 31) / 32)), true));
    if (spans.clash()) return DQ_EINVAL;
    const KeepArgs a{x, rows, cols, xs, nullptr, codes, exponents, key_of(key)};
    return hip_status(launch_keep8(a, kind == DQ_F32, static_cast<hipStream_t>(stream)));
}

dq_status dq_restore8(const int8_t *codes, const uint8_t *exponents, int32_t kind, int64_t rows, int64_t cols, void *y,
                      int64_t ys, void *stream) {
    if (!is_kind(kind) || rows < 0 || cols < 0 || cols > ((int64_t)1 << 31) || bad_rows(rows, ys, cols, true))
        return DQ_EINVAL;
    if (cols > 0 && rows > kMostStride * 1024 / cols) return DQ_EINVAL;
    if (rows == 0 || cols == 0) return DQ_OK;
    if (!codes || !exponents || !y) return DQ_ENULL;
    const int64_t es = (int64_t)elem_bytes(kind);
    if (!aligned(y, es)) return DQ_EINVAL;
    Spans spans;
    spans.add(bytes(codes, (size_t)(rows * cols), false));
    spans.add(bytes(exponents, (size_t)(rows * ((cols + 31) / 32)), false));
    spans.add(span(y, rows, ys, cols, es, true));
    if (spans.clash()) return DQ_EINVAL;
    const RestoreArgs a{codes, exponents, y, rows, cols, ys, nullptr};
    return hip_status(launch_restore8(a, kind == DQ_F32, static_cast<hipStream_t>(stream)));
}

dq_status dq_expert_act(const dq_expert_lists *l, int32_t act, const void *u, int64_t us, const float *gates, void *to,
                        int64_t ts, int32_t kind, int64_t width, int8_t *codes, uint8_t *exponents,
                        const dq_keep_key *key, void *stream) {
    const dq_status bad = check_lists(l);
    if (bad != DQ_OK) return bad;
    const int64_t slots = l->tokens * l->top_k, U = act == DQ_ACT_SWIGLU ? 2 * width : width;
    if (!is_kind(kind) || (act != DQ_ACT_SWIGLU && act != DQ_ACT_RELU) || bad_width(width) ||
        bad_rows(slots, us, U, false) || bad_rows(slots, ts, width, true))
        return DQ_EINVAL;
    if ((codes != nullptr) != (exponents != nullptr) || (codes && !key)) return DQ_ENULL;
    if (codes && bad_key(key)) return DQ_EINVAL;
    if (slots == 0) return DQ_OK;
    if (!u || !gates || !to) return DQ_ENULL;
    const int64_t es = (int64_t)elem_bytes(kind);
    if (!aligned(u, es) || !aligned(to, es) || !aligned(gates, 4)) return DQ_EINVAL;
    Spans spans;
    add_lists(spans, l);
    spans.add(span(u, slots, us, U, es, false));
    spans.add(bytes(gates, 4 * (size_t)slots, false));
    spans.add(span(to, slots, ts, width, es, true));
    if (codes) {
        spans.add(bytes(key->d_round, 4, false));
        spans.add(bytes(codes, (size_t)(slots * U), true));
        spans.add(bytes(exponents, (size_t)(slots * ((U + 31) / 32)), true));
    }
    if (spans.clash()) return DQ_EINVAL;
    ExpertActArgs a{};
    a.l = lists_of(l);
    a.gated = act == DQ_ACT_SWIGLU;
    a.width = (int32_t)width;
    a.u = u;
    a.us = us;
    a.gates = gates;
    a.a = to;
    a.as = ts;
    a.codes = codes;
    a.exponents = exponents;
    if (codes) a.key = key_of(key);
    return hip_status(launch_expert_act(a, kind == DQ_F32, static_cast<hipStream_t>(stream)));
}

dq_status dq_expert_act_backward(const dq_expert_lists *l, int32_t act, const void *u, int64_t us, const int8_t *codes,
                                 const uint8_t *exponents, const void *da, int64_t das, const float *gates, void *du,
                                 int64_t dus, void *again, int64_t as, float *dgates, int32_t kind, int64_t width,
                                 void *stream) {
    const dq_status bad = check_lists(l);
    if (bad != DQ_OK) return bad;
    const int64_t slots = l->tokens * l->top_k, U = act == DQ_ACT_SWIGLU ? 2 * width : width;
    if (!is_kind(kind) || (act != DQ_ACT_SWIGLU && act != DQ_ACT_RELU) || bad_width(width) ||
        bad_rows(slots, us, U, false) || bad_rows(slots, das, width, false) || bad_rows(slots, dus, U, true) ||
        (again && bad_rows(slots, as, width, true)))
        return DQ_EINVAL;
    if ((codes != nullptr) != (exponents != nullptr)) return DQ_ENULL;
    if (slots == 0) return DQ_OK;
    if (codes && u) return DQ_EINVAL;                    // from the one or from the other
    if ((!u && !codes) || !da || !gates || !du) return DQ_ENULL;
    const int64_t es = (int64_t)elem_bytes(kind);
    if (!aligned(u, es) || !aligned(da, es) || !aligned(du, es) || !aligned(again, es) || !aligned(gates, 4) ||
        !aligned(dgates, 4))
        return DQ_EINVAL;
    Spans spans;
    add_lists(spans, l);
    if (codes) {
        spans.add(bytes(codes, (size_t)(slots * U), false));
        spans.add(bytes(exponents, (size_t)(slots * ((U + 31) / 32)), false));
    } else {
        spans.add(span(u, slots, us, U, es, false));
    }
    spans.add(span(da, slots, das, width, es, false));
    spans.add(bytes(gates, 4 * (size_t)slots, false));
    spans.add(span(du, slots, dus, U, es, true));
    spans.add(span(again, slots, as, width, es, true));
    spans.add(bytes(dgates, 4 * (size_t)slots, true));
    if (spans.clash()) return DQ_EINVAL;
    ExpertActArgs a{};
    a.l = lists_of(l);
    a.gated = act == DQ_ACT_SWIGLU;
    a.width = (int32_t)width;
    a.u = u;
    a.us = us;
    a.codes = const_cast<int8_t *>(codes);
    a.exponents = const_cast<uint8_t *>(exponents);
    a.da = da;
    a.das = das;
    a.gates = gates;
    a.du = du;
    a.dus = dus;
    a.a = again;
    a.as = as;
    a.dgates = dgates;
    return hip_status(launch_expert_act_backward(a, kind == DQ_F32, static_cast<hipStream_t>(stream)));
}

dq_status dq_expert_matmul(const dq_expert_lists *l, const void *x, int64_t xs, int32_t flags, const void *w,
                           int64_t we, int64_t ws, void *y, int64_t ys, int32_t kind, int64_t inner, int64_t outer,
                           void *stream) {
    const dq_status bad = check_lists(l);
    if (bad != DQ_OK) return bad;
    const int64_t slots = l->tokens * l->top_k;
    const bool gather = flags & DQ_EXPERT_GATHER, turned = flags & DQ_EXPERT_TURNED;
    const int64_t rows_w = turned ? outer : inner, cols_w = turned ? inner : outer;
    if (!is_kind(kind) || (flags & ~(DQ_EXPERT_GATHER | DQ_EXPERT_TURNED)) || bad_width(inner) || bad_width(outer) ||
        bad_rows(slots, xs, inner, false) || bad_rows(rows_w, ws, cols_w, false) || we < 0 || we > kMostStride ||
        bad_rows(slots, ys, outer, true))
        return DQ_EINVAL;
    if (slots == 0) return DQ_OK;
    if (!x || !w || !y) return DQ_ENULL;
    const int64_t es = (int64_t)elem_bytes(kind);
    if (!aligned(x, es) || !aligned(w, es) || !aligned(y, es)) return DQ_EINVAL;
    Spans spans;
    add_lists(spans, l);
    spans.add(span(x, gather ? l->tokens : slots, xs, inner, es, false));
    spans.add(span_all(w, l->n_experts, we, rows_w, ws, cols_w, es));
    spans.add(span(y, slots, ys, outer, es, true));
    if (spans.clash()) return DQ_EINVAL;
    const ExpertProductArgs a{lists_of(l), x, xs, gather, w, we, ws, turned, y, ys, (int32_t)inner, (int32_t)outer};
    const ExpertPick p = pick_expert_product(a, kind == DQ_F32);
    if (!p.fits) return DQ_EINVAL;
    return hip_status(launch_expert_product(a, p, kind == DQ_F32, static_cast<hipStream_t>(stream)));
}

size_t dq_expert_matmul_grad_bytes(int64_t tokens, int32_t k, int32_t E, int32_t kind, int32_t gather, int64_t inner,
                                   int64_t outer, int32_t kept) {
    if (bad_counts(tokens, k, E) || !is_kind(kind) || bad_width(inner) || bad_width(outer) || gather < 0 ||
        gather > DQ_GATHER_DOUT)
        return 0;
    return kAlign + weights_partial_bytes(tokens * k, E, inner, outer) +
           (kept ? weights_restored_bytes(gather == DQ_GATHER_X ? tokens : tokens * k, tokens * k, E, inner, outer,
                                          kind == DQ_F32)
                 : 0);
}

dq_status dq_expert_matmul_grad(const dq_expert_lists *l, const void *x, int64_t xs, const int8_t *codes,
                                const uint8_t *exponents, const void *dy, int64_t dys, int32_t gather, void *dw,
                                int32_t kind, int32_t out_kind, int64_t inner, int64_t outer, void *work,
                                size_t work_bytes, void *stream) {
    const dq_status bad = check_lists(l);
    if (bad != DQ_OK) return bad;
    const int64_t slots = l->tokens * l->top_k;
    if (!is_kind(kind) || (out_kind != DQ_F32 && out_kind != kind) || gather < 0 || gather > DQ_GATHER_DOUT ||
        bad_width(inner) || bad_width(outer) || bad_rows(slots, xs, inner, false) || bad_rows(slots, dys, outer, false))
        return DQ_EINVAL;
    if ((codes != nullptr) != (exponents != nullptr)) return DQ_ENULL;
    if (codes && x) return DQ_EINVAL;                    // from the one or from the other
    if (!dw || (slots > 0 && ((!x && !codes) || !dy))) return DQ_ENULL;
    const int64_t es = (int64_t)elem_bytes(kind), os = (int64_t)elem_bytes(out_kind);
    if (!aligned(x, es) || !aligned(dy, es) || !aligned(dw, os)) return DQ_EINVAL;
    const size_t need =
        dq_expert_matmul_grad_bytes(l->tokens, l->top_k, l->n_experts, kind, gather, inner, outer, codes != nullptr);
    if (!work || !aligned(work, kAlign) || work_bytes < need) return DQ_EWORKSPACE;
    const int64_t rows_x = gather == DQ_GATHER_X ? l->tokens : slots;
    Spans spans;
    add_lists(spans, l);
    if (codes) {
        spans.add(bytes(codes, (size_t)(rows_x * inner), false));
        spans.add(bytes(exponents, (size_t)(rows_x * ((inner + 31) / 32)), false));
    } else {
        spans.add(span(x, rows_x, xs, inner, es, false));
    }
    spans.add(span(dy, gather == DQ_GATHER_DOUT ? l->tokens : slots, dys, outer, es, false));
    spans.add(bytes(dw, (size_t)(l->n_experts * inner * outer * os), true));
    spans.add(bytes(work, need, true));
    if (spans.clash()) return DQ_EINVAL;
    ExpertWeightsArgs a{};
    a.l = lists_of(l);
    a.x = x;
    a.xs = xs;
    a.codes = codes;
    a.exponents = exponents;
    a.dy = dy;
    a.dys = dys;
    a.gather = gather;
    a.dw = dw;
    a.out_f32 = out_kind == DQ_F32;
    a.K = (int32_t)inner;
    a.N = (int32_t)outer;
    a.partial = static_cast<float *>(work);
    a.parts = expert_weights_parts(slots, l->n_experts, inner, outer);
    RestoreArgs r{};
    if (codes && slots > 0 && weights_restored_bytes(rows_x, slots, l->n_experts, inner, outer, kind == DQ_F32)) {
        // of the rows, those of experts alone
        char *const at = static_cast<char *>(work) + weights_partial_bytes(slots, l->n_experts, inner, outer);
        r = RestoreArgs{codes, exponents, at, rows_x, inner, inner,
                        gather == DQ_GATHER_X ? nullptr : l->d_offsets + l->n_experts};
        a.x = at;
        a.xs = inner;
        a.codes = nullptr;
    }
    const ExpertPick p = pick_expert_weights(a, kind == DQ_F32);
    if (!p.fits) return DQ_EINVAL;
    if (r.y) {
        const hipError_t e = launch_restore8(r, kind == DQ_F32, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return hip_status(e);
    }
    return hip_status(launch_expert_weights(a, p, kind == DQ_F32, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
