// dq_route_backward.hip -- gradient of the router for gfx950: by the logits, from
// the gates' and the balance loss's, in one pass that computes the softmax again.
// fp32 arithmetic, no contraction.
#include "dq_route_device.h"

namespace dq {

namespace {

// LDS traffic between the lanes of one wave: orders it for the compiler too
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The gradient of a row is p_j (a_j - D) + h_j, where h is 0 but for the chosen
// experts: the lanes that hold the choices scatter it into a row of LDS, which is 0
// between rows.  A row is read and written once, its softmax computed again
// (which costs less than reading p); its choices are read a row ahead, so that
// their logits are on the way while the softmax is computed.
//
// Bound: memory, with the VALUs busy 81% of the time.  131072 x 256 bf16, k = 8
// (142 MB with the choices): 27 to 30 us, 4.7 to 5.3 TB/s; 65536 x 256 fp32: 25 to
// 26.5 us, 5.3 to 5.5 TB/s; 8192 tokens 4.1 and 5.9 us.  All blocks read the same few lines of coef first, which
// serialises them: with 16 single loads a lane instead of 4 wide ones the same
// took 33.8, 28.8, 6.9 and 6.7 us (against 27, 25.5, 3.7 and 5.2 in that run).  At most 1024 blocks (4 per CU): each pays for
// its start (2048: 28.1 and 25.5 us).
template <bool F32, int G, int CH, int S, bool VEC>
__global__ __launch_bounds__(256) void k_route_backward(RouteBackwardArgs args) {
    const RouteBackwardWorker &a = args.worker[blockIdx.y];
    typedef Elem<F32> El;
    typedef typename El::type T;
    typedef Slice<F32, G, CH, VEC> L;
    constexpr int V = L::V, W = L::W, C = V * G, R = 256 / G;
    if ((int64_t)blockIdx.x * R >= a.tokens) return;
    __shared__ alignas(16) float rows[R * C];
    const int g = threadIdx.x % G, r = threadIdx.x / G;
    float *h = rows + r * C;
    const T *logits = static_cast<const T *>(a.logits);
    struct Row {
        L l;
        int id[S];
        float dg[S];
        uint8_t mask;
    };
    // lane g holds choices g, g + G, ..; nothing waits for these loads
    const auto load = [&](Row &row, int64_t t) {
        if (t >= a.tokens) t = a.tokens - 1;
        row.l.load(logits + t * a.stride, g, args.E);
        row.mask = 1;
        if (a.mask) row.mask = a.mask[t];
#pragma unroll
        for (int s = 0; s < S; s++) {
            const int64_t at = t * args.k + (s * G + g < args.k ? s * G + g : 0);
            row.id[s] = -1;
            row.dg[s] = 0.0f;
            if (a.dgates) {
                row.id[s] = a.ids[at];
                row.dg[s] = a.dgates[at];
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * R;
    int64_t t = (int64_t)blockIdx.x * R + r;
    Row next;
    load(next, t);
    // dloss coef of the lane's experts; loads of all of them in flight at once
    float up[V];
    const float w = args.coef ? (args.dloss ? *args.dloss : 1.0f) : 0.0f;
    if (VEC && args.coef && reinterpret_cast<uintptr_t>(args.coef) % 16 == 0) {
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const int at = L::expert(v, g);
            const float4 x = *reinterpret_cast<const float4 *>(args.coef + (at < args.E ? at : 0));
            up[v] = x.x;
            up[v + 1] = x.y;
            up[v + 2] = x.z;
            up[v + 3] = x.w;
        }
    } else if (args.coef) {
#pragma unroll
        for (int v = 0; v < V; v++) up[v] = args.coef[min(L::expert(v, g), args.E - 1)];
    } else {
#pragma unroll
        for (int v = 0; v < V; v++) up[v] = 0.0f;
    }
#pragma unroll
    for (int v = 0; v < V; v++) up[v] *= w;
#pragma unroll
    for (int v = 0; v < V; v += 4)
        *reinterpret_cast<float4 *>(__builtin_assume_aligned(h + 4 * g + v * G, 16)) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    wave_lds_sync();
    for (int64_t base = (int64_t)blockIdx.x * R; base < a.tokens; base += step, t += step) {
        Row row = next;
        const bool there = t < a.tokens && row.mask;
        typename El::type ls[S];
#pragma unroll
        for (int s = 0; s < S; s++) {
            if (!there || s * G + g >= args.k || (uint32_t)row.id[s] >= (uint32_t)args.E) row.id[s] = -1;
            ls[s] = logits[(t < a.tokens ? t : a.tokens - 1) * a.stride + (row.id[s] < 0 ? 0 : row.id[s])];
        }
        if (base + step < a.tokens) load(next, t + step);
        row.l.keep(there, g, args.E);
        float m = -INFINITY, e[V], Z;
#pragma unroll
        for (int v = 0; v < V; v++) m = fmaxf(m, row.l.at(v));
        m = group_max<G>(m);
        if (m == -INFINITY) m = 0.0f;
        exponentials(row.l, m, e, Z);
        const float inv = Z == 0.0f ? 0.0f : reciprocal(Z);
        float dots[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; v++) dots[v % 4] = __builtin_fmaf(e[v], up[v], dots[v % 4]);
        float gs[S], top = 0.0f, gd = 0.0f;
#pragma unroll
        for (int s = 0; s < S; s++) {
            gs[s] = row.id[s] >= 0 ? exponential(El::up(ls[s]), m) : 0.0f;
            top += gs[s];
        }
        if (args.renorm) top = group_sum<G>(top);
#pragma unroll
        for (int s = 0; s < S; s++) {
            // with renorm a quotient, so that a choice alone has the gate 1; 0 where
            // a choice that is not the forward pass's has no weight
            gs[s] = !args.renorm ? gs[s] * inv : top == 0.0f ? 0.0f : gs[s] / top;
            if (row.id[s] >= 0) gd = __builtin_fmaf(gs[s], row.dg[s], gd);
        }
        gd = group_sum<G>(gd);
        // p (a - D) = e (a / Z - D / Z)
        float dot = inv * group_sum<G>((dots[0] + dots[1]) + (dots[2] + dots[3]));
        dot = -inv * (dot + (args.renorm ? 0.0f : gd));
#pragma unroll
        for (int s = 0; s < S; s++)
            if (row.id[s] >= 0) h[row.id[s]] = gs[s] * (args.renorm ? row.dg[s] - gd : row.dg[s]);
        wave_lds_sync();
        // the next row is waited for here: after the stores below it would be
        // waited for together with them
        next.l.arrived();
#pragma unroll
        for (int s = 0; s < S; s++) asm volatile("" : "+v"(next.id[s]), "+v"(next.dg[s]));
        if (t < a.tokens) {
            T *out = static_cast<T *>(a.dlogits) + t * a.dstride;
            if (Z == 0.0f) {
                asm volatile("; a token left out: 0, whatever the loss's gradient is");   // a branch, not selects
                const float d[W] = {};
#pragma unroll
                for (int i = 0; i < L::N; i++) {
                    const int at = L::expert(W * i, g);
                    if (at < args.E) L::C::store(out + at, d);
                }
            } else {
#pragma unroll
                for (int i = 0; i < L::N; i++) {
                    const int at = L::expert(W * i, g);
                    float d[W];
                    __builtin_memcpy(d, __builtin_assume_aligned(h + at, W < 4 ? 4 : 16), sizeof d);
#pragma unroll
                    for (int j = 0; j < W; j++)
                        d[j] = __builtin_fmaf(e[W * i + j], __builtin_fmaf(up[W * i + j], inv, dot), d[j]);
                    if (at < args.E) L::C::store(out + at, d);
                }
            }
        }
        wave_lds_sync();
#pragma unroll
        for (int s = 0; s < S; s++)
            if (row.id[s] >= 0) h[row.id[s]] = 0.0f;
    }
}

template <bool F32, int G, int CH, bool VEC>
hipError_t backward_choices(const RouteBackwardArgs &a, hipStream_t s) {
    // choices of a lane: at most all of 8 experts in one lane
    constexpr int R = 256 / G, most = G == 1 ? 8 : G < kRouteMaxTopK ? kRouteMaxTopK / G : 1;
    static_assert(G > 1 || CH == 1, "");
    int64_t want = 0;
    for (int w = 0; w < a.workers; w++) want = a.worker[w].tokens > want ? a.worker[w].tokens : want;
    want = (want + R - 1) / R;
    const int64_t blocks = 1024 / a.workers;
    const dim3 grid((unsigned)(want < blocks ? want : blocks), (unsigned)a.workers), block(256);
    const int each = (a.k + G - 1) / G;
    if (each <= 1 || most == 1) hipLaunchKernelGGL((k_route_backward<F32, G, CH, 1, VEC>), grid, block, 0, s, a);
    else if (each <= 2 || most == 2)
        hipLaunchKernelGGL((k_route_backward<F32, G, CH, most < 2 ? most : 2, VEC>), grid, block, 0, s, a);
    else if (each <= 4 || most == 4)
        hipLaunchKernelGGL((k_route_backward<F32, G, CH, most < 4 ? most : 4, VEC>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_route_backward<F32, G, CH, most, VEC>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <bool F32>
hipError_t backward_experts(const RouteBackwardArgs &a, hipStream_t s) {
    bool vec = true;
    for (int w = 0; w < a.workers; w++)
        vec = vec && rows_on_16(a.worker[w].logits, a.worker[w].stride, a.E, F32) &&
              rows_on_16(a.worker[w].dlogits, a.worker[w].dstride, a.E, F32);
    return by_experts(a.E, [&](auto G, auto CH) {
        return vec ? backward_choices<F32, G.value, CH.value, true>(a, s)
                   : backward_choices<F32, G.value, CH.value, false>(a, s);
    });
}

}  // namespace

hipError_t launch_route_backward(const RouteBackwardArgs &a, int f32, hipStream_t s) {
    return f32 ? backward_experts<true>(a, s) : backward_experts<false>(a, s);
}

}  // namespace dq
