// dq_route.hip -- expert router for gfx950: softmax, choice of the top_k experts,
// gates and balance statistics of every token in one pass over the logits, and
// the balance loss.  fp32 arithmetic, no contraction.
#include <algorithm>

#include "dq_route_device.h"

namespace dq {

namespace {

// Order key of a logit and its expert: keys are distinct, a larger logit has
// the larger key and of equal ones the lower index.  bf16: the bits in signed
// order, then 16 bits of ~index.  fp32: the bits in unsigned order and 20 bits of
// ~index as the mantissa of a double in [1, 2), which has a one-instruction
// maximum.  chunk is for rows without NaN and ranks -0 below +0; make takes
// anything (-0 = +0, NaN above +inf).  inv: ~index, of a chunk's first expert.
template <bool F32>
struct Key;
template <>
struct Key<false> {
    typedef int32_t type;
    static constexpr int32_t kNone = INT32_MIN;
    static __device__ __forceinline__ uint32_t ordered(uint32_t w) {     // both halves; its own inverse
        typedef short s16x2 __attribute__((ext_vector_type(2)));
        const s16x2 sign = __builtin_bit_cast(s16x2, w) >> 15;
        return __builtin_amdgcn_bitop3_b32(__builtin_bit_cast(uint32_t, sign), 0x7FFF7FFFu, w, 0x6A);   // (a & b) ^ c
    }
    static __device__ __forceinline__ void chunk(const Chunk<false, false> &c, uint32_t inv, int32_t key[1]) {
        key[0] = (int32_t)(ordered(c.v) << 16 | inv);
    }
    static __device__ __forceinline__ void chunk(const Chunk<false, true> &c, uint32_t inv, int32_t key[8]) {
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const uint32_t o = ordered(c.w[q]);
            key[2 * q] = (int32_t)(o << 16 | (inv ^ (2 * q)));
            key[2 * q + 1] = (int32_t)((o & 0xFFFF0000u) | (inv ^ (2 * q + 1)));
        }
    }
    static __device__ __forceinline__ int32_t make(float x, uint32_t inv) {
        x += 0.0f;
        const uint32_t o = x != x ? 0x7FFF0000u : ordered(__float_as_uint(x)) & 0xFFFF0000u;
        return (int32_t)(o | inv);
    }
    static __device__ __forceinline__ int32_t hi(int32_t a, int32_t b) { return max(a, b); }
    static __device__ __forceinline__ int32_t lo(int32_t a, int32_t b) { return min(a, b); }
    static __device__ __forceinline__ int32_t flip(int32_t k, uint32_t x) { return (int32_t)((uint32_t)k ^ x); }
    static __device__ __forceinline__ bool open(int32_t k) { return k >= (int32_t)0x80800000u; }   // above -inf
    static __device__ __forceinline__ bool zero(int32_t k) { return (uint32_t)(k + 0x10000) < 0x20000u; }
    static __device__ __forceinline__ int index(int32_t k) { return (int)(~(uint32_t)k & 0xFFFFu); }
    static __device__ __forceinline__ float value(int32_t k) {
        return __uint_as_float(ordered((uint32_t)k) & 0xFFFF0000u);
    }
};
template <>
struct Key<true> {
    typedef double type;
    static constexpr double kNone = 1.0;
    static __device__ __forceinline__ double pack(uint32_t o, uint32_t inv) {
        const uint32_t h = __builtin_amdgcn_alignbit(0x3FFu, o, 12), l = o << 20 | inv;
        return __builtin_bit_cast(double, (uint64_t)h << 32 | l);
    }
    static __device__ __forceinline__ uint32_t ordered(uint32_t u) {
        return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    }
    static __device__ __forceinline__ void chunk(const Chunk<true, false> &c, uint32_t inv, double key[1]) {
        key[0] = pack(ordered(__float_as_uint(c.v)), inv);
    }
    static __device__ __forceinline__ void chunk(const Chunk<true, true> &c, uint32_t inv, double key[4]) {
#pragma unroll
        for (int j = 0; j < 4; j++) key[j] = pack(ordered(__float_as_uint(c.v[j])), inv ^ j);
    }
    static __device__ __forceinline__ double make(float x, uint32_t inv) {
        x += 0.0f;
        return pack(x != x ? 0xFFFFFFFFu : ordered(__float_as_uint(x)), inv);
    }
    // (fmax and fmin would first quiet every operand that they cannot prove to
    // be no signalling NaN)
    static __device__ __forceinline__ double hi(double a, double b) {
        double r;
        asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
        return r;
    }
    static __device__ __forceinline__ double lo(double a, double b) {
        double r;
        asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
        return r;
    }
    static __device__ __forceinline__ double flip(double k, uint32_t x) {
        return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) ^ x);
    }
    static __device__ __forceinline__ uint32_t order(double k) {
        return (uint32_t)(__builtin_bit_cast(uint64_t, k) >> 20);
    }
    static __device__ __forceinline__ bool open(double k) { return order(k) > 0x007FFFFFu; }       // above -inf
    static __device__ __forceinline__ bool zero(double k) { return order(k) - 0x7FFFFFFFu < 2u; }
    static __device__ __forceinline__ int index(double k) {
        return (int)(~(uint32_t)__builtin_bit_cast(uint64_t, k) & 0xFFFFu);
    }
    static __device__ __forceinline__ float value(double k) {
        const uint32_t o = order(k);
        return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
    }
};

template <int G, int D = 1>
__device__ __forceinline__ int32_t group_most(int32_t x) {
    if constexpr (D < G)
        return group_most<G, 2 * D>((int32_t)with_other_half<D>(
            (uint32_t)x, [](uint32_t a, uint32_t b) { return (uint32_t)max((int32_t)a, (int32_t)b); }));
    return x;
}
// of both words of a double, then the larger
template <int G, int D = 1>
__device__ __forceinline__ double group_most(double x) {
    if constexpr (D < G) {
        const uint64_t b = __builtin_bit_cast(uint64_t, x);
        uint32_t own[2] = {(uint32_t)b, (uint32_t)(b >> 32)}, other[2];
#pragma unroll
        for (int i = 0; i < 2; i++)
            with_other_half<D>(own[i], [&](uint32_t p, uint32_t q) {
                own[i] = p;
                other[i] = q;
                return p;
            });
        return group_most<G, 2 * D>(
            Key<true>::hi(__builtin_bit_cast(double, (uint64_t)own[1] << 32 | own[0]),
                          __builtin_bit_cast(double, (uint64_t)other[1] << 32 | other[0])));
    }
    return x;
}

// Falling lists of the KP largest keys.  Sorting: Batcher's odd-even merge
// network; two lists: the larger of a_i and b_(KP-1-i) are the KP largest, a
// bitonic sequence that log2 KP stages sort.
template <bool F32, int KP>
struct Best {
    typedef Key<F32> K;
    typedef typename K::type T;
    static __device__ __forceinline__ void order(T &a, T &b) {
        const T h = K::hi(a, b);
        b = K::lo(a, b);
        a = h;
    }
    static __device__ __forceinline__ void sort(T *v) {
#pragma unroll
        for (int p = 1; p < KP; p *= 2)
#pragma unroll
            for (int q = p; q >= 1; q /= 2)
#pragma unroll
                for (int j = q % p; j + q < KP; j += 2 * q)
#pragma unroll
                    for (int i = 0; i < q; i++)
                        if (i + j + q < KP && (i + j) / (2 * p) == (i + j + q) / (2 * p)) order(v[i + j], v[i + j + q]);
    }
    static __device__ __forceinline__ void settle(T *v) {
#pragma unroll
        for (int d = KP / 2; d >= 1; d /= 2)
#pragma unroll
            for (int i = 0; i < KP; i++)
                if (!(i & d)) order(v[i], v[i | d]);
    }
    // v takes the KP largest of v and w
    static __device__ __forceinline__ void merge(T *v, const T *w) {
#pragma unroll
        for (int i = 0; i < KP; i++) v[i] = K::hi(v[i], w[KP - 1 - i]);
        settle(v);
    }
};

// The KP largest keys of a row in falling order: lane g has the ones at g, g + G,
// .. in mine, all lanes the first in most.  Each lane sorts its own KP largest; then
// KP times the largest head of the G lists is taken off its list.  inv: ~index of
// the lane's first expert
template <int KP, bool F32, int G, int CH, bool VEC>
__device__ __forceinline__ void pick(const Slice<F32, G, CH, VEC> &l, uint32_t inv, int g,
                                     typename Key<F32>::type mine[(KP + G - 1) / G], typename Key<F32>::type &most) {
    typedef Key<F32> K;
    typename K::type best[KP];
    typedef Best<F32, KP> B;
    constexpr int W = Slice<F32, G, CH, VEC>::W, U = KP < 8 ? 8 : KP, N = U / W;   // elements and chunks sorted together
#pragma unroll
    for (int i = 0; i < Slice<F32, G, CH, VEC>::N; i += N) {
        typename K::type key[U];
#pragma unroll
        for (int n = 0; n < N; n++) {
            if (i + n < Slice<F32, G, CH, VEC>::N) {
                K::chunk(l.c[i + n], inv, key + W * n);
                if (n > 0)
#pragma unroll
                    for (int j = 0; j < W; j++) key[W * n + j] = K::flip(key[W * n + j], W * G * n);
            } else {
#pragma unroll
                for (int j = 0; j < W; j++) key[W * n + j] = K::kNone;
            }
        }
        B::sort(key);
#pragma unroll
        for (int v = KP; v < U; v += KP) {
            B::sort(key + v);
            B::merge(key, key + v);
        }
        if (i == 0) {
#pragma unroll
            for (int j = 0; j < KP; j++) best[j] = key[j];
        } else {
            // chunk i's indices
#pragma unroll
            for (int j = 0; j < KP; j++) key[j] = K::flip(key[j], W * G * i);
            B::merge(best, key);
        }
    }
    if constexpr (G == 1) {
#pragma unroll
        for (int i = 0; i < KP; i++) mine[i] = best[i];
        most = best[0];
    } else {
#pragma unroll
        for (int s = 0; s < KP; s++) {
            const typename K::type head = group_most<G>(best[0]);
            if (s == 0) most = head;
            if (g == s % G) mine[s / G] = head;
            const bool taken = best[0] == head;
            typename K::type own = best[0];
#pragma unroll
            for (int i = 0; i + 1 < KP - s; i++) {
                typename K::type next = best[i + 1];
                asm("" : "+v"(next));         // a select of values, not of their places in the list
                best[i] = taken ? next : own;
                own = next;
            }
        }
    }
}

// The same one key at a time, for rows with NaN or with zeros of both signs
// among the choices; the largest key is not needed again
template <int KP, bool F32, int G, int CH, bool VEC>
__device__ __forceinline__ void pick_any(const Slice<F32, G, CH, VEC> &l, uint32_t inv, int g, int k,
                                         typename Key<F32>::type mine[(KP + G - 1) / G]) {
    typedef Key<F32> K;
    typename K::type last = K::kNone;
#pragma nounroll
    for (int s = 0; s < k; s++) {
        typename K::type most = K::kNone;
#pragma unroll
        for (int v = 0; v < 8 * CH; v++) {
            const typename K::type key = K::make(l.at(v), inv ^ Slice<F32, G, CH, VEC>::expert(v, 0));
            if (s == 0 || key < last) most = K::hi(most, key);
        }
        last = group_most<G>(most);
#pragma unroll
        for (int i = 0; i < (KP + G - 1) / G; i++)
            if (s == i * G + g) mine[i] = last;
    }
}

// p = softmax(l), the k largest l, their p (divided by their sum with renorm), and
// per block the sums over its tokens that the balance loss needs: one pass, a
// row is read once.  All of it is per lane but KP + 1 reductions over G lanes (the
// heads of the lists, the softmax's denominator) and with renorm one more.  The
// probabilities are summed in the lanes' registers over all rows of a block and
// meet in LDS at its end; choices are counted in LDS.
//
// Bound: vector instructions.  131072 x 256 bf16, k = 8, takes 25.1 to 26.4 us (in a
// replayed graph of such calls) where the 67 MB alone take 13; 689 instructions per
// 8 tokens, 0.4 of them in sorting and merging, and the VALUs are busy 76% of the
// time (fp32, 65536 x 256: 21.1 to 22.3 us, 88%; 131072 x 64 bf16: 12.0 us where 17 MB
// and the 8 MB of results take 5, 82%).  k = 2 takes 19.6 us.  Rows with zeros among
// the choices go through pick_any: where all logits are 0, as before the first step of
// a router that starts so, the same rows take 59 us (k = 2 31, 64 experts 19).
// Measured and not kept, on the same rows, when they took 26 (gates were products
// then): rows loaded one pass ahead (no faster; the registers cost a wave per SIMD),
// 4 waves per SIMD where registers then spill (31 us), merging whole lists across
// lanes instead of taking heads off them (27.4 us), the blocks' sums added by 64-bit
// atomics (+4 to +10 us); long sums cut by a second sum in LDS (+0.3 to +2.5 us).
template <bool F32, int G, int CH, int KP, bool VEC>
__global__ __launch_bounds__(256, KP == 16 || CH == 4 || !VEC ? 3 : 4) void k_route(RouteArgs args) {
    const RouteWorker &a = args.worker[blockIdx.y];
    if ((int)blockIdx.x >= a.part.nblk) return;
    typedef typename Elem<F32>::type T;
    typedef Key<F32> K;
    typedef typename K::type KT;
    typedef Slice<F32, G, CH, VEC> L;
    constexpr int V = L::V, C = V * G, R = 256 / G;       // per lane; columns; tokens of a block's pass
    constexpr int S = (KP + G - 1) / G;                   // choices of a lane: g, g + G, ..
    __shared__ uint32_t hist[C];
    __shared__ float sums[R * C];
    __shared__ uint32_t routed_of[4];
    const int g = threadIdx.x % G, r = threadIdx.x / G, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int j = threadIdx.x; j < C; j += 256) hist[j] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; v++) acc[v] = 0.0f;
    uint32_t routed = 0;
    const uint32_t inv = 0xFFFFu ^ (uint32_t)L::expert(0, g);
    const int64_t step = (int64_t)a.part.nblk * R;
    int64_t t = (int64_t)blockIdx.x * R + r;
    for (int64_t base = (int64_t)blockIdx.x * R; base < a.tokens; base += step, t += step) {
        L l;
        const int64_t at = t < a.tokens ? t : a.tokens - 1;
        l.load(static_cast<const T *>(a.logits) + at * a.stride, g, args.E);
        const bool there = t < a.tokens && (!a.mask || a.mask[at]);
        if (!__all(there) || args.E < C) {
            asm volatile("; logits that do not exist");
            l.keep(there, g, args.E);
        }
        KT mine[S], most;
        pick<KP>(l, inv, g, mine, most);
        const float m = K::open(most) ? K::value(most) : 0.0f;
        float e[V], Z;
        exponentials(l, m, e, Z);
        bool odd = Z != Z;
#pragma unroll
        for (int s = 0; s < S; s++) odd = odd || (s * G + g < KP && K::zero(mine[s]));
        if (__any(odd)) {
            uint32_t start = inv;
            asm volatile("; NaN, or zeros that may tie" : "+v"(start));   // (opaque: no constants of it are kept)
            pick_any<KP>(l, start, g, args.k, mine);
        }
        const float by_z = Z == 0.0f ? 0.0f : reciprocal(Z);
        if (g == 0) routed += Z != 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++) acc[v] = __builtin_fmaf(e[v], by_z, acc[v]);

        float ge[S], top = 0.0f;
        int id[S];
#pragma unroll
        for (int s = 0; s < S; s++) {
            const bool open = s * G + g < args.k && K::open(mine[s]);
            id[s] = open ? K::index(mine[s]) : -1;
            ge[s] = open ? exponential(K::value(mine[s]), m) : 0.0f;
            top += ge[s];
        }
        // with renorm a quotient, so that a choice alone has the gate 1
        if (args.renorm) top = group_sum<G>(top);
#pragma unroll
        for (int s = 0; s < S; s++) {
            if (s * G + g < args.k && t < a.tokens) {
                a.ids[t * args.k + s * G + g] = id[s];
                const float gate = args.renorm ? ge[s] / top : ge[s] * by_z;
                a.gates[t * args.k + s * G + g] = id[s] < 0 ? 0.0f : Z != Z ? Z : gate;
                if (id[s] >= 0) atomicAdd(&hist[id[s]], 1u);
            }
        }
    }
    // the block's sums: token rows side by side in LDS, then over the rows.  The
    // thread's number is made again: held over the loop for this, it was spilled
    // (& 255 tells the compiler its range).
    const int own = (64 * wave + (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0))) & 255;
#pragma unroll
    for (int v = 0; v < V; v++) sums[own / G * C + L::expert(v, own % G)] = acc[v];
    for (int d = 32; d; d >>= 1) routed += __shfl_xor((int)routed, d, 64);
    if ((own & 63) == 0) routed_of[wave] = routed;
    __syncthreads();
    constexpr int P = C < 256 ? 256 / C : 1;            // threads per column
    for (int j = own; j < C * P; j += 256) {
        const int col = j % C, part = j / C;
        float sum = 0.0f;
        for (int i = part; i < R; i += P) sum += sums[i * C + col];
        if (P > 1) {
            __syncthreads();
            sums[part * C + col] = sum;
            __syncthreads();
            if (part != 0) break;
            for (int i = 1; i < P; i++) sum += sums[i * C + col];
        }
        if (col < args.E) {
            a.part.psum()[(int)blockIdx.x * args.E + col] = sum;
            a.part.count(args.E)[(int)blockIdx.x * args.E + col] = hist[col];
        }
    }
    if (own == 0) {
        a.part.routed(args.E)[blockIdx.x] = routed_of[0] + routed_of[1] + routed_of[2] + routed_of[3];
        if (blockIdx.x == 0) *a.part.done(args.E) = 0;
    }
}

__device__ __forceinline__ double wave_sum(double v, int from = 32) {
    for (int d = from; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// The outputs from the folded parts: thread j has expert j's choices n and summed
// probabilities p of all parts, and all threads the routed tokens N.
__device__ __forceinline__ void balance_outputs(const BalanceArgs &a, double p, double n, double N) {
    __shared__ double shares[16];
    const int j = threadIdx.x;
    if (a.sums) N += a.sums[2 * a.E];
    __syncthreads();                  // a.stats may be a.sums, whose last element all threads read
    const double f = N > 0.0 ? (double)a.E / ((double)a.k * N * N) : 0.0;
    double share = 0.0;
    if (j < a.E) {
        if (a.sums) {
            n += a.sums[j];
            p += a.sums[a.E + j];
        }
        if (a.stats) {
            a.stats[j] = n;
            a.stats[a.E + j] = p;
            if (j == 0) a.stats[2 * a.E] = N;
        }
        const double w = f * n;
        if (a.coef) a.coef[j] = (float)w;
        if (a.counts) a.counts[j] = (int64_t)n;
        share = w * p;
    }
    share = wave_sum(share);
    if ((j & 63) == 0) shares[j >> 6] = share;
    __syncthreads();
    if (j == 0 && a.loss) {
        for (int w = 1; w < 16; w++) share += shares[w];
        *a.loss = (float)share;
    }
}

// Sums column `col` of a part's rows first, first + step, ..: in groups of U rows
// whose loads are all in flight before the first is added.
template <int U>
__device__ __forceinline__ void fold_rows(const RoutePart &part, int E, int col, int first, int step, double &p,
                                          double &n) {
    const int rows = part.nblk;
    const float *psum = part.psum();
    const uint32_t *count = part.count(E);
    for (int b0 = first; b0 < rows; b0 += U * step) {
        float x[U];
        uint32_t m[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int at = min(b0 + u * step, rows - 1) * E + col;
            x[u] = psum[at];
            m[u] = count[at];
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const bool there = b0 + u * step < rows;
            p += there ? x[u] : 0.0f;
            n += there ? m[u] : 0u;
        }
    }
}

// Few rows: one block for all parts, C >= E columns (a power of two) of 1024 / C
// threads.
__global__ __launch_bounds__(1024) void k_balance_few(BalanceArgs a, int C) {
    __shared__ double ps[1024], cs[1024], ts[16];
    const int i = threadIdx.x, j = i & (C - 1), col = j < a.E ? j : 0;
    double p = 0.0, n = 0.0, t = 0.0;
    for (int q = 0; q < a.parts; q++) {
        for (int b = i; b < a.part[q].nblk; b += 1024) t += a.part[q].routed(a.E)[b];
        if (a.part[q].nblk <= 1024 / C) fold_rows<1>(a.part[q], a.E, col, i / C, 1024 / C, p, n);
        else fold_rows<16>(a.part[q], a.E, col, i / C, 1024 / C, p, n);
    }
    t = wave_sum(t);
    ps[i] = p;
    cs[i] = n;
    if ((i & 63) == 0) ts[i >> 6] = t;
    __syncthreads();
    double N = 0.0;
    for (int w = 0; w < 16; w++) N += ts[w];
    if (i < C) {
#pragma unroll 4
        for (int r = C; r < 1024; r += C) {
            p += ps[r + j];
            n += cs[r + j];
        }
    }
    balance_outputs(a, p, n, N);
}

// A block of 16 waves folds 16 experts of one part, 64 threads for each over the
// rows; the last block to finish adds the parts up.  Every sum runs in a fixed
// order.  Bound by latency: the rows' loads, the count, the last block's loads.
// Four parts of 1024 rows by 256 experts (8 MB): 11 us, 23 with a loop over the
// parts in every block.
__global__ __launch_bounds__(1024) void k_balance(BalanceArgs a) {
    constexpr int COLUMNS = kBalanceColumns, STEP = 1024 / COLUMNS;
    __shared__ double ps[16][COLUMNS], cs[16][COLUMNS], ts[16];
    __shared__ bool last;
    const RoutePart &part = a.part[blockIdx.y];
    const int i = threadIdx.x, lane = i & 63, wave = i >> 6, rows = part.nblk;
    const int j = (int)blockIdx.x * COLUMNS + i % COLUMNS, col = j < a.E ? j : 0;
    double p = 0.0, n = 0.0, t = 0.0;
    fold_rows<16>(part, a.E, col, i / COLUMNS, STEP, p, n);
    if (blockIdx.x == 0)
        for (int b = i; b < rows; b += 1024) t += part.routed(a.E)[b];
    static_assert(COLUMNS == 16, "lanes 16 apart hold one expert");
    p += __shfl_xor(p, 32, 64);
    p += __shfl_xor(p, 16, 64);
    n += __shfl_xor(n, 32, 64);
    n += __shfl_xor(n, 16, 64);
    t = wave_sum(t);
    if (lane < COLUMNS) {
        ps[wave][lane] = p;
        cs[wave][lane] = n;
    }
    if (lane == 0) ts[wave] = t;
    __syncthreads();
    const auto put = [&](int at, double v) {
        __hip_atomic_store(part.fold(a.E) + at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    if (i < COLUMNS) {
        p = n = t = 0.0;
        for (int w = 0; w < 16; w++) {
            p += ps[w][i];
            n += cs[w][i];
            t += ts[w];
        }
        if (j < a.E) {
            put(j, n);
            put(a.E + j, p);
        }
        if (j == 0) put(2 * a.E, t);
        // All that passes between blocks goes through agent-scope atomics, which
        // no cache holds back; they have only to be finished before the count.
        // (A release fence would also write back the whole L2: 4 us here.)
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (i == 0)
            last = __hip_atomic_fetch_add(a.part[0].done(a.E), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                   gridDim.x * gridDim.y - 1;
    }
    __syncthreads();
    if (!last) return;
    if (i == 0) __hip_atomic_store(a.part[0].done(a.E), 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    double N = 0.0;
    p = n = 0.0;
    const int e = i < a.E ? i : 0;
    for (int q = 0; q < a.parts; q++) {
        const auto get = [&](int at) {
            return __hip_atomic_load(a.part[q].fold(a.E) + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        };
        n += get(e);
        p += get(a.E + e);
        N += get(2 * a.E);
    }
    balance_outputs(a, p, n, N);
}

template <bool F32, int G, int CH, bool VEC>
hipError_t route_choices(const RouteArgs &a, hipStream_t s) {
    // 8 experts, or long lists of up to 512 experts, are never asked for more than 8
    constexpr int most_choices = G * CH == 1 || (CH == 4 && G < 32) ? 8 : kRouteMaxTopK;
    int most = 1;
    for (int w = 0; w < a.workers; w++) most = a.worker[w].part.nblk > most ? a.worker[w].part.nblk : most;
    const dim3 grid((unsigned)most, (unsigned)a.workers), block(256);
    if (a.k <= 2) hipLaunchKernelGGL((k_route<F32, G, CH, 2, VEC>), grid, block, 0, s, a);
    else if (a.k <= 4) hipLaunchKernelGGL((k_route<F32, G, CH, 4, VEC>), grid, block, 0, s, a);
    else if (a.k <= 8 || most_choices == 8) hipLaunchKernelGGL((k_route<F32, G, CH, 8, VEC>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_route<F32, G, CH, most_choices, VEC>), grid, block, 0, s, a);
    return hipGetLastError();
}

// The same with longer lists in fewer lanes, for bf16 and E > 128: fewer steps
// across lanes per token, but half as many waves (and fp32 keys take twice the
// registers: 23.6 against 22.0 us for 65536 x 256).  bf16, us, long lists and short:
//            131072 x 256  65536 x 512  32768 x 1024  16384 x 256   512         1024
//   k = 2    19.6  21.8    19.7  22.4   21.2  24.4
//   k = 8    25.7  29.3    26.0  31.0   27.7  33.5     6.7  6.7   10.6  11.1  17.3  19.6
//   k = 16   42.8  39.4    43.1  42.4   34.7  45.9     9.8  8.6   15.6  14.8  20.5  25.5
// (k = 16 up to 512 experts: 16 keys beside the lists do not fit the registers), and
// with k = 8 of 256, 8192 tokens 4.9 against 4.8, 1024 tokens 4.6 against 4.0.
constexpr int64_t kManyTokens = 16384;
inline bool long_lists(int64_t tokens, int E, int k) {
    return tokens >= kManyTokens && E > 128 && (k <= 8 || E > 512);
}
template <class F>
auto by_experts_long(int E, F f) {
    if (E <= 256) return shape<8, 4>(f);
    if (E <= 512) return shape<16, 4>(f);
    return shape<32, 4>(f);
}

template <bool F32>
hipError_t route_experts(const RouteArgs &a, hipStream_t s) {
    bool vec = true;
    int64_t tokens = 0;
    for (int w = 0; w < a.workers; w++) {
        vec = vec && rows_on_16(a.worker[w].logits, a.worker[w].stride, a.E, F32);
        tokens += a.worker[w].tokens;
    }
    if constexpr (!F32)
        if (vec && long_lists(tokens, a.E, a.k))
            return by_experts_long(a.E, [&](auto G, auto CH) { return route_choices<F32, G.value, CH.value, true>(a, s); });
    return by_experts(a.E, [&](auto G, auto CH) {
        return vec ? route_choices<F32, G.value, CH.value, true>(a, s)
                   : route_choices<F32, G.value, CH.value, false>(a, s);
    });
}

}  // namespace

int route_blocks(int64_t tokens, int E) {
    // 4 or 6 blocks of 256 threads per CU, about what the chip holds at once (3 of the
    // kernels compiled for 3 waves per SIMD), and more of them where a lane would add
    // more than 64 tokens' probabilities in fp32: one sum of 5461 equal terms was off
    // by 5e-5.  (Up to 2^22 sums, 50 MB a part: 2^24 tokens of 256 experts.)
    const int64_t rows = by_experts(E, [](auto G, auto) { return 256 / G.value; });
    const int64_t chip = by_experts(E, [](auto, auto CH) { return 256 * (CH.value == 1 ? 6 : 4); });
    const int64_t few_terms = std::min((tokens + 64 * rows - 1) / (64 * rows), (int64_t)(1 << 22) / E);
    const int64_t want = (tokens + rows - 1) / rows, most = std::max(chip, few_terms);
    return (int)(want < 1 ? 1 : want < most ? want : most);
}

hipError_t launch_route(const RouteArgs &a, int f32, hipStream_t s) {
    return f32 ? route_experts<true>(a, s) : route_experts<false>(a, s);
}

hipError_t launch_balance(const BalanceArgs &a, hipStream_t s) {
    static_assert(kRouteMaxExperts == 1024, "a block has a thread for each expert");
    int64_t rows = 0;
    for (int q = 0; q < a.parts; q++) rows += a.part[q].nblk;
    int C = 16;
    while (C < a.E) C *= 2;
    // what one block reads in one go (16 rows a thread) needs no second step
    // between blocks: 256 rows of 64 experts take 6.1 us against 7.1
    if (rows * C <= 16 * 1024)
        hipLaunchKernelGGL(k_balance_few, dim3(1), dim3(1024), 0, s, a, C);
    else
        hipLaunchKernelGGL(k_balance,
                           dim3((unsigned)((a.E + kBalanceColumns - 1) / kBalanceColumns), (unsigned)a.parts),
                           dim3(1024), 0, s, a);
    return hipGetLastError();
}

}  // namespace dq
