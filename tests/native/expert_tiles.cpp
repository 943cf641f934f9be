// Prints which kernel computes a product grouped by expert, for shapes on standard input:
//   p FP32 TOKENS TOP_K EXPERTS INNER OUTER GATHER TURNED OFF [STRIDE]      y = x w
//   w FP32 TOKENS TOP_K EXPERTS INNER OUTER GATHER KEPT OFF [STRIDE]        dw = x^T dy
// OFF: elements that x, dy and w lie off 16 bytes; STRIDE: of the rows of x, else the least
// there is.  A line of the result: the tile, whether x and dy are loaded straight into LDS,
// the parts that the rows are split into, whether the blocks fit a launch.  Links with
// csrc/dq_expert_pick.cpp alone.
#include <stdio.h>

#include "dq_experts.h"

using namespace dq;

int main() {
    const char *const names[] = {"Big", "Mid", "Small", "Narrow", "Few", "Any", "FewAny"};
    char op;
    int f32, k, E, gather, last;
    long tokens, K, N, off, xs = 0;
    char line[256];
    while (fgets(line, sizeof(line), stdin) &&
           sscanf(line, " %c %d %ld %d %d %ld %ld %d %d %ld %ld", &op, &f32, &tokens, &k, &E, &K, &N, &gather, &last,
                  &off, &xs) >= 10) {
        const int64_t es = f32 ? 4 : 2, wide = off ? 3 : 0;
        const void *at = reinterpret_cast<const void *>(4096 + off * es);
        const ExpertLists l{nullptr, nullptr, nullptr, tokens, (int32_t)(tokens * k), k, E};
        ExpertPick p;
        int parts = 1;
        if (op == 'p') {
            ExpertProductArgs a{};
            a.l = l;
            a.x = a.w = at;
            a.xs = xs ? xs : K + wide;
            a.gather = gather;
            a.turned = last;
            a.we = K * N;
            a.ws = last ? K : N;
            a.K = (int32_t)K;
            a.N = (int32_t)N;
            p = pick_expert_product(a, f32);
        } else {
            ExpertWeightsArgs a{};
            a.l = l;
            a.x = last ? nullptr : at;
            a.xs = xs ? xs : K + wide;
            a.codes = last ? static_cast<const int8_t *>(at) : nullptr;
            a.dy = at;
            a.dys = N + wide;
            a.gather = gather;
            a.K = (int32_t)K;
            a.N = (int32_t)N;
            a.parts = parts = expert_weights_parts(tokens * k, E, K, N);
            p = pick_expert_weights(a, f32);
        }
        printf("%s %d %d %d %d\n", names[(int)p.tile], p.x_async, p.dy_async, parts, p.fits);
        xs = 0;
    }
    return 0;
}
