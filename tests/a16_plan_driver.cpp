// Prints the launch rules' choices for the shapes on standard input, one line each.
//   a16 b m n r          -> many rows, rows of a CTA, panels of a wave, waves that share K, K slices of T, K slices
//   route b m experts    -> matrix instructions, K slices
//   moe b m f experts k  -> few tokens, shared gate and up, waves that share K, rows of a down tile, K slices
#include <cstdio>
#include <cstring>

#include "twq_moe.h"

int main() {
    char what[16];
    long long b, m, n, r, k;
    while (std::scanf("%15s", what) == 1) {
        if (!std::strcmp(what, "a16")) {
            if (std::scanf("%lld %lld %lld %lld", &b, &m, &n, &r) != 4) return 1;
            const twq::A16Plan p = twq::plan_a16(b, m, n, r);
            std::printf("%d %d %d %d %d %d\n", p.many, p.rows, p.fn, p.kw, p.tks, p.ks);
        } else if (!std::strcmp(what, "route")) {
            if (std::scanf("%lld %lld %lld", &b, &m, &n) != 3) return 1;
            const twq::RoutePlan p = twq::plan_route(b, m, n);
            std::printf("%d %d\n", p.tiled, p.slices);
        } else {
            if (std::scanf("%lld %lld %lld %lld %lld", &b, &m, &n, &r, &k) != 5) return 1;
            const twq::MoePlan p = twq::plan_moe(b, m, n, r, k);
            std::printf("%d %d %d %d %d\n", p.few, p.up_shared, p.up_waves, p.down_rows, p.ks);
        }
    }
    return 0;
}
