// Prints the launch rules' choices for the shapes on standard input, one line each.
//   dx b m n r          -> token rows, wave groups and channel slices of the input gradient; its K stages;
//                          the row tile and K slices of dY L2
//   rows b              -> the plan's row tile and a weight-gradient piece's rows
#include <cstdio>
#include <cstring>

#include "twq_adapters.h"

int main() {
    char what[16];
    long long b, m, n, r;
    while (std::scanf("%15s", what) == 1) {
        if (!std::strcmp(what, "dx")) {
            if (std::scanf("%lld %lld %lld %lld", &b, &m, &n, &r) != 4) return 1;
            const twq::DxPlan p = twq::plan_dx(b, m, n, r);
            std::printf("%d %d %d %lld %d %d\n", p.bt, p.kg, p.ks, (long long)(p.npad / twq::kDxK), twq::tile_rows(b), p.tks);
        } else {
            if (std::scanf("%lld", &b) != 1) return 1;
            std::printf("%d %d\n", twq::tile_rows(b), twq::chunk_rows(b));
        }
    }
    return 0;
}
