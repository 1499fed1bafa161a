// CPU driver for the sanitizer build of adapters_api.cpp: every entry point on buffers of
// exactly the documented sizes, over shapes from one token to many, and the plan's bounds on
// tiles, pieces and partial-sum slots against counts drawn at random.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "twq.h"
#include "twq_adapters.h"

namespace {

int g_fail = 0;
std::vector<void *> g_blocks;

void *buf(size_t bytes) {
    void *p = nullptr;
    if (posix_memalign(&p, 16, bytes ? bytes : 16)) std::abort();
    std::memset(p, 0, bytes ? bytes : 16);
    g_blocks.push_back(p);
    return p;
}

void release() {
    for (void *p : g_blocks) std::free(p);
    g_blocks.clear();
}

#define CHECK(call, want)                                                                                          \
    do {                                                                                                           \
        const int got_ = (call);                                                                                   \
        if (got_ != (want)) {                                                                                      \
            std::fprintf(stderr, "FAIL %s b=%lld m=%lld n=%lld r=%lld count=%lld: %d, expected %d\n", #call,       \
                         (long long)b, (long long)m, (long long)n, (long long)r, (long long)count, got_, (want));  \
            ++g_fail;                                                                                              \
        }                                                                                                          \
    } while (0)

void calls(int64_t b, int64_t m, int64_t n, int64_t r, int64_t count, int type) {
    int32_t *index = (int32_t *)buf(b * 4);
    const size_t pb = twq_adapter_plan_bytes(b, count);
    void *plan = buf(pb);
    CHECK(twq_adapter_plan(index, b, count, plan, pb, nullptr), TWQ_OK);
    CHECK(twq_adapter_plan(index, b, count, plan, pb - 1, nullptr), TWQ_ERR_WORKSPACE);
    void *x = buf(b * m * 2), *y = buf(b * n * 2), *out = buf(b * n * 2), *dx = buf(b * m * 2), *dxo = buf(b * m * 2);
    void *qc = buf(b * m);
    float *sc = (float *)buf(m / 128 * b * 4), *h = (float *)buf(b * r * 4), *scale = (float *)buf(count * 4);
    CHECK(twq_checkpoint_act(x, b, m, type, qc, sc, nullptr), TWQ_OK);
    CHECK(twq_restore_act(qc, sc, b, m, type, x, nullptr), TWQ_OK);
    if (r > 0) {
        void *at = buf(count * r * m * 2), *bt = buf(count * n * r * 2), *dat = buf(count * r * m * 2), *dbt = buf(count * n * r * 2);
        const size_t wf = twq_adapters_workspace_bytes(b, m, n, r, count), wg = twq_adapters_grad_workspace_bytes(b, m, n, r, count);
        void *w1 = buf(wf), *w2 = buf(wg);
        CHECK(twq_adapters(x, at, bt, scale, plan, pb, y, out, h, b, m, n, r, count, type, w1, wf, nullptr), TWQ_OK);
        CHECK(twq_adapters(x, at, bt, nullptr, plan, pb, nullptr, out, nullptr, b, m, n, r, count, type, w1, wf, nullptr), TWQ_OK);
        if (b > 0)
            CHECK(twq_adapters(x, at, bt, scale, plan, pb, y, out, h, b, m, n, r, count, type, w1, wf - 1, nullptr), TWQ_ERR_WORKSPACE);
        CHECK(twq_adapters_grad(y, x, nullptr, nullptr, h, at, bt, scale, plan, pb, dx, dxo, dat, dbt, b, m, n, r, count, type, w2, wg, nullptr), TWQ_OK);
        CHECK(twq_adapters_grad(y, nullptr, qc, sc, h, at, bt, nullptr, plan, pb, nullptr, dxo, dat, dbt, b, m, n, r, count, type, w2, wg, nullptr), TWQ_OK);
        if (wg > 0)
            CHECK(twq_adapters_grad(y, x, nullptr, nullptr, h, at, bt, scale, plan, pb, dx, dxo, dat, dbt, b, m, n, r, count, type, w2, wg - 1, nullptr), TWQ_ERR_WORKSPACE);
    }
    void *qw = buf(n * m / 2), *l1t = buf(r * m * 2), *l2t = buf(n * r * 2);
    float *sw = (float *)buf(n * 4);
    const size_t wd = twq_linear_dx_workspace_bytes(b, m, n, r);
    void *w3 = buf(wd);
    CHECK(twq_linear_dx(y, qw, sw, r ? l1t : nullptr, r ? l2t : nullptr, r, dx, b, m, n, type, w3, wd, nullptr), TWQ_OK);
    if (b > 0) CHECK(twq_linear_dx(y, qw, sw, l1t, l2t, r, dx, b, m, n, type, w3, wd - 1, nullptr), TWQ_ERR_WORKSPACE);
    release();
}

// tiles, pieces and slots of random row counts stay inside the plan's arrays
void bounds() {
    uint32_t s = 12345;
    auto next = [&](uint32_t m) { return (s = s * 1664525u + 1013904223u) >> 8, (s >> 8) % m; };
    for (int it = 0; it < 4000; ++it) {
        const int64_t count = next(40), b = 1 + next(it % 3 == 0 ? 300 : 20000);
        std::vector<int64_t> rows(count + 1, 0);
        const uint32_t used = 1 + next((uint32_t)count + 1);
        for (int64_t left = b; left > 0;) {
            const int64_t take = 1 + next((uint32_t)left);
            rows[next(used)] += take;
            left -= take;
        }
        const twq::PlanLayout L = twq::plan_layout(b, count);
        const int64_t tr = twq::tile_rows(b), ch = twq::chunk_rows(b);
        int64_t tiles = 0, pieces = 0, slots = 0;
        for (int64_t a = 0; a <= count; ++a) {
            tiles += (rows[a] + tr - 1) / tr;
            if (a == count) break;
            pieces += (rows[a] + ch - 1) / ch;
            if (rows[a] > ch) slots += (rows[a] + ch - 1) / ch;
        }
        if (tiles > L.max_tiles || pieces > L.max_chunks || slots > L.max_slots || ch > twq::kMaxChunk) {
            std::fprintf(stderr, "FAIL bounds b=%lld count=%lld\n", (long long)b, (long long)count);
            ++g_fail;
        }
    }
}

}  // namespace

int main() {
    const int64_t shapes[][5] = {{0, 256, 32, 16, 3},  {0, 256, 32, 16, 0},   {1, 128, 16, 16, 1},   {1, 512, 528, 0, 4},
                                 {5, 256, 80, 48, 40}, {16, 4096, 256, 64, 2}, {256, 384, 48, 96, 7}, {257, 256, 64, 256, 3},
                                 {600, 128, 1040, 32, 0}, {2050, 256, 48, 16, 3}, {8200, 128, 32, 32, 5}, {40, 256, 16, 16, 4096}};
    for (const auto &c : shapes)
        for (int type : {TWQ_F16, TWQ_BF16}) calls(c[0], c[1], c[2], c[3], c[4], type);
    bounds();
    if (g_fail) {
        std::fprintf(stderr, "%d check(s) failed\n", g_fail);
        return 1;
    }
    std::printf("adapters_driver: all calls returned the expected status\n");
    return 0;
}
