// CPU driver for the sanitizer build of moe_api.cpp: every entry point on buffers of exactly the
// documented sizes, over shapes from one token to many, with host stand-ins for the launchers
// that read every input region and write every output and scratch region the kernels would, so
// that a wrong size or workspace offset shows under AddressSanitizer. Nothing runs on a GPU.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "twq.h"
#include "twq_adapters.h"
#include "twq_moe.h"

namespace {

int g_fail = 0;
volatile uint8_t g_sink;
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

void rd(const void *p, size_t bytes) {
    if (!p || !bytes) return;
    const volatile uint8_t *q = static_cast<const volatile uint8_t *>(p);
    uint8_t acc = 0;
    for (size_t i = 0; i < bytes; i += 61) acc ^= q[i];
    g_sink = acc ^ q[bytes - 1];
}

void wr(void *p, size_t bytes) {
    if (p && bytes) std::memset(p, 0x5a, bytes);
}

}  // namespace

namespace twq {

int hip_error(hipError_t, const char *) { return TWQ_ERR_HIP; }

hipError_t launch_shrink(const ShrinkArgs &a, hipStream_t) {
    if (a.ks < 1 || a.tiles < 1 || !a.w_f16 || a.tiles * a.ks * 16 > (int64_t(1) << 31)) return hipErrorInvalidValue;
    rd(a.v, a.b * a.k * 2);
    rd(a.w, a.r * a.k * 2);
    wr(a.p, (size_t)a.ks * a.b * a.r * 4);
    return hipSuccess;
}

hipError_t launch_a16_t(const A16Args &a, hipStream_t) {
    if (a.tks < 1 || a.b * a.r > 65536) return hipErrorInvalidValue;
    rd(a.x, a.b * a.m * 2);
    rd(a.l1t, a.r * a.m * 2);
    wr(a.t, (size_t)a.tks * a.b * a.r * 4);
    return hipSuccess;
}

hipError_t launch_a16(const A16Args &a, const A16Plan &p, hipStream_t) {
    if (a.ks < 1 || (p.many && (a.b <= kFewTokens || a.ks > 1))) return hipErrorInvalidValue;
    rd(a.x, a.b * a.m * 2);
    rd(a.qw, a.n * a.m / 2);
    rd(a.sw, a.m / 128 * a.n * 4);
    if (a.r > 0) {
        rd(a.l2t, a.n * a.r * 2);
        rd(a.t, (size_t)a.tks * a.b * a.r * 4);
    }
    if (p.many) {
        wr(a.x16, a.b * a.m * 2);
        wr(a.xe, a.b * 4);
        wr(a.mul, a.m / 128 * a.n * 4);
        wr(a.mask, a.m / 128 * a.n * 4);
        wr(a.unit, a.n * 4);
        if (a.r > 0) {
            wr(a.t16, a.b * a.r * 4);
            wr(a.te, a.b * 4);
        }
    }
    if (a.ks > 1) wr(a.part, (size_t)a.ks * a.b * a.n * 4);
    wr(a.y, a.b * a.n * 2);
    return hipSuccess;
}

hipError_t launch_route(const RouteArgs &a, hipStream_t) {
    rd(a.x, a.b * a.m * 2);
    rd(a.wr, a.experts * a.m * 2);
    rd(a.bias, a.bias ? a.experts * 4 : 0);
    if (a.slices < 1) return hipErrorInvalidValue;
    wr(a.logits, a.slices * a.b * a.experts * 8);
    wr(a.ids, a.b * a.k * 4);
    wr(a.weights, a.b * a.k * 4);
    return hipSuccess;
}

hipError_t launch_moe(const MoeArgs &a, const MoePlan &p, hipStream_t) {
    if (p.slots < 1 || p.slots > a.b * a.k || p.slots > a.experts || a.ks < 1 || p.few != (a.b <= kFewMoe) || (p.few && p.up_shared))
        return hipErrorInvalidValue;
    rd(a.x, a.b * a.m * 2);
    rd(a.ids, a.b * a.k * 4);
    rd(a.weights, a.b * a.k * 4);
    rd(a.q1, a.experts * a.f * a.m);
    rd(a.s1, a.m / 128 * a.experts * 2 * a.f * 4);
    rd(a.q2, a.experts * a.m * a.f / 2);
    rd(a.s2, a.f / 128 * a.experts * a.m * 4);
    wr(a.h, a.b * a.k * a.f * 4);
    if (p.few) {
        wr(a.entries, a.b * a.k * sizeof(MoeEntry));
        wr(a.entry_count, 4);
    } else {
        wr(a.part, a.ks * a.b * a.k * a.m * 4);
    }
    wr(a.y, a.b * a.m * 2);
    return hipSuccess;
}

}  // namespace twq

namespace {

#define CHECK(call, want)                                                                                       \
    do {                                                                                                        \
        const int got_ = (call);                                                                                \
        if (got_ != (want)) {                                                                                   \
            std::fprintf(stderr, "FAIL %s b=%lld m=%lld: %d, expected %d\n", #call, (long long)b, (long long)m, \
                         got_, (want));                                                                         \
            ++g_fail;                                                                                           \
        }                                                                                                       \
    } while (0)

void layer(int64_t b, int64_t m, int64_t n, int64_t r, int type) {
    void *x = buf(b * m * 2), *qw = buf(n * m / 2), *l1t = buf(r * m * 2), *l2t = buf(n * r * 2), *y = buf(b * n * 2);
    float *sw = (float *)buf(m / 128 * n * 4);
    const size_t wsb = twq_linear_a16_workspace_bytes(b, m, n, r, 128);
    void *ws = wsb ? buf(wsb) : nullptr;
    CHECK(twq_linear_a16(x, qw, sw, r ? l1t : nullptr, r ? l2t : nullptr, r, y, b, m, n, 128, type, ws, wsb, nullptr), TWQ_OK);
    if (wsb)
        CHECK(twq_linear_a16(x, qw, sw, l1t, l2t, r, y, b, m, n, 128, type, ws, wsb - 1, nullptr), TWQ_ERR_WORKSPACE);
    release();
}

void routed(int64_t b, int64_t m, int64_t f, int64_t experts, int64_t k, int type) {
    void *x = buf(b * m * 2), *w = buf(experts * m * 2), *q1 = buf(experts * f * m), *q2 = buf(experts * m * f / 2);
    float *s1 = (float *)buf(m / 128 * experts * 2 * f * 4), *s2 = (float *)buf(f / 128 * experts * m * 4);
    float *bias = (float *)buf(experts * 4), *weights = (float *)buf(b * k * 4);
    int32_t *ids = (int32_t *)buf(b * k * 4);
    void *y = buf(b * m * 2);
    const size_t wr = twq_moe_route_workspace_bytes(b, m, experts, k), we = twq_moe_experts_workspace_bytes(b, m, f, experts, k);
    const size_t wm = twq_moe_workspace_bytes(b, m, f, experts, k);
    void *ws = buf(wr);
    CHECK(twq_moe_route(x, w, bias, b, m, experts, k, TWQ_SIGMOID, 1, 1.f, type, ids, weights, ws, wr, nullptr), TWQ_OK);
    ws = buf(we);
    CHECK(twq_moe_experts(x, ids, weights, q1, s1, q2, s2, y, b, m, f, experts, k, 128, type, ws, we, nullptr), TWQ_OK);
    ws = buf(wm);
    CHECK(twq_moe(x, w, nullptr, q1, s1, q2, s2, y, b, m, f, experts, k, 128, TWQ_SOFTMAX, 0, 2.f, type, ws, wm, nullptr), TWQ_OK);
    if (b > 0)
        CHECK(twq_moe(x, w, bias, q1, s1, q2, s2, y, b, m, f, experts, k, 128, TWQ_SOFTMAX, 1, 1.f, type, ws, wm - 1, nullptr), TWQ_ERR_WORKSPACE);
    release();
}

}  // namespace

int main() {
    const int64_t layers[][4] = {{0, 256, 32, 16},    {1, 128, 16, 0},    {1, 512, 512, 16},   {4, 8192, 2048, 128}, {5, 256, 8208, 48},
                                 {16, 4096, 256, 32}, {17, 384, 48, 0},   {32, 4096, 4096, 16}, {33, 256, 80, 256},   {64, 14336, 512, 0},
                                 {65, 256, 16, 16},   {129, 1024, 272, 0}, {600, 128, 1040, 32}, {2050, 256, 4112, 16}, {4100, 512, 288, 0}, {600, 256, 16384, 16}, {500, 128, 16400, 256}};
    for (const auto &c : layers)
        for (int type : {TWQ_F16, TWQ_BF16}) layer(c[0], c[1], c[2], c[3], type);
    const int64_t moes[][5] = {{0, 256, 128, 4, 2}, {1, 128, 128, 1, 1}, {1, 512, 384, 64, 8}, {3, 256, 256, 5, 5}, {17, 384, 128, 60, 4},
                               {256, 128, 128, 16, 16}, {100, 256, 128, 512, 3}, {16, 128, 256, 20, 16}, {20, 128, 8192, 2, 2}, {256, 1024, 128, 300, 4}, {2, 4096, 128, 40, 4}};
    for (const auto &c : moes)
        for (int type : {TWQ_F16, TWQ_BF16}) routed(c[0], c[1], c[2], c[3], c[4], type);
    if (g_fail) {
        std::fprintf(stderr, "%d check(s) failed\n", g_fail);
        return 1;
    }
    std::printf("moe_driver: all calls returned the expected status\n");
    return 0;
}
