// moe_api.cpp -- the C ABI of the layer with 16-bit activations and of the routed layer: argument
// validation, workspace layouts and launches. As in twq_api.cpp every check happens before
// the first HIP call.
#include "twq.h"

#include <hip/hip_runtime.h>

#include "twq_adapters.h"
#include "twq_check.h"
#include "twq_kernels.h"
#include "twq_moe.h"

namespace {

using namespace twq;

constexpr int64_t kMaxA16N = int64_t(1) << 22;
// Outputs of one call: 256 GB, and fewer than 2^24 tiles, so that no grid dimension has 2^32 threads.
constexpr int64_t kMaxOutput = int64_t(1) << 37;

// ids, weights and bias are read and written one by one: rows of a larger batch's may be passed.
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

bool valid_type(int t) { return t == TWQ_F16 || t == TWQ_BF16; }
bool valid_a16(int64_t b, int64_t m, int64_t n, int64_t r) {
    return valid_b(b) && valid_m(m) && n >= 0 && n % 16 == 0 && n <= kMaxA16N && b * n <= kMaxOutput && valid_r(r);
}
bool valid_route(int64_t b, int64_t m, int64_t experts, int64_t k) {
    return b >= 0 && b <= kMaxMoeTokens && valid_m(m) && experts >= 1 && experts <= kMaxExperts && k >= 1 && k <= kMaxTopK && k <= experts;
}
bool valid_experts(int64_t b, int64_t m, int64_t f, int64_t experts, int64_t k) {
    // a token may choose more often than there are experts here: its choices are given
    return b >= 0 && b <= kMaxMoeTokens && valid_m(m) && valid_m(f) && experts >= 1 && experts <= kMaxExperts && k >= 1 &&
           k <= kMaxTopK && experts * 2 * f <= kMaxN && experts * m <= kMaxN;
}

twq_status done(hipError_t e, const char *name) { return e == hipSuccess ? TWQ_OK : (twq_status)hip_error(e, name); }

const uint16_t *u16(const void *p) { return static_cast<const uint16_t *>(p); }

RouteArgs route_args(const void *x, const void *wr, const float *bias, int64_t b, int64_t m, int64_t experts, int64_t k, int score,
                     int norm, float scale, int type, int32_t *ids, float *weights, void *logits) {
    const RoutePlan p = plan_route(b, m, experts);
    RouteArgs a{};
    a.tiled = p.tiled;
    a.slices = p.slices;
    a.x = u16(x);
    a.wr = u16(wr);
    a.bias = bias;
    a.b = b;
    a.m = m;
    a.experts = (int)experts;
    a.k = (int)k;
    a.bf16 = type == TWQ_BF16;
    a.sigmoid = score == TWQ_SIGMOID;
    a.norm = norm != 0;
    a.scale = scale;
    a.logits = static_cast<double *>(logits);
    a.ids = ids;
    a.weights = weights;
    return a;
}

MoeArgs moe_args(const void *x, const int32_t *ids, const float *weights, const void *q1, const float *s1, const void *q2,
                 const float *s2, void *y, int64_t b, int64_t m, int64_t f, int64_t experts, int64_t k, int type, void *workspace,
                 const MoePlan &p) {
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    MoeArgs a{};
    a.x = u16(x);
    a.ids = ids;
    a.weights = weights;
    a.q1 = static_cast<const uint8_t *>(q1);
    a.s1 = s1;
    a.q2 = static_cast<const uint8_t *>(q2);
    a.s2 = s2;
    a.b = b;
    a.m = m;
    a.f = f;
    a.experts = (int)experts;
    a.k = (int)k;
    a.bf16 = type == TWQ_BF16;
    a.h = reinterpret_cast<uint16_t *>(ws + p.h);
    a.ks = p.ks;
    if (!p.few) {
        a.part = reinterpret_cast<float *>(ws + p.part);
    } else {
        a.entries = reinterpret_cast<MoeEntry *>(ws + p.entries);
        a.entry_count = reinterpret_cast<int32_t *>(a.entries + b * k);
    }
    a.y = static_cast<uint16_t *>(y);
    return a;
}

}  // namespace

extern "C" {

size_t twq_linear_a16_workspace_bytes(int64_t b, int64_t m, int64_t n, int64_t r, int64_t g) {
    if (g != 128 || !valid_a16(b, m, n, r) || b == 0 || n == 0) return 0;
    return plan_a16(b, m, n, r).total;
}

twq_status twq_linear_a16(const void *x, const void *qw, const float *sw, const void *l1t, const void *l2t, int64_t r, void *y,
                          int64_t b, int64_t m, int64_t n, int64_t g, int type, void *workspace, size_t workspace_bytes,
                          void *stream) {
    if (!valid_type(type) || g != 128) return TWQ_ERR_UNSUPPORTED;
    if (!valid_a16(b, m, n, r)) return TWQ_ERR_SHAPE;
    if (b == 0 || n == 0) return TWQ_OK;
    if (!x || !qw || !sw || !y || (r > 0 && (!l1t || !l2t))) return TWQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(qw) || !aligned16(sw) || !aligned16(y) || (r > 0 && (!aligned16(l1t) || !aligned16(l2t))))
        return TWQ_ERR_ALIGN;
    const A16Plan p = plan_a16(b, m, n, r);
    if (p.total > 0 && (!workspace || workspace_bytes < p.total)) return TWQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return TWQ_ERR_ALIGN;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    hipError_t e = hipSuccess;
    A16Args a{};
    a.x = u16(x);
    a.qw = static_cast<const uint8_t *>(qw);
    a.sw = sw;
    a.l1t = u16(l1t);
    a.l2t = u16(l2t);
    a.t = reinterpret_cast<float *>(ws + p.t);
    a.tks = p.tks;
    a.x16 = reinterpret_cast<uint16_t *>(ws + p.x16);
    a.xe = reinterpret_cast<int32_t *>(ws + p.xe);
    a.mul = reinterpret_cast<float *>(ws + p.mul);
    a.mask = reinterpret_cast<uint32_t *>(ws + p.mask);
    a.small = reinterpret_cast<uint32_t *>(ws + p.small);
    a.unit = reinterpret_cast<float *>(ws + p.unit);
    a.t16 = reinterpret_cast<uint16_t *>(ws + p.t16);
    a.twide = reinterpret_cast<uint16_t *>(ws + p.twide);
    a.te = reinterpret_cast<int32_t *>(ws + p.te);
    a.ks = p.ks;
    a.part = reinterpret_cast<float *>(ws + p.part);
    a.y = static_cast<uint16_t *>(y);
    a.b = b;
    a.m = m;
    a.n = n;
    a.r = (int)r;
    a.bf16 = type == TWQ_BF16;
    if (p.tks > 0 && !p.shrink) e = launch_a16_t(a, st);
    if (p.tks > 0 && p.shrink) {
        ShrinkArgs s{};
        s.v = u16(x);
        s.w = u16(l1t);
        s.b = b;
        s.k = m;
        s.r = (int)r;
        s.bf16 = type == TWQ_BF16;
        s.w_f16 = 1;
        s.tiles = (b + tile_rows(b) - 1) / tile_rows(b);
        s.ks = p.tks;
        s.p = a.t;
        e = launch_shrink(s, st);
    }
    if (e != hipSuccess) return done(e, "twq_linear_a16");
    return done(launch_a16(a, p, st), "twq_linear_a16");
}

size_t twq_moe_route_workspace_bytes(int64_t b, int64_t m, int64_t experts, int64_t k) {
    if (!valid_route(b, m, experts, k)) return 0;
    return b > 0 ? plan_route(b, m, experts).total : 0;
}

twq_status twq_moe_route(const void *x, const void *wr, const float *bias, int64_t b, int64_t m, int64_t experts, int64_t k,
                         int score, int norm, float scale, int type, int32_t *ids, float *weights, void *workspace,
                         size_t workspace_bytes, void *stream) {
    if (!valid_type(type) || (score != TWQ_SOFTMAX && score != TWQ_SIGMOID)) return TWQ_ERR_UNSUPPORTED;
    if (!valid_route(b, m, experts, k)) return TWQ_ERR_SHAPE;
    if (b == 0) return TWQ_OK;
    if (!x || !wr || !ids || !weights) return TWQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(wr) || !aligned4(bias) || !aligned4(ids) || !aligned4(weights)) return TWQ_ERR_ALIGN;
    const size_t need = plan_route(b, m, experts).total;
    if (!workspace || workspace_bytes < need) return TWQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return TWQ_ERR_ALIGN;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const RouteArgs a = route_args(x, wr, bias, b, m, experts, k, score, norm, scale, type, ids, weights, workspace);
    return done(launch_route(a, st), "twq_moe_route");
}

size_t twq_moe_experts_workspace_bytes(int64_t b, int64_t m, int64_t f, int64_t experts, int64_t k) {
    if (!valid_experts(b, m, f, experts, k)) return 0;
    return plan_moe(b, m, f, experts, k).experts;
}

twq_status twq_moe_experts(const void *x, const int32_t *ids, const float *weights, const void *q1, const float *s1,
                           const void *q2, const float *s2, void *y, int64_t b, int64_t m, int64_t f, int64_t experts, int64_t k,
                           int64_t g, int type, void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_type(type) || g != 128) return TWQ_ERR_UNSUPPORTED;
    if (!valid_experts(b, m, f, experts, k)) return TWQ_ERR_SHAPE;
    if (b == 0) return TWQ_OK;
    if (!x || !ids || !weights || !q1 || !s1 || !q2 || !s2 || !y) return TWQ_ERR_NULL;
    if (!aligned16(x) || !aligned4(ids) || !aligned4(weights) || !aligned16(q1) || !aligned16(s1) || !aligned16(q2) ||
        !aligned16(s2) || !aligned16(y))
        return TWQ_ERR_ALIGN;
    const MoePlan p = plan_moe(b, m, f, experts, k);
    if (!workspace || workspace_bytes < p.experts) return TWQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return TWQ_ERR_ALIGN;
    const MoeArgs a = moe_args(x, ids, weights, q1, s1, q2, s2, y, b, m, f, experts, k, type, workspace, p);
    return done(launch_moe(a, p, static_cast<hipStream_t>(stream)), "twq_moe_experts");
}

size_t twq_moe_workspace_bytes(int64_t b, int64_t m, int64_t f, int64_t experts, int64_t k) {
    if (!valid_experts(b, m, f, experts, k) || !valid_route(b, m, experts, k)) return 0;
    return plan_moe(b, m, f, experts, k).total;
}

twq_status twq_moe(const void *x, const void *wr, const float *bias, const void *q1, const float *s1, const void *q2,
                   const float *s2, void *y, int64_t b, int64_t m, int64_t f, int64_t experts, int64_t k, int64_t g, int score,
                   int norm, float scale, int type, void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_type(type) || g != 128 || (score != TWQ_SOFTMAX && score != TWQ_SIGMOID)) return TWQ_ERR_UNSUPPORTED;
    if (!valid_experts(b, m, f, experts, k) || !valid_route(b, m, experts, k)) return TWQ_ERR_SHAPE;
    if (b == 0) return TWQ_OK;
    if (!x || !wr || !q1 || !s1 || !q2 || !s2 || !y) return TWQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(wr) || !aligned4(bias) || !aligned16(q1) || !aligned16(s1) || !aligned16(q2) ||
        !aligned16(s2) || !aligned16(y))
        return TWQ_ERR_ALIGN;
    const MoePlan p = plan_moe(b, m, f, experts, k);
    if (!workspace || workspace_bytes < p.total) return TWQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return TWQ_ERR_ALIGN;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    const RouteArgs r = route_args(x, wr, bias, b, m, experts, k, score, norm, scale, type, reinterpret_cast<int32_t *>(ws + p.ids),
                                   reinterpret_cast<float *>(ws + p.weights), ws + p.logits);
    const MoeArgs a = moe_args(x, r.ids, r.weights, q1, s1, q2, s2, y, b, m, f, experts, k, type, workspace, p);
    hipError_t e = launch_route(r, st);
    if (e == hipSuccess) e = launch_moe(a, p, st);
    return done(e, "twq_moe");
}

}  // extern "C"
