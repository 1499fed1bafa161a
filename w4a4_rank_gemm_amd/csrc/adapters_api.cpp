// adapters_api.cpp -- the C ABI of the adapter, 8-bit checkpoint and input-gradient entry
// points: argument validation, workspace layouts and launches. As in twq_api.cpp every
// check happens before the first HIP call.
#include "twq.h"

#include <hip/hip_runtime.h>

#include "twq_adapters.h"
#include "twq_check.h"
#include "twq_kernels.h"

namespace {

using namespace twq;

constexpr int64_t kMaxAdapterN = int64_t(1) << 22;  // 32-bit offsets inside a tile
constexpr int64_t kMaxOutput = int64_t(1) << 40;    // elements of Y: grid sizes below 2^31

bool valid_type(int t) { return t == TWQ_F16 || t == TWQ_BF16; }
bool valid_count(int64_t c) { return c >= 0 && c <= kMaxAdapters; }
bool valid_shape(int64_t b, int64_t m, int64_t n, int64_t r) {
    return valid_b(b) && valid_m(m) && n > 0 && n % 16 == 0 && n <= kMaxAdapterN && b * n <= kMaxOutput && valid_r(r);
}
// The largest launches: a tile's 256-column blocks, a piece's 128-column blocks. A grid
// dimension holds fewer than 2^32 threads, 2^24 CTAs of 256.
bool valid_grid(int64_t b, int64_t m, int64_t n, int64_t count) {
    return (b / 64 + count + 1) * ((m + n) / 128 + 2) < int64_t(1) << 24;
}

twq_status done(hipError_t e, const char *name) { return e == hipSuccess ? TWQ_OK : (twq_status)hip_error(e, name); }

const uint16_t *u16(const void *p) { return static_cast<const uint16_t *>(p); }

struct ForwardLayout {
    int ks;
    size_t p, parts, total;
};

struct GradLayout {
    int ks;
    size_t p, parts, g, planes, part, total;
};

ForwardLayout forward_layout(int64_t b, int64_t k, int64_t r, int64_t count) {
    ForwardLayout L{};
    L.ks = shrink_slices(b, k, r, plan_layout(b, count).max_tiles, 4);
    L.p = 0;
    L.parts = align256((size_t)L.ks * b * r * 4);
    L.total = L.parts + align256(expand_parts_bytes(b, r));
    return L;
}

// The two scratch arrays of expand, one behind the other.
void set_parts(ExpandArgs &a, uint8_t *at) {
    a.parts = at;
    a.undo = reinterpret_cast<float *>(at + (size_t)a.b * ((size_t)(a.r + 31) / 32 * 128));
}

GradLayout grad_layout(int64_t b, int64_t m, int64_t n, int64_t r, int64_t count) {
    const PlanLayout pl = plan_layout(b, count);
    GradLayout L{};
    L.ks = b > 0 ? shrink_slices(b, n, r, pl.max_tiles, 4) : 1;
    L.p = 0;
    L.parts = align256((size_t)L.ks * b * r * 4);
    L.g = L.parts + align256(expand_parts_bytes(b, r));
    L.planes = L.g + align256((size_t)b * r * 4);
    L.part = L.planes + align256((size_t)b * r * 8);
    L.total = L.part + align256((size_t)pl.max_slots * r * (m + n) * 4);
    return L;
}

}  // namespace

extern "C" {

size_t twq_adapter_plan_bytes(int64_t b, int64_t count) {
    if (!valid_b(b) || !valid_count(count)) return 0;
    return plan_layout(b, count).total;
}

twq_status twq_adapter_plan(const int32_t *index, int64_t b, int64_t count, void *plan, size_t plan_bytes, void *stream) {
    if (!valid_b(b) || !valid_count(count)) return TWQ_ERR_SHAPE;
    if ((b > 0 && !index) || !plan) return TWQ_ERR_NULL;
    if (!aligned16(index) || !aligned16(plan)) return TWQ_ERR_ALIGN;
    if (plan_bytes < plan_layout(b, count).total) return TWQ_ERR_WORKSPACE;
    return done(launch_adapter_plan(index, b, count, plan, static_cast<hipStream_t>(stream)), "twq_adapter_plan");
}

size_t twq_adapters_workspace_bytes(int64_t b, int64_t m, int64_t n, int64_t r, int64_t count) {
    if (!valid_shape(b, m, n, r) || r == 0 || !valid_count(count) || !valid_grid(b, m, n, count) || b == 0) return 0;
    return forward_layout(b, m, r, count).total;
}

twq_status twq_adapters(const void *x, const void *at, const void *bt, const float *scale, const void *plan,
                        size_t plan_bytes, const void *y, void *out, float *h, int64_t b, int64_t m, int64_t n,
                        int64_t r, int64_t count, int type, void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_type(type)) return TWQ_ERR_UNSUPPORTED;
    if (!valid_shape(b, m, n, r) || r == 0 || !valid_count(count) || !valid_grid(b, m, n, count)) return TWQ_ERR_SHAPE;
    if (b == 0) return TWQ_OK;
    if (!x || !plan || !out || (count > 0 && (!at || !bt))) return TWQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(at) || !aligned16(bt) || !aligned16(scale) || !aligned16(plan) || !aligned16(y) ||
        !aligned16(out) || !aligned16(h))
        return TWQ_ERR_ALIGN;
    const PlanLayout pl = plan_layout(b, count);
    const ForwardLayout L = forward_layout(b, m, r, count);
    if (plan_bytes < pl.total || !workspace || workspace_bytes < L.total) return TWQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return TWQ_ERR_ALIGN;
    const hipStream_t st = static_cast<hipStream_t>(stream);

    ShrinkArgs s{};
    s.v = u16(x);
    s.w = u16(at);
    s.b = b;
    s.k = m;
    s.r = (int)r;
    s.bf16 = type == TWQ_BF16;
    s.plan = plan_view(plan, pl);
    s.tiles = pl.max_tiles;
    s.ks = L.ks;
    s.p = static_cast<float *>(workspace);
    hipError_t e = launch_shrink(s, st);
    if (e != hipSuccess) return done(e, "twq_adapters");

    ExpandArgs x2{};
    x2.p = s.p;
    x2.ks = s.ks;
    x2.w = u16(bt);
    x2.scale = scale;
    x2.b = b;
    x2.n = n;
    x2.r = (int)r;
    x2.bf16 = s.bf16;
    x2.plan = s.plan;
    x2.tiles = pl.max_tiles;
    x2.base = u16(y);
    x2.out = static_cast<uint16_t *>(out);
    x2.sum = h;
    set_parts(x2, static_cast<uint8_t *>(workspace) + L.parts);
    if (b > kFewRows) e = launch_split(x2, st);
    if (e == hipSuccess) e = launch_expand(x2, st);
    return done(e, "twq_adapters");
}

size_t twq_adapters_grad_workspace_bytes(int64_t b, int64_t m, int64_t n, int64_t r, int64_t count) {
    if (!valid_shape(b, m, n, r) || r == 0 || !valid_count(count) || !valid_grid(b, m, n, count)) return 0;
    return grad_layout(b, m, n, r, count).total;
}

twq_status twq_adapters_grad(const void *dy, const void *x, const void *qc, const float *sc, const float *h,
                             const void *at, const void *bt, const float *scale, const void *plan, size_t plan_bytes,
                             const void *dx, void *dx_out, void *dat, void *dbt, int64_t b, int64_t m, int64_t n,
                             int64_t r, int64_t count, int type, void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_type(type)) return TWQ_ERR_UNSUPPORTED;
    if (!valid_shape(b, m, n, r) || r == 0 || !valid_count(count) || !valid_grid(b, m, n, count)) return TWQ_ERR_SHAPE;
    if (b == 0 && count == 0) return TWQ_OK;
    if (!plan || (count > 0 && (!at || !bt || !dat || !dbt))) return TWQ_ERR_NULL;
    if (b > 0 && (!dy || !h || !dx_out || (!x && (!qc || !sc)))) return TWQ_ERR_NULL;
    if (b > 0 && x && qc) return TWQ_ERR_UNSUPPORTED;  // X whole or in 8 bits, not both
    if (!aligned16(dy) || !aligned16(x) || !aligned16(qc) || !aligned16(sc) || !aligned16(h) || !aligned16(at) ||
        !aligned16(bt) || !aligned16(scale) || !aligned16(plan) || !aligned16(dx) || !aligned16(dx_out) ||
        !aligned16(dat) || !aligned16(dbt))
        return TWQ_ERR_ALIGN;
    const PlanLayout pl = plan_layout(b, count);
    const GradLayout L = grad_layout(b, m, n, r, count);
    if (plan_bytes < pl.total || (L.total > 0 && (!workspace || workspace_bytes < L.total))) return TWQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return TWQ_ERR_ALIGN;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    hipError_t e = hipSuccess;

    ShrinkArgs s{};
    s.v = u16(dy);
    s.w = u16(bt);
    s.b = b;
    s.k = n;
    s.r = (int)r;
    s.bf16 = type == TWQ_BF16;
    s.kmajor = 1;
    s.plan = plan_view(plan, pl);
    s.tiles = pl.max_tiles;
    s.ks = L.ks;
    s.p = reinterpret_cast<float *>(ws + L.p);
    if (b > 0) e = launch_shrink(s, st);
    if (e != hipSuccess) return done(e, "twq_adapters_grad");

    ExpandArgs x2{};
    x2.p = s.p;
    x2.ks = s.ks;
    x2.w = u16(at);
    x2.scale = scale;
    x2.b = b;
    x2.n = m;
    x2.r = (int)r;
    x2.bf16 = s.bf16;
    x2.kmajor = 1;
    x2.plan = s.plan;
    x2.tiles = pl.max_tiles;
    x2.base = u16(dx);
    x2.out = static_cast<uint16_t *>(dx_out);
    x2.sum = x ? nullptr : reinterpret_cast<float *>(ws + L.g);
    x2.sum_by_pos = 1;
    x2.planes = reinterpret_cast<uint16_t *>(ws + L.planes);
    x2.h = h;
    set_parts(x2, ws + L.parts);
    // The weight gradients come before the expand where it does not form their factors: their
    // read of dY then finds what the shrink's left in the caches.
    if (b > kFewRows)
        e = launch_split(x2, st);
    else if (b > 0)
        e = launch_expand(x2, st);
    if (e != hipSuccess) return done(e, "twq_adapters_grad");

    OuterArgs o{};
    o.g = x2.sum;
    o.planes = x2.planes;
    o.x = u16(x);
    o.qc = x ? nullptr : static_cast<const int8_t *>(qc);
    o.sc = sc;
    o.dy = u16(dy);
    o.scale = scale;
    o.b = b;
    o.m = m;
    o.n = n;
    o.count = count;
    o.r = (int)r;
    o.bf16 = s.bf16;
    o.plan = s.plan;
    o.chunks = pl.max_chunks;
    o.chunk = chunk_rows(b);
    o.part = reinterpret_cast<float *>(ws + L.part);
    o.dat = static_cast<uint16_t *>(dat);
    o.dbt = static_cast<uint16_t *>(dbt);
    if (count > 0) e = launch_outer(o, st);
    if (e == hipSuccess && b > kFewRows) e = launch_expand(x2, st);
    return done(e, "twq_adapters_grad");
}

twq_status twq_checkpoint_act(const void *x, int64_t b, int64_t m, int type, void *qc, float *sc, void *stream) {
    if (!valid_type(type)) return TWQ_ERR_UNSUPPORTED;
    if (!valid_b(b) || !valid_m(m)) return TWQ_ERR_SHAPE;
    if (b == 0) return TWQ_OK;
    if (!x || !qc || !sc) return TWQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(qc) || !aligned16(sc)) return TWQ_ERR_ALIGN;
    return done(launch_checkpoint(u16(x), b, m, type == TWQ_BF16, static_cast<int8_t *>(qc), sc,
                                  static_cast<hipStream_t>(stream)), "twq_checkpoint_act");
}

twq_status twq_restore_act(const void *qc, const float *sc, int64_t b, int64_t m, int type, void *x, void *stream) {
    if (!valid_type(type)) return TWQ_ERR_UNSUPPORTED;
    if (!valid_b(b) || !valid_m(m)) return TWQ_ERR_SHAPE;
    if (b == 0) return TWQ_OK;
    if (!x || !qc || !sc) return TWQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(qc) || !aligned16(sc)) return TWQ_ERR_ALIGN;
    return done(launch_restore(static_cast<const int8_t *>(qc), sc, b, m, type == TWQ_BF16, static_cast<uint16_t *>(x),
                               static_cast<hipStream_t>(stream)), "twq_restore_act");
}

size_t twq_linear_dx_workspace_bytes(int64_t b, int64_t m, int64_t n, int64_t r) {
    if (!valid_shape(b, m, n, r) || b == 0) return 0;
    return plan_dx(b, m, n, r).total;
}

twq_status twq_linear_dx(const void *dy, const void *qw, const float *sw, const void *l1t, const void *l2t, int64_t r,
                         void *dx, int64_t b, int64_t m, int64_t n, int type, void *workspace, size_t workspace_bytes,
                         void *stream) {
    if (!valid_type(type)) return TWQ_ERR_UNSUPPORTED;
    if (!valid_shape(b, m, n, r)) return TWQ_ERR_SHAPE;
    if (b == 0) return TWQ_OK;
    if (!dy || !qw || !sw || !dx || (r > 0 && (!l1t || !l2t))) return TWQ_ERR_NULL;
    if (!aligned16(dy) || !aligned16(qw) || !aligned16(sw) || !aligned16(dx) || (r > 0 && (!aligned16(l1t) || !aligned16(l2t))))
        return TWQ_ERR_ALIGN;
    const DxPlan p = plan_dx(b, m, n, r);
    if (!workspace || workspace_bytes < p.total) return TWQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return TWQ_ERR_ALIGN;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    hipError_t e = hipSuccess;

    if (r > 0) {
        ShrinkArgs s{};
        s.v = u16(dy);
        s.w = u16(l2t);
        s.b = b;
        s.k = n;
        s.r = (int)r;
        s.bf16 = type == TWQ_BF16;
        s.kmajor = 1;
        s.tiles = (b + tile_rows(b) - 1) / tile_rows(b);
        s.ks = p.tks;
        s.p = reinterpret_cast<float *>(ws + p.t);
        s.sw = sw;
        s.rowmax = reinterpret_cast<float *>(ws + p.rowmax);
        e = launch_shrink(s, st);
        if (e != hipSuccess) return done(e, "twq_linear_dx");
    }
    DxArgs a{};
    a.dy = u16(dy);
    a.qw = static_cast<const uint8_t *>(qw);
    a.sw = sw;
    a.l1t = u16(l1t);
    a.b = b;
    a.m = m;
    a.n = n;
    a.r = (int)r;
    a.bf16 = type == TWQ_BF16;
    a.g = reinterpret_cast<uint16_t *>(ws + p.g);
    a.ge = reinterpret_cast<int32_t *>(ws + p.ge);
    a.rowmax = reinterpret_cast<float *>(ws + p.rowmax);
    a.rks = r > 0 ? p.tks : 1;
    a.t = reinterpret_cast<const float *>(ws + p.t);
    a.tks = p.tks;
    a.t16 = reinterpret_cast<uint16_t *>(ws + p.t16);
    a.ks = p.ks;
    a.part = reinterpret_cast<float *>(ws + p.part);
    a.dx = static_cast<uint16_t *>(dx);
    if (r == 0) e = launch_dx_max(a, st);
    if (e == hipSuccess) e = launch_dx_scale(a, p, st);
    if (e == hipSuccess) e = launch_dx(a, p, st);
    return done(e, "twq_linear_dx");
}

}  // extern "C"
