// Host stand-ins for the adapter, checkpoint and input-gradient launchers: each reads every
// input region and writes every output and scratch region the kernels would, sized from the
// arguments, so that a wrong size or workspace offset of the ABI layer shows under
// AddressSanitizer. Pointers are host memory; nothing runs on a GPU.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstring>

#include "twq.h"
#include "twq_adapters.h"

namespace {

volatile uint8_t g_sink;

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

static void plan_read(const PlanView &v, int64_t b, int64_t tiles) {
    rd(v.head, 8);
    rd(v.order, b * 4);
    rd(v.tiles, tiles * sizeof(PlanItem));
    rd(v.rows, tiles * tile_rows(b) * 4);
}

hipError_t launch_adapter_plan(const int32_t *index, int64_t b, int64_t count, void *plan, hipStream_t) {
    rd(index, b * 4);
    wr(plan, plan_layout(b, count).total);
    return hipSuccess;
}

hipError_t launch_shrink(const ShrinkArgs &a, hipStream_t) {
    if (a.ks < 1 || a.tiles < 1 || a.tiles * a.ks * 16 > (int64_t(1) << 31)) return hipErrorInvalidValue;
    rd(a.v, a.b * a.k * 2);
    if (a.plan.rows)
        plan_read(a.plan, a.b, a.tiles);
    else
        rd(a.w, a.r * a.k * 2);
    if (a.rowmax) {
        rd(a.sw, a.k * 4);
        wr(a.rowmax, (size_t)a.ks * a.b * 4);
    }
    wr(a.p, (size_t)a.ks * a.b * a.r * 4);
    return hipSuccess;
}

static void split(const ExpandArgs &a) {
    rd(a.p, (size_t)a.ks * a.b * a.r * 4);
    wr(a.sum, a.b * a.r * 4);
    if (a.planes) {
        rd(a.h, a.b * a.r * 4);
        wr(a.planes, a.b * a.r * 8);
    }
}

hipError_t launch_split(const ExpandArgs &a, hipStream_t) {
    if (a.b <= kFewRows) return hipErrorInvalidValue;
    plan_read(a.plan, a.b, a.tiles);
    split(a);
    wr(a.parts, a.b * ((a.r + 31) / 32 * 128));
    wr(a.undo, a.b * 4);
    return hipSuccess;
}

hipError_t launch_expand(const ExpandArgs &a, hipStream_t) {
    plan_read(a.plan, a.b, a.tiles);
    if (a.b <= kFewRows) {
        split(a);
    } else {
        rd(a.parts, a.b * ((a.r + 31) / 32 * 128));
        rd(a.undo, a.b * 4);
    }
    rd(a.base, a.b * a.n * 2);
    wr(a.out, a.b * a.n * 2);
    return hipSuccess;
}

hipError_t launch_outer(const OuterArgs &a, hipStream_t) {
    const PlanLayout L = plan_layout(a.b, a.count);
    if (a.chunks != L.max_chunks || a.chunk != chunk_rows(a.b)) return hipErrorInvalidValue;
    rd(a.plan.chunks, L.max_chunks * sizeof(PlanItem));
    rd(a.plan.offsets, (a.count + 2) * 4);
    rd(a.plan.slot0, a.count * 4);
    rd(a.planes, a.b * a.r * 8);
    if (a.qc) {
        rd(a.qc, a.b * a.m);
        rd(a.sc, a.m / 128 * a.b * 4);
        rd(a.g, a.b * a.r * 4);
    } else {
        rd(a.x, a.b * a.m * 2);
    }
    rd(a.dy, a.b * a.n * 2);
    wr(a.part, (size_t)L.max_slots * a.r * (a.m + a.n) * 4);
    wr(a.dat, a.count * a.r * a.m * 2);
    wr(a.dbt, a.count * a.r * a.n * 2);
    return hipSuccess;
}

hipError_t launch_checkpoint(const uint16_t *x, int64_t b, int64_t m, int, int8_t *qc, float *sc, hipStream_t) {
    rd(x, b * m * 2);
    wr(qc, b * m);
    wr(sc, m / 128 * b * 4);
    return hipSuccess;
}

hipError_t launch_restore(const int8_t *qc, const float *sc, int64_t b, int64_t m, int, uint16_t *x, hipStream_t) {
    rd(qc, b * m);
    rd(sc, m / 128 * b * 4);
    wr(x, b * m * 2);
    return hipSuccess;
}

hipError_t launch_dx_max(const DxArgs &a, hipStream_t) {
    rd(a.dy, a.b * a.n * 2);
    wr(a.rowmax, a.b * 4);
    return hipSuccess;
}

hipError_t launch_dx_scale(const DxArgs &a, const DxPlan &p, hipStream_t) {
    rd(a.dy, a.b * a.n * 2);
    rd(a.sw, a.n * 4);
    rd(a.rowmax, (size_t)a.rks * a.b * 4);
    rd(a.t, (size_t)a.tks * a.b * a.r * 4);
    wr(a.g, a.b * p.npad * 2);
    wr(a.ge, a.b * 8);
    wr(a.t16, a.b * ((a.r + 31) / 32 * 32) * 4);
    return hipSuccess;
}

hipError_t launch_dx(const DxArgs &a, const DxPlan &p, hipStream_t) {
    if (p.ks < 1 || p.npad % 64 || p.npad < a.n || (p.bt != 32 && p.bt != 64 && p.bt != 128)) return hipErrorInvalidValue;
    if (p.ks > p.npad / 64) return hipErrorInvalidValue;
    rd(a.g, a.b * p.npad * 2);
    rd(a.ge, a.b * 8);
    rd(a.qw, a.n * a.m / 2);
    rd(a.t16, a.b * ((a.r + 31) / 32 * 32) * 4);
    rd(a.l1t, a.r * a.m * 2);
    if (p.ks > 1) wr(a.part, (size_t)p.ks * a.b * a.m * 4);
    wr(a.dx, a.b * a.m * 2);
    return hipSuccess;
}

}  // namespace twq
