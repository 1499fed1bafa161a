// twq_adapters.h -- launch interface of the adapter, 8-bit checkpoint and
// input-gradient kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace twq {

// ---- the plan of a batch: its token rows sorted by adapter ---------------------------

// Token rows of one tile (never two adapters in one): 16 up to 256 rows, which the kernels
// for few rows take (no launch that splits the rows' sums); 64 above; 128 for many (the weights of
// a tile are read once a tile). Measured, forward (8 adapters):
//   b=256, 4096 -> 4096, 32 ranks      16-row tiles 12.0 us, 64-row 14.7
//   b=512, 4096 -> 4096, 32 ranks      14.5, 17.7;  8192 -> 28672, 128 ranks 67, 55
//   b=2048, 4096 -> 14336, 64 ranks    64-row tiles 55.6 us, 128-row 60.4
//   b=4096, the same                   89 and 92; its gradients 129 and 124
constexpr int kFewRows = 256, kManyRows = 2048;
inline int tile_rows(int64_t b) { return b <= kFewRows ? 16 : b <= kManyRows ? 64 : 128; }
constexpr int64_t kMaxAdapters = 4096;

// Rows of one piece of an adapter's tokens in the weight-gradient kernel. Longer pieces
// write fewer partial sums, shorter ones share the work better. At 8192 rows of 16 ragged
// adapters (4096 -> 14336, 64 ranks) pieces of 2048, 1024 and 512 rows took 87, 94 and 103 us
// with the joining of the sums; at 2048 rows of 8 (32 ranks) 1024 and 512 rows 24.6 and 28 us.
constexpr int kMaxChunk = 2048;
inline int chunk_rows(int64_t b) { return b >= 8192 ? kMaxChunk : b >= 2048 ? 1024 : 512; }

// One tile or piece: adapter (-1: the rows without one), first position in `order`, rows (a
// piece of none: the adapter has none), and for a piece the slot of its partial sums (-1: the only piece of its adapter, which
// needs none).
struct PlanItem {
    int32_t adapter, first, rows, slot;
};

// Byte offsets inside the plan block, from b and count alone.
struct PlanLayout {
    size_t head;     // int32: tiles, pieces
    size_t order;    // int32 [b]: token rows sorted by adapter (stable), those without one last
    size_t offsets;  // int32 [count + 2]: first position of each adapter; of the rows without; b
    size_t slot0;    // int32 [count]: first partial-sum slot of each adapter
    size_t tiles;    // PlanItem [max_tiles]
    size_t rows;     // int32 [max_tiles][tile_rows(b)]: each tile's token rows, the last one repeated to the end
    size_t chunks;   // PlanItem [max_chunks]
    int64_t max_tiles, max_chunks, max_slots;
    size_t total;
};

inline PlanLayout plan_layout(int64_t b, int64_t count) {
    auto up = [](size_t v) { return (v + 63) & ~size_t(63); };
    PlanLayout L{};
    // sum over adapters of ceil(n_a / T) <= b / T + the number of adapters with tokens
    L.max_tiles = b / tile_rows(b) + (count + 1 < b ? count + 1 : b);
    L.max_chunks = b / chunk_rows(b) + count;
    // adapters of several pieces only: ceil(n / T) < 2 n / T for n > T
    L.max_slots = 2 * b / chunk_rows(b);
    L.head = 0;
    L.order = 64;
    L.offsets = up(L.order + (size_t)b * 4);
    L.slot0 = up(L.offsets + (size_t)(count + 2) * 4);
    L.tiles = up(L.slot0 + (size_t)count * 4);
    L.rows = up(L.tiles + (size_t)L.max_tiles * sizeof(PlanItem));
    L.chunks = up(L.rows + (size_t)L.max_tiles * tile_rows(b) * 4);
    L.total = up(L.chunks + (size_t)L.max_chunks * sizeof(PlanItem));
    return L;
}

struct PlanView {
    const int32_t *head, *order, *offsets, *slot0, *rows;
    const PlanItem *tiles, *chunks;
};

inline PlanView plan_view(const void *plan, const PlanLayout &L) {
    const uint8_t *p = static_cast<const uint8_t *>(plan);
    return PlanView{reinterpret_cast<const int32_t *>(p + L.head),    reinterpret_cast<const int32_t *>(p + L.order),
                    reinterpret_cast<const int32_t *>(p + L.offsets), reinterpret_cast<const int32_t *>(p + L.slot0),
                    reinterpret_cast<const int32_t *>(p + L.rows),
                    reinterpret_cast<const PlanItem *>(p + L.tiles),  reinterpret_cast<const PlanItem *>(p + L.chunks)};
}

hipError_t launch_adapter_plan(const int32_t *index, int64_t b, int64_t count, void *plan, hipStream_t stream);

// ---- first product: P[s][pos][r] = partial sums over K slices of V W ------------------

struct ShrinkArgs {
    const uint16_t *v;   // [b][k] fp16 or bf16 rows
    const uint16_t *w;   // per adapter [r][k], or [k][r] (kmajor)
    int64_t b, k;
    int r;
    int bf16;            // type of v and w (rowmax: w is fp16)
    int w_f16;           // w is fp16 whatever v is ([r][k] only)
    int kmajor;
    const float *sw;     // with rowmax: [k]
    float *rowmax;       // [ks][b]: largest |v sw| of a row over a slice, or NULL (the plain products)
    PlanView plan;       // rows == NULL: one adapter, positions are rows
    int64_t tiles;       // grid bound
    int ks;              // K slices
    float *p;            // [ks][b][r]
};
int shrink_slices(int64_t b, int64_t k, int64_t r, int64_t tiles, int64_t least);  // plan.cpp
hipError_t launch_shrink(const ShrinkArgs &a, hipStream_t stream);

// ---- second product: out[row] = base[row] + c (sum_s P[s][pos]) W ---------------------

struct ExpandArgs {
    const float *p;      // [ks][b][r]
    int ks;
    const uint16_t *w;   // per adapter [n][r], or [r][n] (kmajor)
    const float *scale;  // [count] or NULL (1)
    int64_t b, n;
    int r;
    int bf16;
    int kmajor;
    PlanView plan;
    int64_t tiles;
    const uint16_t *base;  // [b][n] or NULL (0)
    uint16_t *out;         // [b][n]; may be base
    float *sum;            // sum_s P (unscaled) [b][r], or NULL
    int sum_by_pos;        // sum is by position in the plan instead of by token row
    uint16_t *planes;      // bf16 [4][b][r] by position: c sum_s P as hi + lo, c h as hi + lo; or NULL
    const float *h;        // with planes: [b][r] by token row
    uint8_t *parts;        // more than kFewRows rows: [b][r rounded up to 32][2] 16-bit scratch
    float *undo;           // more than kFewRows rows: [b] scratch
};
inline size_t expand_parts_bytes(int64_t b, int64_t r) {
    return b > kFewRows ? (size_t)b * ((size_t)(r + 31) / 32 * 128 + 4) : 0;
}
// More than kFewRows rows: the split forms the sums' parts (and planes and sums), the expand uses
// them. Up to kFewRows rows the expand does both.
hipError_t launch_split(const ExpandArgs &a, hipStream_t stream);
hipError_t launch_expand(const ExpandArgs &a, hipStream_t stream);

// ---- weight gradients -------------------------------------------------------------------

struct OuterArgs {
    const float *g;        // [b][r] by position: dY B (unscaled); with qc
    const uint16_t *planes;  // bf16 [4][b][r] by position: c dY B as hi + lo, c X A as hi + lo
    const uint16_t *x;     // [b][m], or NULL: qc, sc
    const int8_t *qc;      // [b][m] codes
    const float *sc;       // [m / 128][b]
    const uint16_t *dy;    // [b][n]
    const float *scale;
    int64_t b, m, n, count;
    int r;
    int bf16;
    PlanView plan;
    int64_t chunks;        // grid bound
    int chunk;             // rows of a piece
    float *part;           // [slots][r (m + n)] fp32, for adapters of several pieces
    uint16_t *dat;         // [count][r][m]
    uint16_t *dbt;         // [count][n][r]
};
hipError_t launch_outer(const OuterArgs &a, hipStream_t stream);

// ---- 8-bit checkpoints -----------------------------------------------------------------

hipError_t launch_checkpoint(const uint16_t *x, int64_t b, int64_t m, int bf16, int8_t *qc, float *sc,
                             hipStream_t stream);
hipError_t launch_restore(const int8_t *qc, const float *sc, int64_t b, int64_t m, int bf16, uint16_t *x,
                          hipStream_t stream);

// ---- input gradient of the frozen layer ------------------------------------------------

struct DxArgs {
    const uint16_t *dy;  // [b][n]
    const uint8_t *qw;   // panels
    const float *sw;     // [n]
    const uint16_t *l1t; // [r][m]
    int64_t b, m, n;
    int r;
    int bf16;            // type of dy and dx
    uint16_t *g;         // [b][npad] fp16: dY s_W 2^-e, permuted along n
    int32_t *ge;         // [b][2] exponents of g and of t16
    float *rowmax;       // [rks][b] largest |dY s_W| of a row over a slice
    int rks;
    const float *t;      // [tks][b][r] partial sums of dY L2
    int tks;
    uint16_t *t16;       // [b][r rounded up to 32][2]: dY L2 2^-e in two fp16 parts, 8 hi, 8 lo
    int ks;              // slices of n
    float *part;         // [ks][b][m] fp32 when ks > 1
    uint16_t *dx;        // [b][m]
};
constexpr int kDxM = 256;  // input columns of a CTA: 64 a wave
constexpr int kDxK = 64;   // output channels of a stage: four panels

struct DxPlan {
    int bt;          // token rows a CTA
    int kg;          // groups of four waves that share the channels of a CTA (2: bt = 128 only)
    int ks;          // slices of n
    int64_t npad;    // n rounded up to a K stage
    int tks;         // K slices of dY L2
    size_t g, ge, rowmax, t, t16, part, total;
};
DxPlan plan_dx(int64_t b, int64_t m, int64_t n, int64_t r);  // plan.cpp
hipError_t launch_dx_max(const DxArgs &a, hipStream_t stream);  // r == 0: rowmax, one slice
hipError_t launch_dx_scale(const DxArgs &a, const DxPlan &p, hipStream_t stream);
hipError_t launch_dx(const DxArgs &a, const DxPlan &p, hipStream_t stream);

}  // namespace twq
