// plan.cpp -- host-side planning of the launches (no device code): how the activation
// launch splits T = X L1 and the quantizer, and which decode tiling a few-token shape
// takes. Kept apart from the kernels so it builds with any host compiler (the CPU
// sanitizer tests build it with g++ -fsanitize=address,undefined).
#include <stddef.h>
#include <stdint.h>

#include "twq_adapters.h"
#include "twq_kernels.h"
#include "twq_moe.h"

namespace twq {

static int64_t pow2_floor(int64_t v) {
    int64_t p = 1;
    while (p * 2 <= v) p *= 2;
    return p;
}

ActPlan plan_act(int64_t b, int64_t m, int64_t r) {
    ActPlan pl{};
    pl.ks = 1;
    pl.nsl = 1;
    if (b == 0) return pl;
    if (b > 128) {
        // many tokens: 128-row tiles x all ranks; K slices (steps of 32, at least 512
        // long, at most 32 of them) until about 256 CTAs
        pl.mode = 0;
        pl.row_tile = 128;
        pl.row_tiles = (int)((b + 127) / 128);
        int64_t ks = 1;
        if (r > 0)
            while ((int64_t)pl.row_tiles * ks < 256 && ks < 32 && m / (ks * 2) >= 512 && m % (ks * 2 * 32) == 0)
                ks *= 2;
        pl.ks = (int)ks;
    } else {
        // few tokens: every token x one 16-rank tile x one K slice per CTA, slices of
        // about 32 KB of X and L1 each (a compute unit streams only tens of GB/s, so
        // the read is spread wide; smaller slices measured slower, their partial sums
        // costing more than they spread); each short token row is quantized by nsl CTAs
        pl.mode = 1;
        pl.fm = (int)((b + 15) / 16);
        pl.row_tile = pl.fm * 16;
        pl.row_tiles = (int)(r / 16);
        const int64_t bytes = m * (16 * pl.fm + 16) * 2;
        int64_t ks = pow2_floor(bytes / 32768 > 0 ? bytes / 32768 : 1);
        const int64_t max_ks = m / 128 < 32 ? m / 128 : 32;  // each wave keeps at least one step
        while (ks > max_ks) ks /= 2;
        pl.ks = r > 0 ? (int)ks : 1;
        int64_t nsl = 1;
        while (b * nsl < 128 && (m / 8) / (nsl * 2) >= 32) nsl *= 2;
        pl.nsl = (int)nsl;
    }
    // a row of m fp16 is m / 8 chunks of 16 bytes over 256 threads
    const int64_t per_thread = (m / 8 + 255) / 256;
    pl.jq = per_thread <= 1 ? 1 : per_thread <= 2 ? 2 : per_thread <= 4 ? 4 : per_thread <= 8 ? 8 : 0;
    if (r > 0 && pl.ks > 1) {
        const int64_t rows_pad = pl.mode == 0 ? (int64_t)pl.row_tiles * 128 : (int64_t)pl.fm * 16;
        pl.workspace_bytes = (size_t)pl.ks * rows_pad * r * sizeof(float);
    }
    return pl;
}

// Decode tiles (FN x FM blocks of 16 channels x 16 tokens per CTA, FM = ceil(b / 16)):
// the widest channel tile that still leaves at least 192 CTAs, at most 2 blocks for 16
// tokens and 4 for 64; for 32 tokens 2 blocks, or 8 where the grid stays that wide and
// K is long enough (m >= 8192) for each of the eight waves of such a CTA to stream at
// least 8 pieces. Wider tiles read Q_X from L2 fewer times; fewer CTAs than that leave
// compute units idle. Measured on MI355X (same-process sweeps of 6 tilings on each of
// 37 few-token shapes, m and n from 4096 to 28672, weights cold): within 6% of the best
// tiling on every shape. false: many tokens, the LDS-ring kernel.
bool decode_shape(int64_t b, int64_t m, int64_t n, int &fn, int &fm) {
    if (b > 64) return false;
    fm = b <= 16 ? 1 : b <= 32 ? 2 : 4;
    if (fm == 2) {
        fn = n / 128 >= 192 && m >= 8192 ? 8 : n / 32 >= 192 ? 2 : 1;
        return true;
    }
    const int cap = fm == 1 ? 2 : 4;
    for (fn = 1; fn < cap && n / (32 * fn) >= 192; fn *= 2) {}
    return true;
}

int dual_max_t_slices(int64_t b, int64_t m, int64_t n, int r) {
    int fn, fm;
    if (r == 0 || !decode_shape(b, m, n, fn, fm) || fn * fm > 4) return 1;  // the epilogue reads T whole
    const int rs = r <= 32 ? 1 : r <= 64 ? 2 : r <= 128 ? 4 : 8;
    return kMaxTSlices / rs;
}

FoldLayout fold_layout(int64_t m, int64_t n, int64_t r) {
    auto al = [](size_t v) { return (v + 255) & ~size_t(255); };
    FoldLayout L{};
    L.ur = 0;
    L.vr = L.ur + al((size_t)(m * r) * 8);
    L.t1 = L.vr + al((size_t)(r * n) * 8);
    L.aug = L.t1 + al((size_t)(m * r) * 8);
    L.ginv = L.aug + al((size_t)(2 * r * r) * 8);
    L.total = L.ginv + al((size_t)(r * r) * 8);
    return L;
}

// ---- adapters and the input gradient ----

// K slices: enough CTAs to fill the 256 compute units twice (once with 128-row tiles, whose
// CTAs are twice as large), at least `least` stages of 128 each, at most 16 (the partial sums are
// read again). Half and twice as many CTAs: b=8192, 4096 -> 14336, 64 ranks, gradients 272 and
// 215 us against 210; b=4096, 4096 -> 4096, 32 ranks, 63 and 64 against 60. At most 8 instead of
// 16: one row, 14336 -> 4096, 64 ranks, 12.5 against 11.2 us; at most 32: 12.0.
// `least`: 4 for adapters (b=256, 4096 -> 4096: 2, 3, 4 and 8 stages took 11.9, 12.0, 10.3 and
// 12.4 us), 2 for the input gradient, whose slices also find the rows' maxima (b=512, 1024 x 4096,
// 64 ranks: 2, 4 and 8 stages 34, 37 and 44 us).
int shrink_slices(int64_t b, int64_t k, int64_t r, int64_t tiles, int64_t least) {
    const bool many = b > kManyRows;
    const int64_t rt = r <= 32 ? 1 : many ? (r + 127) / 128 : (r + 63) / 64, steps = (k + 127) / 128;
    int64_t ks = (many ? 256 : 512) / (tiles * rt);
    if (ks > steps / least) ks = steps / least;
    if (ks > 16) ks = 16;
    return ks < 1 ? 1 : (int)ks;
}

// Token rows a CTA, by the work in 128-row tiles x stages: small tiles fill the chip, large ones
// expand each code for more rows. With 32, 64 and 128 rows (us):
//   b=128,  512 x 512     17, 20, 27       b=256,  4096 x 14336  62, 58, 62
//   b=512,  1024 x 4096   34, 42, 43       b=2048, 1024 x 4096   57, 58, 62
//   b=64,   8192 x 28672  78, 85, 98       b=1024, 4096 x 14336  177, 153, 143
//   b=128,  8192 x 28672  118, 104, 112    b=4096, 8192 x 28672  2242, 1871, 1792
// Up to one 128-row tile a compute unit, two groups of waves share its channels (4096 x 4096, one
// group and two: b=2048 104 and 90 us; b=4096, 512 tiles, 155 and 170).
// Channel slices where the compute units are not full (two CTAs of one group each, or one of
// two), at least four stages each and at most 16 (b=16, 4096 x 14336: at most 4 and 16 took 47 and
// 29 us; at most 32, as 16); below 16 stages in all the joining launch costs more than the slices
// save.
DxPlan plan_dx(int64_t b, int64_t m, int64_t n, int64_t r) {
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    DxPlan p{};
    const int64_t mtiles = (m + kDxM - 1) / kDxM;
    p.npad = (n + kDxK - 1) / kDxK * kDxK;
    const int64_t stages = p.npad / kDxK, work = (b + 127) / 128 * mtiles * stages;
    p.bt = b <= 64 || work < 4096 ? 32 : b <= 128 || work < 8192 ? 64 : 128;
    const int64_t ctas = (b + p.bt - 1) / p.bt * mtiles;
    p.kg = p.bt == 128 && ctas <= 256 && stages >= 16 ? 2 : 1;
    int64_t ks = (p.kg == 2 ? 256 : 512) / ctas;
    if (ks > stages / 4 / p.kg) ks = stages < 16 ? 1 : stages / 4 / p.kg;
    if (ks > 16) ks = 16;
    p.ks = ks < 1 ? 1 : (int)ks;
    p.tks = r > 0 ? shrink_slices(b, n, r, (b + tile_rows(b) - 1) / tile_rows(b), 2) : 0;
    p.g = 0;
    p.ge = up((size_t)b * p.npad * 2);
    p.rowmax = p.ge + up((size_t)b * 8);
    p.t = p.rowmax + up((size_t)(r > 0 ? p.tks : 1) * b * 4);
    p.t16 = p.t + up((size_t)p.tks * b * r * 4);
    p.part = p.t16 + up((size_t)b * ((r + 31) / 32 * 32) * 4);
    p.total = p.part + (p.ks > 1 ? up((size_t)p.ks * b * m * 4) : 0);
    return p;
}

// ---- the layer with 16-bit activations ----

// Every CTA of the few-row kernels forms T for itself instead of reading what a launch before it left.
// With m r = 8192, 16384, 32768 and 65536 (m = n = 512, 1024, 2048, 2048; one token, fp16) 5.2, 6.1, 7.6
// and 10.2 us, with the launch 6.9, 7.3, 7.7 and 7.8; 16 tokens 5.9, 6.9, 9.8, 13.3 and 7.8, 8.6, 10.2,
// 10.0. A launch also costs the host 4 us.
static bool a16_own_t(int64_t b, int64_t m, int64_t r) { return b <= 16 && r <= kOwnRanks && m * r <= 32768; }

A16Plan plan_a16(int64_t b, int64_t m, int64_t n, int64_t r) {
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    A16Plan p{};
    const int64_t panels = n / 16, pieces = m / 128, blocks = (b + 63) / 64, plain = (panels + 7) / 8 * blocks;
    p.many = b > kFewTokens && plain > kFewTiles;
    // X L1 by the adapters' kernel, which reads L1 once for 64 or 128 rows: 2048 x 2048 -> 2048, 128 ranks 47.0 us,
    // a16_t_kernel 50.0; 4096 x 4096 -> 512, 64 ranks 48.9 and 69.3; with 65536 sums (2048 x 32, 4096 x 16) 34.8
    // and 34.2, 14.5 and 13.0; before the tile kernel 2048 x 4096 -> 4096, 32 ranks 90.4 and 93.5.
    p.shrink = p.many || b * r > 65536;
    if (r > 0 && p.shrink) p.tks = shrink_slices(b, m, r, (b + tile_rows(b) - 1) / tile_rows(b), 4);
    // T of few rows in slices of 1024: one token, 8192 -> 28672, 128 ranks 38.1 us; slices of 512, 2048 and
    // 4096: 41.7, 38.8, 40.6 (16 tokens, 4096 -> 4096, 32 ranks: 12.1; 11.3, 13.6, 17.1)
    if (r > 0 && !p.shrink && !a16_own_t(b, m, r)) p.tks = m >= 16384 ? 16 : (int)((m + 1023) / 1024);
    p.ks = 1;
    p.x16 = up((size_t)p.tks * b * r * 4);
    p.total = p.x16;
    if (!p.many) {
        p.rows = b <= 4 ? 4 : b <= 16 ? 16 : b <= 32 ? 32 : 64;
        if (p.rows <= 16) {
            // 5 to 16 rows: two panels a wave from 512 on (8192 channels). 4096 -> 8192: 9.7 us, one panel 9.9;
            // 4096 -> 14336: 11.7 and 15.4; 14336 -> 4096: 17.1 and 14.5; 8 rows 4096 -> 4096: 8.1 and 6.9.
            // Waves that share K: until there are 12 (6 of the 16-row kernel) a compute unit. One row,
            // 4096 -> 14336 with 1, 2, 4, 8: 14.1, 10.9, 10.0, 10.9; 8192 -> 28672 32.7, 28.0, 31.0 (1, 2, 4);
            // 14336 -> 4096 14.7, 10.8 (4, 8); 16 rows, 8192 -> 28672 56.5, 35.3, 36.0 (1, 2, 4).
            p.fn = p.rows == 4 || panels < 512 ? 1 : 2;
            const int64_t units = (panels + p.fn - 1) / p.fn;
            p.kw = 1;
            while (p.kw < 8 && units * p.kw < 256 * (p.rows == 4 ? 12 : 6) && pieces >= p.kw * 2) p.kw *= 2;
        } else {
            // Two panels a wave where one would give a compute unit more than one CTA and two do not: 768 x 4096 -> 4096
            // (384 CTAs, 192) 42.4 us, one panel 44.2; 200 x 4096 -> 14336 (448, 224) 41.7 and 46.4; 8000 x 4096 -> 512
            // (500, 250) 49 and 57; 12000 x 4096 -> 192 (376, 188) 46.9 and 50.1. With 256 CTAs or fewer of one panel:
            // 512 x 4096 -> 4096 (256) 29.3 and 25.4, 64 x 4096 -> 28672 (224) 34.5 and 27, 64 x 8192 -> 28672 50.8
            // and 50.2. With more than 256 of two, where waves of narrow layers own no second panel: 17000 x 4096 ->
            // 128 (266, 266) 88 and 53, 10000 x 4096 -> 272 (471, 314) 83 and 52, 10000 x 1024 -> 384 (471, 314) 28.2
            // and 18.9, 20000 x 2048 -> 16 (313, 313) 47 and 27.4.
            // Wave pairs that split K make CTAs of four panels, so that fewer K slices and no join fill the GPU.
            // More than 32 rows: 256 x 4096 -> 4096 (128 CTAs without) 17.9 us, without 21.8; 64 x 4096 -> 14336 (112)
            // 20.0 and 22.8; 512 x 4096 -> 4096 (256) 28.8 and 25.4, 128 x 4096 -> 14336 (224) 28.4 and 25.0;
            // longer rows of X: 61 x 14336 -> 4096 22.5 and 20.9, 128 x 14336 -> 4096 32.5 and 27.9.
            // 32 rows: 4096 -> 6144, 8192, 14336 11.3, 11.7, 13.4 and 11.5, 12.2, 15.8; 4096 -> 4096 9.1 and 9.0,
            // 14336 -> 4096 16.1 and 15.2, 4096 -> 22016 22.0 and 19.3.
            p.fn = p.rows == 64 && plain > 256 && (panels + 15) / 16 * blocks <= 256 ? 2 : 1;
            p.kw = p.rows == 32 ? panels >= 384 && panels <= 1024 ? 2 : 1 : p.fn == 1 && plain < 192 && m <= 8192 ? 2 : 1;
            const int64_t per = 8 / p.kw * p.fn, ctas = (panels + per - 1) / per * blocks;
            // K slices: as many as leave one CTA a compute unit. 61 rows, 14336 -> 4096 with 4, 8, 16 (rule: 8)
            // 28.7, 21.4, 25.1 us; 32 rows, 4096 -> 4096 with 4, 8 (8) 10.2, 9.8.
            int64_t ks = 256 / ctas;
            if (ks > pieces / 4) ks = pieces / 4;
            if (pieces < 16) ks = 1;  // 256 x 1024 -> 1024 with 1, 2: 7.4, 8.7
            p.ks = ks < 1 ? 1 : ks > 16 ? 16 : (int)ks;
        }
        p.part = p.x16;
        p.total = p.part + (p.ks > 1 ? up((size_t)p.ks * b * n * 4) : 0);
        return p;
    }
    const int64_t groups = m / 128, ntiles = (n + kA16N - 1) / kA16N;
    p.rows = 128;
    // Tiles of 64 rows while those of 128 give a compute unit at most 1.5 on average (two fit): 2048 x 4096 -> 4096
    // 83 and 100 us (256 tiles of 128), 1536 x 4096 -> 8192 124 and 127 (384); 1024 x 4096 -> 14336 141 and 137
    // (448), 2048 x 4096 -> 8192 152 and 140 (512).
    if ((b + 127) / 128 * ntiles <= 384) p.rows = 64;
    p.xe = p.x16 + up((size_t)b * m * 2);
    p.mul = p.xe + up((size_t)b * 4);
    p.mask = p.mul + up((size_t)groups * n * 4);
    p.small = p.mask + up((size_t)groups * n * 4);
    p.unit = p.small + up((size_t)n * 4);
    p.t16 = p.unit + up((size_t)n * 4);
    p.twide = p.t16 + up((size_t)b * r * 4);
    p.te = p.twide + up((size_t)b * r * 4);
    p.total = p.te + up((size_t)b * 4);
    return p;
}

RoutePlan plan_route(int64_t b, int64_t m, int64_t experts) {
    RoutePlan p{};
    p.slices = 1;
    // Tokens, experts, m: 128, 128, 4096 13.7 us tiled, 19.2 else; 64, 256, 4096 14.7 and 20.3; 32, 512, 4096
    // 16.3 and 21.2; 256, 256, 7168 29 and 75; below: 64, 128, 2048 12.6 and 12.1, 32, 256, 7168 18.6 and 17.2.
    p.tiled = b * experts >= 16384;
    if (p.tiled) {
        const int64_t tiles = (experts + 31) / 32 * ((b + 31) / 32);
        // at most one tile a compute unit: 256, 64, 4096 with 2, 4, 8 (rule: 8) 25.4, 17.2, 13.2; 256, 256, 7168 (4)
        // 39.6, 28.6, 31.4; 72, 512, 4096 (4) 28.4, 20.5, 23.4; and 512 elements a slice: 256, 64, 2048 (4) 16.9,
        // 12.5, 13.2
        while (p.slices < 8 && tiles * p.slices * 2 <= 256 && m / 512 >= p.slices * 2) p.slices *= 2;
    }
    p.total = ((size_t)(p.slices * b * experts) * 8 + 255) & ~size_t(255);
    return p;
}

MoePlan plan_moe(int64_t b, int64_t m, int64_t f, int64_t experts, int64_t k) {
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    MoePlan p{};
    const int64_t pairs = b * k, slots = pairs < experts ? pairs : experts;
    // Layers below: A 8 of 64 experts, 2048 -> 768, bf16; B 2 of 8, 4096 -> 14336, fp16; C 4 of 60, 2048 -> 1408, bf16;
    // D 8 of 128, 4096 -> 1408, fp16; us of a whole call, the router's launches among them.
    // The down kernel that sums a token's outputs itself against the shared one with its join: 1 token A 23.0 and 26.0,
    // B 57 and 63; 2 tokens A 29.0 and 30.1, B 91 and 102; 4 tokens B 124 and 155, D 78 and 80, but A 39.2 and 37.5,
    // C 37.7 and 36.7. Its list holds four.
    p.few = b <= kFewMoe;
    p.slots = (int)slots;
    // CTAs that share an expert's rows from 4 rows an expert on average. Shared, and waves with rows of their own: 256
    // tokens A (32 rows an expert) 121 and 155, B (64) 557 and 859; 64 B (16) 216 and 292; 128 C (8) 99 and 111, D
    // (8) 284 and 307; 6 rows A (48) 65 and 63, C (90) 94 and 96, D (96) 283 and 288; 4 rows A (32) 62.5 and 61, C
    // (60) 88.5 and 84.5, D (64) 263 and 280, B (16) 195 and 192; 2 rows D (32) 229 and 220, 1 row C (13)
    // 59.4 and 58.8. And where there are CTAs of 128 inner channels for the compute units: waves that split K
    // fill the GPU with fewer (256 tokens, 2 of 8 experts of 2048 -> 768: 75 and 65; 2 of 4 of 4096 -> 2048: 192 and
    // 141). Short K loses by that: 200 tokens, 8 of 10 of 1024 -> 768 105 and 116; 256, 4 of 16 of 512 -> 256 45 and 57.
    p.up_shared = !p.few && pairs >= experts * 4 && f / 128 * slots >= 256;
    // Waves that share K, 1, 2, 4, 8: one token A 29.6, 25.1, 22.7, 23.0 (rule: 4), C 28.7, 24.0, 21.6, 22.0 (4), B 56, 56,
    // 56, 59 (4), D 41, 34, 35, 34.5 (8); 4 tokens A 38, 39, 39, 42.5 (4); 8 tokens B 169, 163, 162, 182 (1), 2 of 4 of
    // 4096 -> 2048, bf16 47.6, 36.3, 31, 31.4 (8); 13 tokens C 57.7, 58.9, 61, 69.5 (2).
    p.up_waves = 1;
    while (p.up_waves < 8 && f / 16 * slots * p.up_waves < 5000 && m / 128 >= p.up_waves * 8) p.up_waves *= 2;
    // Rows of a down tile, 16 or 32: 8 rows an expert A (64) 68 and 70.6, B (32) 196 and 211, D (128) 282-325 and
    // 310-337, C (120) 101 and 99.6; 10 A (80) 73.5 and 73.2, B (40) 197 and 216; 12 A (96) 77 and 74, B (48) 262 and 216,
    // D (192) 303-330 and 321-335, C (180) 111 and 109; 32 A (256) 131 and 122.
    p.down_rows = pairs >= experts * 12 ? 32 : 16;
    p.ks = 1;
    if (!p.few)
        while (p.ks < 8 && m / 128 * slots * p.ks < 256 && f / 128 >= p.ks * 8) p.ks *= 2;
    p.h = 0;
    p.part = up((size_t)(pairs * f) * 4);
    p.entries = p.part;
    p.experts = !p.few ? p.part + up((size_t)(p.ks * pairs * m) * 4) : p.entries + up((size_t)pairs * sizeof(MoeEntry) + 16);
    p.logits = p.experts;
    p.ids = p.logits + plan_route(b, m, experts).total;
    p.weights = p.ids + up((size_t)pairs * 4);
    p.total = p.weights + up((size_t)pairs * 4);
    return p;
}

}  // namespace twq
