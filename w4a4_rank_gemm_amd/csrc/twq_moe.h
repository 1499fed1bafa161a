// twq_moe.h -- launch interface of the layer with 16-bit activations and of the routed layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace twq {

// ---- the layer with 16-bit activations ------------------------------------------------------

// With few rows the product is bound by the weights' read (a few-row kernel); above by the
// matrix cores (a tile kernel, which wants X in fp16 in the order of the expanded codes, and
// the scales as ratios of neighbouring groups). More rows take the few-row kernel too, in blocks of 64, while
// blocks of 64 rows x 128 channels are at most kFewTiles, two a compute unit. Few-row and tile
// kernel: 256 x 4096 -> 14336 (448) 40.6 and 53.7 us, 1024 x 4096 -> 4096 (512) 42.3 and 56.6, 2048 x 2048 -> 2048
// (512) 33 and 43, 128 x 8192 -> 28672 (448) 77 and 133; 384 x 4096 -> 14336 (672) 74 and 73, 160 x 8192 -> 28672
// (672) 142 and 138, 100 x 1024 -> 131072 (2048) 66 and 58.
constexpr int64_t kFewTokens = 64, kFewTiles = 512;
constexpr int kOwnRanks = 128;  // of X L1 that a few-row CTA may form for itself
constexpr int kA16N = 256;  // channels of a tile CTA: 64 a wave

struct A16Args {
    const uint16_t *x;    // [b][m]
    const uint8_t *qw;    // panels
    const float *sw;      // [m / 128][n]
    const uint16_t *l1t;  // [r][m] fp16
    const uint16_t *l2t;  // [n][r] fp16
    float *t;             // [tks][b][r] partial sums of X L1
    int tks;
    uint16_t *y;          // [b][n]
    int64_t b, m, n;
    int r;
    int bf16;             // type of x and y
    // tile kernel
    uint16_t *x16;        // [b][m] fp16: X 2^-xe, eight elements in the order 0 4 1 5 2 6 3 7
    int32_t *xe;          // [b] (bf16)
    float *mul;           // [m / 128][n]: unit of the group before over this group's
    uint32_t *mask;       // [m / 128][n]: all ones, or 0 for a group with little or no weight
    uint32_t *small;      // [n]: 1 where a group with weight is masked
    float *unit;          // [n]: unit of the last group
    uint16_t *t16;        // [b][r / 8][2][8]: X L1 2^-(te / 2) in two fp16 parts; zeros where te is odd
    uint16_t *twide;      // the same of X L1 in two bf16 parts, in rows where te is odd
    int32_t *te;          // [b]
    // few rows
    int ks;               // slices of K
    float *part;          // [ks][b][n] when ks > 1
};

struct A16Plan {
    int many;      // the tile kernel
    int shrink;    // X L1 by the adapters' kernel
    int rows;      // token rows a CTA
    int fn, kw;    // few rows: panels of a wave, and neighbouring waves that share their K
    int tks;       // K slices of X L1, 0: formed by the product's CTAs (or r = 0)
    int ks;        // K slices of the product
    size_t t, x16, xe, mul, mask, small, unit, t16, twide, te, part, total;
};
A16Plan plan_a16(int64_t b, int64_t m, int64_t n, int64_t r);  // plan.cpp
hipError_t launch_a16_t(const A16Args &a, hipStream_t stream);  // t, with few sums
hipError_t launch_a16(const A16Args &a, const A16Plan &p, hipStream_t stream);

// ---- the routed layer ------------------------------------------------------------------------

constexpr int64_t kMaxMoeTokens = 256, kMaxExperts = 512, kMaxTopK = 16;

struct RouteArgs {
    const uint16_t *x;    // [b][m]
    const uint16_t *wr;   // [experts][m]
    const float *bias;    // [experts] or NULL
    int64_t b, m;
    int experts, k;
    int bf16;
    int sigmoid;          // scores: sigmoid (1) or softmax (0) of the logits
    int norm;             // weights divided by their sum
    float scale;
    int tiled;            // logits on matrix instructions
    int slices;           // K slices of the logits
    double *logits;       // [slices][b][experts]
    int32_t *ids;         // [b][k]
    float *weights;       // [b][k]
};
struct RoutePlan {
    int tiled, slices;
    size_t total;  // logits
};
RoutePlan plan_route(int64_t b, int64_t m, int64_t experts);  // plan.cpp
hipError_t launch_route(const RouteArgs &a, hipStream_t stream);

// Tokens whose outputs the down kernel sums by itself, from a work list of at most kFewPairs entries.
constexpr int kFewMoe = 4, kFewPairs = kFewMoe * (int)kMaxTopK;
struct alignas(16) MoeEntry {
    int32_t expert, rows;     // rows: its pairs (token, choice), in order
    int16_t pair[kFewMoe];
    int8_t place[kFewMoe];    // of each token: which of the pairs is its own, or -1
};
static_assert(sizeof(MoeEntry) == 32, "read in 16-byte pieces");

struct MoeArgs {
    const uint16_t *x;    // [b][m]
    const int32_t *ids;   // [b][k], outside [0, experts): none
    const float *weights; // [b][k]
    const uint8_t *q1;    // [experts] panels of 2 f channels: f gate, f up
    const float *s1;      // [m / 128][experts 2 f]
    const uint8_t *q2;    // [experts] panels of m channels
    const float *s2;      // [f / 128][experts m]
    int64_t b, m, f;
    int experts, k;
    int bf16;             // type of x and y
    uint16_t *h;          // [b k][f / 128][2][128] bf16: the experts' inner rows, upper and lower parts
    int ks;               // K slices of the down product above kFewMoe tokens
    float *part;          // [ks][b k][m]: weighted outputs of each token's choices, above kFewMoe tokens
    MoeEntry *entries;    // [b k], up to kFewMoe tokens
    int32_t *entry_count;
    uint16_t *y;          // [b][m]
};

struct MoePlan {
    int few;         // the down kernel sums a token's outputs by itself
    int slots;       // rows of CTAs: pairs (token, choice) or experts
    int up_shared;   // gate and up: a CTA's waves share rows and K
    int up_waves;    // or: waves that share a panel's K
    int down_rows;   // above kFewMoe tokens: rows of a tile
    int ks;
    size_t h, part, entries, experts;    // workspace of the experts' products, its size
    size_t logits, ids, weights, total;  // of the whole layer, behind it
};
MoePlan plan_moe(int64_t b, int64_t m, int64_t f, int64_t experts, int64_t k);  // plan.cpp
hipError_t launch_moe(const MoeArgs &a, const MoePlan &p, hipStream_t stream);

}  // namespace twq
