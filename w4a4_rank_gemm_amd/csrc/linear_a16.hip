// linear_a16.hip -- the packed layer with unquantized 16-bit activations (gfx950).
//
//   y[i][j] = sum_G s_W[G][j] sum_{k in G} x[i][k] q[j][k] + sum_t (sum_k x[i][k] L1[k][t]) L2[t][j]
//
// G: groups of 128 input channels. X is fp16 or bf16 and used as it is; codes are exact in both
// types, so the only roundings are those of the binary32 sums, of T = X L1 to 16 or more bits and
// the output's. T comes in partial sums over K slices from a launch of its own (with few sums
// a16_t_kernel, otherwise the adapters' shrink kernel), or from the product's own CTAs where L1 is small.
#include "twq_few_device.h"
#include "twq_moe.h"

namespace twq {

constexpr int kFewWaves = 8;
constexpr int kTWaves = 16, kTSteps = 4;

// One wave's part of T = X L1 for 16 rows and 16 ranks: K steps s0 .. s1 - 1 of 32, a few steps'
// loads in flight. A fp16 L1 meets bf16 rows as two exact bf16 parts. Result: lane (li, g)
// holds row li, ranks 4 g .. 4 g + 3.
template <class T>
__device__ __forceinline__ v4f t_part(const A16Args &a, int64_t rank0, int64_t row0, int s0, int s1) {
    const int lane = threadIdx.x % kWave, li = lane & 15, g = lane >> 4;
    const int64_t row = row0 + li;
    const uint16_t *w = a.l1t + (rank0 + li) * a.m + g * 8, *x = a.x + (row < a.b ? row : a.b - 1) * a.m + g * 8;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    for (int s = s0; s < s1; s += kTSteps) {
        v4i wv[kTSteps], xv[kTSteps];
#pragma unroll
        for (int u = 0; u < kTSteps; ++u) {
            const int q = s + u < s1 ? s + u : s1 - 1;
            wv[u] = load16(w + q * 32);
            xv[u] = load16(x + q * 32);
        }
#pragma unroll
        for (int u = 0; u < kTSteps; ++u) {
            if (s + u >= s1) break;
            if constexpr (T::kBf16) {
                v4i hi, lo;
                split_f16(wv[u], hi, lo);
                acc = T::mfma(lo, xv[u], acc);
                acc = T::mfma(hi, xv[u], acc);
            } else {
                acc = T::mfma(wv[u], xv[u], acc);
            }
        }
    }
    return acc;
}

// T in a launch of its own, with few sums: a CTA owns 16 rows x 16 ranks over a slice of K, which
// its 16 waves split; their sums are added in wave order. Bound by its start and one round of loads:
// 4.8 us for one token of 8192 with 128 ranks and for 16 of 4096 with 32.
template <class T>
__global__ __launch_bounds__(kTWaves *kWave) void a16_t_kernel(A16Args a) {
    __shared__ v4f red[kTWaves][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, li = lane & 15, g = lane >> 4;
    const int64_t rank0 = (int64_t)blockIdx.x * 16, row0 = (int64_t)blockIdx.y * 16, slice = blockIdx.z;
    const int steps = (int)(a.m / 32), parts = a.tks * kTWaves, part = (int)slice * kTWaves + wave;
    v4f acc = t_part<T>(a, rank0, row0, (int)((int64_t)part * steps / parts), (int)((int64_t)(part + 1) * steps / parts));
    red[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int q = 1; q < kTWaves; ++q) {
        const v4f o = red[q][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += o[e];
    }
    if (row0 + li < a.b) *reinterpret_cast<v4f *>(a.t + (slice * a.b + row0 + li) * a.r + rank0 + g * 4) = acc;
}

hipError_t launch_a16_t(const A16Args &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.r / 16), (unsigned)((a.b + 15) / 16), (unsigned)a.tks);
    if (a.bf16)
        a16_t_kernel<BF16><<<grid, kTWaves * kWave, 0, stream>>>(a);
    else
        a16_t_kernel<F16><<<grid, kTWaves * kWave, 0, stream>>>(a);
    return hipGetLastError();
}

// Partial sums of T: [slices][rows][r].
struct TSums {
    const float *t;
    int64_t stride;  // rows r
    int slices;
};

// Eight ranks k .. k + 7 of row `row` of T, summed over its slices in order, as two bf16 parts
// (16 significant bits); zeros past the last rank.
__device__ __forceinline__ void few_t(const TSums &ts, int r, int64_t row, int k, v4i &hi, v4i &lo) {
    const float *p = ts.t + row * r + (k < r ? k : 0);
    const v4f t[2] = {sum_slices(p, ts.stride, ts.slices), sum_slices(p + 4, ts.stride, ts.slices)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float v0 = k < r ? t[e / 2][e % 2 * 2] : 0.f, v1 = k < r ? t[e / 2][e % 2 * 2 + 1] : 0.f;
        const uint16_t h0 = BF16::from_f32(v0), h1 = BF16::from_f32(v1);
        const uint16_t l0 = BF16::from_f32(v0 - BF16::to_f32(h0)), l1 = BF16::from_f32(v1 - BF16::to_f32(h1));
        hi[e] = (int)((uint32_t)h0 | (uint32_t)h1 << 16);
        lo[e] = (int)((uint32_t)l0 | (uint32_t)l1 << 16);
    }
}

// acc += T L2 for 16 FM rows and FN panels, a wave's blocks of 32 ranks share, share + shares, .. L2
// is taken as its two exact bf16 parts: the four products are T L2 up to 2^-18 of T. `rank8` gives
// eight ranks of a row (few_t, or what stage_t left).
template <int FN, int FM, class F>
__device__ __forceinline__ void few_lowrank(const A16Args &a, F &&rank8, const int64_t (&chan)[FN], int share, int shares,
                                            v4f (&acc)[FN][FM]) {
    const int lane = threadIdx.x % kWave, li = lane & 15, g = lane >> 4;
    for (int rb = share; rb * 32 < a.r; rb += shares) {
        const int k = rb * 32 + g * 8, kc = k < a.r ? k : a.r - 8;
        v4i wh[FN], wl[FN];
#pragma unroll
        for (int f = 0; f < FN; ++f) split_f16(load16(a.l2t + (chan[f] + li) * a.r + kc), wh[f], wl[f]);
#pragma unroll
        for (int c = 0; c < FM; ++c) {
            v4i th, tl;
            rank8(c * 16 + li, k, th, tl);
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                acc[f][c] = BF16::mfma(wl[f], tl, acc[f][c]);
                acc[f][c] = BF16::mfma(wl[f], th, acc[f][c]);
                acc[f][c] = BF16::mfma(wh[f], tl, acc[f][c]);
                acc[f][c] = BF16::mfma(wh[f], th, acc[f][c]);
            }
        }
    }
}

// T's parts of the R rows from row0 on to LDS, [r / 8][R rows][hi, lo], by the whole CTA: each of its waves would
// otherwise read T's slices again (64 tokens, fp16: 4096 -> 14336, 64 ranks 38.5 us, this way 27.5; 8192 -> 28672,
// 128 ranks 111 and 64).
template <int R>
__device__ __forceinline__ void stage_t(const A16Args &a, int64_t row0, uint8_t *lds) {
    __syncthreads();
    const int eights = a.r / 8, rows = (int)(a.b - row0 < R ? a.b - row0 : R);
    for (int i = threadIdx.x; i < rows * eights; i += kFewWaves * kWave) {
        const int row = i / eights, k8 = i % eights;
        v4i hi, lo;
        few_t({a.t, a.b * a.r, a.tks}, a.r, row0 + row, k8 * 8, hi, lo);
        *reinterpret_cast<v4i *>(lds + (k8 * R + row) * 32) = hi;
        *reinterpret_cast<v4i *>(lds + (k8 * R + row) * 32 + 16) = lo;
    }
    __syncthreads();
}
template <int R>
__device__ __forceinline__ void staged_t(const uint8_t *lds, int r, int row, int k, v4i &hi, v4i &lo) {
    const uint8_t *p = lds + ((k < r ? k : r - 8) / 8 * R + row) * 32;
    const v4i zero = {0, 0, 0, 0};
    hi = k < r ? load16(p) : zero;
    lo = k < r ? load16(p + 16) : zero;
}

// T of at most 16 rows and kOwnRanks ranks by the CTA's eight waves: a wave takes 16 ranks and a share
// of K, its sums go to t [slices][b][r].
template <class T>
__device__ __forceinline__ TSums own_t(const A16Args &a, float *t, int wave) {
    const int blocks = a.r / 16, lane = threadIdx.x % kWave, li = lane & 15, g = lane >> 4;
    const int slices = blocks > 4 ? 1 : blocks > 2 ? 2 : blocks > 1 ? 4 : 8, per = kFewWaves / slices;
    const int block = wave & (per - 1), slice = wave / per, steps = (int)(a.m / 32);
    if (block < blocks) {
        const v4f s = t_part<T>(a, block * 16, 0, slice * steps / slices, (slice + 1) * steps / slices);
        if (li < a.b) *reinterpret_cast<v4f *>(t + (slice * a.b + li) * a.r + block * 16 + g * 4) = s;
    }
    return {t, a.b * a.r, slices};
}

// Stores the row blocks c = share, share + shares, .. of FN panels: Y, or this slice's sums.
template <class T, int FN, int FM>
__device__ __forceinline__ void a16_store(const A16Args &a, const v4f (&acc)[FN][FM], int64_t row0, int64_t panel0, int64_t slice,
                                          int shares, int share) {
    const int64_t panels = a.n / 16;
    const int lane = threadIdx.x % kWave, li = lane & 15, g = lane >> 4;
#pragma unroll
    for (int c = 0; c < FM; ++c) {
        const int64_t row = row0 + c * 16 + li;
        if (c % shares != share || row >= a.b) continue;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            if (panel0 + f >= panels) continue;
            const int64_t at = row * a.n + (panel0 + f) * 16 + g * 4;
            const v4f s = acc[f][c];
            if (a.ks > 1)
                *reinterpret_cast<v4f *>(a.part + slice * a.b * a.n + at) = s;
            else
                *reinterpret_cast<uint2 *>(a.y + at) = make_uint2((uint32_t)T::from_f32(s[0]) | (uint32_t)T::from_f32(s[1]) << 16,
                                                                  (uint32_t)T::from_f32(s[2]) | (uint32_t)T::from_f32(s[3]) << 16);
        }
    }
}

// Up to 16 rows: groups of kw waves (a power of two) own FN panels of 16 channels each and split their
// K; the waves' sums are added in wave order. Bound by the weights' read: 1 x 8192 -> 28672, 128 ranks
// (132 MB) 35-38 us, 3.6 TB/s; 16 x 4096 -> 4096, 32 ranks (11 MB) 8.0 us, start and drain.
template <class T, int FN, int XR, int U>
__global__ __launch_bounds__(kFewWaves *kWave) void a16_few_kernel(A16Args a, int kw) {
    typedef FewRows<T, FN, XR, 1, U> Rows;
    static_assert(Rows::FM == 1 && kFewWaves * Rows::LDS >= XR * 4 * 256, "T's parts of 256 ranks");
    __shared__ __align__(16) uint8_t smem[kFewWaves * Rows::LDS];
    __shared__ __align__(16) float tsums[XR * kOwnRanks];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), share = wave & (kw - 1);
    const int64_t panels = a.n / 16, pieces = a.m / 128, panel0 = ((int64_t)blockIdx.x * kFewWaves + wave) / kw * FN;
    Rows rows;
    int64_t chan[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f) {
        const int64_t p = panel0 + f < panels ? panel0 + f : panels - 1;
        chan[f] = p * 16;
        rows.w[f] = a.qw + p * pieces * 1024;
        rows.s[f] = a.sw + p * 16;
    }
    rows.s_stride = a.n;
    rows.x = a.x;
#pragma unroll
    for (int j = 0; j < Rows::XL; ++j) {
        const int row = 4 * j + lane / 16;
        rows.row[j] = (uint32_t)((row < a.b ? row : a.b - 1) * a.m * 2);
    }
    v4f acc[FN][1] = {};
    const bool own = a.r > 0 && a.tks == 0;
    TSums ts = {a.t, a.b * a.r, a.tks};
    auto rank8 = [&](int row, int k, v4i &hi, v4i &lo) { few_t(ts, a.r, row < a.b ? row : a.b - 1, k, hi, lo); };
    auto between = [&] {
        if (own) ts = own_t<T>(a, tsums, wave);
        if (XR == 4 && a.r > 0 && !own) few_lowrank<FN, 1>(a, rank8, chan, share, kw, acc);
    };
    if (panel0 < panels)
        rows.run((int)(share * pieces / kw), (int)((share + 1) * pieces / kw), smem + wave * Rows::LDS, acc, between);
    else if (own)
        own_t<T>(a, tsums, wave);
    if (own) {
        __syncthreads();
        if (panel0 < panels) few_lowrank<FN, 1>(a, rank8, chan, share, kw, acc);
    } else if (XR > 4 && a.r > 0) {
        stage_t<16>(a, 0, smem);
        auto staged = [&](int row, int k, v4i &hi, v4i &lo) { staged_t<16>(smem, a.r, row, k, hi, lo); };
        if (panel0 < panels) few_lowrank<FN, 1>(a, staged, chan, share, kw, acc);
    }
    join_waves(smem, kw, wave, acc);
    a16_store<T, FN, 1>(a, acc, 0, panel0, 0, kw, share);
}

// From 17 rows on, in blocks of XR: the CTA's eight waves, in groups of KG, own FN panels each and share
// the rows and a slice of K. 32 x 8192 -> 28672 37 us (3.3 TB/s of weights), 64 rows 50, 128 rows 77,
// 1024 x 4096 -> 4096 46-48 (0.75 PFLOP/s). Bound by the steps themselves, which turn rows through LDS, expand
// codes and feed chains of matrix instructions with two waves a SIMD: with rows and codes that come from a
// cache, 61 x 14336 -> 4096 took 18.0 us instead of 18.8, 32 x 4096 -> 14336 10.9 of 12.6, 512 x 4096 -> 4096 24.1 of
// 26.1, 128 x 8192 -> 28672 74 of 79 (matrix cores busy 23%, LDS in use for 31% of the cycles in the first; reading
// row operands for two panels at once, or two steps ahead, gained nothing). Joining eight slices of the first
// takes 4.7 us.
template <class T, int FN, int XR, int U, int KG>
__global__ __launch_bounds__(kSharedWaves *kWave) void a16_shared_kernel(A16Args a) {
    typedef SharedRows<T, FN, XR, 1, U, KG> Rows;
    constexpr int FM = Rows::FM;
    static_assert(Rows::LDS >= XR * 4 * 256, "T's parts of 256 ranks");
    static_assert(KG == 1 || Rows::LDS >= kSharedWaves * FN * FM * 1024, "sums of wave pairs");
    static_assert(kSharedWaves == kFewWaves, "stage_t's threads");
    __shared__ __align__(16) uint8_t smem[Rows::LDS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t panels = a.n / 16, pieces = a.m / 128, slice = blockIdx.y;
    // Row blocks of the same panels are neighbours on an XCD and share their weights' read in its L2 (128 x 8192 ->
    // 28672 95 us one block after the other, 77 so).
    const uint32_t id = (uint32_t)xcd_range(blockIdx.x, gridDim.x), blocks = (uint32_t)((a.b + XR - 1) / XR);
    const int64_t row0 = (int64_t)(id % blocks) * XR;
    const int64_t panel0 = ((int64_t)(id / blocks) * (kSharedWaves / KG) + wave / KG) * FN;
    Rows rows;
    int64_t chan[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f) {
        const int64_t p = panel0 + f < panels ? panel0 + f : panels - 1;
        chan[f] = p * 16;
        rows.w[f] = a.qw + p * pieces * 1024;
        rows.s[f] = a.sw + p * 16;
    }
    rows.s_stride = a.n;
    rows.x = a.x + row0 * a.m;
#pragma unroll
    for (int j = 0; j < Rows::PER; ++j) {
        const int64_t row = Rows::row_of(j);
        rows.row[j] = (uint32_t)((row < a.b - row0 ? row : a.b - row0 - 1) * a.m * 2);
    }
    v4f acc[FN][FM] = {};
    rows.run((int)(slice * pieces / a.ks), (int)((slice + 1) * pieces / a.ks), smem, acc);
    if (a.r > 0 && slice == 0) {
        stage_t<XR>(a, row0, smem);
        auto staged = [&](int row, int k, v4i &hi, v4i &lo) { staged_t<XR>(smem, a.r, row, k, hi, lo); };
        few_lowrank<FN, FM>(a, staged, chan, wave % KG, KG, acc);
    }
    join_waves(smem, KG, wave, acc);
    a16_store<T, FN, FM>(a, acc, row0, panel0, slice, KG, wave % KG);
}

// Y = the slices' sums in slice order, rounded once.
template <class T>
__global__ __launch_bounds__(256) void a16_join_kernel(const float *part, int ks, int64_t total, uint16_t *y) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= total) return;
    const v4f s = sum_slices(part + at, total, ks);
    *reinterpret_cast<uint2 *>(y + at) = make_uint2((uint32_t)T::from_f32(s[0]) | (uint32_t)T::from_f32(s[1]) << 16,
                                                    (uint32_t)T::from_f32(s[2]) | (uint32_t)T::from_f32(s[3]) << 16);
}

template <class T>
static hipError_t a16_join(const A16Args &a, hipStream_t stream) {
    const int64_t total = a.b * a.n;
    a16_join_kernel<T><<<dim3((unsigned)((total / 4 + 255) / 256)), 256, 0, stream>>>(a.part, a.ks, total, a.y);
    return hipGetLastError();
}

template <class T, int FN, int XR, int U>
static hipError_t a16_few(const A16Args &a, const A16Plan &p, hipStream_t stream) {
    const int64_t groups = (a.n / 16 + FN - 1) / FN, per = kFewWaves / p.kw;
    a16_few_kernel<T, FN, XR, U><<<dim3((unsigned)((groups + per - 1) / per)), kFewWaves * kWave, 0, stream>>>(a, p.kw);
    return hipGetLastError();
}

template <class T, int FN, int XR, int U, int KG>
static hipError_t a16_shared(const A16Args &a, hipStream_t stream) {
    const int64_t groups = (a.n / 16 + FN - 1) / FN, per = kSharedWaves / KG;
    const dim3 grid((unsigned)((groups + per - 1) / per * ((a.b + XR - 1) / XR)), (unsigned)a.ks);
    a16_shared_kernel<T, FN, XR, U, KG><<<grid, kSharedWaves * kWave, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || a.ks == 1 ? e : a16_join<T>(a, stream);
}

template <class T>
static hipError_t a16_rows(const A16Args &a, const A16Plan &p, hipStream_t stream) {
    if (p.rows == 4) return a16_few<T, 1, 4, 2>(a, p, stream);
    if (p.rows == 16) return p.fn == 1 ? a16_few<T, 1, 16, 1>(a, p, stream) : a16_few<T, 2, 16, 1>(a, p, stream);
    if (p.rows == 32) return p.kw == 1 ? a16_shared<T, 1, 32, 2, 1>(a, stream) : a16_shared<T, 1, 32, 4, 2>(a, stream);
    if (p.fn == 2) return a16_shared<T, 2, 64, 2, 1>(a, stream);
    return p.kw == 1 ? a16_shared<T, 1, 64, 2, 1>(a, stream) : a16_shared<T, 1, 64, 2, 2>(a, stream);
}

// ---- many rows ---------------------------------------------------------------------------

__device__ __forceinline__ v16f mfma_bf16_32(v4i a, v4i b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// What the tile kernel reads: X in fp16, the scales as ratios, T in two parts. One pass over each,
// bound by memory: 4001 x 8192 (bf16, 28672 channels, 128 ranks) 46.5 us, 2048 x 4096 (fp16, 14336, 32) 11 us.
//
// The tile kernel multiplies its sums by mul[G] = unit[G - 1] / unit[G] before group G, so that
// they are in units of the group's scale when its products (codes times X) are added: one
// multiplication a sum and group, no second set of sums. unit[G] is s_W[G]; where that is below
// 2^-90 of the channel's largest (zero among it) the group's codes are masked and the unit is the
// largest. Sums then stay below 7 2^17 2^16 2^90 < 2^126. A masked group with weight marks its channel in
// `small`: its products are added after the main loop, since X may be zero where the scales are large.
constexpr int kPrepRows = 4, kPrepChannels = 32;

template <class T>
__device__ __forceinline__ void prepare_row(const A16Args &a, int64_t row) {
    const int lane = threadIdx.x % kWave;
    const uint16_t *x = a.x + row * a.m;
    uint16_t *out = a.x16 + row * a.m;
    float f = 1.f;
    if constexpr (T::kBf16) {  // to a largest element in [2^14, 2^15): exact down to 2^-28 of it, off by 2^-39 of it below
        uint32_t mx = 0;
        for (int64_t k = lane * 8; k < a.m; k += kWave * 8) {
            const v4i v = load16(x + k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = (uint32_t)v[e] << 16 & 0x7FFFFFFFu, hi = (uint32_t)v[e] & 0x7FFF0000u;
                mx = mx > lo ? mx : lo;
                mx = mx > hi ? mx : hi;
            }
        }
        const int e = scale_exponent(__builtin_bit_cast(float, wave_max_u32(mx)));
        f = pow2(14 - e);
        if (lane == 0) a.xe[row] = e - 14;
    }
    for (int64_t k = lane * 8; k < a.m; k += kWave * 8) {
        v4i v = load16(x + k);
        if constexpr (T::kBf16) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = (int)((uint32_t)F16::from_f32(T::to_f32(half_of(v[e], 0)) * f) |
                             (uint32_t)F16::from_f32(T::to_f32(half_of(v[e], 1)) * f) << 16);
        }
        *reinterpret_cast<v4i *>(out + k) = Codes<F16>::order(v);
    }
}

__device__ __forceinline__ void prepare_scales(const A16Args &a, int64_t block, float *red) {
    const int groups = (int)(a.m / 128), gl = threadIdx.x / kPrepChannels;
    const int64_t c = block * kPrepChannels + threadIdx.x % kPrepChannels, cc = c < a.n ? c : a.n - 1;
    float top = 0.f;
    for (int g = gl; g < groups; g += 256 / kPrepChannels) top = __builtin_fmaxf(top, __builtin_fabsf(a.sw[g * a.n + cc]));
    red[threadIdx.x] = top;
    __syncthreads();
    for (int q = 0; q < 256 / kPrepChannels; ++q) top = __builtin_fmaxf(top, red[q * kPrepChannels + threadIdx.x % kPrepChannels]);
    const float least = top * 0x1p-90f;
    bool small = false;
    auto on = [&](float s) { return s != 0.f && !(__builtin_fabsf(s) < least); };
    auto unit = [&](float s) { return on(s) ? s : top == 0.f ? 1.f : top; };
    for (int g = gl; c < a.n && g < groups; g += 256 / kPrepChannels) {
        const float s = a.sw[g * a.n + c], before = a.sw[(g > 0 ? g - 1 : 0) * a.n + c];
        a.mul[g * a.n + c] = unit(before) / unit(s);
        a.mask[g * a.n + c] = on(s) ? 0xFFFFFFFFu : 0u;
        if (s != 0.f && !on(s)) {  // codes of zeros (pruned, under a least scale) need no adding
            const uint8_t *const w = a.qw + (c / 16 * groups + g) * 1024 + c % 16 * 64;
            v4i any = load16(w);
#pragma unroll
            for (int e = 1; e < 4; ++e) any |= load16(w + e * 16);
            small |= (any[0] | any[1] | any[2] | any[3]) != 0;
        }
        if (g + 1 == groups) a.unit[c] = unit(s);
    }
    __syncthreads();
    red[threadIdx.x] = small ? 1.f : 0.f;
    __syncthreads();
    if (gl > 0 || c >= a.n) return;
    for (int q = 1; q < 256 / kPrepChannels; ++q) small |= red[q * kPrepChannels + threadIdx.x] != 0.f;
    a.small[c] = small;
}

// 16 rows, 16 threads a row: T summed over its slices in order, under a power of two a row, in two
// fp16 parts (22 significant bits of elements within 2^-17 of the row's largest, 16 within 2^-22). A row with smaller
// elements is left as it is, in two bf16 parts (16 significant bits of all of them) in an array of its
// own and zeros in the other's place. te: exponent times two, plus one for such a row.
__device__ __forceinline__ void prepare_t(const A16Args &a, int64_t block) {
    const int q = threadIdx.x % 16;
    const int64_t row = block * 16 + threadIdx.x / 16, rc = row < a.b ? row : a.b - 1;
    float t[16], mx = 0.f;  // ranks q, q + 16, ..
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        t[u] = 0.f;
        if (u * 16 >= a.r) continue;
        for (int s = 0; s < a.tks; ++s) t[u] += a.t[(s * a.b + rc) * a.r + u * 16 + q];
        mx = __builtin_fmaxf(mx, __builtin_fabsf(t[u]));
    }
    for (int off = 8; off > 0; off >>= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, off, kWave));
    const int e = scale_exponent(mx);
    const float scale = pow2(14 - e);  // to a largest element in [2^14, 2^15)
    bool small = false;                // the second fp16 part ends at 2^-24
#pragma unroll
    for (int u = 0; u < 16; ++u) small |= t[u] != 0.f && __builtin_fabsf(t[u] * scale) < 0x1p-8f;
    const bool wide = (__ballot(small) >> (threadIdx.x % kWave & 48) & 0xFFFF) != 0;
    if (row >= a.b) return;
    if (q == 0) a.te[row] = wide ? 1 : (e - 14) * 2;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        if (u * 16 >= a.r) continue;
        const int k = u * 16 + q;
        const float v = t[u] * scale;
        const uint16_t hi = F16::from_f32(v), lo = F16::from_f32(v - F16::to_f32(hi));
        const int64_t at = (row * a.r + k / 8 * 8) * 2 + k % 8;
        a.t16[at] = wide ? 0 : hi;
        a.t16[at + 8] = wide ? 0 : lo;
    }
    if (__builtin_expect(wide, 0)) {
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            if (u * 16 >= a.r) continue;
            const int64_t at = (row * a.r + (u * 16 + q) / 8 * 8) * 2 + q % 8;
            const uint16_t hi = BF16::from_f32(t[u]);
            a.twide[at] = hi;
            a.twide[at + 8] = BF16::from_f32(t[u] - BF16::to_f32(hi));
        }
    }
}

template <class T>
__global__ __launch_bounds__(256) void a16_prepare_kernel(A16Args a, int64_t row_ctas, int64_t scale_ctas) {
    __shared__ float red[256];
    int64_t id = blockIdx.x;
    if (id < row_ctas) {
        const int64_t row = id * kPrepRows + threadIdx.x / kWave;
        if (row < a.b) prepare_row<T>(a, row);
        return;
    }
    id -= row_ctas;
    if (id < scale_ctas)
        prepare_scales(a, id, red);
    else
        prepare_t(a, id - scale_ctas);
}

// The X operands of two matrix steps (addresses a0, a1) for TB token blocks, 8 KB apart, completed
// before returning (one statement, so that no other in-flight direct-to-LDS load is waited for).
template <int TB, int OFF>
__device__ __forceinline__ void a16_read(uint32_t a0, uint32_t a1, v4i (&r)[2][TB]) {
    static_assert(TB == 2 || TB == 4, "token blocks");
    if constexpr (TB == 4)
        asm volatile(
            "ds_read_b128 %0, %8 offset:%10\n\t"
            "ds_read_b128 %1, %8 offset:%11\n\t"
            "ds_read_b128 %2, %8 offset:%12\n\t"
            "ds_read_b128 %3, %8 offset:%13\n\t"
            "ds_read_b128 %4, %9 offset:%10\n\t"
            "ds_read_b128 %5, %9 offset:%11\n\t"
            "ds_read_b128 %6, %9 offset:%12\n\t"
            "ds_read_b128 %7, %9 offset:%13\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[0][2]), "=&v"(r[0][3]), "=&v"(r[1][0]), "=&v"(r[1][1]), "=&v"(r[1][2]),
              "=&v"(r[1][3])
            : "v"(a0), "v"(a1), "n"(OFF), "n"(OFF + 8192), "n"(OFF + 16384), "n"(OFF + 24576)
            : "memory");
    else
        asm volatile(
            "ds_read_b128 %0, %4 offset:%6\n\t"
            "ds_read_b128 %1, %4 offset:%7\n\t"
            "ds_read_b128 %2, %5 offset:%6\n\t"
            "ds_read_b128 %3, %5 offset:%7\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[1][0]), "=&v"(r[1][1])
            : "v"(a0), "v"(a1), "n"(OFF), "n"(OFF + 8192)
            : "memory");
}

// A CTA owns 32 TB tokens x 256 channels; its four waves take 64
// channels each and share the tokens' operands. A group of X (8 TB KB) goes to LDS by direct
// loads, one group ahead, in 256-byte lines with the 16-byte chunk index XORed by row % 8 and 8
// ((row / 16) % 2) (one 16-byte read serves lanes 0-7 with 16-23 in a pass). Each wave reads its own
// codes straight from memory to registers, one group ahead: lane l of a 32-channel block holds
// channel l % 32, and of each half group the 32 codes of K quarter l / 32. Tokens are the
// rows of the result and channels its columns, so that a group's scale is one register a lane.
// A wave's group is 64 matrix instructions (2048 cycles) and beside them 128 multiplications by scale
// ratios and 144 operations of expansion (1090 cycles). 4001 x 8192 -> 28672 1.66-1.82 ms, 1.1 PFLOP/s:
// matrix cores busy 60% of the cycles at about 1.9 GHz, no LDS conflicts. 2048 x 4096 -> 14336 by itself
// 262-295 us (clocks differ by card and by what ran before; the whole call, with two passes before it, 255-286): 896
// tiles on 512 places, 53%. Interleaving the multiplications with the matrix instructions by
// hand was 3-10% slower than leaving it to two waves a SIMD.
template <class T, int TB>
__global__ __launch_bounds__(256, 2) void a16_tile_kernel(A16Args a, int64_t ntiles, int64_t ttiles) {
    constexpr int ROWS = 32 * TB, XBYTES = ROWS * 256, XL = 2 * TB;
    __shared__ __align__(1024) uint8_t ring[2 * XBYTES];
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int col = lane % 32, half = lane / 32;
    // neighbours on an XCD: bands of eight token tiles, channel tile by channel tile
    const int64_t id = xcd_range(blockIdx.x, ntiles * ttiles), band = id / (8 * ntiles), in = id % (8 * ntiles);
    const int64_t deep = ttiles - band * 8 < 8 ? ttiles - band * 8 : 8;
    const int64_t tok0 = (band * 8 + in % deep) * ROWS, n0 = in / deep * kA16N + wave * 64;
    const int64_t groups = a.m / 128;

    const int panels = (int)(a.n / 16), panel0 = (int)(n0 / 16) < panels ? (int)(n0 / 16) : panels - 1;
    uint32_t chan[2], woff[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int p = panel0 + q * 2 + col / 16, pc = p < panels ? p : panels - 1;
        chan[q] = pc * 16 + col % 16;
        woff[q] = (uint32_t)((pc - panel0) * groups * 1024) + col % 16 * 64 + half * 16;
    }
    const uint8_t *wbase = a.qw + panel0 * groups * 1024;
    uint32_t xoff[XL];  // block j * 4 + wave of 1 KB: four rows, 16 chunks each
#pragma unroll
    for (int j = 0; j < XL; ++j) {
        const int row = (j * 4 + wave) * 4 + lane / 16, swz = (row & 7) | (row >> 4 & 1) << 3;
        const int64_t rel = tok0 + row < a.b ? row : a.b - 1 - tok0;
        xoff[j] = (uint32_t)(rel * a.m * 2 + (lane % 16 ^ swz) * 16);
    }
    const uint16_t *xbase = a.x16 + tok0 * a.m;
    v4i wn[2][2];
    float mn[2];
    uint32_t kn[2];
    auto fetch = [&](int64_t g, int slot) {
        const __amdgpu_buffer_rsrc_t rx =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(xbase + g * 128), 0, 0x7fffffff, 0x00020000);
#pragma unroll
        for (int j = 0; j < XL; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rx, (__attribute__((address_space(3))) void *)(ring + slot * XBYTES + (j * 4 + wave) * 1024), 16, (int)xoff[j], 0, 0, 0);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            wn[q][0] = load16(wbase + g * 1024 + woff[q]);
            wn[q][1] = load16(wbase + g * 1024 + 32 + woff[q]);
            mn[q] = (a.mul + g * a.n)[chan[q]];
            kn[q] = (a.mask + g * a.n)[chan[q]];
        }
    };
    const DequantConst dq = dequant_const();
    v16f acc[2][TB];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[q][t][e] = 0.f;
    // read address of matrix step s of half group st: chunk 8 st + 4 half + s of row `col`; st flips bit 7
    const int swz = (col & 7) | (col >> 4 & 1) << 3;
    uint32_t at[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) at[s] = lds_offset(ring) + col * 256 + ((half * 4 + s) ^ swz) * 16;

    fetch(0, 0);
    for (int64_t c0 = 0; c0 < groups; c0 += 2) {
        static_for(std::make_integer_sequence<int, 2>{}, [&](auto u) {
            constexpr int U = decltype(u)::value, OFF = U * XBYTES;
            const int64_t g = c0 + U;
            if (g >= groups) return;
            wait_vmcnt<0>();  // issued a group ago
            stage_barrier();  // group g has landed for every wave, and group g - 1 is read
            v4i w[2][2];
            float mul[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                mul[q] = mn[q];
                w[q][0] = wn[q][0];
                w[q][1] = wn[q][1];
            }
            if (__builtin_expect(__ballot((kn[0] & kn[1]) == 0) != 0, 0)) {  // rarely a group without weight
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[q][h][e] &= (int)kn[q];
            }
            if (g + 1 < groups) fetch(g + 1, 1 - U);
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int t = 0; t < TB; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[q][t][e] *= mul[q];
            static_for(std::make_integer_sequence<int, 4>{}, [&](auto pv) {
                constexpr int P = decltype(pv)::value;
                v4i x[2][TB];
                a16_read<TB, OFF>(at[P % 2 * 2] ^ (P / 2 * 128), at[P % 2 * 2 + 1] ^ (P / 2 * 128), x);
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const v8h wf = __builtin_bit_cast(v8h, dequant8((uint32_t)w[q][P / 2][P % 2 * 2 + s], dq));
#pragma unroll
                        for (int t = 0; t < TB; ++t) acc[q][t] = mfma_f16_32(__builtin_bit_cast(v8h, x[s][t]), wf, acc[q][t]);
                    }
            });
        });
    }
    __syncthreads();

    // true values; then the low-rank term, T L2 2^te; then the stores, turned in this wave's LDS
    uint16_t *const turn = reinterpret_cast<uint16_t *>(ring) + wave * ROWS * 64;
    const int64_t last = a.b - 1;
    const bool small = __ballot((a.small[chan[0]] | a.small[chan[1]]) != 0) != 0;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        const int64_t tok = tok0 + t * 32 + half * 4;  // + 8 (v / 4) + v % 4
        const int64_t i = tok0 + t * 32 + col;
        int xe[16];
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int64_t i = tok + v / 4 * 8 + v % 4;
            xe[v] = T::kBf16 ? a.xe[i < last ? i : last] : 0;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            // fraction and exponents apart: the unit's and the row's may each leave the range that their product is in
            const float u = a.unit[chan[q]], fraction = T::kBf16 ? __builtin_amdgcn_frexp_mantf(u) : u;
            const int ue = T::kBf16 ? __builtin_amdgcn_frexp_expf(u) : 0;
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                acc[q][t][v] *= fraction;
                if constexpr (T::kBf16) acc[q][t][v] = __builtin_ldexpf(acc[q][t][v], ue + xe[v]);
            }
        }
        if (__builtin_expect(small, 0)) {  // rarely: masked groups with a scale, the products of each by themselves
            const uint16_t *xp = a.x16 + (i < last ? i : last) * a.m + half * 32;
            const DequantConst dc = dequant_const();  // and the codes' addresses again: none of them is held over the main loop
            for (int64_t g = 0; g < groups; ++g)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float s = (a.mask + g * a.n)[chan[q]] == 0 ? (a.sw + g * a.n)[chan[q]] : 0.f;
                    if (__ballot(s != 0.f) == 0) continue;
                    v16f p;
#pragma unroll
                    for (int v = 0; v < 16; ++v) p[v] = 0.f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const v4i c = load16(a.qw + (chan[q] / 16 * groups + g) * 1024 + chan[q] % 16 * 64 + half * 16 + h * 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            p = mfma_f16_32(__builtin_bit_cast(v8h, load16(xp + g * 128 + h * 64 + e * 8)),
                                            __builtin_bit_cast(v8h, dequant8((uint32_t)c[e], dc)), p);
                    }
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[q][t][v] += s != 0.f ? s * (T::kBf16 ? p[v] * pow2(xe[v]) : p[v]) : 0.f;
                }
        }
        if (a.r > 0) {
            v16f low[2];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int v = 0; v < 16; ++v) low[q][v] = 0.f;
            const uint16_t *tp = a.t16 + ((i < last ? i : last) * a.r + half * 8) * 2;
            const int wide = -(a.te[i < last ? i : last] & 1);  // all ones: a row in bf16 parts
            for (int k = 0; k < a.r; k += 16) {
                const v8h hi = __builtin_bit_cast(v8h, load16(tp + k * 2)), lo = __builtin_bit_cast(v8h, load16(tp + k * 2 + 8));
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const v8h l2 = __builtin_bit_cast(v8h, load16(a.l2t + chan[q] * a.r + k + half * 8));
                    low[q] = mfma_f16_32(lo, l2, low[q]);
                    low[q] = mfma_f16_32(hi, l2, low[q]);
                }
            }
            if (__builtin_expect(__ballot(wide) != 0, 0)) {
                const uint16_t *wp = a.twide + (tp - a.t16);
#pragma unroll 1
                for (int k = 0; k < a.r; k += 16) {
                    v4i hi = load16(wp + k * 2), lo = load16(wp + k * 2 + 8);
#pragma unroll
                    for (int e = 0; e < 4; ++e) hi[e] &= wide, lo[e] &= wide;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        v4i wh, wl;
                        split_f16(load16(a.l2t + chan[q] * a.r + k + half * 8), wh, wl);
                        low[q] = mfma_bf16_32(lo, wl, low[q]);
                        low[q] = mfma_bf16_32(hi, wl, low[q]);
                        low[q] = mfma_bf16_32(lo, wh, low[q]);
                        low[q] = mfma_bf16_32(hi, wh, low[q]);
                    }
                }
            }
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int64_t i2 = tok + v / 4 * 8 + v % 4;
                const float te = pow2(a.te[i2 < last ? i2 : last] >> 1);
#pragma unroll
                for (int q = 0; q < 2; ++q) acc[q][t][v] += low[q][v] * te;
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int row = t * 32 + half * 4 + v / 4 * 8 + v % 4;
                turn[row * 64 + q * 32 + col] = T::from_f32(acc[q][t][v]);
            }
    }
    wave_fence();
#pragma unroll
    for (int j = 0; j < ROWS / 8; ++j) {
        const int row = j * 8 + lane / 8;
        const int64_t c = n0 + lane % 8 * 8;
        if (tok0 + row < a.b && c < a.n)
            *reinterpret_cast<v4i *>(a.y + (tok0 + row) * a.n + c) = load16(turn + row * 64 + lane % 8 * 8);
    }
}

template <class T>
static hipError_t a16_many(const A16Args &a, const A16Plan &p, hipStream_t stream) {
    const int64_t row_ctas = (a.b + kPrepRows - 1) / kPrepRows, scale_ctas = (a.n + kPrepChannels - 1) / kPrepChannels;
    const int64_t t_ctas = a.r > 0 ? (a.b + 15) / 16 : 0;
    a16_prepare_kernel<T><<<dim3((unsigned)(row_ctas + scale_ctas + t_ctas)), 256, 0, stream>>>(a, row_ctas, scale_ctas);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t ntiles = (a.n + kA16N - 1) / kA16N, ttiles = (a.b + p.rows - 1) / p.rows;
    const unsigned grid = (unsigned)(ntiles * ttiles);
    if (p.rows == 128)
        a16_tile_kernel<T, 4><<<grid, 256, 0, stream>>>(a, ntiles, ttiles);
    else
        a16_tile_kernel<T, 2><<<grid, 256, 0, stream>>>(a, ntiles, ttiles);
    return hipGetLastError();
}

hipError_t launch_a16(const A16Args &a, const A16Plan &p, hipStream_t stream) {
    if (p.many) return a.bf16 ? a16_many<BF16>(a, p, stream) : a16_many<F16>(a, p, stream);
    return a.bf16 ? a16_rows<BF16>(a, p, stream) : a16_rows<F16>(a, p, stream);
}

}  // namespace twq
