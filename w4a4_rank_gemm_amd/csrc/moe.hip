// moe.hip -- a routed layer of packed 4-bit experts for a few tokens (gfx950).
//
//   l_i = Wr x_i,  p_i = softmax(l_i) or sigmoid(l_i),  e_ij: the k experts with the largest l_i (or p_i + bias)
//   h_ij = silu(G_e x_i) * (U_e x_i),  y_i = sum_j w_ij D_e h_ij,   e = e_ij
//
// with G, U (one array of 2 f rows an expert) and D in the layer's packed format with group-wise
// scales. Launches: the logits; the choice; gate, up and the activation; down; the sum over a token's
// choices. One token is bound by the read of its experts' codes and by the chain of launches, more tokens by the
// work of the CTAs (see the kernels).
#include "twq_few_device.h"
#include "twq_moe.h"

namespace twq {

// ---- router ------------------------------------------------------------------------------

// Logits in binary64: the products of two 16-bit values are exact in it and their sums all but
// exact, so that the choice of experts is that of the formula (binary32 sums would swap experts
// whose logits differ by less than their rounding).
//
// Few products: a CTA owns one expert and kRouteTokens tokens, its waves and lanes split K, four
// loads in flight. One token, 64 experts of 2048: 4.6 us, a start and one round of loads.
constexpr int kRouteTokens = 4, kRouteWaves = 4;

template <class T>
__global__ __launch_bounds__(kRouteWaves *kWave) void route_logits_kernel(RouteArgs a) {
    __shared__ double red[kRouteWaves][kRouteTokens];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, e = blockIdx.x;
    const int64_t t0 = (int64_t)blockIdx.y * kRouteTokens;
    const uint16_t *w = a.wr + (int64_t)e * a.m, *x[kRouteTokens];
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t) x[t] = a.x + (t0 + t < a.b ? t0 + t : a.b - 1) * a.m;
    double acc[kRouteTokens] = {};
    for (int64_t k0 = threadIdx.x * 8; k0 < a.m; k0 += kRouteWaves * kWave * 8 * 4) {
        v4i wv[4], xv[4][kRouteTokens];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t k = k0 + u * kRouteWaves * kWave * 8, kc = k < a.m ? k : 0;
            wv[u] = load16(w + kc);
#pragma unroll
            for (int t = 0; t < kRouteTokens; ++t) xv[u][t] = load16(x[t] + kc);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (k0 + u * kRouteWaves * kWave * 8 >= a.m) break;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const double wd = T::to_f32(half_of(wv[u][q / 2], q % 2));
#pragma unroll
                for (int t = 0; t < kRouteTokens; ++t)
                    acc[t] = __builtin_fma((double)T::to_f32(half_of(xv[u][t][q / 2], q % 2)), wd, acc[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t) {
        for (int off = 32; off > 0; off >>= 1) acc[t] += __shfl_xor(acc[t], off, kWave);
        if (lane == 0) red[wave][t] = acc[t];
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < kRouteTokens && t0 + t < a.b) {
        double s = red[0][t];
        for (int q = 1; q < kRouteWaves; ++q) s += red[q][t];
        a.logits[(t0 + t) * a.experts + e] = s;
    }
}

// Many products: tiles of 32 experts x 32 tokens on binary64 matrix instructions (16 x 16 x 4, four a
// wave, so that an element is converted for two of them), K split over slices and the CTA's 16
// waves, whose sums are added in wave order. Element e of a lane's eight goes to instruction e, for both
// operands. Result: lane (li, g) holds token li, experts 4 v + g of a 16 x 16 block. 256 tokens, 256
// experts of 7168: 24.4 us, of which the binary64 matrix instructions alone take 12.6; they are busy
// 57% of the cycles, and each element takes two conversions on the way.
typedef double v4d __attribute__((ext_vector_type(4)));
constexpr int kTileWaves = 16;

template <class T>
__global__ __launch_bounds__(kTileWaves *kWave) void route_logits_tile_kernel(RouteArgs a) {
    __shared__ double red[kTileWaves][4][4][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, li = lane & 15, g = lane >> 4;
    const int64_t e0 = (int64_t)blockIdx.x * 32, t0 = (int64_t)blockIdx.y * 32, slice = blockIdx.z;
    const int steps = (int)(a.m / 32), parts = a.slices * kTileWaves, part = (int)slice * kTileWaves + wave;
    const int s0 = (int)((int64_t)part * steps / parts), s1 = (int)((int64_t)(part + 1) * steps / parts);
    const uint16_t *w[2], *x[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int64_t e = e0 + q * 16 + li, t = t0 + q * 16 + li;
        w[q] = a.wr + (e < a.experts ? e : a.experts - 1) * a.m + g * 8;
        x[q] = a.x + (t < a.b ? t : a.b - 1) * a.m + g * 8;
    }
    v4d acc[2][2] = {};
    v4i wn[2], xn[2];
    auto load = [&](int s) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            wn[q] = load16(w[q] + s * 32);
            xn[q] = load16(x[q] + s * 32);
        }
    };
    if (s0 < s1) load(s0);
    for (int s = s0; s < s1; ++s) {
        const v4i wc[2] = {wn[0], wn[1]}, xc[2] = {xn[0], xn[1]};
        if (s + 1 < s1) load(s + 1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            double wd[2], xd[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                wd[q] = T::to_f32(half_of(wc[q][e / 2], e % 2));
                xd[q] = T::to_f32(half_of(xc[q][e / 2], e % 2));
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int t = 0; t < 2; ++t) acc[q][t] = __builtin_amdgcn_mfma_f64_16x16x4f64(wd[q], xd[t], acc[q][t], 0, 0, 0);
        }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) red[wave][q * 2 + t][v][lane] = acc[q][t][v];
    __syncthreads();
    const int blk = wave / 4, v = wave % 4;
    double sum = red[0][blk][v][lane];
    for (int q = 1; q < kTileWaves; ++q) sum += red[q][blk][v][lane];
    const int64_t t = t0 + blk % 2 * 16 + li, e = e0 + blk / 2 * 16 + 4 * v + g;
    if (t < a.b && e < a.experts) a.logits[(slice * a.b + t) * a.experts + e] = sum;
}

// Maximum over the 64 lanes, uniform: the upper halves first, the lower ones among those that tie.
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
    const uint32_t hi = (uint32_t)(v >> 32), top = wave_max_u32(hi);
    const uint64_t tied = __ballot(hi == top);
    const uint32_t low = tied & (tied - 1) ? wave_max_u32(hi == top ? (uint32_t)v : 0)
                                           : (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, __builtin_ctzll(tied));
    return (uint64_t)top << 32 | low;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

// The k best experts of a token by one wave; lane l holds experts l, l + 64, .. as keys whose
// unsigned order is the order of the values (0: none or taken, 1: NaN). Each round takes the largest
// key, the lowest index among equals. Probabilities of all experts are formed only where they
// are asked for: with a bias, or softmax weights that are not divided by their sum. Bound by the rounds'
// dependent maxima over lanes: k = 8 of 64 experts 4-5 us, of 256 over four slices 6.8.
__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 to 0
    return v == v ? u ^ ((u >> 63) ? ~uint64_t(0) : uint64_t(1) << 63) : 1;
}
__device__ __forceinline__ double key_value(uint64_t k) {
    return __builtin_bit_cast(double, k >> 63 ? k ^ uint64_t(1) << 63 : ~k);
}

template <int H>
__device__ __forceinline__ void choose_experts(const RouteArgs &a, int64_t tok) {
    const int lane = threadIdx.x % kWave;
    double l[H], p[H];
    const auto logit = [&](int slice, int i) {
        const int e = i * kWave + lane;
        return a.logits[(slice * a.b + tok) * a.experts + (e < a.experts ? e : 0)];
    };
#pragma unroll
    for (int i = 0; i < H; ++i) l[i] = logit(0, i);
    for (int q = 1; q < a.slices; q += 4) {  // four slices' loads in flight
        double v[4][H];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < H; ++i) v[u][i] = logit(q + u < a.slices ? q + u : q, i);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < H; ++i) l[i] += q + u < a.slices ? v[u][i] : 0.0;
    }
    uint64_t key[H], best = 0;
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const int e = i * kWave + lane;
        key[i] = e < a.experts ? order_key(l[i]) : 0;
        p[i] = 0;
        best = best > key[i] ? best : key[i];
    }
    const bool every = a.bias || (!a.sigmoid && !a.norm);
    double top = 0, sum = 1;
    if (every && !a.sigmoid) {
        top = key_value(wave_max_u64(best));
        sum = 0;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            p[i] = key[i] ? exp(l[i] - top) : 0.0;
            sum += p[i];
        }
        sum = wave_sum_f64(sum);
    }
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int e = i * kWave + lane;
            p[i] = a.sigmoid ? 1.0 / (1.0 + exp(-l[i])) : p[i] / sum;
            key[i] = e < a.experts ? order_key(p[i] + (double)a.bias[e]) : 0;
        }
    }
    int mine = 0;
    double value = 0, first = 0;  // of lane j's choice j: its logit, or with a bias its probability
    for (int j = 0; j < a.k; ++j) {
        uint64_t k = 0;
#pragma unroll
        for (int i = 0; i < H; ++i) k = k > key[i] ? k : key[i];
        k = wave_max_u64(k);
        int at = -1;
        double v = key_value(k);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const uint64_t hit = __ballot(key[i] == k);
            if (at >= 0 || hit == 0) continue;
            const int o = __builtin_ctzll(hit);
            at = i * kWave + o;
            if (lane == o) key[i] = 0;
            if (a.bias) v = __shfl(p[i], o, kWave);
        }
        if (j == 0) first = v;
        if (lane == j) mine = at, value = v;
    }
    double w = 0;
    if (lane < a.k) w = a.bias ? value : a.sigmoid ? 1.0 / (1.0 + exp(-value)) : exp(value - (every ? top : first)) / sum;
    const double total = wave_sum_f64(w);
    if (lane < a.k) {
        a.ids[tok * a.k + lane] = mine;
        a.weights[tok * a.k + lane] = (float)((a.norm ? (total == 0 ? 0.0 : w / total) : w) * a.scale);
    }
}

__global__ __launch_bounds__(kWave) void route_choose_kernel(RouteArgs a) {
    if (a.experts <= kWave)
        choose_experts<1>(a, blockIdx.x);
    else if (a.experts <= 2 * kWave)
        choose_experts<2>(a, blockIdx.x);
    else if (a.experts <= 4 * kWave)
        choose_experts<4>(a, blockIdx.x);
    else
        choose_experts<8>(a, blockIdx.x);
}

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
    const unsigned b = (unsigned)a.b;
    if (a.tiled) {
        const dim3 grid((unsigned)((a.experts + 31) / 32), (b + 31) / 32, (unsigned)a.slices);
        if (a.bf16)
            route_logits_tile_kernel<BF16><<<grid, kTileWaves * kWave, 0, stream>>>(a);
        else
            route_logits_tile_kernel<F16><<<grid, kTileWaves * kWave, 0, stream>>>(a);
    } else {
        const dim3 grid((unsigned)a.experts, (b + kRouteTokens - 1) / kRouteTokens);
        if (a.bf16)
            route_logits_kernel<BF16><<<grid, kRouteWaves * kWave, 0, stream>>>(a);
        else
            route_logits_kernel<F16><<<grid, kRouteWaves * kWave, 0, stream>>>(a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_choose_kernel<<<b, kWave, 0, stream>>>(a);
    return hipGetLastError();
}

// ---- experts -----------------------------------------------------------------------------

constexpr int kMoeWaves = 8, kMoeThreads = kMoeWaves * kWave, kMaxPairs = kMaxMoeTokens * kMaxTopK;

// The pairs (token, choice) of this CTA's expert, in order, in `list`; returns their number. With at
// most as many pairs as experts a slot is a pair, and the first pair of an expert takes all of its
// pairs; otherwise a slot is an expert. All threads call it. Up to 64 pairs every wave writes the
// whole list for itself.
__device__ __forceinline__ int expert_pairs(const MoeArgs &a, int slot, int &expert, uint16_t *list, int *count) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, n = (int)a.b * a.k;
    const uint64_t below = (uint64_t(1) << lane) - 1;
    int have = 0;
    if (n <= kWave) {
        const int id = lane < n ? a.ids[lane] : -1;
        expert = n <= a.experts ? __builtin_amdgcn_readlane(id, slot) : slot;
        if ((unsigned)expert >= (unsigned)a.experts) return 0;
        const uint64_t hit = __ballot(lane < n && id == expert);
        if (hit >> lane & 1) list[__popcll(hit & below)] = (uint16_t)lane;
        wave_fence();
        have = __popcll(hit);
        return n <= a.experts && __builtin_ctzll(hit) != slot ? 0 : have;
    }
    int id = tid < n ? a.ids[tid] : -1;
    expert = n <= a.experts ? __builtin_amdgcn_readfirstlane(a.ids[slot]) : slot;
    if ((unsigned)expert >= (unsigned)a.experts) return 0;
    for (int i0 = 0; i0 < n; i0 += kMoeThreads) {
        const int i = i0 + tid;
        if (i0 > 0) id = i < n ? a.ids[i] : -1;
        const uint64_t hit = __ballot(i < n && id == expert);
        if (lane == 0) count[wave] = __popcll(hit);
        __syncthreads();
        int before = have;
#pragma unroll
        for (int w = 0; w < kMoeWaves; ++w) {
            before += w < wave ? count[w] : 0;
            have += count[w];
        }
        if (hit >> lane & 1) list[before + __popcll(hit & below)] = (uint16_t)i;
        __syncthreads();
    }
    return n <= a.experts && list[0] != slot ? 0 : have;
}

// h = silu(gate) up of four channels of a panel and one pair, as two bf16 parts (16 significant bits:
// one would round as coarsely as a bf16 output, and the type of an fp16 layer could overflow).
__device__ __forceinline__ void store_inner(const MoeArgs &a, const v4f &gate, const v4f &up, int pair, int64_t panel) {
    uint16_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float h = gate[e] / (1.f + __expf(-gate[e])) * up[e];
        hi[e] = BF16::from_f32(h);
        lo[e] = BF16::from_f32(h - BF16::to_f32(hi[e]));
    }
    const int64_t c = panel * 16 + threadIdx.x % kWave / 16 * 4;
    uint16_t *p = a.h + ((int64_t)pair * (a.f / 128) + c / 128) * 256 + c % 128;
    *reinterpret_cast<uint2 *>(p) = make_uint2((uint32_t)hi[0] | (uint32_t)hi[1] << 16, (uint32_t)hi[2] | (uint32_t)hi[3] << 16);
    *reinterpret_cast<uint2 *>(p + 128) = make_uint2((uint32_t)lo[0] | (uint32_t)lo[1] << 16, (uint32_t)lo[2] | (uint32_t)lo[3] << 16);
}

// Gate and up rows of one panel of 16 inner channels, kw waves to a panel.
template <class T, int XR, int U>
__device__ __forceinline__ void up_tile(const MoeArgs &a, int expert, const uint16_t *list, int rows, uint8_t *smem, int wave_lds, int kw) {
    typedef FewRows<T, 2, XR, 1, U> Rows;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), share = wave & (kw - 1);
    const int64_t pieces = a.m / 128, half = a.f / 16, unit = ((int64_t)blockIdx.x * kMoeWaves + wave) / kw;
    Rows r;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int64_t p = expert * 2 * half + f * half + (unit < half ? unit : half - 1);  // gate, up
        r.w[f] = a.q1 + p * pieces * 1024;
        r.s[f] = a.s1 + p * 16;
    }
    r.s_stride = a.experts * 2 * a.f;
    r.x = a.x;
#pragma unroll
    for (int j = 0; j < Rows::XL; ++j) {
        const int i = 4 * j + lane / 16;
        r.row[j] = (uint32_t)((list[i < rows ? i : rows - 1] / a.k) * a.m * 2);
    }
    v4f acc[2][1] = {};
    if (unit < half)
        r.run((int)(share * pieces / kw), (int)((share + 1) * pieces / kw), smem + wave * wave_lds, acc, [] {});
    join_waves(smem, kw, wave, acc);
    if (share == 0 && unit < half && lane % 16 < rows) store_inner(a, acc[0][0], acc[1][0], list[lane % 16], unit);
}

// The work list of the down kernel for few tokens: the experts asked for, each with its pairs, at most
// one a token (an expert that a token names again is another entry). One CTA, in its LDS.
struct EntryScratch {
    int32_t id[kFewPairs], again[kFewPairs], number[kFewPairs];
    MoeEntry entries[kFewPairs];
};
__device__ __forceinline__ void expert_entries(const MoeArgs &a, EntryScratch &s) {
    const int i = threadIdx.x, n = (int)a.b * a.k;  // at most kFewPairs, fewer than threads
    const int id = i < n ? a.ids[i] : -1;
    const bool on = (unsigned)id < (unsigned)a.experts;
    if (i < n) s.id[i] = id;
    __syncthreads();
    int turn = 0, first = i, at = 0;  // how often its token named the expert before; the entry's first pair; place in the entry
    if (on)
        for (int j = i / a.k * a.k; j < i; ++j) turn += s.id[j] == id;
    if (i < n) s.again[i] = turn;
    __syncthreads();
    if (on)
        for (int j = i - 1; j >= 0; --j)
            if (s.id[j] == id && s.again[j] == turn) first = j, ++at;
    if (i < n) s.number[i] = on && first == i;
    __syncthreads();
    int entry = 0, rows = 0, all = 0;
    for (int j = 0; on && j < n; ++j) {
        entry += j < first ? s.number[j] : 0;
        rows += s.id[j] == id && s.again[j] == turn;
    }
    MoeEntry &e = s.entries[entry];
    if (on && first == i) {
        e.expert = id;
        e.rows = rows;
        for (int t = 0; t < kFewMoe; ++t) e.place[t] = -1;
    }
    for (int j = 0; i == 0 && j < n; ++j) all += s.number[j];
    __syncthreads();
    if (on) {
        e.pair[at] = (int16_t)i;
        e.place[i / a.k] = (int8_t)at;
    }
    if (i == 0) *a.entry_count = all;
    __syncthreads();
    for (int j = i; j < n * (int)(sizeof(MoeEntry) / 16); j += kMoeThreads)
        reinterpret_cast<v4i *>(a.entries)[j] = reinterpret_cast<const v4i *>(s.entries)[j];
}

// kw waves to a panel of gate and up rows. One more row of CTAs than there are slots (few tokens)
// makes the down kernel's work list. One token, 2 of 8 experts of 4096 -> 14336 (125 MB): 30.6 us, 4.1
// TB/s; 13 tokens, 4 of 60 of 2048 -> 1408 (71 MB) 24, and 21.6 with rows and codes that
// come from a cache: the CTAs' start, search and steps; one token, 8 of 64 of 2048 -> 768 (14 MB) 8.9.
template <class T>
__global__ __launch_bounds__(kMoeThreads, 4) void moe_up_kernel(MoeArgs a, int slots, int kw) {
    // one place a wave, whatever the rows of a tile: waves may be at different tiles
    constexpr int LDS = FewRows<T, 2, 16, 1, 1>::LDS;
    static_assert(LDS >= FewRows<T, 2, 4, 1, 2>::LDS && LDS >= 2 * 1024 && kMoeWaves * LDS >= (int)sizeof(EntryScratch), "shared buffer");
    __shared__ __align__(16) uint8_t smem[kMoeWaves * LDS];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count[kMoeWaves];
    if ((int)blockIdx.y == slots) {
        if (blockIdx.x == 0) expert_entries(a, *reinterpret_cast<EntryScratch *>(smem));
        return;
    }
    int expert;
    const int n = expert_pairs(a, blockIdx.y, expert, list, count);
    for (int i = 0; i < n; i += 16) {
        const int rows = n - i < 16 ? n - i : 16;
        if (rows <= 4)
            up_tile<T, 4, 2>(a, expert, list + i, rows, smem, LDS, kw);
        else
            up_tile<T, 16, 1>(a, expert, list + i, rows, smem, LDS, kw);
        if (kw > 1) __syncthreads();
    }
}

// Few tokens: a CTA owns a panel of 16 output channels and all of the work list, whose pieces its 16
// waves split evenly; a wave adds its products to its tokens' sums with their weights, the waves'
// sums are added in wave order and rounded once. No partial output reaches memory. One token, 2 experts of
// 14336 -> 4096 (63 MB): 20.5 us, 3.1 TB/s; 8 of 768 -> 2048 (7 MB) 7.7.
constexpr int kDownWaves = 16, kDownThreads = kDownWaves * kWave;

template <class T>
__global__ __launch_bounds__(kDownThreads) void moe_down_few_kernel(MoeArgs a) {
    typedef FewRows<BF16, 1, kFewMoe, 2, 2> Rows;
    __shared__ __align__(16) uint8_t smem[kDownWaves * Rows::LDS];
    __shared__ MoeEntry entries[kFewPairs];
    __shared__ float weights[kFewPairs];
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave), n = (int)a.b * a.k;
    const int li = lane & 15, g = lane >> 4;
    if (tid < n) weights[tid] = a.weights[tid];
    if (tid < n * (int)(sizeof(MoeEntry) / 16))  // entries past the last are not used
        reinterpret_cast<v4i *>(entries)[tid] = load16(reinterpret_cast<const uint8_t *>(a.entries) + tid * 16);
    const int pieces = (int)(a.f / 128), all = *a.entry_count * pieces, u1 = (int)((int64_t)(wave + 1) * all / kDownWaves);
    const int64_t panel = xcd_range(blockIdx.x, gridDim.x);  // neighbours share lines of scales
    __syncthreads();
    v4f sum[1][1] = {};
    for (int u = (int)((int64_t)wave * all / kDownWaves); u < u1;) {
        const MoeEntry &e = entries[u / pieces];
        const int p0 = u % pieces, p1 = pieces - p0 < u1 - u ? pieces : p0 + u1 - u;
        const int64_t p = __builtin_amdgcn_readfirstlane(e.expert) * (a.m / 16) + panel;
        Rows r;
        r.w[0] = a.q2 + p * pieces * 1024;
        r.s[0] = a.s2 + p * 16;
        r.s_stride = a.experts * a.m;
        r.x = a.h;
        r.row[0] = (uint32_t)(e.pair[g < e.rows ? g : e.rows - 1] * a.f * 4);
        v4f acc[1][1] = {};
        r.run(p0, p1, smem + wave * Rows::LDS, acc, [] {});
        const int place = li < kFewMoe ? e.place[li] : -1;  // column of this lane's token
        const float w = place < 0 ? 0.f : weights[e.pair[place]];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float v = __shfl(acc[0][0][q], (lane & 48) + (place < 0 ? 0 : place), kWave);
            if (place >= 0) sum[0][0][q] += w * v;
        }
        u += p1 - p0;
    }
    join_waves(smem, kDownWaves, wave, sum);
    if (wave == 0 && li < a.b) {
        const v4f s = sum[0][0];
        *reinterpret_cast<uint2 *>(a.y + li * a.m + panel * 16 + g * 4) =
            make_uint2((uint32_t)T::from_f32(s[0]) | (uint32_t)T::from_f32(s[1]) << 16,
                       (uint32_t)T::from_f32(s[2]) | (uint32_t)T::from_f32(s[3]) << 16);
    }
}

// Many rows an expert, or many experts: the CTA's eight waves share an expert's rows and K, and own
// eight panels of inner (output) channels together. 128 tokens, 8 of 128 experts of 4096 and 1408: gate and
// up 158-189 us for 798 MB (4.2-5.0 TB/s), down 104-130 for 444 MB (3.4-4.3): its CTAs have 11 steps only,
// and finding the expert's rows and the first loads are a larger part of them. With many rows an expert a CTA takes
// its tiles of 32 one after the other and expands the same codes for each: 256 tokens, 8 of 64 of 2048 -> 768 60 and
// 44 us, 58.6 and 43 with rows and codes that come from a cache; 2 of 8 of 4096 -> 14336 266 and 285, 245 and 257.
// Two panels a wave, wave pairs that split K and two pieces a step were all slower with 128 tokens (1-7%).
template <class T>
__global__ __launch_bounds__(kMoeThreads) void moe_up_shared_kernel(MoeArgs a) {
    constexpr int XR = 32;
    typedef SharedRows<T, 2, XR, 1, 1, 1> Rows;
    __shared__ __align__(16) uint8_t smem[Rows::LDS];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count[kMoeWaves];
    int expert;
    const int n = expert_pairs(a, blockIdx.y, expert, list, count);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t pieces = a.m / 128, half = a.f / 16, panel = (int64_t)blockIdx.x * kMoeWaves + wave;  // f is a multiple of 128
    Rows r;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int64_t p = expert * 2 * half + f * half + panel;
        r.w[f] = a.q1 + p * pieces * 1024;
        r.s[f] = a.s1 + p * 16;
    }
    r.s_stride = a.experts * 2 * a.f;
    r.x = a.x;
    for (int i = 0; i < n; i += XR) {
        const int rows = n - i < XR ? n - i : XR;
#pragma unroll
        for (int j = 0; j < Rows::PER; ++j) {
            const int row = Rows::row_of(j);
            r.row[j] = (uint32_t)((list[i + (row < rows ? row : rows - 1)] / a.k) * a.m * 2);
        }
        v4f acc[2][Rows::FM] = {};
        r.run(0, (int)pieces, smem, acc);
#pragma unroll
        for (int c = 0; c < Rows::FM; ++c)
            if (c * 16 + lane % 16 < rows) store_inner(a, acc[0][c], acc[1][c], list[i + c * 16 + lane % 16], panel);
        __syncthreads();
    }
}

template <int XR>
__global__ __launch_bounds__(kMoeThreads) void moe_down_shared_kernel(MoeArgs a) {
    typedef SharedRows<BF16, 1, XR, 2, 1, 1> Rows;
    __shared__ __align__(16) uint8_t smem[Rows::LDS];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count[kMoeWaves];
    int expert;
    const int n = expert_pairs(a, blockIdx.y, expert, list, count);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t pieces = a.f / 128, panel = (int64_t)blockIdx.x * kMoeWaves + wave;  // m is a multiple of 128
    const int64_t p = expert * (a.m / 16) + panel;
    const int64_t slice = blockIdx.z;
    Rows r;
    r.w[0] = a.q2 + p * pieces * 1024;
    r.s[0] = a.s2 + p * 16;
    r.s_stride = a.experts * a.m;
    r.x = a.h;
    for (int i = 0; i < n; i += XR) {
        const int rows = n - i < XR ? n - i : XR;
#pragma unroll
        for (int j = 0; j < Rows::PER; ++j) {
            const int row = Rows::row_of(j);
            r.row[j] = (uint32_t)(list[i + (row < rows ? row : rows - 1)] * a.f * 4);  // at most 4095 x 2^19
        }
        v4f acc[1][Rows::FM] = {};
        r.run((int)(slice * pieces / a.ks), (int)((slice + 1) * pieces / a.ks), smem, acc);
#pragma unroll
        for (int c = 0; c < Rows::FM; ++c)
            if (c * 16 + lane % 16 < rows) {
                const int pair = list[i + c * 16 + lane % 16];
                const float w = a.weights[pair];
                v4f s = acc[0][c];
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] *= w;
                *reinterpret_cast<v4f *>(a.part + ((slice * a.b * a.k + pair) * a.m + panel * 16 + lane / 16 * 4)) = s;
            }
        __syncthreads();
    }
}

// y = the sum of a token's weighted parts, in the order of its choices and of K's slices, rounded once.
template <class T>
__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs a) {
    const int64_t tok = blockIdx.y, c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (c >= a.m) return;
    v4f s = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.k; ++j) {
        if ((unsigned)a.ids[tok * a.k + j] >= (unsigned)a.experts) continue;
        for (int q = 0; q < a.ks; ++q) {
            const v4f o = *reinterpret_cast<const v4f *>(a.part + ((q * a.b + tok) * a.k + j) * a.m + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += o[e];
        }
    }
    *reinterpret_cast<uint2 *>(a.y + tok * a.m + c) = make_uint2((uint32_t)T::from_f32(s[0]) | (uint32_t)T::from_f32(s[1]) << 16,
                                                                 (uint32_t)T::from_f32(s[2]) | (uint32_t)T::from_f32(s[3]) << 16);
}

template <class T>
static hipError_t moe_typed(const MoeArgs &a, const MoePlan &p, hipStream_t stream) {
    const dim3 up((unsigned)((a.f / 16 * p.up_waves + kMoeWaves - 1) / kMoeWaves), (unsigned)(p.slots + p.few));
    if (p.up_shared)
        moe_up_shared_kernel<T><<<dim3((unsigned)(a.f / 128), (unsigned)p.slots), kMoeThreads, 0, stream>>>(a);
    else
        moe_up_kernel<T><<<up, kMoeThreads, 0, stream>>>(a, p.slots, p.up_waves);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.few) {
        moe_down_few_kernel<T><<<(unsigned)(a.m / 16), kDownThreads, 0, stream>>>(a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)(a.m / 128), (unsigned)p.slots, (unsigned)p.ks);
    if (p.down_rows == 16)
        moe_down_shared_kernel<16><<<grid, kMoeThreads, 0, stream>>>(a);
    else
        moe_down_shared_kernel<32><<<grid, kMoeThreads, 0, stream>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    moe_join_kernel<T><<<dim3((unsigned)((a.m + 1023) / 1024), (unsigned)a.b), 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe(const MoeArgs &a, const MoePlan &p, hipStream_t stream) {
    return a.bf16 ? moe_typed<BF16>(a, p, stream) : moe_typed<F16>(a, p, stream);
}

}  // namespace twq
