// moe.hip -- a routed layer of packed 4-bit experts for a few tokens (gfx950).
//
//   l_i = Wr x_i,  p_i = softmax(l_i) or sigmoid(l_i),  e_ij: the k experts with the largest l_i (or p_i + bias)
//   h_ij = silu(G_e x_i) * (U_e x_i),  y_i = sum_j w_ij D_e h_ij,   e = e_ij
//
// with G, U (one array of 2 f rows an expert) and D in the layer's packed format with group-wise
// scales. Launches: the logits; the choice; gate, up and the activation; down; the sum over a token's
// choices. Bound by the read of the chosen experts' codes.
#include "twq_few_device.h"
#include "twq_moe.h"

namespace twq {

// ---- router ------------------------------------------------------------------------------

// Logits in binary64: the products of two 16-bit values are exact in it and their sums all but
// exact, so that the choice of experts is that of the formula (binary32 sums would swap experts
// whose logits differ by less than their rounding). A wave owns one expert and kRouteTokens
// tokens, its lanes split K.
constexpr int kRouteTokens = 4, kRouteWaves = 4;

template <class T>
__global__ __launch_bounds__(kRouteWaves *kWave) void route_logits_kernel(RouteArgs a) {
    const int lane = threadIdx.x % kWave, e = blockIdx.x * kRouteWaves + threadIdx.x / kWave;
    if (e >= a.experts) return;
    const int64_t t0 = (int64_t)blockIdx.y * kRouteTokens;
    const uint16_t *w = a.wr + (int64_t)e * a.m, *x[kRouteTokens];
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t) x[t] = a.x + (t0 + t < a.b ? t0 + t : a.b - 1) * a.m;
    double acc[kRouteTokens] = {};
    for (int64_t k = lane * 8; k < a.m; k += kWave * 8) {
        const v4i wv = load16(w + k);
        v4i xv[kRouteTokens];
#pragma unroll
        for (int t = 0; t < kRouteTokens; ++t) xv[t] = load16(x[t] + k);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const double wd = T::to_f32(half_of(wv[q / 2], q % 2));
#pragma unroll
            for (int t = 0; t < kRouteTokens; ++t) acc[t] = __builtin_fma((double)T::to_f32(half_of(xv[t][q / 2], q % 2)), wd, acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t) {
        for (int off = 32; off > 0; off >>= 1) acc[t] += __shfl_xor(acc[t], off, kWave);
        if (lane == 0 && t0 + t < a.b) a.logits[(t0 + t) * a.experts + e] = acc[t];
    }
}

// The k best experts of a token, one wave a token: lane l holds experts l, l + 64, .. Each round
// takes the largest of what is left, the lowest index among equals. A NaN counts as lowest.
constexpr int kHeld = kMaxExperts / kWave;

__global__ __launch_bounds__(kRouteWaves *kWave) void route_choose_kernel(RouteArgs a) {
    const int lane = threadIdx.x % kWave;
    const int64_t tok = (int64_t)blockIdx.x * kRouteWaves + threadIdx.x / kWave;
    if (tok >= a.b) return;
    const double none = -__builtin_inf();
    double l[kHeld], p[kHeld], mx = none;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int e = i * kWave + lane;
        const double v = e < a.experts ? a.logits[tok * a.experts + e] : none;
        l[i] = v == v ? v : none;
        mx = l[i] > mx ? l[i] : mx;
    }
    for (int off = 32; off > 0; off >>= 1) {
        const double o = __shfl_xor(mx, off, kWave);
        mx = o > mx ? o : mx;
    }
    double sum = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        p[i] = i * kWave + lane >= a.experts ? 0.0 : a.sigmoid ? 1.0 / (1.0 + exp(-l[i])) : exp(l[i] - mx);
        sum += p[i];
    }
    if (!a.sigmoid) {
        for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, kWave);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) p[i] /= sum;
    }
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int e = i * kWave + lane;
            const double v = e < a.experts ? p[i] + (double)a.bias[e] : none;
            l[i] = v == v ? v : none;
        }
    }
    uint32_t taken = 0;
    int mine = 0;
    double weight = 0, total = 0;  // lane j: choice j
    for (int j = 0; j < a.k; ++j) {
        double best = none, prob = 0;
        int at = INT32_MAX;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int e = i * kWave + lane;
            if (e < a.experts && !(taken >> i & 1) && (l[i] > best || at == INT32_MAX)) best = l[i], at = e, prob = p[i];
        }
        for (int off = 32; off > 0; off >>= 1) {
            const double o = __shfl_xor(best, off, kWave), q = __shfl_xor(prob, off, kWave);
            const int w = __shfl_xor(at, off, kWave);
            if (w != INT32_MAX && (at == INT32_MAX || o > best || (o == best && w < at))) best = o, at = w, prob = q;
        }
        if (at % kWave == lane) taken |= 1u << at / kWave;
        total += prob;
        if (lane == j) mine = at, weight = prob;
    }
    if (lane < a.k) {
        a.ids[tok * a.k + lane] = mine;
        a.weights[tok * a.k + lane] = (float)((a.norm ? (total > 0 ? weight / total : 0.0) : weight) * a.scale);
    }
}

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.experts + kRouteWaves - 1) / kRouteWaves), (unsigned)((a.b + kRouteTokens - 1) / kRouteTokens));
    if (a.bf16)
        route_logits_kernel<BF16><<<grid, kRouteWaves * kWave, 0, stream>>>(a);
    else
        route_logits_kernel<F16><<<grid, kRouteWaves * kWave, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_choose_kernel<<<dim3((unsigned)((a.b + kRouteWaves - 1) / kRouteWaves)), kRouteWaves * kWave, 0, stream>>>(a);
    return hipGetLastError();
}

// ---- experts -----------------------------------------------------------------------------

constexpr int kMoeWaves = 8, kMoeThreads = kMoeWaves * kWave, kMaxPairs = kMaxMoeTokens * kMaxTopK;

// The pairs (token, choice) of this CTA's expert, in order, in `list`; returns their number. With at
// most as many pairs as experts a slot is a pair, and the first pair of an expert takes all of its
// pairs; otherwise a slot is an expert. All threads call it.
__device__ __forceinline__ int expert_pairs(const MoeArgs &a, int slot, int &expert, uint16_t *list, int *count) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, n = (int)a.b * a.k;
    int id = tid < n ? a.ids[tid] : -1;
    expert = n <= a.experts ? a.ids[slot] : slot;
    if ((unsigned)expert >= (unsigned)a.experts) return 0;
    int have = 0;
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
        if (hit >> lane & 1) list[before + __popcll(hit & ((uint64_t(1) << lane) - 1))] = (uint16_t)i;
        __syncthreads();
    }
    return n <= a.experts && list[0] != slot ? 0 : have;
}

// The waves' sums, in wave order: element t of FN x 64 lanes for thread t.
template <int FN>
__device__ __forceinline__ v4f join_waves(v4f *red, const v4f (&acc)[FN][1], int t) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    __syncthreads();
#pragma unroll
    for (int f = 0; f < FN; ++f) red[(wave * FN + f) * kWave + lane] = acc[f][0];
    __syncthreads();
    v4f s = red[t];
#pragma unroll
    for (int w = 1; w < kMoeWaves; ++w) {
        const v4f o = red[w * FN * kWave + t];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += o[e];
    }
    return s;
}

template <class T, int XR, int U>
__device__ __forceinline__ void up_tile(const MoeArgs &a, int expert, const uint16_t *list, int rows, uint8_t *smem) {
    typedef FewRows<T, 2, XR, 1, U> Rows;
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int64_t pieces = a.m / 128, half = a.f / 16, panel = blockIdx.x;
    Rows r;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int64_t p = expert * 2 * half + f * half + panel;  // gate, up
        r.w[f] = a.q1 + p * pieces * 1024;
        r.s[f] = a.s1 + p * 16;
    }
    r.s_stride = a.experts * 2 * a.f;
#pragma unroll
    for (int j = 0; j < Rows::XL; ++j) {
        const int i = 4 * j + lane / 16;
        r.x[j] = a.x + (int64_t)(list[i < rows ? i : rows - 1] / a.k) * a.m + lane % 16 * 8;
    }
    v4f acc[2][1] = {};
    r.template run<false>((int)(wave * pieces / kMoeWaves), (int)((wave + 1) * pieces / kMoeWaves), smem + wave * Rows::LDS, acc);
    v4f *const red = reinterpret_cast<v4f *>(smem);
    const v4f s = join_waves<2>(red, acc, tid % (2 * kWave));
    __syncthreads();
    if (tid < 2 * kWave) red[tid] = s;
    __syncthreads();
    // h = silu(gate) up, as two bf16 parts (16 significant bits: one would round as coarsely as a
    // bf16 output, and the type of an fp16 layer could overflow)
    if (tid < kWave && tid % 16 < rows) {
        const v4f gate = red[tid], up = red[kWave + tid];
        uint16_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float h = gate[e] / (1.f + __expf(-gate[e])) * up[e];
            hi[e] = BF16::from_f32(h);
            lo[e] = BF16::from_f32(h - BF16::to_f32(hi[e]));
        }
        const int64_t c = panel * 16 + tid / 16 * 4;
        uint16_t *p = a.h + ((int64_t)list[tid % 16] * (a.f / 128) + c / 128) * 256 + c % 128;
        *reinterpret_cast<uint2 *>(p) = make_uint2((uint32_t)hi[0] | (uint32_t)hi[1] << 16, (uint32_t)hi[2] | (uint32_t)hi[3] << 16);
        *reinterpret_cast<uint2 *>(p + 128) = make_uint2((uint32_t)lo[0] | (uint32_t)lo[1] << 16, (uint32_t)lo[2] | (uint32_t)lo[3] << 16);
    }
}

template <class T>
__global__ __launch_bounds__(kMoeThreads) void moe_up_kernel(MoeArgs a) {
    constexpr int LDS = kMoeWaves * FewRows<T, 2, 16, 1, 2>::LDS;
    static_assert(LDS >= kMoeWaves * FewRows<T, 2, 4, 1, 4>::LDS && LDS >= kMoeWaves * 2 * 1024, "shared buffer");
    __shared__ __align__(16) uint8_t smem[LDS];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count[kMoeWaves];
    int expert;
    const int n = expert_pairs(a, blockIdx.y, expert, list, count);
    for (int i = 0; i < n; i += 16) {
        const int rows = n - i < 16 ? n - i : 16;
        if (rows <= 4)
            up_tile<T, 4, 4>(a, expert, list + i, rows, smem);
        else
            up_tile<T, 16, 2>(a, expert, list + i, rows, smem);
        __syncthreads();
    }
}

template <int XR, int U>
__device__ __forceinline__ void down_tile(const MoeArgs &a, int expert, const uint16_t *list, int rows, uint8_t *smem) {
    typedef FewRows<BF16, 2, XR, 2, U> Rows;
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int64_t pieces = a.f / 128, panels = a.m / 16, panel0 = (int64_t)blockIdx.x * 2;
    Rows r;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int64_t p = expert * panels + panel0 + f;  // m is a multiple of 128
        r.w[f] = a.q2 + p * pieces * 1024;
        r.s[f] = a.s2 + p * 16;
    }
    r.s_stride = a.experts * a.m;
#pragma unroll
    for (int j = 0; j < Rows::XL; ++j) {
        const int i = 4 * j + lane / 16;
        r.x[j] = a.h + (int64_t)list[i < rows ? i : rows - 1] * a.f * 2 + lane % 16 * 8;
    }
    v4f acc[2][1] = {};
    r.template run<false>((int)(wave * pieces / kMoeWaves), (int)((wave + 1) * pieces / kMoeWaves), smem + wave * Rows::LDS, acc);
    v4f s = join_waves<2>(reinterpret_cast<v4f *>(smem), acc, tid % (2 * kWave));
    if (tid < 2 * kWave && tid % 16 < rows) {
        const int pair = list[tid % 16];
        const float w = a.weights[pair];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] *= w;
        *reinterpret_cast<v4f *>(a.part + (int64_t)pair * a.m + (panel0 + tid / kWave) * 16 + tid % kWave / 16 * 4) = s;
    }
}

__global__ __launch_bounds__(kMoeThreads) void moe_down_kernel(MoeArgs a) {
    constexpr int LDS = kMoeWaves * FewRows<BF16, 2, 16, 2, 1>::LDS;
    static_assert(LDS >= kMoeWaves * FewRows<BF16, 2, 4, 2, 2>::LDS && LDS >= kMoeWaves * 2 * 1024, "shared buffer");
    __shared__ __align__(16) uint8_t smem[LDS];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count[kMoeWaves];
    int expert;
    const int n = expert_pairs(a, blockIdx.y, expert, list, count);
    for (int i = 0; i < n; i += 16) {
        const int rows = n - i < 16 ? n - i : 16;
        if (rows <= 4)
            down_tile<4, 2>(a, expert, list + i, rows, smem);
        else
            down_tile<16, 1>(a, expert, list + i, rows, smem);
        __syncthreads();
    }
}

// y = the sum of a token's weighted parts, in the order of its choices, rounded once.
template <class T>
__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs a) {
    const int64_t tok = blockIdx.y, c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (c >= a.m) return;
    v4f s = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.k; ++j) {
        if ((unsigned)a.ids[tok * a.k + j] >= (unsigned)a.experts) continue;
        const v4f o = *reinterpret_cast<const v4f *>(a.part + (tok * a.k + j) * a.m + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += o[e];
    }
    *reinterpret_cast<uint2 *>(a.y + tok * a.m + c) = make_uint2((uint32_t)T::from_f32(s[0]) | (uint32_t)T::from_f32(s[1]) << 16,
                                                                 (uint32_t)T::from_f32(s[2]) | (uint32_t)T::from_f32(s[3]) << 16);
}

hipError_t launch_moe(const MoeArgs &a, hipStream_t stream) {
    const int64_t pairs = a.b * a.k;
    const unsigned slots = (unsigned)(pairs < a.experts ? pairs : a.experts);
    const dim3 up((unsigned)(a.f / 16), slots), down((unsigned)(a.m / 32), slots);
    if (a.bf16)
        moe_up_kernel<BF16><<<up, kMoeThreads, 0, stream>>>(a);
    else
        moe_up_kernel<F16><<<up, kMoeThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    moe_down_kernel<<<down, kMoeThreads, 0, stream>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 join((unsigned)((a.m + 1023) / 1024), (unsigned)a.b);
    if (a.bf16)
        moe_join_kernel<BF16><<<join, 256, 0, stream>>>(a);
    else
        moe_join_kernel<F16><<<join, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace twq
