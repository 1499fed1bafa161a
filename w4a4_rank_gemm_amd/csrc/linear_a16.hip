// linear_a16.hip -- the packed layer with unquantized 16-bit activations (gfx950).
//
//   y[i][j] = sum_G s_W[G][j] sum_{k in G} x[i][k] q[j][k] + sum_t (sum_k x[i][k] L1[k][t]) L2[t][j]
//
// G: groups of 128 input channels. X is fp16 or bf16 and used as it is; codes are exact in both
// types, so the only roundings are those of the binary32 sums and the output's. T = X L1 comes from
// a launch of its own (the adapters' shrink kernel), in partial sums over K slices.
#include "twq_few_device.h"
#include "twq_moe.h"

namespace twq {

constexpr int kFewWaves = 8;

// acc += T L2 for 16 FM rows and FN panels, this wave's share of the ranks (blocks of 32). T is
// summed over its slices in order and taken as two bf16 parts (16 significant bits), L2 as its
// two exact ones: the four products are T L2 up to 2^-17 of T.
template <int FN, int FM>
__device__ __forceinline__ void few_lowrank(const A16Args &a, int64_t row0, int64_t last, const int64_t (&chan)[FN], int wave,
                                            v4f (&acc)[FN][FM]) {
    const int lane = threadIdx.x % kWave, li = lane & 15, g = lane >> 4;
    for (int rb = wave; rb * 32 < a.r; rb += kFewWaves) {
        const int k = rb * 32 + g * 8, kc = k < a.r ? k : a.r - 8;
        v4i wh[FN], wl[FN];
#pragma unroll
        for (int f = 0; f < FN; ++f) split_f16(load16(a.l2t + (chan[f] + li) * a.r + kc), wh[f], wl[f]);
#pragma unroll
        for (int c = 0; c < FM; ++c) {
            const int64_t row = row0 + c * 16 + li < last ? row0 + c * 16 + li : last - 1;
            const float *p = a.t + row * a.r + kc;
            v4f t0 = sum_slices(p, a.b * a.r, a.ks), t1 = sum_slices(p + 4, a.b * a.r, a.ks);
            v4i th, tl;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v0 = k < a.r ? (e < 2 ? t0[2 * e] : t1[2 * e - 4]) : 0.f;
                const float v1 = k < a.r ? (e < 2 ? t0[2 * e + 1] : t1[2 * e - 3]) : 0.f;
                const uint16_t h0 = BF16::from_f32(v0), h1 = BF16::from_f32(v1);
                th[e] = (int)((uint32_t)h0 | (uint32_t)h1 << 16);
                const uint16_t l0 = BF16::from_f32(v0 - BF16::to_f32(h0)), l1 = BF16::from_f32(v1 - BF16::to_f32(h1));
                tl[e] = (int)((uint32_t)l0 | (uint32_t)l1 << 16);
            }
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

// Few rows: a CTA owns FN panels of 16 channels and up to XR rows; its eight waves split K and
// their sums are added in wave order.
template <class T, int FN, int XR, int U>
__global__ __launch_bounds__(kFewWaves *kWave) void a16_few_kernel(A16Args a) {
    typedef FewRows<T, FN, XR, 1, U> Rows;
    constexpr int FM = Rows::FM, RED = kFewWaves * FN * FM * 1024;
    __shared__ __align__(16) uint8_t smem[kFewWaves * Rows::LDS > RED ? kFewWaves * Rows::LDS : RED];
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int64_t panels = a.n / 16, pieces = a.m / 128, panel0 = (int64_t)blockIdx.x * FN, row0 = (int64_t)blockIdx.y * XR;
    const int64_t last = row0 + XR < a.b ? row0 + XR : a.b;
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
#pragma unroll
    for (int j = 0; j < Rows::XL; ++j) {
        const int64_t row = row0 + 4 * j + lane / 16;
        rows.x[j] = a.x + (row < last ? row : last - 1) * a.m + lane % 16 * 8;
    }
    v4f acc[FN][FM] = {};
    rows.template run<true>((int)(wave * pieces / kFewWaves), (int)((wave + 1) * pieces / kFewWaves), smem + wave * Rows::LDS, acc);
    if (a.r > 0) few_lowrank<FN, FM>(a, row0, last, chan, wave, acc);
    __syncthreads();
    v4f *const red = reinterpret_cast<v4f *>(smem);
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int c = 0; c < FM; ++c) red[((wave * FN + f) * FM + c) * kWave + lane] = acc[f][c];
    __syncthreads();
    for (int t = tid; t < FN * FM * kWave; t += kFewWaves * kWave) {
        v4f s = red[t];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) {
            const v4f o = red[w * FN * FM * kWave + t];
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += o[e];
        }
        const int64_t panel = panel0 + t / kWave / FM, row = row0 + t / kWave % FM * 16 + t % 16;
        if (panel < panels && row < last)
            *reinterpret_cast<uint2 *>(a.y + row * a.n + panel * 16 + t % kWave / 16 * 4) =
                make_uint2((uint32_t)T::from_f32(s[0]) | (uint32_t)T::from_f32(s[1]) << 16,
                           (uint32_t)T::from_f32(s[2]) | (uint32_t)T::from_f32(s[3]) << 16);
    }
}

template <class T, int FN>
static hipError_t a16_few(const A16Args &a, const A16Plan &p, hipStream_t stream) {
    const dim3 grid((unsigned)((a.n / 16 + FN - 1) / FN), (unsigned)((a.b + p.rows - 1) / p.rows));
    constexpr int NT = kFewWaves * kWave;
    if (p.rows == 4)
        a16_few_kernel<T, FN, 4, 4><<<grid, NT, 0, stream>>>(a);
    else if (p.rows == 16)
        a16_few_kernel<T, FN, 16, 2><<<grid, NT, 0, stream>>>(a);
    else if (p.rows == 32)
        a16_few_kernel<T, FN, 32, 1><<<grid, NT, 0, stream>>>(a);
    else
        a16_few_kernel<T, FN, 64, 1><<<grid, NT, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_a16(const A16Args &a, const A16Plan &p, hipStream_t stream) {
    if (p.fn == 1) return a.bf16 ? a16_few<BF16, 1>(a, p, stream) : a16_few<F16, 1>(a, p, stream);
    return a.bf16 ? a16_few<BF16, 2>(a, p, stream) : a16_few<F16, 2>(a, p, stream);
}

}  // namespace twq
