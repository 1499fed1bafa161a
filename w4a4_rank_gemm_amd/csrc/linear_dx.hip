// linear_dx.hip -- the frozen layer's input gradient (gfx950).
//
//   dX = dY W^T,  W^T = diag(s_W) Q_W + L2 L1 (as [n][m]):
//   dX[i][k] = sum_j dY[i][j] s_W[j] Q_W[j][k] + sum_t (sum_j dY[i][j] L2[t][j]) L1[k][t]
//
// The long sum runs over the output channels j, the slow axis of the packed weight. Packed
// 4-bit codes go to LDS as they lie (a 16-channel panel piece is 16 rows of K) and are read
// transposed as nibbles: a lane gets 16 channels of one input column in 8 bytes, which are
// expanded to fp16 in registers. Codes are exact in fp16; the per-channel scale is folded into dY by a
// first kernel, G[i][j] = fp16(dY[i][j] s_W[j] 2^-e_i) with a power of two per token that brings the
// row's largest element to [2^14, 2^15) (from 2^-112 up; a smaller row is scaled by 2^126): one
// rounding, and no gradient too small or too large for fp16. Elements below 2^-28 of the row's largest
// are subnormal there and off by up to 2^-39 of the largest; a T below 2^-40 of G is off by up to
// 2^-79 of G's largest. In an fp16 dX that rounding weighs as much as the output's own (the 2-norm off
// by 2.9e-4 instead of 2.1e-4 where the low-rank part is small), in a bf16 one nothing. It is the
// error of a weight dequantized to fp16 (code times scale rounded to 11 bits); a second part of G
// would double the matrix work. T = dY L2 (the adapters' shrink kernel) is held in binary32, then in
// two fp16 parts, and joins the same accumulator after the long sum.
// Together: 4096 tokens, 8192 x 28672, 128 ranks 1.67-1.76 ms (1963 GFLOP, 1.1-1.2
// PFLOP/s; a library fp16 product of 8192^3 runs at 1.33); 2048 tokens, 4096 x 14336, 32 ranks 242-254 us.
#include <utility>

#include "twq_adapters.h"
#include "twq_adapters_device.h"

namespace twq {

constexpr int kDxStages = 3;

// ---- G and T in fp16 -------------------------------------------------------------------

// The largest |dY s_W| of each row (without a low-rank pair; otherwise the shrink kernel finds
// it while it reads dY). One CTA a row, 2^23 along a grid dimension (it holds fewer than 2^32
// threads).
template <class T>
__global__ __launch_bounds__(256) void dx_max_kernel(DxArgs a) {
    __shared__ uint32_t red[4];
    const int tid = threadIdx.x;
    const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (row >= a.b) return;
    uint32_t mx = 0;
    for (int64_t c = tid * 8; c < a.n; c += 2048) {
        const v4i v = load16(a.dy + row * a.n + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float f = T::to_f32(half_of(v[e / 2], e % 2)) * a.sw[c + e];
            const uint32_t m = __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu;
            mx = mx > m ? mx : m;
        }
    }
    mx = wave_max_u32(mx);
    if (tid % kWave == 0) red[tid / kWave] = mx;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < 4; ++w) mx = mx > red[w] ? mx : red[w];
        a.rowmax[row] = __builtin_bit_cast(float, mx);
    }
}

hipError_t launch_dx_max(const DxArgs &a, hipStream_t stream) {
    const int64_t most = int64_t(1) << 23;
    const dim3 grid((unsigned)(a.b < most ? a.b : most), (unsigned)((a.b + most - 1) / most));
    if (a.bf16)
        dx_max_kernel<BF16><<<grid, 256, 0, stream>>>(a);
    else
        dx_max_kernel<F16><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

constexpr int kScaleRows = 16, kScaleCols = 2048;

// Exponent of a row of G, from the largest |dY s_W| of its slices (at most 16): lane q of the
// row's 16 reads slice q, so that the slices are not waited for one after the other
// (b=16, 4096 x 14336, 16 slices here and in t_parts: 37 to 29 us for the whole call).
__device__ __forceinline__ int g_exponent(const DxArgs &a, int64_t row, int q) {
    const uint32_t m = __builtin_bit_cast(uint32_t, a.rowmax[(q < a.rks ? q : a.rks - 1) * a.b + row]);
    return scale_exponent(__builtin_bit_cast(float, row16_max(m)));  // magnitudes: ordered as integers, NaN last
}

// T = dY L2 of 16 rows, 16 threads a row: the slices' sum, its largest magnitude, two fp16 parts.
__device__ __forceinline__ void t_parts(const DxArgs &a, int64_t row0, int nrows) {
    const int i = threadIdx.x / 16, q = threadIdx.x % 16, r32 = (a.r + 31) / 32 * 32;
    const int64_t row = row0 + (i < nrows ? i : 0);
    float t[16], mx = 0.f;  // ranks q, q + 16, ..
#pragma unroll
    for (int u = 0; u < 16; ++u) t[u] = 0.f;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        if (u * 16 >= a.r) continue;
        for (int s = 0; s < a.tks; s += 8) {  // eight slices in flight
            float p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = a.t[((s + j < a.tks ? s + j : s) * a.b + row) * a.r + u * 16 + q];
#pragma unroll
            for (int j = 0; j < 8; ++j) t[u] += s + j < a.tks ? p[j] : 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < 16; ++u) mx = __builtin_fmaxf(mx, __builtin_fabsf(t[u]));
    for (int off = 8; off > 0; off >>= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, off, kWave));
    const int ge = g_exponent(a, row, q);
    // the two exponents meet in one accumulator: far below G, T keeps fewer bits (a G of zeros has
    // the least exponent, and T its own)
    int te = mx > 0.f ? scale_exponent(mx) : ge;
    te = te < ge - 40 ? ge - 40 : te;
    if (i >= nrows) return;
#pragma unroll
    for (int u = 0; u < 16; ++u)
        if (u * 16 < r32) {  // r is a multiple of 16: the last half step is zero
            const float f = t[u] * pow2(14 - te);
            const uint16_t hi = F16::from_f32(f), lo = F16::from_f32(f - F16::to_f32(hi));
            const int k = u * 16 + q;
            uint16_t *p = a.t16 + (row * r32 + k / 8 * 8) * 2 + k % 8;
            p[0] = hi;
            p[8] = lo;
        }
    if (q == 0) {
        a.ge[row * 2] = ge - 14;
        a.ge[row * 2 + 1] = te - 14;
    }
}

// 16 token rows x 2048 channels a CTA, eight channels a thread with their scales in
// registers; bound by the read of dY and the write of G (4096 x 28672: 470 MB in 80 us, 5.9
// TB/s, part of dY from the last-level cache after the shrink's read). Eight consecutive channels are stored
// in the order 0 4 1 5 2 6 3 7, in which expanded codes come (dequant8). One more CTA per 16
// rows brings T to fp16 and stores the exponents.
template <class T>
__global__ __launch_bounds__(256) void dx_scale_kernel(DxArgs a, int64_t npad) {
    __shared__ int exps[kScaleRows];
    const int tid = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * kScaleRows;
    const int nrows = (int)(a.b - row0 < kScaleRows ? a.b - row0 : kScaleRows);
    if (blockIdx.y + 1 == gridDim.y) return t_parts(a, row0, nrows);
    const int64_t c = (int64_t)blockIdx.y * kScaleCols + tid * 8;
    const bool on = c < a.n;
    v4i v[kScaleRows];
#pragma unroll
    for (int i = 0; i < kScaleRows; ++i) v[i] = load16(a.dy + (row0 + (i < nrows ? i : 0)) * a.n + (on ? c : 0));
    const float *swp = a.sw + (on ? c : 0);
    const v4f s0 = *reinterpret_cast<const v4f *>(swp), s1 = *reinterpret_cast<const v4f *>(swp + 4);
    const int ge = g_exponent(a, row0 + (tid / 16 < nrows ? tid / 16 : 0), tid % 16);
    if (tid % 16 == 0) exps[tid / 16] = ge;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kScaleRows; ++i) {
        const float gf = pow2(14 - exps[i]);
        v4i o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint16_t f0 = F16::from_f32(T::to_f32(half_of(v[i][e / 2], e % 2)) * s0[e] * gf);
            const uint16_t f1 = F16::from_f32(T::to_f32(half_of(v[i][(e + 4) / 2], e % 2)) * s1[e] * gf);
            o[e] = (int)((uint32_t)f0 | (uint32_t)f1 << 16);
        }
        if (i < nrows && c < npad) *reinterpret_cast<v4i *>(a.g + (row0 + i) * npad + c) = on ? o : v4i{0, 0, 0, 0};
    }
}

hipError_t launch_dx_scale(const DxArgs &a, const DxPlan &p, hipStream_t stream) {
    const dim3 grid((unsigned)((a.b + kScaleRows - 1) / kScaleRows), (unsigned)((p.npad + kScaleCols - 1) / kScaleCols + 1));
    if (a.bf16)
        dx_scale_kernel<BF16><<<grid, 256, 0, stream>>>(a, p.npad);
    else
        dx_scale_kernel<F16><<<grid, 256, 0, stream>>>(a, p.npad);
    return hipGetLastError();
}

// ---- main kernel -----------------------------------------------------------------------

// One pair of panels (32 channels): the codes of two 32-column blocks (addresses w0, w1) and
// the two operands of each of TB 32-token blocks (addresses g0, g1), completed before
// returning (one statement, so that no other in-flight direct-to-LDS load is waited for).
template <int TB, int WOFF, int GOFF>
__device__ __forceinline__ void dx_read(uint32_t w0, uint32_t w1, uint32_t g0, uint32_t g1, v2i (&w)[2], v4i (&r)[2 * TB]) {
    static_assert(TB == 1 || TB == 2 || TB == 4, "token blocks");
    if constexpr (TB == 4)
        asm volatile(
            "ds_read_b64_tr_b4 %0, %10 offset:%14\n\t"
            "ds_read_b64_tr_b4 %1, %11 offset:%14\n\t"
            "ds_read_b128 %2, %12 offset:%15\n\t"
            "ds_read_b128 %3, %13 offset:%15\n\t"
            "ds_read_b128 %4, %12 offset:%16\n\t"
            "ds_read_b128 %5, %13 offset:%16\n\t"
            "ds_read_b128 %6, %12 offset:%17\n\t"
            "ds_read_b128 %7, %13 offset:%17\n\t"
            "ds_read_b128 %8, %12 offset:%18\n\t"
            "ds_read_b128 %9, %13 offset:%18\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(w[0]), "=&v"(w[1]), "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]),
              "=&v"(r[6]), "=&v"(r[7])
            : "v"(w0), "v"(w1), "v"(g0), "v"(g1), "n"(WOFF), "n"(GOFF), "n"(GOFF + 4096), "n"(GOFF + 8192), "n"(GOFF + 12288)
            : "memory");
    else if constexpr (TB == 2)
        asm volatile(
            "ds_read_b64_tr_b4 %0, %6 offset:%10\n\t"
            "ds_read_b64_tr_b4 %1, %7 offset:%10\n\t"
            "ds_read_b128 %2, %8 offset:%11\n\t"
            "ds_read_b128 %3, %9 offset:%11\n\t"
            "ds_read_b128 %4, %8 offset:%12\n\t"
            "ds_read_b128 %5, %9 offset:%12\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(w[0]), "=&v"(w[1]), "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
            : "v"(w0), "v"(w1), "v"(g0), "v"(g1), "n"(WOFF), "n"(GOFF), "n"(GOFF + 4096)
            : "memory");
    else
        asm volatile(
            "ds_read_b64_tr_b4 %0, %4 offset:%8\n\t"
            "ds_read_b64_tr_b4 %1, %5 offset:%8\n\t"
            "ds_read_b128 %2, %6 offset:%9\n\t"
            "ds_read_b128 %3, %7 offset:%9\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(w[0]), "=&v"(w[1]), "=&v"(r[0]), "=&v"(r[1])
            : "v"(w0), "v"(w1), "v"(g0), "v"(g1), "n"(WOFF), "n"(GOFF)
            : "memory");
}

// The low-rank term and the stores of TB token blocks of a wave, its sums in acc: lane holds
// token lane % 32 of each block, columns 8 (v / 4) + 4 half + v % 4. All NT threads of the CTA
// call it (L1 goes through their LDS).
template <class T, int TB, int NT>
__device__ __forceinline__ void dx_finish(const DxArgs &a, v16f (&acc)[2][TB], uint8_t *ring, int64_t tok0, int64_t m0,
                                          int64_t slice, int wave) {
    const int tid = threadIdx.x, lane = tid % kWave, li = lane & 15, half = lane >> 5;
    float fin[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        const int64_t tok = tok0 + t * 32 + lane % 32, tc = tok < a.b ? tok : a.b - 1;
        int e = a.ge[tc * 2];
        if (a.r > 0 && slice == 0) {
            const int te = a.ge[tc * 2 + 1], d = e - te;
            const float f = pow2(d < -126 ? -126 : d > 127 ? 127 : d);
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[q][t][v] *= f;
            e = te;
        }
        fin[t] = pow2(e);
    }
    if (a.r > 0 && slice == 0) {
        const int r32 = (a.r + 31) / 32 * 32;
        uint16_t *const l1 = reinterpret_cast<uint16_t *>(ring);  // [32 ranks][256 columns]
        for (int k0 = 0; k0 < a.r; k0 += 32) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 1024 / NT; ++j) {
                const int c = j * NT + tid, k = k0 + c / 32;
                const int64_t col = m0 + c % 32 * 8;
                *reinterpret_cast<v4i *>(l1 + c * 8) =
                    load16(a.l1t + (int64_t)(k < a.r ? k : a.r - 1) * a.m + (col < a.m ? col : a.m - 8));
            }
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // ranks 16 h + 8 half .. + 7
                v4i wf[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint16_t *p = l1 + (h * 16 + half * 8 + li / 4) * 256 + wave * 64 + q * 32 + ((lane >> 4) & 1) * 16 + (li % 4) * 4;
                    const v4s p0 = read_tr16(p), p1 = read_tr16(p + 4 * 256);
                    wf[q] = join(p0, p1);
                }
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    const int64_t tok = tok0 + t * 32 + lane % 32, tc = tok < a.b ? tok : a.b - 1;
                    const uint16_t *tp = a.t16 + (tc * r32 + k0 + h * 16 + half * 8) * 2;
                    const v4i hi = load16(tp), lo = load16(tp + 8);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        acc[q][t] = mfma_f16_32(__builtin_bit_cast(v8h, wf[q]), __builtin_bit_cast(v8h, lo), acc[q][t]);
                        acc[q][t] = mfma_f16_32(__builtin_bit_cast(v8h, wf[q]), __builtin_bit_cast(v8h, hi), acc[q][t]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        const int64_t tok = tok0 + t * 32 + lane % 32;
        if (tok >= a.b) continue;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int64_t col = m0 + wave * 64 + q * 32 + v * 8 + half * 4;
                if (col >= a.m) continue;
                v4f o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = acc[q][t][v * 4 + e] * fin[t];
                if (a.ks > 1)
                    *reinterpret_cast<v4f *>(a.part + (slice * a.b + tok) * a.m + col) = o;
                else
                    *reinterpret_cast<uint2 *>(a.dx + tok * a.m + col) =
                        make_uint2((uint32_t)T::from_f32(o[0]) | (uint32_t)T::from_f32(o[1]) << 16,
                                   (uint32_t)T::from_f32(o[2]) | (uint32_t)T::from_f32(o[3]) << 16);
            }
    }
}

// A CTA owns 32 TB tokens x 256 input columns over a slice of the channels; its four waves
// take 64 columns each and share the tokens' operands. A stage of 64 channels is 8 KB of
// codes and 4 TB KB of G, by direct-to-LDS loads into a ring of three stages (two in
// flight). G rows are 128-byte lines with the 16-byte chunk index XORed by row % 8 and by
// (row / 16) % 2 (one 16-byte read serves lanes 0-7 with 16-23 in a pass), code rows 64 bytes
// with the chunk XORed by (row / 4) % 4. No bank conflicts to speak of (0.6% of LDS cycles).
//
// Bound by the matrix cores and the expansion of the codes, whose cycles add up (a wave waits for
// its LDS reads before its matrix instructions, with two waves a SIMD to fill in): 4096 tokens, 8192 x
// 28672: 1.54-1.70 ms, matrix cores busy 1.85 of the kernel's 2.80 million cycles, 0.70 of those in which
// their compute unit is. 2048 tokens, 4096 x 14336: 207-262 us, medians of runs 210 to 250; 0.60.
//
// KG = 2: eight waves in two groups, each with its own ring and half of the channels; their
// sums meet in LDS. That fills a compute unit with one CTA where the tiles are too few for two,
// without sums in memory and a launch to join them (b=2048, 4096 x 14336: 271 to 261 us).
template <class T, int TB, int KG>
__global__ __launch_bounds__(256 * KG, 2 / KG) void dx_kernel(DxArgs a, int64_t npad, int64_t mtiles) {
    constexpr int BT = 32 * TB, WBYTES = kDxK / 16 * 2048, GBYTES = BT * 128, STAGE = WBYTES + GBYTES;
    constexpr int GL = GBYTES / 4096, LOADS = 2 + GL;  // direct-to-LDS loads of a wave per stage
    constexpr int RING = kDxStages * STAGE;
    __shared__ __align__(1024) uint8_t ring_lds[KG * RING];
    const int tid = threadIdx.x, lane = tid % kWave, wave_id = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wave = wave_id % 4, grp = KG == 1 ? 0 : wave_id / 4;
    uint8_t *const ring = ring_lds + grp * RING;
    const int li = lane & 15, half = lane >> 5;
    const int64_t mt = blockIdx.x % mtiles, tt = blockIdx.x / mtiles, slice = blockIdx.y;
    const int64_t tok0 = tt * BT, m0 = mt * kDxM, pieces = a.m / 128, panels = a.n / 16;
    const int64_t nst = npad / kDxK, parts = (int64_t)a.ks * KG, part = slice * KG + grp;
    const int64_t s0 = part * nst / parts, s1 = (part + 1) * nst / parts;

    // direct-to-LDS: lane l of a 1 KB block fetches row l / 8, chunk (l % 8) ^ row ^ (block / 2) of G (8
    // rows), or row l / 4, chunk (l % 4) ^ (row / 4) of a panel piece (16 rows)
    uint32_t goff[GL];
#pragma unroll
    for (int j = 0; j < GL; ++j) {
        const int64_t row = (j * 4 + wave) * 8 + lane / 8, rel = tok0 + row < a.b ? row : a.b - 1 - tok0;
        goff[j] = (uint32_t)(rel * npad * 2 + ((lane % 8) ^ (lane / 8) ^ ((j * 4 + wave) / 2 % 2)) * 16);
    }
    const uint32_t woff = (lane / 4) * 64 + ((lane % 4) ^ (lane / 16)) * 16;
    const uint8_t *gbase = reinterpret_cast<const uint8_t *>(a.g + tok0 * npad);
    auto issue = [&](int64_t st, int slot) {
        uint8_t *dst = ring + slot * STAGE;
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // eight pieces a stage, two a wave
            const int p = wave, pc = j;
            const int64_t panel = st * 4 + p < panels ? st * 4 + p : panels - 1;  // past n: G is zero
            const int64_t piece = m0 / 128 + pc < pieces ? m0 / 128 + pc : pieces - 1;
            const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint8_t *>(a.qw + (panel * pieces + piece) * 1024), 0, 1024, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (__attribute__((address_space(3))) void *)(dst + (p * 2 + pc) * 1024), 16,
                                                     (int)woff, 0, 0, 0);
        }
        const __amdgpu_buffer_rsrc_t rg =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(gbase + st * kDxK * 2), 0, 0x7fffffff, 0x00020000);
#pragma unroll
        for (int j = 0; j < GL; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rg, (__attribute__((address_space(3))) void *)(dst + WBYTES + (j * 4 + wave) * 1024), 16, (int)goff[j], 0, 0, 0);
    };

    const DequantConst dq = dequant_const();
    v16f acc[2][TB];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[q][t][e] = 0.f;

    // read addresses: codes of column block q: panel 2 pair + half, this wave's piece, row li,
    // chunk 2 (wave % 2) + q; G: token lane % 32, chunk 4 pair + 2 half + h
    const uint32_t ring0 = lds_offset(ring);
    uint32_t wa[2], ga[2][2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
        wa[q] = ring0 + (half * 2 + wave / 2) * 1024 + li * 64 + (((wave % 2) * 2 + q) ^ (li / 4)) * 16 + ((lane >> 4) & 1) * 8;
#pragma unroll
    for (int pr = 0; pr < 2; ++pr)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            ga[pr][h] = ring0 + WBYTES + (lane % 32) * 128 + ((pr * 4 + half * 2 + h) ^ (lane % 8) ^ (lane / 16 % 2)) * 16;

    const int64_t n_st = s1 - s0, rounds = KG == 1 ? n_st : (nst + parts - 1) / parts;  // the groups meet at barriers
    if (n_st > 0) issue(s0, 0);
    if (n_st > 1) issue(s0 + 1, 1);
    for (int64_t c0 = 0; c0 < rounds; c0 += kDxStages) {
        static_for(std::make_integer_sequence<int, kDxStages>{}, [&](auto u) {
            constexpr int U = decltype(u)::value, OFF = U * STAGE;
            const int64_t c = c0 + U;
            if (c >= rounds) return;
            if (c + 1 < n_st)
                wait_vmcnt<LOADS>();
            else
                wait_vmcnt<0>();
            stage_barrier();  // stage c has landed for every wave, and stage c - 1 is read
            if (KG > 1 && c >= n_st) return;
            if (c + 2 < n_st) issue(s0 + c + 2, (U + 2) % kDxStages);
            static_for(std::make_integer_sequence<int, 2>{}, [&](auto pv) {
                constexpr int PR = decltype(pv)::value;
                v2i w[2];
                v4i r[2 * TB];
                dx_read<TB, OFF + PR * 4096, OFF>(wa[0], wa[1], ga[PR][0], ga[PR][1], w, r);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const v8h wf = __builtin_bit_cast(v8h, dequant8((uint32_t)w[q][h], dq));
#pragma unroll
                        for (int t = 0; t < TB; ++t) acc[q][t] = mfma_f16_32(wf, __builtin_bit_cast(v8h, r[2 * t + h]), acc[q][t]);
                    }
            });
        });
    }

    if constexpr (KG == 2) {
        // group 0 finishes the first half of the token blocks, group 1 the second: each puts its
        // sums of the other's half in LDS, [4 waves][2 column blocks][TB / 2][4][64 lanes] a group
        constexpr int H = TB / 2;
        v4f *const swap = reinterpret_cast<v4f *>(ring_lds);
        auto slot = [&](int g, int q, int t, int v) { return swap + (((g * 4 + wave) * 2 + q) * H + t) * 4 * kWave + v * kWave + lane; };
        auto put = [&](auto first) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int t = 0; t < H; ++t)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const v16f &s = acc[q][decltype(first)::value + t];
                        *slot(grp, q, t, v) = v4f{s[4 * v], s[4 * v + 1], s[4 * v + 2], s[4 * v + 3]};
                    }
        };
        __syncthreads();  // every wave is done with the rings
        if (grp == 0)
            put(std::integral_constant<int, H>{});
        else
            put(std::integral_constant<int, 0>{});
        __syncthreads();
        v16f fold[2][H];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int t = 0; t < H; ++t)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const v4f o = *slot(1 - grp, q, t, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e)  // group 0's sum first, whichever group adds
                        fold[q][t][4 * v + e] = (grp == 0 ? acc[q][t][4 * v + e] : o[e]) + (grp == 0 ? o[e] : acc[q][H + t][4 * v + e]);
                }
        dx_finish<T, H, 512>(a, fold, ring_lds, tok0 + grp * H * 32, m0, slice, wave);
    } else {
        dx_finish<T, TB, 256>(a, acc, ring_lds, tok0, m0, slice, wave);
    }
}

// dX = the slices' sums in slice order, rounded once.
template <class T>
__global__ __launch_bounds__(256) void dx_join_kernel(const float *part, int ks, int64_t total, uint16_t *dx) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= total) return;
    const v4f s = sum_slices(part + at, total, ks);
    *reinterpret_cast<uint2 *>(dx + at) = make_uint2((uint32_t)T::from_f32(s[0]) | (uint32_t)T::from_f32(s[1]) << 16,
                                                     (uint32_t)T::from_f32(s[2]) | (uint32_t)T::from_f32(s[3]) << 16);
}

template <class T>
static hipError_t dx_typed(const DxArgs &a, const DxPlan &p, hipStream_t stream) {
    const int64_t mtiles = (a.m + kDxM - 1) / kDxM;
    const dim3 grid((unsigned)(mtiles * ((a.b + p.bt - 1) / p.bt)), (unsigned)p.ks);
    if (p.bt == 32)
        dx_kernel<T, 1, 1><<<grid, 256, 0, stream>>>(a, p.npad, mtiles);
    else if (p.bt == 64)
        dx_kernel<T, 2, 1><<<grid, 256, 0, stream>>>(a, p.npad, mtiles);
    else if (p.kg == 1)
        dx_kernel<T, 4, 1><<<grid, 256, 0, stream>>>(a, p.npad, mtiles);
    else
        dx_kernel<T, 4, 2><<<grid, 512, 0, stream>>>(a, p.npad, mtiles);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.ks == 1) return e;
    const int64_t total = a.b * a.m;
    dx_join_kernel<T><<<dim3((unsigned)((total / 4 + 255) / 256)), 256, 0, stream>>>(a.part, p.ks, total, a.dx);
    return hipGetLastError();
}

hipError_t launch_dx(const DxArgs &a, const DxPlan &p, hipStream_t stream) {
    return a.bf16 ? dx_typed<BF16>(a, p, stream) : dx_typed<F16>(a, p, stream);
}

}  // namespace twq
