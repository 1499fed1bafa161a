// checkpoint.hip -- activations kept in 8 bits between forward and backward (gfx950).
//
// Per token row and group of 128 elements: s = fl32(max|x| / 127), q = round-half-even
// (fl32(x / s)); the restored value is s q. It is eq. (1) with k = 8 on groups: an outlier
// channel coarsens its own group only. Both kernels read and write each byte once and are
// bound by memory: 8192 x 14336 takes 82-103 us to keep (357 MB, 3.5-4.4 TB/s) and to restore 56-58 us
// right after (6.3 TB/s, part of it from the last-level cache), 55-64, median 62 (5.8), when five other
// such tensors were kept in between.
#include "twq_adapters.h"
#include "twq_adapters_device.h"

namespace twq {

constexpr int kCkRows = 16, kCkGroups = 8;  // a CTA: 16 token rows x 8 groups

// 16 lanes a group, 16 bytes a lane; 128 threads cover a row's eight groups. All loads are
// issued first, past the end from other rows and groups (under a condition each load would be
// waited for before the next). The scales
// gather in LDS, because a group's scales of consecutive tokens are neighbours in memory.
template <class T>
__global__ __launch_bounds__(256) void checkpoint_kernel(const uint16_t *x, int64_t b, int64_t m, int8_t *qc, float *sc, unsigned ncol) {
    __shared__ float scl[kCkGroups][kCkRows];
    const int tid = threadIdx.x, rhalf = tid / 128, gl = tid % 128 / 16;
    const int64_t row0 = (int64_t)(blockIdx.x / ncol) * kCkRows, grp0 = (int64_t)(blockIdx.x % ncol) * kCkGroups;
    const int64_t ngrp = m / 128, col = grp0 * 128 + tid % 128 * 8;
    const bool on = grp0 + gl < ngrp;
    uint4 v[kCkRows / 2];
#pragma unroll
    for (int j = 0; j < kCkRows / 2; ++j) {
        const int64_t row = row0 + 2 * j + rhalf;
        v[j] = *reinterpret_cast<const uint4 *>(x + (row < b ? row : row0) * m + (on ? col : 0));
    }
#pragma unroll
    for (int j = 0; j < kCkRows / 2; ++j) {
        __builtin_amdgcn_sched_barrier(0);  // one row at a time: fewer registers, more waves
        const int64_t row = row0 + 2 * j + rhalf;
        const uint32_t mx = row16_max(absmax8_bits(v[j], 0));
        const bool finite = mx < (T::kBf16 ? 0x7F80u : 0x7C00u);
        float s;
        {
#pragma clang fp contract(off)
            s = T::to_f32((uint16_t)mx) / kQMax8;
        }
        const float inv = 1.0f / s;
        const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
        uint32_t out[2] = {0, 0};
        // q = rint(x inv) unless that lies within 2^-15 of a half-integer, where the division decides
        // (quant_code8_fast's argument); one rare branch for the eight elements. A subnormal s,
        // whose reciprocal may overflow, always divides.
        float f[8], q[8];
        bool near = s < 0x1p-126f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma clang fp contract(off)
            f[e] = T::to_f32(half_of((int)w[e / 2], e % 2));
            const float t = f[e] * inv;
            q[e] = __builtin_rintf(t);
            near |= __builtin_fabsf(t - q[e]) >= 0.5f - 0x1p-15f;
        }
        if (near && s > 0.f && finite) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                __builtin_amdgcn_sched_barrier(0);
                q[e] = __builtin_fminf(__builtin_fmaxf(__builtin_rintf(f[e] / s), -kQMax8), kQMax8);
            }
        }
        if (s > 0.f && finite) {
#pragma unroll
            for (int e = 0; e < 8; ++e) out[e / 4] |= ((uint32_t)(int)q[e] & 0xFFu) << (8 * (e % 4));
        }
        if (on && row < b) *reinterpret_cast<uint2 *>(qc + row * m + col) = make_uint2(out[0], out[1]);
        if (tid % 16 == 0) scl[gl][2 * j + rhalf] = finite ? s : __builtin_nanf("");
    }
    __syncthreads();
    if (tid < kCkGroups * kCkRows) {
        const int64_t g = grp0 + tid / kCkRows, row = row0 + tid % kCkRows;
        if (g < ngrp && row < b) sc[g * b + row] = scl[tid / kCkRows][tid % kCkRows];
    }
}

hipError_t launch_checkpoint(const uint16_t *x, int64_t b, int64_t m, int bf16, int8_t *qc, float *sc, hipStream_t stream) {
    const unsigned ncol = (unsigned)((m / 128 + kCkGroups - 1) / kCkGroups), grid = (unsigned)((b + kCkRows - 1) / kCkRows) * ncol;
    if (bf16)
        checkpoint_kernel<BF16><<<grid, 256, 0, stream>>>(x, b, m, qc, sc, ncol);
    else
        checkpoint_kernel<F16><<<grid, 256, 0, stream>>>(x, b, m, qc, sc, ncol);
    return hipGetLastError();
}

// The same tile: 8 codes a thread and row.
template <class T>
__global__ __launch_bounds__(256) void restore_kernel(const int8_t *qc, const float *sc, int64_t b, int64_t m, uint16_t *x,
                                                      unsigned ncol) {
    __shared__ float scl[kCkGroups][kCkRows];
    const int tid = threadIdx.x, rhalf = tid / 128, gl = tid % 128 / 16;
    const int64_t row0 = (int64_t)(blockIdx.x / ncol) * kCkRows, grp0 = (int64_t)(blockIdx.x % ncol) * kCkGroups;
    const int64_t ngrp = m / 128, col = grp0 * 128 + tid % 128 * 8;
    const bool on = grp0 + gl < ngrp;
    uint2 v[kCkRows / 2];
#pragma unroll
    for (int j = 0; j < kCkRows / 2; ++j) {
        const int64_t row = row0 + 2 * j + rhalf;
        v[j] = *reinterpret_cast<const uint2 *>(qc + (row < b ? row : row0) * m + (on ? col : 0));
    }
    if (tid < kCkGroups * kCkRows) {
        const int64_t g = grp0 + tid / kCkRows, row = row0 + tid % kCkRows;
        scl[tid / kCkRows][tid % kCkRows] = g < ngrp && row < b ? sc[g * b + row] : 0.f;
    }
    __syncthreads();
    if (!on) return;
#pragma unroll
    for (int j = 0; j < kCkRows / 2; ++j) {
        const int64_t row = row0 + 2 * j + rhalf;
        if (row >= b) break;
        const float s = scl[gl][2 * j + rhalf];
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t p = (e < 2 ? v[j].x : v[j].y) >> (16 * (e % 2));
            const float f0 = s * (float)(int8_t)p, f1 = s * (float)(int8_t)(p >> 8);
            w[e] = (uint32_t)T::from_f32(f0) | (uint32_t)T::from_f32(f1) << 16;
        }
        *reinterpret_cast<uint4 *>(x + row * m + col) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

hipError_t launch_restore(const int8_t *qc, const float *sc, int64_t b, int64_t m, int bf16, uint16_t *x, hipStream_t stream) {
    const unsigned ncol = (unsigned)((m / 128 + kCkGroups - 1) / kCkGroups), grid = (unsigned)((b + kCkRows - 1) / kCkRows) * ncol;
    if (bf16)
        restore_kernel<BF16><<<grid, 256, 0, stream>>>(qc, sc, b, m, x, ncol);
    else
        restore_kernel<F16><<<grid, 256, 0, stream>>>(qc, sc, b, m, x, ncol);
    return hipGetLastError();
}

}  // namespace twq
