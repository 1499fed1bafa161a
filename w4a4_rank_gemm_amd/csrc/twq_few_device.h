// twq_few_device.h -- the product of a few 16-bit rows with packed 4-bit weights of group-wise
// scales, one wave's share of it (gfx950): the layer with 16-bit activations for few tokens
// and the experts of the routed layer.
#pragma once

#include "twq_adapters_device.h"

namespace twq {

// The packed codes as matrix operands of a 16-bit type. Eight codes of one dword become four
// pairs, in an order that `order` gives eight elements of a row too; the operand's values are
// the codes times kTimes.
template <class T>
struct Codes;

template <>
struct Codes<F16> {  // pairs (0, 4), (1, 5), (2, 6), (3, 7)
    static constexpr float kTimes = 1.f;
    DequantConst c = dequant_const();
    __device__ __forceinline__ v4i operator()(uint32_t d) const { return dequant8(d, c); }
    static __device__ __forceinline__ v4i order(v4i x) {
        return v4i{(int)__builtin_amdgcn_perm((uint32_t)x[2], (uint32_t)x[0], 0x05040100u),
                   (int)__builtin_amdgcn_perm((uint32_t)x[2], (uint32_t)x[0], 0x07060302u),
                   (int)__builtin_amdgcn_perm((uint32_t)x[3], (uint32_t)x[1], 0x05040100u),
                   (int)__builtin_amdgcn_perm((uint32_t)x[3], (uint32_t)x[1], 0x07060302u)};
    }
};

// bf16 has no packed arithmetic here: a nibble at the top of a byte is an int8 of 16 times the
// code, which converts to binary32 exactly and lies in its upper 16 bits.
template <>
struct Codes<BF16> {  // pairs (0, 1), (2, 3), ..
    static constexpr float kTimes = 16.f;
    __device__ __forceinline__ v4i operator()(uint32_t d) const {
        const uint32_t even = (d << 4) & 0xF0F0F0F0u, odd = d & 0xF0F0F0F0u;
        v4i r;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t lo = __builtin_bit_cast(uint32_t, (float)(int8_t)(even >> (8 * t)));
            const uint32_t hi = __builtin_bit_cast(uint32_t, (float)(int8_t)(odd >> (8 * t)));
            r[t] = (int)__builtin_amdgcn_perm(hi, lo, 0x07060302u);
        }
        return r;
    }
    static __device__ __forceinline__ v4i order(v4i x) { return x; }
};

// LDS written by this wave is read by its other lanes: LDS operations of a wave stay in order,
// the compiler has to keep them so.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Zeros that stay in registers, as the first addend of a chain of matrix instructions: a constant
// would be moved into each chain's result first.
__device__ __forceinline__ v4f held_zero() {
    v4f z = {0.f, 0.f, 0.f, 0.f};
    asm("" : "+v"(z));
    return z;
}

// LDS holds a piece of 16 or more rows as 16 slots, one for each (instruction d, quarter g), with 16
// bytes a row; within 16 rows a row's place is XORed with this, and a step of d has 16 bytes more. A
// 16-byte access serves 16 lanes in one pass, 0-3, 12-15, 20-23, 24-27 or 4-11, 16-19, 28-31 of each
// half: reading, those are the 16 rows of two neighbouring quarters, in 16 different places. Neither
// reads nor writes conflict (slots of 16 bytes more instead: half of the LDS cycles; 64 x 4096 -> 14336 20.4
// and 19.5 us, 61 x 14336 -> 4096 21.7 and 20.9).
__device__ __forceinline__ int row_turn(int g) { return ((g ^ g >> 1) & 1) << 2 | (g & 1) << 3; }

// One wave's share of Y = X W^T for up to XR rows and FN panels of 16 channels: pieces (groups
// of 128 elements of K) p0 .. p1 - 1, U in flight at a time. For each piece
//
//   acc[f][c] += s_W[piece][channel] (codes of the piece, panel f) . (rows 16 c .. 16 c + 15)
//
// on 16 x 16 x 32 matrix instructions: the product of one group is exact up to binary32 sums,
// its scale multiplies the sum. A piece of a panel is 1 KB of contiguous memory, one 16-byte
// load a lane, and goes to the matrix operands without LDS: lane (channel li, quarter g) holds
// codes 32 g .. 32 g + 31, eight for each of four instructions. Rows are read along K (16 lanes a
// row's piece) and turned through the wave's own LDS, so no wave waits for another; a piece's
// scales too. PARTS = 2: a row's piece is 128 upper and then 128 lower parts of its elements, and
// both take part in the sum.
// acc: lane (li, g) holds row 16 c + li, channels 4 g .. 4 g + 3 of panel f.
template <class T, int FN, int XR, int PARTS, int U>
struct FewRows {
    static_assert(XR % 4 == 0 && U <= 4, "rows in fours; a batch's scales are one load");
    static constexpr int FM = (XR + 15) / 16;
    static constexpr int XL = XR / 4;                 // row loads of a piece and part
    static constexpr int SLOT = XR * 16 + (XR < 16 ? 16 : 0);  // of one instruction and quarter
    static constexpr int STEP = 4 * SLOT + (XR < 16 ? 0 : 16), PIECE = PARTS * 4 * STEP;
    static constexpr int LDS = U * PIECE + FN * 256;  // bytes of a wave

    // Pointers are the same in all lanes, and lanes add 32-bit offsets, so that a piece's addresses
    // cost no vector instructions.
    const uint8_t *w[FN];      // this wave's panels, at piece 0
    const float *s[FN];        // scales of the panels' first channels, group 0
    int64_t s_stride;          // floats between groups
    const uint16_t *x;         // rows
    uint32_t row[XL];          // bytes to this lane's rows 4 j + lane / 16 (rows lie within 4 GB)

    // `between` runs after the first loads are issued.
    template <class F>
    __device__ __forceinline__ void run(int p0, int p1, uint8_t *lds, v4f (&acc)[FN][FM], F &&between) const {
        const int lane = threadIdx.x % kWave, li = lane & 15, g = lane >> 4;
        const Codes<T> codes;
        const v4f zero = held_zero();
        v4i wn[U][FN], xn[U][PARTS][XL];
        float sn[FN];
        const uint32_t woff = li * 64 + g * 16, soff = li * 4;
        uint32_t xoff[XL];
#pragma unroll
        for (int j = 0; j < XL; ++j) xoff[j] = row[j] + li * 16;
        const int64_t s_step = s_stride * 4;
        auto load = [&](int p) {  // pieces past the last are read again and scaled by zero
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t q = p + u < p1 ? p + u : p1 - 1;
#pragma unroll
                for (int f = 0; f < FN; ++f) {
                    const uint8_t *const a = w[f] + q * 1024;
                    wn[u][f] = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(a + woff));
                }
#pragma unroll
                for (int h = 0; h < PARTS; ++h)
#pragma unroll
                    for (int j = 0; j < XL; ++j) xn[u][h][j] = load16(reinterpret_cast<const uint8_t *>(x) + (q * PARTS + h) * 256 + xoff[j]);
            }
            const uint32_t q = (U == 1 ? 0 : p + g < p1 ? g : p1 - 1 - p) * (uint32_t)s_step;  // U neighbouring groups
#pragma unroll
            for (int f = 0; f < FN; ++f)
                sn[f] = *reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(s[f]) + p * s_step + (q + soff));
        };
        if (p0 >= p1) return between();
        load(p0);
        between();
        float *const scales = reinterpret_cast<float *>(lds + U * PIECE);
        int put[XL];
#pragma unroll
        for (int j = 0; j < XL; ++j) {
            const int d = lane & 3, q = lane >> 2 & 3;  // chunk lane % 16 = 4 quarter + instruction
            put[j] = d * STEP + q * SLOT + ((j * 4 + g) ^ (XR < 16 ? 0 : row_turn(q))) * 16;
        }
        const int get = g * SLOT + (XR < 16 ? li < XR ? li : XR - 1 : li ^ row_turn(g)) * 16;
        for (int p = p0; p < p1; p += U) {
            v4i wc[U][FN];
            wave_fence();
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int f = 0; f < FN; ++f) wc[u][f] = wn[u][f];
#pragma unroll
                for (int h = 0; h < PARTS; ++h)
#pragma unroll
                    for (int j = 0; j < XL; ++j)
                        *reinterpret_cast<v4i *>(lds + u * PIECE + h * 4 * STEP + put[j]) = Codes<T>::order(xn[u][h][j]);
            }
#pragma unroll
            for (int f = 0; f < FN; ++f) scales[f * 64 + lane] = p + g < p1 ? sn[f] * (1.f / Codes<T>::kTimes) : 0.f;
            if (p + U < p1) load(p + U);
            wave_fence();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v4f t[FN][FM];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    v4i xf[PARTS][FM];
#pragma unroll
                    for (int h = 0; h < PARTS; ++h)
#pragma unroll
                        for (int c = 0; c < FM; ++c)
                            xf[h][c] = load16(lds + u * PIECE + (h * 4 + d) * STEP + get + c * 256);
#pragma unroll
                    for (int f = 0; f < FN; ++f) {
                        const v4i wf = codes((uint32_t)wc[u][f][d]);
#pragma unroll
                        for (int c = 0; c < FM; ++c)
#pragma unroll
                            for (int h = 0; h < PARTS; ++h)
                                t[f][c] = T::mfma(wf, xf[h][c], h == 0 && d == 0 ? zero : t[f][c]);
                    }
                }
#pragma unroll
                for (int f = 0; f < FN; ++f) {
                    const v4f sc = *reinterpret_cast<const v4f *>(scales + f * 64 + u * 16 + g * 4);
#pragma unroll
                    for (int c = 0; c < FM; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[f][c][e] += sc[e] * t[f][c][e];
                }
            }
        }
        wave_fence();
    }
};

// The same product for the eight waves of a CTA that own neighbouring panel groups and share rows
// and K: the rows' pieces p0 .. p1 - 1 go through LDS once for all of them, U at a time into one of
// two buffers, with one barrier a step. All waves call it with the same pieces. KG neighbouring waves
// own the same FN panels and take U / KG pieces of a step each (join_waves adds their sums).
constexpr int kSharedWaves = 8;

template <class T, int FN, int XR, int PARTS, int U, int KG>
struct SharedRows {
    static_assert(XR % 16 == 0 && U <= 4 && U % KG == 0, "a batch's scales are one load");
    static constexpr int UW = U / KG;  // pieces of a step that are this wave's
    static constexpr int NT = kSharedWaves * kWave, FM = XR / 16;
    static constexpr int CHUNKS = U * PARTS * XR * 16, PER = CHUNKS / NT;  // 16-byte chunks of a step, and a thread's
    static_assert(CHUNKS % NT == 0, "every thread loads the same number of chunks");
    static constexpr int SLOT = XR * 16, STEP = 4 * SLOT + 16, PIECE = PARTS * 4 * STEP;
    static constexpr int LDS = 2 * U * PIECE + kSharedWaves * FN * 256;

    const uint8_t *w[FN];    // this wave's panels, at piece 0
    const float *s[FN];      // scales of the panels' first channels, group 0
    int64_t s_stride;        // floats between groups
    const uint16_t *x;       // rows
    uint32_t row[PER];       // bytes to row row_of(j) (rows lie within 4 GB)

    // Row of this thread's chunk j.
    static __device__ __forceinline__ int row_of(int j) { return (j * NT + (int)threadIdx.x) / 16 % XR; }

    __device__ __forceinline__ void run(int p0, int p1, uint8_t *lds, v4f (&acc)[FN][FM]) const {
        const int tid = threadIdx.x, lane = tid % kWave, li = lane & 15, g = lane >> 4;
        const Codes<T> codes;
        const v4f zero = held_zero();
        v4i wn[UW][FN], xn[PER];
        const int mine = __builtin_amdgcn_readfirstlane(tid / kWave) % KG * UW;  // this wave's first
        float sn[FN];
        const uint32_t woff = li * 64 + g * 16, soff = li * 4;
        uint32_t xoff[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) xoff[j] = row[j] + (j * NT + tid) / (16 * XR) % PARTS * 256 + tid % 16 * 16;
        const int64_t s_step = s_stride * 4;
        auto load = [&](int p) {  // pieces past the last are read again and scaled by zero
            const uint8_t *const xp = reinterpret_cast<const uint8_t *>(x) + (int64_t)p * (256 * PARTS);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int u = (j * NT + tid) / (16 * XR * PARTS);
                xn[j] = load16(xp + (xoff[j] + (U == 1 ? 0 : p + u < p1 ? u : p1 - 1 - p) * (256 * PARTS)));
            }
#pragma unroll
            for (int u = 0; u < UW; ++u) {
                const int64_t q = p + mine + u < p1 ? p + mine + u : p1 - 1;
#pragma unroll
                for (int f = 0; f < FN; ++f) {
                    const uint8_t *const a = w[f] + q * 1024;
                    wn[u][f] = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(a + woff));
                }
            }
            const uint32_t q = (U == 1 ? 0 : p + g < p1 ? g : p1 - 1 - p) * (uint32_t)s_step;
#pragma unroll
            for (int f = 0; f < FN; ++f)
                sn[f] = *reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(s[f]) + p * s_step + (q + soff));
        };
        if (p0 >= p1) return;
        load(p0);
        float *const scales = reinterpret_cast<float *>(lds + 2 * U * PIECE) + tid / kWave * FN * 64;
        int put[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int d = tid & 3, quarter = tid >> 2 & 3, q = (j * NT + tid) / 16;  // chunk 4 quarter + instruction of row q % XR
            put[j] = (q / XR * 4 + d) * STEP + quarter * SLOT + ((q % XR) ^ row_turn(quarter)) * 16;
        }
        const int get = g * SLOT + (li ^ row_turn(g)) * 16;
        uint8_t *buf = lds;
        for (int p = p0; p < p1; p += U) {
            v4i wc[UW][FN];
            wave_fence();
#pragma unroll
            for (int j = 0; j < PER; ++j) *reinterpret_cast<v4i *>(buf + put[j]) = Codes<T>::order(xn[j]);
#pragma unroll
            for (int u = 0; u < UW; ++u)
#pragma unroll
                for (int f = 0; f < FN; ++f) wc[u][f] = wn[u][f];
#pragma unroll
            for (int f = 0; f < FN; ++f) scales[f * 64 + lane] = p + g < p1 ? sn[f] * (1.f / Codes<T>::kTimes) : 0.f;
            if (p + U < p1) load(p + U);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            stage_barrier();  // this step's rows are written, and the other buffer is read
#pragma unroll
            for (int u = 0; u < UW; ++u) {
                const uint8_t *const rows = buf + (mine + u) * PIECE;
                v4f t[FN][FM];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    v4i xf[PARTS][FM];
#pragma unroll
                    for (int h = 0; h < PARTS; ++h)
#pragma unroll
                        for (int c = 0; c < FM; ++c)
                            xf[h][c] = load16(rows + (h * 4 + d) * STEP + get + c * 256);
#pragma unroll
                    for (int f = 0; f < FN; ++f) {
                        const v4i wf = codes((uint32_t)wc[u][f][d]);
#pragma unroll
                        for (int c = 0; c < FM; ++c)
#pragma unroll
                            for (int h = 0; h < PARTS; ++h)
                                t[f][c] = T::mfma(wf, xf[h][c], h == 0 && d == 0 ? zero : t[f][c]);
                    }
                }
#pragma unroll
                for (int f = 0; f < FN; ++f) {
                    const v4f sc = *reinterpret_cast<const v4f *>(scales + f * 64 + (mine + u) * 16 + g * 4);
#pragma unroll
                    for (int c = 0; c < FM; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[f][c][e] += sc[e] * t[f][c][e];
                }
            }
            buf = buf == lds ? lds + U * PIECE : lds;
        }
        wave_fence();
    }
};

// The sums of the KW waves (a power of two) that share a panel group's K, neighbours `wave / KW`
// in a CTA: wave kw of them gets the sums of row blocks c = kw, kw + KW, .. in acc, added in wave
// order. All threads of the CTA call it; `red` holds FN FM KB a wave.
template <int FN, int FM>
__device__ __forceinline__ void join_waves(uint8_t *smem, int kw_count, int wave, v4f (&acc)[FN][FM]) {
    if (kw_count == 1) return;
    const int lane = threadIdx.x % kWave;
    v4f *const red = reinterpret_cast<v4f *>(smem) + lane;
    __syncthreads();
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int c = 0; c < FM; ++c) red[((wave * FN + f) * FM + c) * kWave] = acc[f][c];
    __syncthreads();
    const int first = wave & -kw_count;
#pragma unroll
    for (int c = 0; c < FM; ++c) {
        if (c % kw_count != wave - first) continue;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            v4f s = red[((first * FN + f) * FM + c) * kWave];
            for (int w = 1; w < kw_count; ++w) {
                const v4f o = red[(((first + w) * FN + f) * FM + c) * kWave];
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] += o[e];
            }
            acc[f][c] = s;
        }
    }
}

}  // namespace twq
