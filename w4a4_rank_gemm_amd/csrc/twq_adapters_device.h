// twq_adapters_device.h -- 16-bit element types, transposing LDS reads and the expansion of
// 4-bit codes of the adapter, input-gradient and 16-bit-activation kernels (gfx950).
#pragma once

#include "twq_device.h"

namespace twq {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef int v2i __attribute__((ext_vector_type(2)));

// A 16-bit element type: its matrix instruction and its conversions. Operands travel as
// v4i (eight elements of one K run).
struct F16 {
    static constexpr bool kBf16 = false;
    static __device__ __forceinline__ v4f mfma(v4i a, v4i b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ float to_f32(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ __forceinline__ uint16_t from_f32(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};
struct BF16 {
    static constexpr bool kBf16 = true;
    static __device__ __forceinline__ v4f mfma(v4i a, v4i b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ float to_f32(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t from_f32(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};

__device__ __forceinline__ v4i load16(const void *p) { return *reinterpret_cast<const v4i *>(p); }

// 16-bit element e (0 or 1) of a dword
__device__ __forceinline__ uint16_t half_of(int w, int e) { return (uint16_t)((uint32_t)w >> (16 * e)); }

// Eight fp16 values as bf16 hi + lo: hi is the value cut to its upper 8 significant
// bits, lo the rest (3 bits). The sum is the fp16 value exactly (the smallest fp16
// subnormals are far inside bf16's range).
__device__ __forceinline__ void split_f16(v4i v, v4i &hi, v4i &lo) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t f0 = __builtin_bit_cast(uint32_t, F16::to_f32(half_of(v[e], 0)));
        const uint32_t f1 = __builtin_bit_cast(uint32_t, F16::to_f32(half_of(v[e], 1)));
        hi[e] = (int)__builtin_amdgcn_perm(f1, f0, 0x07060302u);
        const float l0 = __builtin_bit_cast(float, f0) - __builtin_bit_cast(float, f0 & 0xFFFF0000u);
        const float l1 = __builtin_bit_cast(float, f1) - __builtin_bit_cast(float, f1 & 0xFFFF0000u);
        lo[e] = (int)__builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, l1), __builtin_bit_cast(uint32_t, l0), 0x07060302u);
    }
}

// Transposing LDS reads. The 16 lanes of a group address a block of 16-bit elements, 4
// rows (K) x 16 columns: lane i gives the address of columns 4 (i % 4) .. + 3 of row
// i / 4 (each quarter row anywhere), and receives column i's four rows.
__device__ __forceinline__ v4s read_tr16(const void *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)p);
}
// The same for bytes: 8 rows x 16 columns, lane i gives columns 8 (i % 2) .. + 7 of row
// i / 2 and receives column i's eight rows.
__device__ __forceinline__ v2i read_tr8(const void *p) {
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) v2i *)p);
}
// The same for 4-bit codes: 16 rows x 16 columns, lane i gives row i (8 bytes) and
// receives column i's sixteen rows, the first in the lowest nibble.
__device__ __forceinline__ v2i read_tr4(const void *p) {
    return __builtin_amdgcn_ds_read_tr4_b64_v2i32((__attribute__((address_space(3))) v2i *)p);
}
__device__ __forceinline__ v4i join(v4s a, v4s b) {
    return __builtin_bit_cast(v4i, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Sum of `count` slices, `stride` floats apart, in order, eight in flight.
__device__ __forceinline__ v4f sum_slices(const float *p, int64_t stride, int count) {
    v4f s = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < count; i += 8) {
        v4f v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const v4f *>(p + (i + j < count ? i + j : i) * stride);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += i + j < count ? v[j][e] : 0.f;
    }
    return s;
}

// CTA b runs on XCD b % 8 (they are dealt out in turn). XCD x gets a contiguous range of `ctas`
// ids, the first ctas % 8 XCDs one more: a bijection of [0, ctas), in which neighbours, which
// share operands, share an L2.
__device__ __forceinline__ int64_t xcd_range(int64_t b, int64_t ctas) {
    const int64_t x = b % 8, more = ctas % 8;
    return ctas / 8 * x + (x < more ? x : more) + b / 8;
}

// Power of two 2^e, e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// Exponent by which a row with the largest magnitude v is scaled: e with 2^e <= v < 2^(e + 1),
// at least -112, so that 2^(14 - e) and 2^(e - 14) lie in the range of pow2 (subnormals and 0 are
// scaled by 2^126 too); 0 for infinities and NaN, which pass unscaled.
__device__ __forceinline__ int scale_exponent(float v) {
    const int e = (int)((__builtin_bit_cast(uint32_t, v) >> 23) & 0xFFu);
    return e == 255 ? 0 : e < 15 ? -112 : e - 127;
}

// Maximum over the 16 lanes of a row of lanes, in every one of them.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    uint32_t t;
    t = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);   // quad_perm [1, 0, 3, 2]
    v = v > t ? v : t;
    t = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);   // quad_perm [2, 3, 0, 1]
    v = v > t ? v : t;
    t = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false);  // row_half_mirror
    v = v > t ? v : t;
    t = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false);  // row_mirror
    return v > t ? v : t;
}

// Eight codes of a dword (two's complement nibbles q, nibble k = channel k) as fp16 pairs
// (0, 4), (1, 5), (2, 6), (3, 7): q + 8 in the low mantissa bits of 1024 (or, four bits up,
// times 16), then the offset taken off. Exact. One three-input logic operation
// ((d & mask) ^ c) per pair masks the nibbles, flips their sign bits and sets the exponent; its
// constants come in registers (the instruction takes one scalar operand), in `c`. The loop's
// matrix and vector cycles add up to its time, so this matters: the 70B kernel took 1640 us with
// the fourteen operations the compiler made of the plain expression, 1600 with these nine.
struct DequantConst {
    uint32_t lo, hi;  // 1024 with the sign bit of the nibble at bits 0-3, at bits 4-7
};
__device__ __forceinline__ DequantConst dequant_const() {
    DequantConst c{0x64086408u, 0x64806480u};
    asm("" : "+v"(c.lo), "+v"(c.hi));
    return c;
}
__device__ __forceinline__ v4i dequant8(uint32_t d, const DequantConst &c) {
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    const uint32_t s = d >> 8;
    const v2h one = {(_Float16)1032.f, (_Float16)1032.f}, six = {(_Float16)0.0625f, (_Float16)0.0625f};
    const v2h off = {(_Float16)72.f, (_Float16)72.f};
    constexpr uint32_t AND_XOR = 0x6A;  // (a & b) ^ c
    const v2h p0 = __builtin_bit_cast(v2h, __builtin_amdgcn_bitop3_b32(d, 0x000F000Fu, c.lo, AND_XOR)) - one;
    const v2h p1 = __builtin_bit_cast(v2h, __builtin_amdgcn_bitop3_b32(d, 0x00F000F0u, c.hi, AND_XOR)) * six - off;
    const v2h p2 = __builtin_bit_cast(v2h, __builtin_amdgcn_bitop3_b32(s, 0x000F000Fu, c.lo, AND_XOR)) - one;
    const v2h p3 = __builtin_bit_cast(v2h, __builtin_amdgcn_bitop3_b32(s, 0x00F000F0u, c.hi, AND_XOR)) * six - off;
    return v4i{__builtin_bit_cast(int, p0), __builtin_bit_cast(int, p1), __builtin_bit_cast(int, p2), __builtin_bit_cast(int, p3)};
}

}  // namespace twq
