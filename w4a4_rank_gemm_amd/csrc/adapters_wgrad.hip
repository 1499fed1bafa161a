// adapters_wgrad.hip -- the weight gradients of low-rank adapters (gfx950).
//
//   dA_a = c_a sum_i G[i] x_i^T   [r][m]        dB_a = c_a sum_i dy_i H[i]^T   [n][r]
//
// over the token rows i of adapter a: products whose long axis K is the tokens, so both
// operands lie with K as the slow index. They are staged in LDS row by row and read
// transposed. One CTA takes a piece of one adapter's rows and 128 columns of X or dY;
// both gradients are one launch. Each element of X and dY is read once (up to 128 ranks); X may
// come as an 8-bit checkpoint, whose codes are made bf16 in registers.
//
// Bound by memory up to about 32 ranks, then by LDS and the matrix cores as well: 8192 rows, 4096
// (codes) + 14336 columns with 16, 32, 64 and 128 ranks take 52, 55, 73 and 133 us (268 MB of rows:
// 5.1 to 2.0 TB/s), LDS active in 38 to 53% of the compute units' busy cycles, a third of that bank
// conflicts, matrix cores in 11, 21, 29 and 31%. 2048 rows, 32 ranks 18-21 us. Wider tiles read the factor
// less often but are fewer: 256 and 512 columns a CTA were equal to 45% slower.
//
// The binary32 factor, c_a G or c_a H, comes as two bf16 parts, 16 significant bits together
// (expand's planes); with a checkpoint c_a G still takes the group's scale of the token and is
// split here. Codes (at most 127) and bf16 elements are exact in bf16, fp16 elements are split
// exactly into two parts. bf16 rather than fp16: gradients span more binades than fp16 has.
#include "twq_adapters.h"
#include "twq_adapters_device.h"

namespace twq {

constexpr int kStep = 32;    // token rows of one matrix instruction

enum Src { kSrcF16, kSrcBF16, kSrcI8 };

// Columns of X or dY a CTA, 32 a wave; of a checkpoint that is one group.
constexpr int kCols = 128, kBlocks = 2;

// Eight codes (one column's eight rows) to bf16, exactly.
__device__ __forceinline__ v4i codes_to_bf16(v2i c) {
    v4i r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t p = (uint32_t)c[e / 2] >> (16 * (e % 2));
        const float f0 = (float)(int8_t)p, f1 = (float)(int8_t)(p >> 8);
        r[e] = (int)__builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, f1), __builtin_bit_cast(uint32_t, f0), 0x07060302u);
    }
    return r;
}

// OUT[s][c] (RB rank blocks x the column blocks of a wave) += P^T Z over the piece's rows.
// RANKS_M: ranks are the rows of the result blocks (dB, stored with ranks contiguous), else
// the columns of Z are (dA).
template <int RB, Src SRC, bool RANKS_M>
__device__ __forceinline__ void outer_piece(const OuterArgs &a, const PlanItem &it, int col0, int rank0, const int *rows,
                                            uint8_t *smem, v4f (&acc)[kBlocks][RB]) {
    constexpr int ZB = SRC == kSrcI8 ? 1 : 2;                  // bytes of an element of Z
    constexpr int ZROW = kCols * ZB + 16, PROW = RB * 32 + 16; // padded LDS rows
    constexpr int ZBYTES = kStep * ZROW, PBYTES = kStep * PROW, BUF = ZBYTES + 2 * PBYTES;
    constexpr int ZN = kStep * kCols * ZB / 16 / 256;          // 16-byte chunks of Z a thread
    // the factor's chunks of a step: four binary32 ranks (codes), or eight bf16 ranks of a plane
    constexpr int PC = SRC == kSrcI8 ? RB * 4 : RB * 2, PALL = kStep * PC * (SRC == kSrcI8 ? 1 : 2), PN = (PALL + 255) / 256;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, li = lane & 15, g = lane >> 4;
    const uint32_t ld = (uint32_t)(RANKS_M ? a.n : a.m);
    const uint8_t *z = SRC == kSrcI8 ? reinterpret_cast<const uint8_t *>(a.qc)
                                     : reinterpret_cast<const uint8_t *>(RANKS_M ? a.dy : a.x);
    const float scale = SRC == kSrcI8 && a.scale ? a.scale[it.adapter] : 1.f;
    const uint16_t *planes = a.planes + (RANKS_M ? 2 : 0) * a.b * a.r + (int64_t)it.first * a.r + rank0;
    const float *sc = SRC == kSrcI8 ? a.sc + (int64_t)(col0 / 128) * a.b : nullptr;
    const int nst = (it.rows + kStep - 1) / kStep;

    v4i zr2[2][ZN];
    v4f pr2[2][PN];
    float ps2[2][PN];
    // Unconditional, with clamped addresses: a load under a condition would leave the number of
    // loads in flight open, and the wait for the older step would wait for the newer one too.
    // Rows and ranks past the end re-read others and are cleared when stored.
    auto load = [&](int st, auto slot) {
        constexpr int S = decltype(slot)::value;
        v4i (&zr)[ZN] = zr2[S];
        v4f (&pr)[PN] = pr2[S];
        float (&ps)[PN] = ps2[S];
#pragma unroll
        for (int j = 0; j < ZN; ++j) {
            constexpr int PER = kCols * ZB / 16;
            const int q = j * 256 + tid, i = st * kStep + q / PER;
            const uint32_t row = (uint32_t)rows[i < it.rows ? i : it.rows - 1];
            const uint32_t c = col0 + q % PER * (16 / ZB);
            zr[j] = load16(z + ((uint64_t)row * (ld * ZB) + (c < ld ? c : ld - 16 / ZB) * ZB));
        }
#pragma unroll
        for (int j = 0; j < PN; ++j) {
            const int q = j * 256 + tid, i0 = st * kStep + q / PC % kStep, i = i0 < it.rows ? i0 : it.rows - 1;
            if constexpr (SRC == kSrcI8) {
                const int rank = rank0 + q % PC * 4;
                pr[j] = *reinterpret_cast<const v4f *>(a.g + (int64_t)(it.first + i) * a.r + (rank < a.r ? rank : 0));
                ps[j] = sc[rows[i]];
            } else {
                const int rank = q % PC * 8;
                pr[j] = *reinterpret_cast<const v4f *>(planes + q / (kStep * PC) % 2 * a.b * a.r +
                                                       (uint64_t)(uint32_t)i * (uint32_t)a.r + (rank0 + rank < a.r ? rank : 0));
            }
        }
    };
    auto store = [&](int st, auto slot) {
        constexpr int S = decltype(slot)::value;
        const v4i (&zr)[ZN] = zr2[S];
        const v4f (&pr)[PN] = pr2[S];
        const float (&ps)[PN] = ps2[S];
        uint8_t *buf = smem + S * BUF;
#pragma unroll
        for (int j = 0; j < ZN; ++j) {
            constexpr int PER = kCols * ZB / 16;
            const int q = j * 256 + tid;
            *reinterpret_cast<v4i *>(buf + q / PER * ZROW + q % PER * 16) = zr[j];
        }
#pragma unroll
        for (int j = 0; j < PN; ++j) {
            const int q = j * 256 + tid, rank = rank0 + q % PC * (SRC == kSrcI8 ? 4 : 8);
            if (PALL % 256 && q >= PALL) break;
            const bool live = st * kStep + q / PC % kStep < it.rows && rank < a.r;
            if constexpr (SRC != kSrcI8) {
                *reinterpret_cast<v4f *>(buf + ZBYTES + q / (kStep * PC) * PBYTES + q / PC % kStep * PROW + q % PC * 16) =
                    live ? pr[j] : v4f{0.f, 0.f, 0.f, 0.f};
                continue;
            }
            const float f = live ? scale * ps[j] : 0.f;
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float v0 = live ? pr[j][2 * e] * f : 0.f, v1 = live ? pr[j][2 * e + 1] * f : 0.f;
                const uint16_t h0 = BF16::from_f32(v0), h1 = BF16::from_f32(v1);
                const uint16_t l0 = BF16::from_f32(v0 - BF16::to_f32(h0)), l1 = BF16::from_f32(v1 - BF16::to_f32(h1));
                hi[e] = (uint32_t)h0 | (uint32_t)h1 << 16;
                lo[e] = (uint32_t)l0 | (uint32_t)l1 << 16;
            }
            uint8_t *p = buf + ZBYTES + q / PC * PROW + q % PC * 8;
            *reinterpret_cast<uint2 *>(p) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2 *>(p + PBYTES) = make_uint2(lo[0], lo[1]);
        }
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    auto step = [&](int st, auto slot) {
        __builtin_amdgcn_sched_barrier(0);  // keep this step's waits from moving before the last step's work
        store(st, slot);  // the buffer was last read in step st - 2, before the barrier of st - 1
        load(st + 2, slot);
        __syncthreads();
        const uint8_t *buf = smem + decltype(slot)::value * BUF;
        v4i zf[kBlocks], zl[kBlocks];
#pragma unroll
        for (int s = 0; s < kBlocks; ++s) {
            const int c = (wave * kBlocks + s) * 16;
            if constexpr (SRC == kSrcI8) {
                zf[s] = codes_to_bf16(read_tr8(buf + (g * 8 + li / 2) * ZROW + c + (li % 2) * 8));
            } else {
                const uint8_t *p = buf + (g * 8 + li / 4) * ZROW + (c + (li % 4) * 4) * 2;
                const v4s z0 = read_tr16(p), z1 = read_tr16(p + 4 * ZROW);
                zf[s] = join(z0, z1);
                if constexpr (SRC == kSrcF16) split_f16(zf[s], zf[s], zl[s]);
            }
        }
#pragma unroll
        for (int c = 0; c < RB; ++c) {
            const uint8_t *p = buf + ZBYTES + (g * 8 + li / 4) * PROW + (c * 16 + (li % 4) * 4) * 2;
            const v4s h0 = read_tr16(p), h1 = read_tr16(p + 4 * PROW);
            const v4s l0 = read_tr16(p + PBYTES), l1 = read_tr16(p + PBYTES + 4 * PROW);
            const v4i hi = join(h0, h1), lo = join(l0, l1);
#pragma unroll
            for (int s = 0; s < kBlocks; ++s) {
                auto add = [&](v4i p16, v4i z16) {
                    acc[s][c] = RANKS_M ? BF16::mfma(p16, z16, acc[s][c]) : BF16::mfma(z16, p16, acc[s][c]);
                };
                if constexpr (SRC == kSrcF16) add(lo, zl[s]), add(hi, zl[s]);
                add(lo, zf[s]);
                add(hi, zf[s]);
            }
        }
    };
    // Two steps of rows in flight; an odd last step is followed by one of cleared rows, so that
    // the loop has no branch (which would cost a wait for every load at its end).
    load(0, S0{});
    load(1, S1{});
    for (int st = 0; st < nst; st += 2) {
        step(st, S0{});
        step(st + 1, S1{});
    }
}

// A result block's four values of this lane, to the gradient (rounded) or its partial sum.
template <class T>
__device__ __forceinline__ void outer_put(const OuterArgs &a, uint16_t *out, float *part, int64_t at, const v4f &v) {
    if (part) {
        *reinterpret_cast<v4f *>(part + at) = v;
    } else {
        *reinterpret_cast<uint2 *>(out + at) =
            make_uint2((uint32_t)T::from_f32(v[0]) | (uint32_t)T::from_f32(v[1]) << 16,
                       (uint32_t)T::from_f32(v[2]) | (uint32_t)T::from_f32(v[3]) << 16);
    }
}

template <class T, int RB, bool CODES>
__global__ __launch_bounds__(256) void outer_kernel(OuterArgs a) {
    constexpr Src ZS = T::kBf16 ? kSrcBF16 : kSrcF16, XS = CODES ? kSrcI8 : ZS;
    constexpr int BUF = kStep * (kCols * 2 + 16) + 2 * kStep * (RB * 32 + 16);
    __shared__ __align__(16) uint8_t smem[2 * BUF];
    __shared__ int rows[kMaxChunk];
    const int nt = (int)((a.n + kCols - 1) / kCols), ct = nt + (int)(a.m / kCols), tile = (int)(blockIdx.x % ct);
    const int64_t piece = blockIdx.x / ct;
    if (piece >= a.plan.head[1]) return;
    const PlanItem it = a.plan.chunks[piece];
    if (it.rows > 0) {
        int in[kMaxChunk / 256];
#pragma unroll
        for (int j = 0; j < kMaxChunk / 256; ++j) {
            const int i = j * 256 + threadIdx.x;
            in[j] = a.plan.order[it.first + (i < it.rows ? i : it.rows - 1)];
        }
#pragma unroll
        for (int j = 0; j < kMaxChunk / 256; ++j) rows[j * 256 + threadIdx.x] = in[j];
    }
    __syncthreads();
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, li = lane & 15, g = lane >> 4;
    const int rank0 = blockIdx.y * RB * 16;
    float *const part = it.slot < 0 ? nullptr : a.part + (int64_t)it.slot * a.r * (a.m + a.n);
    if (tile >= nt) {
        v4f acc[kBlocks][RB] = {};
        const int col0 = (tile - nt) * kCols;
        if (it.rows > 0) outer_piece<RB, XS, false>(a, it, col0, rank0, rows, smem, acc);
        uint16_t *const out = a.dat + (int64_t)it.adapter * a.r * a.m;
#pragma unroll
        for (int c = 0; c < RB; ++c) {
            const int rank = rank0 + c * 16 + li;
            if (rank >= a.r) continue;
#pragma unroll
            for (int s = 0; s < kBlocks; ++s) {
                const int64_t col = col0 + (wave * kBlocks + s) * 16 + g * 4;
                outer_put<T>(a, out, part, (int64_t)rank * a.m + col, acc[s][c]);
            }
        }
    } else {
        v4f acc[kBlocks][RB] = {};
        const int col0 = tile * kCols;
        if (it.rows > 0) outer_piece<RB, ZS, true>(a, it, col0, rank0, rows, smem, acc);
        uint16_t *const out = a.dbt + (int64_t)it.adapter * a.r * a.n;
        float *const bp = part ? part + (int64_t)a.r * a.m : nullptr;
#pragma unroll
        for (int c = 0; c < RB; ++c) {
            const int rank = rank0 + c * 16 + g * 4;
            if (rank >= a.r) continue;
#pragma unroll
            for (int s = 0; s < kBlocks; ++s) {
                const int64_t col = col0 + (wave * kBlocks + s) * 16 + li;
                if (col < a.n) outer_put<T>(a, out, bp, col * a.r + rank, acc[s][c]);
            }
        }
    }
}

// Gradients of adapters whose rows were several pieces: the pieces' sums in order (no atomics).
// The others were written whole. 16 adapters, 64 x (4096 + 14336) each, 8.8 us.
template <class T>
__global__ __launch_bounds__(256) void outer_join_kernel(OuterArgs a) {
    const int ad = blockIdx.y;
    const int rows = a.plan.offsets[ad + 1] - a.plan.offsets[ad], parts = (rows + a.chunk - 1) / a.chunk;
    if (parts < 2) return;
    const int64_t per = (int64_t)a.r * (a.m + a.n), e4 = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e4 * 4 >= per) return;
    const v4f s = sum_slices(a.part + (int64_t)a.plan.slot0[ad] * per + e4 * 4, per, parts);
    const int64_t at = e4 * 4, na = (int64_t)a.r * a.m;
    if (at < na)
        outer_put<T>(a, a.dat + ad * na, nullptr, at, s);
    else
        outer_put<T>(a, a.dbt + (int64_t)ad * a.r * a.n, nullptr, at - na, s);
}

template <class T, bool CODES>
static hipError_t outer_ranks(const OuterArgs &a, hipStream_t stream) {
    const int rb = a.r <= 16 ? 1 : a.r <= 32 ? 2 : a.r <= 64 ? 4 : 8;
    const dim3 grid((unsigned)(a.chunks * (a.m / kCols + (a.n + kCols - 1) / kCols)), (unsigned)((a.r + 16 * rb - 1) / (16 * rb)));
    if (rb == 1)
        outer_kernel<T, 1, CODES><<<grid, 256, 0, stream>>>(a);
    else if (rb == 2)
        outer_kernel<T, 2, CODES><<<grid, 256, 0, stream>>>(a);
    else if (rb == 4)
        outer_kernel<T, 4, CODES><<<grid, 256, 0, stream>>>(a);
    else
        outer_kernel<T, 8, CODES><<<grid, 256, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.b <= a.chunk) return e;  // no adapter has two pieces
    const int64_t per4 = (int64_t)a.r * (a.m + a.n) / 4;
    outer_join_kernel<T><<<dim3((unsigned)((per4 + 255) / 256), (unsigned)a.count), 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_outer(const OuterArgs &a, hipStream_t stream) {
    if (a.bf16) return a.qc ? outer_ranks<BF16, true>(a, stream) : outer_ranks<BF16, false>(a, stream);
    return a.qc ? outer_ranks<F16, true>(a, stream) : outer_ranks<F16, false>(a, stream);
}

}  // namespace twq
