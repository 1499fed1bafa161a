// adapters.hip -- low-rank adapters of many requests beside a shared projection (gfx950).
//
//   H[i] = A_a x_i,   out[i] = y_i + c_a B_a H[i]        a = adapter of token row i
//
// and the two products of its gradient that have one row per token,
//
//   G[i] = B_a^T dy_i,   dX[i] = dx_i + c_a A_a^T G[i].
//
// Token rows are grouped by adapter (the plan), so a tile of up to 64 rows shares one
// adapter's weights, whatever the order of the requests in the batch; no row is moved.
// Each product is a pair of launches: shrink (K = the long axis, partial sums over K
// slices) and expand (K = the rank). Both are bound by memory: shrink by the rows and the
// adapters' first factors, expand by the read and write of the output rows. All sums
// are in binary32 and in a fixed order, so equal calls give equal bits.
#include "twq_adapters.h"
#include "twq_adapters_device.h"

namespace twq {

// ---- plan ----------------------------------------------------------------------------

// CTA a owns adapter a (CTA `count`: the rows without one). It counts every adapter's
// rows, from which its own first position, first tile and first piece follow, then
// scans the index again and writes its rows in token order.
__global__ __launch_bounds__(256) void adapter_plan_kernel(const int32_t *index, int64_t b, int count, uint8_t *plan,
                                                           PlanLayout L, int chunk) {
    __shared__ int hist[kMaxAdapters + 1];
    __shared__ int red[4][4];
    __shared__ int wsum[4];
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const int a = blockIdx.x;
    for (int k = tid; k <= count; k += 256) hist[k] = 0;
    __syncthreads();
    for (int64_t i = tid; i < b; i += 256) {
        const int key = index[i];
        atomicAdd(&hist[(unsigned)key < (unsigned)count ? key : count], 1);
    }
    __syncthreads();
    int s[4] = {0, 0, 0, 0};  // rows, tiles, pieces, partial-sum slots before adapter a
    for (int k = tid; k < a; k += 256) {
        const int c = hist[k];
        s[0] += c;
        s[1] += (c + kTileRows - 1) / kTileRows;
        s[2] += (c + chunk - 1) / chunk;
        s[3] += c > chunk ? (c + chunk - 1) / chunk : 0;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        for (int off = 32; off > 0; off >>= 1) s[q] += __shfl_xor(s[q], off, kWave);
        if (lane == 0) red[q][wave] = s[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = red[q][0] + red[q][1] + red[q][2] + red[q][3];
    const int rows = hist[a], ntiles = (rows + kTileRows - 1) / kTileRows, nparts = (rows + chunk - 1) / chunk;
    int32_t *head = reinterpret_cast<int32_t *>(plan + L.head), *order = reinterpret_cast<int32_t *>(plan + L.order);
    int32_t *offsets = reinterpret_cast<int32_t *>(plan + L.offsets), *slot0 = reinterpret_cast<int32_t *>(plan + L.slot0);
    PlanItem *tiles = reinterpret_cast<PlanItem *>(plan + L.tiles), *chunks = reinterpret_cast<PlanItem *>(plan + L.chunks);
    if (tid == 0) {
        offsets[a] = s[0];
        if (a < count) slot0[a] = s[3];
        if (a == count) {
            offsets[count + 1] = s[0] + rows;
            head[0] = s[1] + ntiles;
            head[1] = s[2];
        }
    }
    for (int j = tid; j < ntiles; j += 256) {
        const int left = rows - j * kTileRows;
        tiles[s[1] + j] = PlanItem{a == count ? -1 : a, s[0] + j * kTileRows, left < kTileRows ? left : kTileRows, -1};
    }
    if (a < count)
        for (int j = tid; j < nparts; j += 256) {
            const int left = rows - j * chunk;
            chunks[s[2] + j] = PlanItem{a, s[0] + j * chunk, left < chunk ? left : chunk, nparts > 1 ? s[3] + j : -1};
        }
    if (rows == 0) return;
    int pos = s[0];
    for (int64_t i0 = 0; i0 < b; i0 += 256) {
        const int64_t i = i0 + tid;
        bool mine = false;
        if (i < b) {
            const int key = index[i];
            mine = ((unsigned)key < (unsigned)count ? key : count) == a;
        }
        const uint64_t mask = __ballot(mine);
        if (lane == 0) wsum[wave] = __popcll(mask);
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            before += w < wave ? wsum[w] : 0;
            all += wsum[w];
        }
        if (mine) order[pos + before + __popcll(mask & ((uint64_t(1) << lane) - 1))] = (int32_t)i;
        pos += all;
        __syncthreads();
    }
}

hipError_t launch_adapter_plan(const int32_t *index, int64_t b, int64_t count, void *plan, hipStream_t stream) {
    adapter_plan_kernel<<<dim3((unsigned)(count + 1)), 256, 0, stream>>>(index, b, (int)count, static_cast<uint8_t *>(plan),
                                                                        plan_layout(b, count), chunk_rows(b));
    return hipGetLastError();
}

// ---- shrink --------------------------------------------------------------------------

struct Tile {
    int adapter, rows;
    int64_t first;
};

// Tile t of the plan (rows == 0: none); without a plan, rows 64 t .. of one adapter.
__device__ __forceinline__ Tile tile_of(const PlanView &p, int64_t t, int64_t b) {
    if (p.order == nullptr) {
        const int64_t left = b - t * kTileRows;
        return Tile{0, (int)(left < kTileRows ? left : kTileRows), t * kTileRows};
    }
    if (t >= p.head[0]) return Tile{-1, 0, 0};
    const PlanItem it = p.tiles[t];
    return Tile{it.adapter, it.rows, it.first};
}

// One tile of up to 16 NG rows x 16 RB ranks over steps [s0, s1) of 64 elements of K; the
// four waves take batches of U steps in turn. A lane holds 16 elements of a step in two
// operands (lane group g: elements 16 g .. + 15), the same for rows and weights, so every
// 128-byte line of a row is read whole by its four lanes. KMAJOR weights ([k][r], ranks
// contiguous) pass through this wave's own LDS and come back transposed. XW: bf16 rows on
// fp16 weights, the weights split exactly into two bf16 parts.
template <class T, int NG, int RB, int U, bool KMAJOR, bool XW>
__device__ __forceinline__ void shrink_tile(const ShrinkArgs &a, const Tile &t, int rank0, int64_t s0, int64_t s1,
                                            uint8_t *smem, v4f (&acc)[NG][RB]) {
    static_assert(!KMAJOR || U == 1, "one step at a time through LDS");
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, li = lane & 15, g = lane >> 4;
    const uint16_t *w = a.w + (int64_t)t.adapter * a.r * a.k;
    const uint16_t *row[NG];
#pragma unroll
    for (int q = 0; q < NG; ++q) {
        const int i = q * 16 + li < t.rows ? q * 16 + li : t.rows - 1;
        const int64_t pos = t.first + i;
        row[q] = a.v + (a.plan.order ? (int64_t)a.plan.order[pos] : pos) * a.k;
    }
    const uint16_t *wrow[RB];
    if constexpr (!KMAJOR) {
#pragma unroll
        for (int c = 0; c < RB; ++c) {
            const int rank = rank0 + c * 16 + li;
            wrow[c] = w + (int64_t)(rank < a.r ? rank : a.r - 1) * a.k;
        }
    }
    // KMAJOR: this wave's [64 steps of K][16 RB ranks]
    uint16_t *const wl = reinterpret_cast<uint16_t *>(smem) + wave * 64 * 16 * RB;
    const int64_t nst = s1 - s0, nb = (nst + 4 * U - 1) / (4 * U);
    v4i xb[2][U][NG][2], wb[2][U][RB][2];
    auto load = [&](int64_t bt, auto slot) {
        constexpr int S = decltype(slot)::value;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t st = s0 + (bt * 4 + wave) * U + u;
            // steps and runs past the end re-read valid elements and are zeroed in use
            const int64_t k0 = (st < s1 ? st : s1 - 1) * 64, kc = k0 + g * 16 < a.k ? k0 + g * 16 : a.k - 16;
#pragma unroll
            for (int q = 0; q < NG; ++q) {
                xb[S][u][q][0] = load16(row[q] + kc);
                xb[S][u][q][1] = load16(row[q] + kc + 8);
            }
            if constexpr (!KMAJOR) {
#pragma unroll
                for (int c = 0; c < RB; ++c) {
                    wb[S][u][c][0] = load16(wrow[c] + kc);
                    wb[S][u][c][1] = load16(wrow[c] + kc + 8);
                }
            } else {
                // chunk q of 8 ranks: row q / (2 RB), ranks 8 (q % (2 RB)) ..
#pragma unroll
                for (int c = 0; c < RB; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int q = (c * 2 + e) * kWave + lane, kr = q / (2 * RB), rr = rank0 + q % (2 * RB) * 8;
                        const int64_t kk = k0 + kr < a.k ? k0 + kr : a.k - 1;
                        wb[S][u][c][e] = load16(w + kk * a.r + (rr < a.r ? rr : a.r - 8));
                    }
            }
        }
    };
    auto use = [&](int64_t bt, auto slot) {
        constexpr int S = decltype(slot)::value;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t st = s0 + (bt * 4 + wave) * U + u;
            const bool live = st < s1 && st * 64 + g * 16 < a.k;
            if (!live) {
#pragma unroll
                for (int q = 0; q < NG; ++q) xb[S][u][q][0] = xb[S][u][q][1] = v4i{0, 0, 0, 0};
            }
            if constexpr (KMAJOR) {
#pragma unroll
                for (int c = 0; c < RB; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<v4i *>(wl + ((c * 2 + e) * kWave + lane) * 8) = wb[S][u][c][e];
                __builtin_amdgcn_wave_barrier();
                // lane group g reads rows 16 g + 4 q + (li / 4), q = 0..3: its 16 elements of K
#pragma unroll
                for (int c = 0; c < RB; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint16_t *p = wl + (g * 16 + e * 8 + li / 4) * 16 * RB + c * 16 + (li % 4) * 4;
                        const v4s lo4 = read_tr16(p), hi4 = read_tr16(p + 4 * 16 * RB);
                        wb[S][u][c][e] = join(lo4, hi4);
                    }
                __builtin_amdgcn_wave_barrier();
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int c = 0; c < RB; ++c) {
                    if constexpr (XW) {
                        v4i hi, lo;
                        split_f16(wb[S][u][c][e], hi, lo);
#pragma unroll
                        for (int q = 0; q < NG; ++q) {
                            acc[q][c] = T::mfma(lo, xb[S][u][q][e], acc[q][c]);
                            acc[q][c] = T::mfma(hi, xb[S][u][q][e], acc[q][c]);
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < NG; ++q) acc[q][c] = T::mfma(wb[S][u][c][e], xb[S][u][q][e], acc[q][c]);
                    }
                }
        }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    if (nb > 0) load(0, I0{});
    for (int64_t bt = 0; bt < nb; bt += 2) {
        if (bt + 1 < nb) load(bt + 1, I1{});
        use(bt, I0{});
        if (bt + 1 >= nb) break;
        if (bt + 2 < nb) load(bt + 2, I0{});
        use(bt + 1, I1{});
    }
}

// The waves' sums, added in wave order through LDS, to this slice's rows of P.
template <int NG, int RB>
__device__ __forceinline__ void shrink_store(const ShrinkArgs &a, const Tile &t, int rank0, int64_t slice, uint8_t *smem,
                                             const v4f (&acc)[NG][RB]) {
    v4f *const red = reinterpret_cast<v4f *>(smem);  // [4 waves][RB][64 lanes]
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
#pragma unroll
    for (int q = 0; q < NG; ++q) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < RB; ++c) red[(wave * RB + c) * kWave + lane] = acc[q][c];
        __syncthreads();
        if (tid < RB * kWave) {
            const int c = tid / kWave, i = q * 16 + (tid & 15), rank = rank0 + c * 16 + (tid % kWave) / 16 * 4;
            v4f s = red[tid];
#pragma unroll
            for (int w = 1; w < 4; ++w) {
                const v4f o = red[w * RB * kWave + tid];
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] += o[e];
            }
            if (i < t.rows && rank < a.r)
                *reinterpret_cast<v4f *>(a.p + ((slice * a.b + t.first + i) * a.r + rank)) = s;
        }
    }
}

template <class T, int RB, bool KMAJOR, bool XW>
__global__ __launch_bounds__(256) void shrink_kernel(ShrinkArgs a) {
    __shared__ __align__(16) uint8_t smem[KMAJOR ? 4 * 64 * 16 * RB * 2 : 4 * RB * kWave * 16];
    const Tile t = tile_of(a.plan, blockIdx.x, a.b);
    if (t.rows == 0 || t.adapter < 0) return;
    const int rank0 = blockIdx.y * 16 * RB;
    const int64_t slice = blockIdx.z, nst = (a.k + 63) / 64;
    const int64_t s0 = slice * nst / a.ks, s1 = (slice + 1) * nst / a.ks;
    if (t.rows <= 16) {
        v4f acc[1][RB] = {};
        shrink_tile<T, 1, RB, KMAJOR ? 1 : (RB == 1 ? 4 : 2), KMAJOR, XW>(a, t, rank0, s0, s1, smem, acc);
        shrink_store<1, RB>(a, t, rank0, slice, smem, acc);
    } else {
        v4f acc[4][RB] = {};
        shrink_tile<T, 4, RB, 1, KMAJOR, XW>(a, t, rank0, s0, s1, smem, acc);
        shrink_store<4, RB>(a, t, rank0, slice, smem, acc);
    }
}

// K slices: enough CTAs to fill the 256 compute units twice, at least four steps of 64 a
// wave-quartet, at most 16 (their partial sums are read again by every expand CTA).
int shrink_slices(int64_t b, int64_t k, int64_t r, int64_t tiles) {
    (void)b;
    const int64_t rt = r <= 16 ? 1 : r <= 32 ? 1 : (r + 63) / 64, steps = (k + 63) / 64;
    int64_t ks = 512 / (tiles * rt);
    if (ks > steps / 4) ks = steps / 4;
    if (ks > 16) ks = 16;
    return ks < 1 ? 1 : (int)ks;
}

template <class T, bool KMAJOR, bool XW>
static hipError_t shrink_ranks(const ShrinkArgs &a, hipStream_t stream) {
    const int rb = a.r <= 16 ? 1 : a.r <= 32 ? 2 : 4;
    const dim3 grid((unsigned)a.tiles, (unsigned)((a.r + 16 * rb - 1) / (16 * rb)), (unsigned)a.ks);
    if (rb == 1)
        shrink_kernel<T, 1, KMAJOR, XW><<<grid, 256, 0, stream>>>(a);
    else if (rb == 2)
        shrink_kernel<T, 2, KMAJOR, XW><<<grid, 256, 0, stream>>>(a);
    else
        shrink_kernel<T, 4, KMAJOR, XW><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_shrink(const ShrinkArgs &a, hipStream_t stream) {
    if (a.bf16 && !a.wbf16) return a.kmajor ? shrink_ranks<BF16, true, true>(a, stream) : hipErrorInvalidValue;
    if (a.bf16) return a.kmajor ? shrink_ranks<BF16, true, false>(a, stream) : shrink_ranks<BF16, false, false>(a, stream);
    return a.kmajor ? shrink_ranks<F16, true, false>(a, stream) : shrink_ranks<F16, false, false>(a, stream);
}

// ---- expand --------------------------------------------------------------------------

// The tile's rows of the first product, summed over the slices, times the adapter's
// scale, as two 16-bit parts hi + lo in LDS: 8 ranks are 32 bytes, hi then lo. One part
// would round H to the element type, an error of the size of the output's own rounding;
// the second part costs a matrix instruction on operands at hand. fp16 rows are first
// scaled by a power of two to a largest element in [2^13, 2^14), so neither part can
// overflow and only elements below 2^-27 of the largest lose bits; rexp holds the exponent
// to undo. Ranks past r (the last half step) are zero.
template <class T, int NG>
__device__ __forceinline__ void expand_rows(const ExpandArgs &a, const Tile &t, float scale, uint8_t *hl, int stride,
                                            float *rfac, bool store_sum) {
    constexpr int TPR = 256 / (16 * NG);  // threads a row
    const int tid = threadIdx.x, i = tid / TPR, q = tid % TPR;
    const bool live = i < t.rows;
    const int64_t pos = t.first + (live ? i : 0);
    const float *src = a.p + pos * a.r;
    uint8_t *dst = hl + i * stride;
    float mx = 0.f;
    for (int c = q * 8; c < a.r; c += TPR * 8) {
        v4f s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
        if (live) {
            for (int s = 0; s < a.ks; ++s) {
                const v4f p0 = *reinterpret_cast<const v4f *>(src + s * a.b * a.r + c);
                const v4f p1 = *reinterpret_cast<const v4f *>(src + s * a.b * a.r + c + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) s0[e] += p0[e], s1[e] += p1[e];
            }
            if (store_sum) {
                const int64_t to = a.sum_by_pos || !a.plan.order ? pos : (int64_t)a.plan.order[pos];
                *reinterpret_cast<v4f *>(a.sum + to * a.r + c) = s0;
                *reinterpret_cast<v4f *>(a.sum + to * a.r + c + 4) = s1;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s0[e] *= scale, s1[e] *= scale;
            mx = __builtin_fmaxf(mx, __builtin_fmaxf(__builtin_fabsf(s0[e]), __builtin_fabsf(s1[e])));
        }
        *reinterpret_cast<v4f *>(dst + c * 4) = s0;
        *reinterpret_cast<v4f *>(dst + c * 4 + 16) = s1;
    }
    float f = 1.f;
    if constexpr (!T::kBf16) {
        for (int off = TPR / 2; off > 0; off >>= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, off, kWave));
        int e = exponent_or_zero(mx);
        e = e < -100 ? -100 : e;  // 13 - e <= 113, inside the range of pow2
        f = mx > 0.f && mx < __builtin_inff() ? pow2(13 - e) : 1.f;
        if (q == 0) rfac[i] = mx > 0.f && mx < __builtin_inff() ? pow2(e - 13) : 1.f;
    }
    for (int c = q * 8; c < a.r; c += TPR * 8) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = *reinterpret_cast<const float *>(dst + c * 4 + e * 4) * f;
        v4i hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint16_t h0 = T::from_f32(v[2 * e]), h1 = T::from_f32(v[2 * e + 1]);
            const uint16_t l0 = T::from_f32(v[2 * e] - T::to_f32(h0)), l1 = T::from_f32(v[2 * e + 1] - T::to_f32(h1));
            hi[e] = (int)((uint32_t)h0 | (uint32_t)h1 << 16);
            lo[e] = (int)((uint32_t)l0 | (uint32_t)l1 << 16);
        }
        *reinterpret_cast<v4i *>(dst + c * 4) = hi;
        *reinterpret_cast<v4i *>(dst + c * 4 + 16) = lo;
    }
    if (a.r % 32)
        for (int c = a.r + q * 8; c < (a.r + 31) / 32 * 32; c += TPR * 8)
            *reinterpret_cast<v4i *>(dst + c * 4) = *reinterpret_cast<v4i *>(dst + c * 4 + 16) = v4i{0, 0, 0, 0};
}

// 64 output columns from col0 of the tile's rows, by one wave. Sub-tile s (of four) of
// the matrix product holds columns 16 (i / 4) + 4 s + i % 4, i = 0..15, so a lane ends
// with 16 consecutive columns of one row: two 16-byte loads and stores.
template <class T, int NG, bool KMAJOR>
__device__ __forceinline__ void expand_block(const ExpandArgs &a, const Tile &t, const uint16_t *w, int64_t col0,
                                             const uint8_t *hl, int stride, const float *rfac, const int *rows,
                                             uint16_t *wl) {
    const int lane = threadIdx.x % kWave, li = lane & 15, g = lane >> 4;
    v4f acc[NG][4] = {};
    const int64_t mycol = col0 + g * 16;
    v4i base[NG][2];
#pragma unroll
    for (int q = 0; q < NG; ++q) {
        const int i = q * 16 + li;
        if (a.base && i < t.rows && mycol < a.n) {
            const uint16_t *p = a.base + (int64_t)rows[i] * a.n + mycol;
            base[q][0] = load16(p);
            base[q][1] = load16(p + 8);
        } else {
            base[q][0] = base[q][1] = v4i{0, 0, 0, 0};
        }
    }
    for (int k0 = 0; k0 < a.r; k0 += 32) {
        v4i wf[4];
        if constexpr (!KMAJOR) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int64_t col = col0 + (li / 4) * 16 + s * 4 + li % 4;
                const int k = k0 + g * 8 < a.r ? k0 + g * 8 : a.r - 8;
                wf[s] = load16(w + (col < a.n ? col : a.n - 1) * a.r + k);
            }
        } else {
            // 32 ranks x 64 columns to this wave's LDS, eight columns a chunk
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = j * kWave + lane, k = k0 + c / 8;
                const int64_t col = col0 + c % 8 * 8;
                const v4i v = load16(w + (int64_t)(k < a.r ? k : a.r - 1) * a.n + (col < a.n ? col : a.n - 8));
                *reinterpret_cast<v4i *>(wl + c * 8) = v;
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint16_t *p = wl + (g * 8 + li / 4) * 64 + (li % 4) * 16 + s * 4;
                const v4s p0 = read_tr16(p), p1 = read_tr16(p + 4 * 64);
                wf[s] = join(p0, p1);
            }
            __builtin_amdgcn_wave_barrier();
        }
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            const uint8_t *p = hl + (q * 16 + li) * stride + (k0 + g * 8) * 4;
            const v4i hi = load16(p), lo = load16(p + 16);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                acc[q][s] = T::mfma(wf[s], lo, acc[q][s]);
                acc[q][s] = T::mfma(wf[s], hi, acc[q][s]);
            }
        }
    }
    if (mycol >= a.n) return;
#pragma unroll
    for (int q = 0; q < NG; ++q) {
        const int i = q * 16 + li;
        if (i >= t.rows) continue;
        const float f = T::kBf16 ? 1.f : rfac[i];
        v4i o[2];
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int word = base[q][s / 2][(s % 2) * 2 + e];
                const float v0 = T::to_f32(half_of(word, 0)) + acc[q][s][2 * e] * f;
                const float v1 = T::to_f32(half_of(word, 1)) + acc[q][s][2 * e + 1] * f;
                o[s / 2][(s % 2) * 2 + e] = (int)((uint32_t)T::from_f32(v0) | (uint32_t)T::from_f32(v1) << 16);
            }
        uint16_t *p = a.out + (int64_t)rows[i] * a.n + mycol;
        *reinterpret_cast<v4i *>(p) = o[0];
        *reinterpret_cast<v4i *>(p + 8) = o[1];
    }
}

// Rows without an adapter: out = base (or 0), sums 0.
__device__ __forceinline__ void expand_plain(const ExpandArgs &a, const int *rows, int nrows, int64_t c0, int64_t c1,
                                             bool store_sum) {
    if (store_sum && !a.sum_by_pos)
        for (int j = threadIdx.x; j < nrows * (a.r / 4); j += 256)
            *reinterpret_cast<v4f *>(a.sum + (int64_t)rows[j / (a.r / 4)] * a.r + j % (a.r / 4) * 4) = v4f{0.f, 0.f, 0.f, 0.f};
    if (a.base == a.out) return;
    const int per = (int)((c1 - c0) / 8);
    for (int j = threadIdx.x; j < nrows * per; j += 256) {
        const int64_t at = (int64_t)rows[j / per] * a.n + c0 + j % per * 8;
        *reinterpret_cast<v4i *>(a.out + at) = a.base ? load16(a.base + at) : v4i{0, 0, 0, 0};
    }
}

template <class T, bool KMAJOR>
__global__ __launch_bounds__(256) void expand_kernel(ExpandArgs a, int64_t nc) {
    extern __shared__ __align__(16) uint8_t dyn[];
    const Tile t = tile_of(a.plan, blockIdx.x, a.b);
    if (t.rows == 0) return;
    int *const rows = reinterpret_cast<int *>(dyn);             // [64] token rows
    float *const rfac = reinterpret_cast<float *>(dyn + 256);   // [64]
    uint16_t *const wl = reinterpret_cast<uint16_t *>(dyn + 512) + (threadIdx.x / kWave) * (KMAJOR ? 2048 : 0);
    uint8_t *const hl = dyn + 512 + (KMAJOR ? 16384 : 0);
    if ((int)threadIdx.x < t.rows)
        rows[threadIdx.x] = (int)(a.plan.order ? a.plan.order[t.first + threadIdx.x] : t.first + threadIdx.x);
    const int64_t c0 = blockIdx.y * nc, c1 = c0 + nc < a.n ? c0 + nc : a.n;
    const bool store_sum = a.sum && blockIdx.y == 0;
    if (t.adapter < 0) {
        __syncthreads();
        expand_plain(a, rows, t.rows, c0, c1, store_sum);
        return;
    }
    const float scale = a.scale ? a.scale[t.adapter] : 1.f;
    const int stride = (a.r + 31) / 32 * 128 + 16;
    const uint16_t *w = a.w + (int64_t)t.adapter * a.r * a.n;
    const int wave = threadIdx.x / kWave;
    if (t.rows <= 16) {
        expand_rows<T, 1>(a, t, scale, hl, stride, rfac, store_sum);
        __syncthreads();
        for (int64_t c = c0 + wave * 64; c < c1; c += 256) expand_block<T, 1, KMAJOR>(a, t, w, c, hl, stride, rfac, rows, wl);
    } else {
        expand_rows<T, 4>(a, t, scale, hl, stride, rfac, store_sum);
        __syncthreads();
        for (int64_t c = c0 + wave * 64; c < c1; c += 256) expand_block<T, 4, KMAJOR>(a, t, w, c, hl, stride, rfac, rows, wl);
    }
}

template <class T, bool KMAJOR>
static hipError_t expand_launch(const ExpandArgs &a, hipStream_t stream) {
    // columns a CTA: 256 (64 a wave), more where that still leaves four CTAs a compute unit
    int64_t nc = 256;
    while (nc < 1024 && a.tiles * ((a.n + 2 * nc - 1) / (2 * nc)) >= 1024) nc *= 2;
    const size_t lds = 512 + (KMAJOR ? 16384 : 0) + (size_t)kTileRows * ((a.r + 31) / 32 * 128 + 16);
    const dim3 grid((unsigned)a.tiles, (unsigned)((a.n + nc - 1) / nc));
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(expand_kernel<T, KMAJOR>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    expand_kernel<T, KMAJOR><<<grid, 256, lds, stream>>>(a, nc);
    return hipGetLastError();
}

hipError_t launch_expand(const ExpandArgs &a, hipStream_t stream) {
    if (a.bf16) return a.kmajor ? expand_launch<BF16, true>(a, stream) : expand_launch<BF16, false>(a, stream);
    return a.kmajor ? expand_launch<F16, true>(a, stream) : expand_launch<F16, false>(a, stream);
}

}  // namespace twq
