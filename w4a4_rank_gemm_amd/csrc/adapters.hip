// adapters.hip -- low-rank adapters of many requests beside a shared projection (gfx950).
//
//   H[i] = A_a x_i,   out[i] = y_i + c_a B_a H[i]        a = adapter of token row i
//
// and the two products of its gradient that have one row per token,
//
//   G[i] = B_a^T dy_i,   dX[i] = dx_i + c_a A_a^T G[i].
//
// Token rows are grouped by adapter (the plan), so a tile of 16, 64 or 128 rows shares one
// adapter's weights, whatever the order of the requests in the batch; no row is moved.
// A product is two launches, shrink (K = the long axis, partial sums over K slices) and expand
// (K = the rank), with a split of the sums between them for many rows. All are bound by memory:
// shrink by the rows and the adapters' first factors, expand by the read and write of the
// output rows. All sums are in binary32 and in a fixed order, so equal calls give equal bits.
#include "twq_adapters.h"
#include "twq_adapters_device.h"

namespace twq {

// ---- plan ----------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;

// CTA a owns adapter a (CTA `count`: the rows without one). It counts every adapter's
// rows, from which its own first position, first tile and first piece follow, then
// scans the index again and writes its rows in token order. Every CTA repeats the count, so that
// one launch does without a sum across CTAs; bound by the second scan's steps of 1024 rows, one
// after the other (one row 6 us, 4096 rows of 6 adapters 12-14, 8192 of 16 16-21; 2^20 of 16 1.25 ms,
// 2^24 of 3 21 ms, of 256 32 ms; made once for all layers of a batch).
__global__ __launch_bounds__(kPlanThreads) void adapter_plan_kernel(const int32_t *index, int64_t b, int count, uint8_t *plan,
                                                           PlanLayout L, int chunk, int trows) {
    __shared__ int hist[kMaxAdapters + 1];
    __shared__ int red[9][kPlanThreads / kWave];
    __shared__ int wsum[kPlanThreads / kWave];
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const int a = blockIdx.x;
    for (int k = tid; k <= count; k += kPlanThreads) hist[k] = 0;
    __syncthreads();
    for (int64_t i = tid; i < b; i += kPlanThreads) {
        const int key = index[i];
        atomicAdd(&hist[(unsigned)key < (unsigned)count ? key : count], 1);
    }
    __syncthreads();
    const int rows = hist[a], rest = rows % chunk;
    // Rows, tiles, whole pieces and partial-sum slots before adapter a; all whole pieces; the
    // shorter pieces before a's; all shorter pieces; the adapters without rows before a; all of
    // those. Pieces lie longest first, so that no long one starts last; an adapter without rows
    // has one of no rows, for its zeros.
    int s[9] = {0, 0, 0, 0, 0, 0, 0, 0, 0};
    for (int k = tid; k <= count; k += kPlanThreads) {
        const int c = hist[k];
        if (k < a) {
            s[0] += c;
            s[1] += (c + trows - 1) / trows;
            s[2] += c / chunk;
            s[3] += c > chunk ? (c + chunk - 1) / chunk : 0;
        }
        if (k < count) {
            s[4] += c / chunk;
            const int other = c % chunk;
            s[5] += other > rest || (other == rest && k < a);
            s[6] += other > 0;
            s[7] += c == 0 && k < a;
            s[8] += c == 0;
        }
    }
#pragma unroll
    for (int q = 0; q < 9; ++q) {
        for (int off = 32; off > 0; off >>= 1) s[q] += __shfl_xor(s[q], off, kWave);
        if (lane == 0) red[q][wave] = s[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 9; ++q) {
        s[q] = 0;
        for (int w = 0; w < kPlanThreads / kWave; ++w) s[q] += red[q][w];
    }
    const int ntiles = (rows + trows - 1) / trows, nparts = (rows + chunk - 1) / chunk;
    int32_t *head = reinterpret_cast<int32_t *>(plan + L.head), *order = reinterpret_cast<int32_t *>(plan + L.order);
    int32_t *offsets = reinterpret_cast<int32_t *>(plan + L.offsets), *slot0 = reinterpret_cast<int32_t *>(plan + L.slot0);
    PlanItem *tiles = reinterpret_cast<PlanItem *>(plan + L.tiles), *chunks = reinterpret_cast<PlanItem *>(plan + L.chunks);
    if (tid == 0) {
        offsets[a] = s[0];
        if (a < count) slot0[a] = s[3];
        if (a == count) {
            offsets[count + 1] = s[0] + rows;
            head[0] = s[1] + ntiles;
            head[1] = s[4] + s[6] + s[8];
        }
    }
    for (int j = tid; j < ntiles; j += kPlanThreads) {
        const int left = rows - j * trows;
        tiles[s[1] + j] = PlanItem{a == count ? -1 : a, s[0] + j * trows, left < trows ? left : trows, -1};
    }
    if (a < count)
        for (int j = tid; j < nparts; j += kPlanThreads) {
            const int left = rows - j * chunk;
            chunks[left < chunk ? s[4] + s[5] : s[2] + j] =
                PlanItem{a, s[0] + j * chunk, left < chunk ? left : chunk, nparts > 1 ? s[3] + j : -1};
        }
    if (rows == 0) {
        if (a < count && tid == 0) chunks[s[4] + s[6] + s[7]] = PlanItem{a, s[0], 0, -1};
        return;
    }
    int pos = s[0];
    for (int64_t i0 = 0; i0 < b; i0 += kPlanThreads) {
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
        for (int w = 0; w < kPlanThreads / kWave; ++w) {
            before += w < wave ? wsum[w] : 0;
            all += wsum[w];
        }
        if (mine) {
            const int at = pos + before + __popcll(mask & ((uint64_t(1) << lane) - 1)), local = at - s[0];
            order[at] = (int32_t)i;
            int32_t *tr = reinterpret_cast<int32_t *>(plan + L.rows) + (int64_t)(s[1] + local / trows) * trows;
            tr[local % trows] = (int32_t)i;
            if (local == rows - 1)
                for (int k = local % trows + 1; k < trows; ++k) tr[k] = (int32_t)i;
        }
        pos += all;
        __syncthreads();
    }
}

hipError_t launch_adapter_plan(const int32_t *index, int64_t b, int64_t count, void *plan, hipStream_t stream) {
    adapter_plan_kernel<<<dim3((unsigned)(count + 1)), kPlanThreads, 0, stream>>>(index, b, (int)count, static_cast<uint8_t *>(plan),
                                                                        plan_layout(b, count), chunk_rows(b), tile_rows(b));
    return hipGetLastError();
}

// ---- shrink --------------------------------------------------------------------------

struct Tile {
    int adapter, rows;
    int64_t first;
    const int32_t *row;  // its token rows, the last repeated up to R; NULL: first, first + 1, ..
    __device__ __forceinline__ int64_t token(int i) const { return row ? (int64_t)row[i] : first + (i < rows ? i : rows - 1); }
};

// Tile t of the plan (rows == 0: none); without a plan, rows R t .. of one adapter. The
// plan's entries lie at places known from t alone, so that a CTA's first loads are all in
// flight together; entries past the last tile are not used.
template <int R>
__device__ __forceinline__ Tile tile_of(const PlanView &p, int64_t t, int64_t b) {
    if (p.rows == nullptr) {
        const int64_t left = b - t * R;
        return Tile{0, (int)(left < R ? left : R), t * R, nullptr};
    }
    const PlanItem it = p.tiles[t];
    return Tile{it.adapter, t < p.head[0] ? it.rows : 0, it.first, p.rows + t * R};
}

// A tile of 16 NG rows x 16 RB ranks over a slice of K, in stages of 128 elements through
// LDS. Global loads run along the rows (sixteen lanes to a row's 256 bytes): matrix operands
// loaded straight to registers put neighbouring lanes on different rows (4096 x 14336, 64 ranks:
// 40 us against 33). The next stage is on its way to registers while this one is used; two
// stages ahead, or one LDS buffer and two or three CTAs a compute unit, gained nothing. With 64
// or 128 rows (NG = 4, 8) a wave owns 16 rows; with 16 (NG = 1) a quarter of each stage, and the
// waves' sums are added in wave order. More rows read the weights less often, and all ranks up to
// 128 in one pass the rows once.
// Bound by the read of V with few ranks, with more of them by LDS as well: every wave reads a stage's
// whole weights from LDS for its 16 rows. 8192 x 14336 by 16, 32, 64 and 128 ranks takes 55, 59, 66 and
// 87 us (4.3 to 2.7 TB/s of V; a 1 GiB copy moves 5.1), LDS active in 25, 32, 42 and 56% of the
// compute units' busy cycles, 34 to 40% of that bank conflicts. 4096 x 14336, 64 ranks, 31 us; 32
// rows of 32 adapters, 8192 x 64 each, 9.4 us (3.6 TB/s of weights).
// KMAJOR weights ([k][r], ranks contiguous) are read back from LDS transposed. W16 (the layer's own
// pair): fp16 weights whatever the rows, split exactly into two bf16 parts for bf16 rows. DX (the
// frozen layer's input gradient): the rows' largest |v sw| on the way.
template <class T, int NG, int RB, bool KMAJOR, bool DX, bool W16>
__global__ __launch_bounds__(NG == 8 ? 512 : 256) void shrink_kernel(ShrinkArgs a) {
    constexpr int NT = NG == 8 ? 512 : 256, XN = 256 * NG / NT, WN = (256 * RB + NT - 1) / NT;  // threads; chunks a thread
    constexpr int SK = 128, XS = SK * 2 + 16;                         // elements of a stage; padded LDS row of X
    constexpr int WROWS = KMAJOR ? SK : 16 * RB, WCH = KMAJOR ? 2 * RB : SK / 8;  // rows and 16-byte chunks a row of W
    constexpr int WS = WCH * 16 + 16;
    constexpr int XB = 16 * NG * XS, BUF = XB + WROWS * WS;
    constexpr int RED = NG == 1 ? 4 * RB * kWave * 16 : 0;
    __shared__ __align__(16) uint8_t smem[2 * BUF > RED ? 2 * BUF : RED];
    // Tiles of one slice, and so of one adapter's weights, on one XCD. With many rows the plan's
    // own number of tiles is dealt out, not the grid's bound on it, so that no XCD gets only
    // empty ones; with few that would be one more load to wait for.
    const int rtiles = (a.r + 16 * RB - 1) / (16 * RB);
    const int64_t tiles = NG > 1 && a.plan.rows ? a.plan.head[0] : a.tiles, ctas = tiles * rtiles * a.ks;
    if (blockIdx.x >= ctas) return;
    const int64_t id = xcd_range(blockIdx.x, ctas);
    const Tile t = tile_of<16 * NG>(a.plan, id % tiles, a.b);
    if (t.rows == 0 || t.adapter < 0) return;
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave, li = lane & 15, g = lane >> 4;
    const int rank0 = (int)(id / tiles % rtiles) * 16 * RB;
    const int64_t slice = id / tiles / rtiles, nst = (a.k + SK - 1) / SK;
    const int64_t s0 = slice * nst / a.ks, s1 = (slice + 1) * nst / a.ks;

    // chunk j of this thread: row (NT j + tid) / 16, elements 8 (tid % 16) of a stage
    int64_t at[XN];
    if (t.row) {
#pragma unroll
        for (int j = 0; j < XN; ++j) at[j] = t.row[(j * NT + tid) / 16];
    } else {
#pragma unroll
        for (int j = 0; j < XN; ++j) at[j] = t.token((j * NT + tid) / 16);
    }
    const uint16_t *xp[XN], *wp[WN];
    const uint16_t *w = a.w + (int64_t)t.adapter * a.r * a.k;
#pragma unroll
    for (int j = 0; j < XN; ++j) xp[j] = a.v + at[j] * a.k;
#pragma unroll
    for (int j = 0; j < WN; ++j) {
        const int c = (j * NT + tid) % (256 * RB);
        const int rr = rank0 + (KMAJOR ? c % WCH * 8 : c / WCH);
        wp[j] = w + (KMAJOR ? (rr < a.r ? rr : a.r - 8) : (int64_t)(rr < a.r ? rr : a.r - 1) * a.k);
    }
    v4i xr[XN], wr[WN];
    v4f sr[2];
    uint32_t mx[XN] = {};
    auto load = [&](int64_t st) {
        const int64_t k0 = st * SK;
        const int left = (int)(a.k - k0 < SK ? a.k - k0 : SK);  // elements of this stage
        const int64_t kx = tid % 16 * 8 < left ? k0 + tid % 16 * 8 : 0;  // past K: re-read, cleared when stored
#pragma unroll
        for (int j = 0; j < XN; ++j) xr[j] = load16(xp[j] + kx);
#pragma unroll
        for (int j = 0; j < WN; ++j) {
            if constexpr (KMAJOR) {
                const int kk = (j * NT + tid) % (256 * RB) / WCH;
                wr[j] = load16(wp[j] + (k0 + (kk < left ? kk : 0)) * a.r);
            } else {
                wr[j] = load16(wp[j] + kx);
            }
        }
        if constexpr (DX) {
            const float *s = a.sw + kx;
            sr[0] = *reinterpret_cast<const v4f *>(s);
            sr[1] = *reinterpret_cast<const v4f *>(s + 4);
        }
    };
    v4f acc[RB] = {};
    if (s0 < s1) load(s0);
    for (int64_t st = s0; st < s1; ++st) {
        uint8_t *buf = smem + (st & 1) * BUF;  // last read two stages ago, before the previous barrier
        if (KMAJOR && st * SK + tid % 16 * 8 >= a.k) {
#pragma unroll
            for (int j = 0; j < XN; ++j) xr[j] = v4i{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < XN; ++j) *reinterpret_cast<v4i *>(buf + (j * NT + tid) / 16 * XS + tid % 16 * 16) = xr[j];
        if constexpr (DX) {  // magnitudes in the order of their bit patterns, NaN above all
#pragma unroll
            for (int j = 0; j < XN; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = T::to_f32(half_of(xr[j][e / 2], e % 2)) * sr[e / 4][e % 4];
                    const uint32_t m = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
                    mx[j] = mx[j] > m ? mx[j] : m;
                }
        }
#pragma unroll
        for (int j = 0; j < WN; ++j) {
            const int c = j * NT + tid;
            if (256 * RB % NT == 0 || c < 256 * RB) *reinterpret_cast<v4i *>(buf + XB + c / WCH * WS + c % WCH * 16) = wr[j];
        }
        if (st + 1 < s1) load(st + 1);
        __syncthreads();
        if (NG > 1 && wave * 16 >= t.rows) continue;
#pragma unroll
        for (int u = 0; u < (NG > 1 ? 4 : 1); ++u) {
            const int e = (NG > 1 ? u : wave) * 32;  // elements e + 8 g .. + 7
            const v4i xf = load16(buf + ((NG > 1 ? wave * 16 : 0) + li) * XS + (e + g * 8) * 2);
#pragma unroll
            for (int c = 0; c < RB; ++c) {
                v4i wf;
                if constexpr (KMAJOR) {
                    const uint8_t *p = buf + XB + (e + g * 8 + li / 4) * WS + (c * 16 + (li % 4) * 4) * 2;
                    const v4s w0 = read_tr16(p), w1 = read_tr16(p + 4 * WS);
                    wf = join(w0, w1);
                } else {
                    wf = load16(buf + XB + (c * 16 + li) * WS + (e + g * 8) * 2);
                }
                if constexpr (W16 && T::kBf16) {
                    v4i hi, lo;
                    split_f16(wf, hi, lo);
                    acc[c] = T::mfma(lo, xf, acc[c]);
                    acc[c] = T::mfma(hi, xf, acc[c]);
                } else {
                    acc[c] = T::mfma(wf, xf, acc[c]);
                }
            }
        }
    }
    if constexpr (DX) {
        if (rank0 == 0) {
#pragma unroll
            for (int j = 0; j < XN; ++j) {
                const uint32_t m = row16_max(mx[j]);
                const int i = (j * NT + tid) / 16;
                if (tid % 16 == 0 && i < t.rows) a.rowmax[slice * a.b + t.first + i] = __builtin_bit_cast(float, m);
            }
        }
    }
    // lane: row li, ranks 4 g .. + 3 of each block
    if constexpr (NG > 1) {
        const int i = wave * 16 + li;
#pragma unroll
        for (int c = 0; c < RB; ++c) {
            const int rank = rank0 + c * 16 + g * 4;
            if (i < t.rows && rank < a.r) *reinterpret_cast<v4f *>(a.p + ((slice * a.b + t.first + i) * a.r + rank)) = acc[c];
        }
    } else {
        v4f *const red = reinterpret_cast<v4f *>(smem);  // [4 waves][RB][64 lanes]
        __syncthreads();
#pragma unroll
        for (int c = 0; c < RB; ++c) red[(wave * RB + c) * kWave + lane] = acc[c];
        __syncthreads();
        if (tid < RB * kWave) {
            const int i = tid & 15, rank = rank0 + tid / kWave * 16 + tid % kWave / 16 * 4;
            v4f s = red[tid];
#pragma unroll
            for (int q = 1; q < 4; ++q) {
                const v4f o = red[q * RB * kWave + tid];
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] += o[e];
            }
            if (i < t.rows && rank < a.r) *reinterpret_cast<v4f *>(a.p + ((slice * a.b + t.first + i) * a.r + rank)) = s;
        }
    }
}

template <class T, int NG, bool KMAJOR, bool DX, bool W16>
static hipError_t shrink_ranks(const ShrinkArgs &a, hipStream_t stream) {
    const int rb = a.r <= 16 ? 1 : a.r <= 32 ? 2 : a.r <= 64 || NG < 8 ? 4 : 8;
    const unsigned grid = (unsigned)(a.tiles * ((a.r + 16 * rb - 1) / (16 * rb)) * a.ks);
    constexpr int NT = NG == 8 ? 512 : 256;
    if (rb == 1)
        shrink_kernel<T, NG, 1, KMAJOR, DX, W16><<<grid, NT, 0, stream>>>(a);
    else if (rb == 2)
        shrink_kernel<T, NG, 2, KMAJOR, DX, W16><<<grid, NT, 0, stream>>>(a);
    else if (rb == 4)
        shrink_kernel<T, NG, 4, KMAJOR, DX, W16><<<grid, NT, 0, stream>>>(a);
    else if constexpr (NG == 8)
        shrink_kernel<T, NG, 8, KMAJOR, DX, W16><<<grid, NT, 0, stream>>>(a);
    return hipGetLastError();
}

template <class T, bool KMAJOR, bool DX, bool W16>
static hipError_t shrink_rows(const ShrinkArgs &a, hipStream_t stream) {
    if (a.b <= kFewRows) return shrink_ranks<T, 1, KMAJOR, DX, W16>(a, stream);
    return a.b <= kManyRows ? shrink_ranks<T, 4, KMAJOR, DX, W16>(a, stream) : shrink_ranks<T, 8, KMAJOR, DX, W16>(a, stream);
}

hipError_t launch_shrink(const ShrinkArgs &a, hipStream_t stream) {
    if (a.rowmax) return a.bf16 ? shrink_rows<BF16, true, true, true>(a, stream) : shrink_rows<F16, true, true, true>(a, stream);
    if (a.bf16 && a.w_f16) return shrink_rows<BF16, false, false, true>(a, stream);
    if (a.bf16) return a.kmajor ? shrink_rows<BF16, true, false, false>(a, stream) : shrink_rows<BF16, false, false, false>(a, stream);
    return a.kmajor ? shrink_rows<F16, true, false, false>(a, stream) : shrink_rows<F16, false, false, false>(a, stream);
}

// ---- expand --------------------------------------------------------------------------

// Four binary32 values as bf16 hi + lo (16 significant bits) to two arrays.
__device__ __forceinline__ void put_planes(uint16_t *hi, uint16_t *lo, const v4f &v) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint16_t h0 = BF16::from_f32(v[2 * e]), h1 = BF16::from_f32(v[2 * e + 1]);
        const uint16_t l0 = BF16::from_f32(v[2 * e] - BF16::to_f32(h0)), l1 = BF16::from_f32(v[2 * e + 1] - BF16::to_f32(h1));
        h[e] = (uint32_t)h0 | (uint32_t)h1 << 16;
        l[e] = (uint32_t)l0 | (uint32_t)l1 << 16;
    }
    *reinterpret_cast<uint2 *>(hi) = make_uint2(h[0], h[1]);
    *reinterpret_cast<uint2 *>(lo) = make_uint2(l[0], l[1]);
}

// A row of the first product, summed over the slices, times the adapter's scale, as two
// 16-bit parts hi + lo (8 ranks are 32 bytes, hi then lo), by the TPR threads q of a row.
// One part would round H to the element type, an error of the size of the output's own
// rounding; the second costs a matrix instruction on operands at hand. fp16 rows are first
// scaled by a power of two to a largest element in [2^13, 2^14), so neither part can
// overflow and only elements below 2^-27 of the largest lose bits; the return value is
// the factor that undoes it. Ranks past r (the last half step) are zero. dst also holds
// the binary32 sums in between.
template <class T, int TPR>
__device__ __forceinline__ float split_row(const ExpandArgs &a, int64_t pos, int64_t row, bool live, int q, float scale,
                                           bool store_sum, uint8_t *dst) {
    const float *src = a.p + pos * a.r;
    float mx = 0.f;
    for (int c = q * 8; c < a.r; c += TPR * 8) {
        v4f s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
        if (live) {
            for (int s = 0; s < a.ks; s += 8) {  // eight slices in flight
                v4f p0[8], p1[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float *ps = src + (s + j < a.ks ? s + j : s) * a.b * a.r + c;
                    p0[j] = *reinterpret_cast<const v4f *>(ps);
                    p1[j] = *reinterpret_cast<const v4f *>(ps + 4);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (s + j < a.ks) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) s0[e] += p0[j][e], s1[e] += p1[j][e];
                    }
            }
            if (store_sum && a.sum) {
                const int64_t to = (a.sum_by_pos ? pos : row) * a.r + c;
                *reinterpret_cast<v4f *>(a.sum + to) = s0;
                *reinterpret_cast<v4f *>(a.sum + to + 4) = s1;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s0[e] *= scale, s1[e] *= scale;
            mx = __builtin_fmaxf(mx, __builtin_fmaxf(__builtin_fabsf(s0[e]), __builtin_fabsf(s1[e])));
        }
        if (store_sum && live && a.planes) {
            const int64_t n = a.b * a.r, to = pos * a.r + c;
            put_planes(a.planes + to, a.planes + n + to, s0);
            put_planes(a.planes + to + 4, a.planes + n + to + 4, s1);
            v4f h0 = *reinterpret_cast<const v4f *>(a.h + row * a.r + c), h1 = *reinterpret_cast<const v4f *>(a.h + row * a.r + c + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) h0[e] *= scale, h1[e] *= scale;
            put_planes(a.planes + 2 * n + to, a.planes + 3 * n + to, h0);
            put_planes(a.planes + 2 * n + to + 4, a.planes + 3 * n + to + 4, h1);
        }
        *reinterpret_cast<v4f *>(dst + c * 4) = s0;
        *reinterpret_cast<v4f *>(dst + c * 4 + 16) = s1;
    }
    float f = 1.f, undo = 1.f;
    if constexpr (!T::kBf16) {
        for (int off = TPR / 2; off > 0; off >>= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, off, kWave));
        const int e = scale_exponent(mx);
        if (mx > 0.f && mx < __builtin_inff()) f = pow2(13 - e), undo = pow2(e - 13);
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
    for (int c = a.r + q * 8; c < (a.r + 31) / 32 * 32; c += TPR * 8)
        *reinterpret_cast<v4i *>(dst + c * 4) = *reinterpret_cast<v4i *>(dst + c * 4 + 16) = v4i{0, 0, 0, 0};
    return undo;
}

// Bytes of a row's parts.
__host__ __device__ inline int parts_bytes(int r) { return (r + 31) / 32 * 128; }

// Many rows: every column block of expand needs the rows' parts, so one launch forms them
// once, 16 threads a row. (With few rows expand forms them itself and saves the launch.) Bound by
// its start and two dependent reads: 4096 rows of 64 ranks, 6 slices, 5.3 us; 8192 rows with the
// weight gradients' parts 8.3 us.
template <class T, int R>
__global__ __launch_bounds__(256) void split_kernel(ExpandArgs a) {
    constexpr int G = R / 16;
    const Tile t = tile_of<R>(a.plan, blockIdx.x / G, a.b);
    const int i = (blockIdx.x % G) * 16 + threadIdx.x / 16, q = threadIdx.x % 16;
    if (i >= t.rows) return;
    const int64_t pos = t.first + i, row = t.row[i];
    if (t.adapter < 0) {
        if (a.sum && !a.sum_by_pos)
            for (int c = q * 4; c < a.r; c += 64) *reinterpret_cast<v4f *>(a.sum + row * a.r + c) = v4f{0.f, 0.f, 0.f, 0.f};
        return;
    }
    const float undo = split_row<T, 16>(a, pos, row, true, q, a.scale ? a.scale[t.adapter] : 1.f, true,
                                        a.parts + pos * parts_bytes(a.r));
    if (q == 0) a.undo[pos] = undo;
}

// The weights of 64 output columns from col0, for one wave: KS steps of 32 ranks x four
// sub-tiles of 16 columns. Memory is read along its rows ([n][r], or [r][n] if KMAJOR) into
// registers (fetch); then, 32 KP ranks a pass, through this wave's LDS into matrix operands
// (place), transposed if KMAJOR.
template <int KS, bool KMAJOR, int KP>
struct Weights {
    static constexpr int STRIDE = KMAJOR ? 64 * 2 + 16 : KP * 64 + 16;  // padded LDS row
    static constexpr int BYTES = (KMAJOR ? 32 : 64) * STRIDE;
    v4i in[KS / KP][KP * 4];
    __device__ __forceinline__ void fetch(const ExpandArgs &a, const uint16_t *w, int64_t col0) {
        const int lane = threadIdx.x % kWave;
#pragma unroll
        for (int p = 0; p < KS / KP; ++p)
#pragma unroll
            for (int j = 0; j < KP * 4; ++j) {
                const int c = j * kWave + lane;
                if constexpr (KMAJOR) {
                    const int k = p * 32 + c / 8;
                    const int64_t col = col0 + c % 8 * 8;
                    in[p][j] = load16(w + (int64_t)(k < a.r ? k : a.r - 1) * a.n + (col < a.n ? col : a.n - 8));
                } else {
                    const int k = p * KP * 32 + c % (KP * 4) * 8;  // past r: parts are zero
                    const int64_t col = col0 + c / (KP * 4);
                    in[p][j] = load16(w + (col < a.n ? col : a.n - 1) * a.r + (k < a.r ? k : a.r - 8));
                }
            }
    }
    __device__ __forceinline__ void place(uint8_t *wl, v4i (&wf)[KS][4]) const {
        const int lane = threadIdx.x % kWave, li = lane & 15, g = lane >> 4;
        constexpr int CH = KMAJOR ? 8 : KP * 4;  // 16-byte chunks a row
#pragma unroll
        for (int p = 0; p < KS / KP; ++p) {
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < KP * 4; ++j) {
                const int c = j * kWave + lane;
                *reinterpret_cast<v4i *>(wl + c / CH * STRIDE + c % CH * 16) = in[p][j];
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if constexpr (KMAJOR) {
                        const uint8_t *q = wl + (g * 8 + li / 4) * STRIDE + (s * 16 + (li % 4) * 4) * 2;
                        const v4s q0 = read_tr16(q), q1 = read_tr16(q + 4 * STRIDE);
                        wf[p][s] = join(q0, q1);
                    } else {
                        wf[p * KP + k][s] = load16(wl + (s * 16 + li) * STRIDE + (k * 32 + g * 8) * 2);
                    }
                }
        }
        __builtin_amdgcn_wave_barrier();
    }
};

// Rows without an adapter: out = base (or 0), sums 0.
__device__ __forceinline__ void expand_plain(const ExpandArgs &a, const Tile &t, int64_t c0, int64_t c1, bool store_sum) {
    if (store_sum && !a.sum_by_pos)
        for (int j = threadIdx.x; j < t.rows * (a.r / 4); j += 256)
            *reinterpret_cast<v4f *>(a.sum + (int64_t)t.row[j / (a.r / 4)] * a.r + j % (a.r / 4) * 4) =
                v4f{0.f, 0.f, 0.f, 0.f};
    if (a.base == a.out) return;
    const int per = (int)((c1 - c0) / 8);
    for (int j = threadIdx.x; j < t.rows * per; j += 256) {
        const int64_t at = (int64_t)t.row[j / per] * a.n + c0 + j % per * 8;
        *reinterpret_cast<v4i *>(a.out + at) = a.base ? load16(a.base + at) : v4i{0, 0, 0, 0};
    }
}

// 16 rows x 64 columns of one wave: products with the rows' parts in LDS (i0: the first row),
// turned in this wave's LDS so that eight lanes hold one row's 64 columns, added to the base
// and stored. rows[h], base[h]: this lane's row 8 h + lane / 8 of the 16 (negative: none) and
// its base at columns col0 + 8 (lane % 8).
template <class T, int KS, int STRIDE>
__device__ __forceinline__ void expand_store(const ExpandArgs &a, const uint8_t *parts, const float *undo, int i0, int last,
                                             const int64_t (&rows)[2], int64_t col0, const v4i (&wf)[KS][4],
                                             const v4i (&base)[2], uint8_t *wl) {
    constexpr int TS = 64 * 4 + 16;  // padded row of the turned block
    const int lane = threadIdx.x % kWave, li = lane & 15, g = lane >> 4;
    const int i = i0 + li < last ? i0 + li : last;
    v4f acc[4] = {};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
        if (k * 32 >= a.r) break;  // r = 96: the last step has no parts
        const uint8_t *p = parts + i * STRIDE + (k * 32 + g * 8) * 4;
        const v4i hi = load16(p), lo = load16(p + 16);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            acc[s] = T::mfma(wf[k][s], lo, acc[s]);
            acc[s] = T::mfma(wf[k][s], hi, acc[s]);
        }
    }
    const float f = T::kBf16 ? 1.f : undo[i];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[s][e] *= f;
        *reinterpret_cast<v4f *>(wl + li * TS + (s * 16 + g * 4) * 4) = acc[s];
    }
    __builtin_amdgcn_wave_barrier();
    const int64_t col = col0 + lane % 8 * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint8_t *p = wl + (h * 8 + lane / 8) * TS + lane % 8 * 32;
        const v4f d0 = *reinterpret_cast<const v4f *>(p), d1 = *reinterpret_cast<const v4f *>(p + 16);
        v4i o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x0 = e < 2 ? d0[2 * e] : d1[2 * e - 4], x1 = e < 2 ? d0[2 * e + 1] : d1[2 * e - 3];
            const float v0 = T::to_f32(half_of(base[h][e], 0)) + x0, v1 = T::to_f32(half_of(base[h][e], 1)) + x1;
            o[e] = (int)((uint32_t)T::from_f32(v0) | (uint32_t)T::from_f32(v1) << 16);
        }
        if (rows[h] >= 0 && col < a.n) *reinterpret_cast<v4i *>(a.out + rows[h] * a.n + col) = o;
    }
}

// This lane's rows 8 h + lane / 8 of the 16 from row i0 of the tile (past its end: the
// complement of the last row).
__device__ __forceinline__ void expand_rows(const ExpandArgs &a, const Tile &t, int i0, int64_t (&rows)[2]) {
    const int lane = threadIdx.x % kWave;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = i0 + h * 8 + lane / 8;
        const int32_t row = t.row[i];
        rows[h] = i < t.rows ? row : ~row;
    }
}

// Their base at this lane's eight columns (0 without a base). Rows and columns past the end
// re-read others.
__device__ __forceinline__ void expand_base(const ExpandArgs &a, const int64_t (&rows)[2], int64_t col0, v4i (&base)[2]) {
    const int64_t col = col0 + threadIdx.x % 8 * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        base[h] = a.base ? load16(a.base + (rows[h] < 0 ? ~rows[h] : rows[h]) * a.n + (col < a.n ? col : a.n - 8)) : v4i{0, 0, 0, 0};
}

constexpr int kTurnBytes = 16 * (64 * 4 + 16);

// Many rows: 64 rows (a tile of the plan or half of one) x 256 columns, 64 a wave. Row numbers,
// bases, weights and the rows' parts (split_kernel's, to LDS) are all requested before the first
// is used, and nothing is loaded after the first store (loads and stores share a counter).
// Weights pass through LDS 32 ranks at a time: up to 64 ranks that leaves room for four CTAs a
// compute unit (with 64 ranks a pass, three: 4096 x 4096, 64 ranks, 26.6 against 22.9 us).
// Bound by the base and output rows: that case moves 76 MB, 3.3 TB/s; 8192 x 4096, 64 ranks,
// 36.8 us (4.1 TB/s).
template <class T, int KS, bool KMAJOR, int TR>
__global__ __launch_bounds__(256, KS <= 2 ? 4 : 1) void expand_kernel(ExpandArgs a, int ncol) {
    using W = Weights<KS, KMAJOR, 1>;
    constexpr int R = 64, STRIDE = KS * 128 + 16, NQ = R / 16;  // padded LDS row of parts
    constexpr int WB = W::BYTES > kTurnBytes ? W::BYTES : kTurnBytes;
    __shared__ __align__(16) uint8_t parts[R * STRIDE];
    __shared__ float undo[R];
    __shared__ __align__(16) uint8_t wlds[4][WB];
    const int64_t ctas = (int64_t)a.plan.head[0] * (TR / R) * ncol;
    if (blockIdx.x >= ctas) return;
    const int64_t id = xcd_range(blockIdx.x, ctas);  // a tile's columns, and one adapter's weights, on one XCD
    Tile t = tile_of<TR>(a.plan, id / ncol / (TR / R), a.b);
    if constexpr (TR > R) {
        const int i0 = (int)(id / ncol % (TR / R)) * R, left = t.rows - i0;
        t.rows = left < 0 ? 0 : left < R ? left : R;
        t.first += i0;
        t.row += i0;
    }
    if (t.rows == 0) return;
    const int64_t c0 = id % ncol * 256, c1 = c0 + 256 < a.n ? c0 + 256 : a.n;
    if (t.adapter < 0) return expand_plain(a, t, c0, c1, false);
    const int tid = threadIdx.x, wave = tid / kWave;
    const int64_t col0 = c0 + wave * 64;

    int64_t rows[NQ][2];
#pragma unroll
    for (int q = 0; q < NQ; ++q) expand_rows(a, t, q * 16, rows[q]);
    v4i base[NQ][2], wf[KS][4];
#pragma unroll
    for (int q = 0; q < NQ; ++q) expand_base(a, rows[q], col0, base[q]);
    W in;
    in.fetch(a, a.w + (int64_t)t.adapter * a.r * a.n, col0);
    const int per = parts_bytes(a.r) / 16, total = t.rows * per;
    const uint8_t *src = a.parts + t.first * parts_bytes(a.r);
    constexpr int N = R * KS * 8 / 256;
    v4i pin[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = j * 256 + tid;
        pin[j] = load16(src + (c < total ? c : total - 1) * 16);
    }
    const float u = a.undo[t.first + (tid < t.rows ? tid : 0)];
    in.place(wlds[wave], wf);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = j * 256 + tid;
        if (c < total) *reinterpret_cast<v4i *>(parts + c / per * STRIDE + c % per * 16) = pin[j];
    }
    if (tid < R) undo[tid] = u;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        if (q * 16 >= t.rows) break;
        expand_store<T, KS, STRIDE>(a, parts, undo, q * 16, t.rows - 1, rows[q], col0, wf, base[q], wlds[wave]);
    }
}

// Few rows: a tile of 16 x `blocks` runs of 256 columns, 64 a wave. The rows' parts are
// formed here, once for all the runs, while the first run's weights are on their way; the
// next run's weights are requested before this one's are used. Bound by the weights: 32 rows of
// 32 adapters, 28672 x 64 each, 26 us (4.6 TB/s). Up to 64 ranks a pass through LDS here: the
// registers allow no fourth CTA, and 32 ranks a pass took 28 us.
template <class T, int KS, bool KMAJOR>
__global__ __launch_bounds__(256, KS == 1 ? 4 : 1) void expand_few_kernel(ExpandArgs a, int ncol, int blocks) {
    using W = Weights<KS, KMAJOR, KMAJOR || KS < 2 ? 1 : 2>;
    constexpr int STRIDE = KS * 128 + 16;
    constexpr int WB = W::BYTES > kTurnBytes ? W::BYTES : kTurnBytes;
    __shared__ __align__(16) uint8_t parts[16 * STRIDE];
    __shared__ float undo[16];
    __shared__ __align__(16) uint8_t wlds[4][WB];
    const Tile t = tile_of<16>(a.plan, blockIdx.x / ncol, a.b);
    if (t.rows == 0) return;
    const int64_t c0 = (int64_t)(blockIdx.x % ncol) * 256 * blocks, c1 = c0 + 256 * blocks < a.n ? c0 + 256 * blocks : a.n;
    const bool store_sum = c0 == 0;
    if (t.adapter < 0) return expand_plain(a, t, c0, c1, store_sum && a.sum);
    const int tid = threadIdx.x, wave = tid / kWave;
    const uint16_t *w = a.w + (int64_t)t.adapter * a.r * a.n;
    int64_t col0 = c0 + wave * 64, rows[2];
    v4i base[2], wf[KS][4];
    W in;
    in.fetch(a, w, col0);
    expand_rows(a, t, 0, rows);
    {
        const int i = tid / 16, q = tid % 16;
        const int64_t pos = t.first + (i < t.rows ? i : 0);
        const float u = split_row<T, 16>(a, pos, t.row[i], i < t.rows, q,
                                         a.scale ? a.scale[t.adapter] : 1.f, store_sum, parts + i * STRIDE);
        if (q == 0) undo[i] = u;
    }
    __syncthreads();
    for (; col0 < c1; col0 += 256) {
        in.place(wlds[wave], wf);
        expand_base(a, rows, col0, base);
        if (col0 + 256 < c1) in.fetch(a, w, col0 + 256);
        expand_store<T, KS, STRIDE>(a, parts, undo, 0, t.rows - 1, rows, col0, wf, base, wlds[wave]);
    }
}

template <class T, int KS, bool KMAJOR>
static hipError_t expand_launch(const ExpandArgs &a, hipStream_t stream) {
    if (a.b > kFewRows) {
        const int ncol = (int)((a.n + 255) / 256);
        if (a.b > kManyRows)
            expand_kernel<T, KS, KMAJOR, 128><<<(unsigned)(a.tiles * 2 * ncol), 256, 0, stream>>>(a, ncol);
        else
            expand_kernel<T, KS, KMAJOR, 64><<<(unsigned)(a.tiles * ncol), 256, 0, stream>>>(a, ncol);
        return hipGetLastError();
    }
    // Runs a CTA: as many as leave the CTAs all resident at once (the registers allow 4, 3, 2
    // or 1 a compute unit). 32 tiles of 28672 columns, 64 ranks: 1, 2, 4, 5 and 8 runs took 36, 32,
    // 33, 27 and 29 us (the one shape measured).
    constexpr int resident = 256 * (KS == 1 ? 4 : KS == 2 ? 3 : KS == 4 ? 2 : 1);
    const int64_t runs = (a.n + 255) / 256, blocks64 = (a.tiles * runs + resident - 1) / resident;
    const int blocks = (int)(blocks64 < runs ? blocks64 : runs);
    const int ncol = (int)((a.n + 256 * blocks - 1) / (256 * blocks));
    expand_few_kernel<T, KS, KMAJOR><<<(unsigned)(a.tiles * ncol), 256, 0, stream>>>(a, ncol, blocks);
    return hipGetLastError();
}

template <class T, bool KMAJOR>
static hipError_t expand_ranks(const ExpandArgs &a, hipStream_t stream) {
    if (a.r <= 32) return expand_launch<T, 1, KMAJOR>(a, stream);
    if (a.r <= 64) return expand_launch<T, 2, KMAJOR>(a, stream);
    if (a.r <= 128) return expand_launch<T, 4, KMAJOR>(a, stream);
    return expand_launch<T, 8, KMAJOR>(a, stream);
}

template <class T>
static hipError_t split_typed(const ExpandArgs &a, hipStream_t stream) {
    if (a.b > kManyRows)
        split_kernel<T, 128><<<(unsigned)(a.tiles * 8), 256, 0, stream>>>(a);
    else
        split_kernel<T, 64><<<(unsigned)(a.tiles * 4), 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_split(const ExpandArgs &a, hipStream_t stream) {
    return a.bf16 ? split_typed<BF16>(a, stream) : split_typed<F16>(a, stream);
}

hipError_t launch_expand(const ExpandArgs &a, hipStream_t stream) {
    if (a.bf16) return a.kmajor ? expand_ranks<BF16, true>(a, stream) : expand_ranks<BF16, false>(a, stream);
    return a.kmajor ? expand_ranks<F16, true>(a, stream) : expand_ranks<F16, false>(a, stream);
}

}  // namespace twq
