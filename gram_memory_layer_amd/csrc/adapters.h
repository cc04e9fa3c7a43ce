// Low-rank adapters beside the shared projection: what the projection's
// kernels need to add one to their output tiles.
//
//   kv[m][n] = bf16( sum_k a[m][k] w[n][k] + sum_r up[j][n][r] * u[m][r] ),
//   u[m][r]  = scale[j] * sum_k down[j][r][k] a[m][k],   j = ids[(m0 + m) / seg].
//
// u comes from a kernel of its own (adapters.hip) in fp32 and is kept as a bf16
// pair, hi = bf16(u) and lo = bf16(u - hi), which leaves 2^-16 of it: the second
// product then runs on the matrix cores, up . hi + up . lo on top of the
// projection's fp32 accumulators, and there is one rounding to bf16 at the end.
//
// A position's output never touches another adapter's weights, so that a NaN
// or an infinity in them stays with the requests that use them: where the 32
// (or 16) positions of an MFMA do not all have the adapter, the product goes to
// a copy of the accumulators and only the lanes that ask for it take it over.
// The sum is the same either way, whatever the positions around it ask for.
#pragma once

#include "tiles.h"

namespace engram {

// No adapters: the projection alone, rows in order.
struct NoAdapters {
    static constexpr bool on = false;
};

struct AddAdapters {
    static constexpr bool on = true;
    const uint16_t* up;   // [n][n_out][rank], at this launch's first column
    const uint16_t* u;    // [M][rp / 8][hi, lo][8]
    const int32_t* ids;   // position m of this launch takes ids[(first + m) / seg]
    // [M up to a multiple of 256] (position, adapter or -1) of each tile row,
    // positions of one adapter together; rows behind the last one hold
    // (M - 1, -1).  Null: positions in order.
    const int2* tile;
    int64_t first;
    int n, rank, rp, seg;
    int64_t up_stride;  // n_out * rank

    __device__ __forceinline__ int raw(int64_t m) const {
        return ids[seg == 1 ? first + m : (first + m) / seg];
    }
    __device__ __forceinline__ int id_of(int64_t m) const {
        const int j = raw(m);
        return j >= 0 && j < n ? j : -1;
    }
    // whether position m's id is one that is neither an adapter nor -1
    __device__ __forceinline__ bool bad(int64_t m) const {
        const int j = raw(m);
        return j < -1 || j >= n;
    }
    // u's 8 ranks from r on, as hi or lo
    __device__ __forceinline__ const uint16_t* pair(int64_t m, int r, int lo) const {
        return u + (m * rp + r) * 2 + lo * 8;
    }

    // For a kernel without free LDS: straight from memory.
    // acc[jt][it]: output columns n0 + 32 jt .. (of N) and tile rows
    // m0 + 32 it ..; lane: row m0 + 32 it + lane % 32, columns
    // 8 (v / 4) + 4 (lane / 32) + v % 4
    template <int TI, int TJ>
    __device__ __forceinline__ void add(f32x16 (&acc)[TJ][TI], int64_t m0, int n0, int N,
                                        int lane) const {
        const int lrow = lane & 31, lhalf = lane >> 5;
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            const int2 own = tile[m0 + i * 32 + lrow];
            const int64_t m = own.x;
            const int mine = own.y;
            uint64_t todo = __ballot(mine >= 0);
            while (todo) {
                const int j = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
                const bool hit = mine == j;
                todo &= ~__ballot(hit);
                const uint16_t* upj = up + j * up_stride;
#pragma unroll
                for (int t = 0; t < TJ; ++t) {
                    const int col = n0 + t * 32 + lrow;
                    f32x16 d = acc[t][i];
                    for (int r0 = 0; r0 < rp; r0 += 16) {
                        const int r = r0 + 8 * lhalf;
                        const bf16x8 hi = *reinterpret_cast<const bf16x8*>(pair(m, r, 0));
                        const bf16x8 lo = *reinterpret_cast<const bf16x8*>(pair(m, r, 1));
                        bf16x8 b = {};
                        if (col < N && r < rank)
                            b = *reinterpret_cast<const bf16x8*>(upj + (int64_t)col * rank + r);
                        d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, hi, d, 0, 0, 0);
                        d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, lo, d, 0, 0, 0);
                    }
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[t][i][v] = hit ? d[v] : acc[t][i][v];
                }
            }
        }
    }
};

// 16-byte slot of logical chunk c in an LDS row of 4 (the pairs of 16 ranks) or 2
// chunks (an up row's 16 ranks): XORed with the row so that one chunk of
// consecutive rows is spread over the banks.
__device__ __forceinline__ int slot_pair(int row, int c) {
    return c ^ (((row >> 1) & 3) ^ ((row >> 3) & 1));
}
__device__ __forceinline__ int slot_up(int row, int c) { return c ^ ((row >> 2) & 1); }

// The adapters of a whole BT x BT tile (rows p0 .. of M, columns n0 .. of N),
// through LDS in up to 64 ranks at a time: the rows' pairs, and the up rows of
// as many of the tile's adapters as fit, arrive by DMA in groups of 16 ranks
// (whole 1 KiB pieces; loaded straight into the fragment layout, every wave
// fetches 32 lines a load), then each wave multiplies as in the projection's
// own k-steps.  The pairs of the first 64 ranks are fetched beside the
// projection's last k-tile, into the LDS stage that it leaves free.
//   own[k]: position and adapter of row p0 + 64 k + lane
// NW waves, the calling one at rows wm * 32 TI, columns wn * 32 TJ.
constexpr int kPairBytes = 64, kUpBytes = 32;  // of a row in a group of 16 ranks

template <int BT, int NW>
__device__ __forceinline__ void load_pairs(const AddAdapters& ad, const int2 (&own)[BT / 64],
                                           int64_t M, int wave, int lane, int r0, uint8_t* pairs) {
    constexpr int LU = BT / 16;  // DMA instructions of a group: 16 rows of 4 chunks
    static_assert(LU % NW == 0, "DMA shares");
    const __amdgpu_buffer_rsrc_t ru = make_rsrc(ad.u, (uint32_t)(M * ad.rp * 4));
    const int groups = min(4, (ad.rp - r0) / 16);
#pragma unroll
    for (int i = 0; i < LU / NW; ++i) {
        const int seg = (LU / NW) * wave + i;
        const int row = seg * 16 + (lane >> 2);
        const int c = slot_pair(row, lane & 3);
        int m = 0;
#pragma unroll
        for (int k = 0; k < BT / 64; ++k) {
            const int x = __shfl(own[k].x, row & 63, 64);
            m = (row >> 6) == k ? x : m;
        }
        const uint32_t off = (uint32_t)m * (uint32_t)(ad.rp * 4) + (uint32_t)(r0 * 4 + c * 16);
        for (int g = 0; g < groups; ++g)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ru, (lds_void*)(pairs + g * (BT * kPairBytes) + seg * 1024), 16, off, g * 64, 0, 0);
    }
}

// whether a row of the tile has an adapter (every wave holds the same rows)
template <int R>
__device__ __forceinline__ bool any_adapter(const int2 (&own)[R]) {
    bool any = false;
#pragma unroll
    for (int k = 0; k < R; ++k) any |= __ballot(own[k].y >= 0) != 0;
    return any;
}

// `pairs`: BT * 256 bytes, holding the first ranks' (or on their way there);
// `ups`: BT * 256 bytes, free.  Both are free afterwards.
template <int BT, int NW, int TI, int TJ>
__device__ __forceinline__ void add_tile(const AddAdapters& ad, f32x16 (&acc)[TJ][TI],
                                         const int2 (&own)[BT / 64], int64_t M, int n0, int N,
                                         int wm, int wn, int wave, int lane, uint8_t* pairs,
                                         uint8_t* ups) {
    // DMA instructions of an adapter's group: 32 rows of 2 chunks
    constexpr int LB = BT / 32, EACH = LB > NW ? LB / NW : 1;
    static_assert(LB % NW == 0 || LB < NW, "DMA shares");
    const int lrow = lane & 31, lhalf = lane >> 5;
    if (!any_adapter(own)) return;
    for (int r0 = 0; r0 < ad.rp; r0 += 64) {
        const int groups = min(4, (ad.rp - r0) / 16);
        const int fit = 8 / groups;  // adapters at once
        if (r0) load_pairs<BT, NW>(ad, own, M, wave, lane, r0, pairs);
        uint64_t todo[BT / 64];
#pragma unroll
        for (int k = 0; k < BT / 64; ++k) todo[k] = __ballot(own[k].y >= 0);
        // the next adapter of `left`, which loses it; -1: none
        auto next = [&](uint64_t (&left)[BT / 64], uint64_t (&has)[BT / 64]) {
            int j = -1;
#pragma unroll
            for (int k = BT / 64 - 1; k >= 0; --k)
                if (left[k]) j = __builtin_amdgcn_readlane(own[k].y, __builtin_ctzll(left[k]));
#pragma unroll
            for (int k = 0; k < BT / 64; ++k) {
                has[k] = __ballot(own[k].y == j);
                left[k] &= ~has[k];
            }
            return j;
        };
        for (;;) {
            uint64_t load[BT / 64], has[BT / 64];
#pragma unroll
            for (int k = 0; k < BT / 64; ++k) load[k] = todo[k];
            int taken = 0;
            for (; taken < fit; ++taken) {
                const int j = next(load, has);
                if (j < 0) break;
                const __amdgpu_buffer_rsrc_t rb =
                    make_rsrc(ad.up + j * ad.up_stride + (int64_t)n0 * ad.rank,
                              (uint32_t)(min(BT, N - n0) * ad.rank * 2));
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    const int seg = EACH * wave + i;
                    if (LB < NW && seg >= LB) break;
                    const int row = seg * 32 + (lane >> 1);
                    const int c = slot_up(row, lane & 1);
                    for (int g = 0; g < groups; ++g) {
                        // (ranks past the last read as zeros)
                        const int r = r0 + 16 * g + 8 * c;
                        const uint32_t off =
                            r < ad.rank ? (uint32_t)(row * ad.rank + r) * 2u : 0xFFFFFFF0u;
                        __builtin_amdgcn_raw_ptr_buffer_load_lds(
                            rb,
                            (lds_void*)(ups + (taken * groups + g) * (BT * kUpBytes) + seg * 1024),
                            16, off, 0, 0, 0);
                    }
                }
            }
            if (taken == 0) break;
            __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
            __syncthreads();
            for (int x = 0; x < taken; ++x) {
                next(todo, has);
#pragma unroll
                for (int i = 0; i < TI; ++i) {
                    const int first = (wm * TI + i) * 32;  // this wave's 32 rows
                    uint64_t h = 0;
#pragma unroll
                    for (int k = 0; k < BT / 64; ++k) h = (first >> 6) == k ? has[k] : h;
                    const uint32_t mask = (uint32_t)(h >> (first & 32));
                    if (mask == 0) continue;
                    const bool hit = (mask >> lrow) & 1;
                    const int row = first + lrow;
                    f32x16 d[TJ];
#pragma unroll
                    for (int t = 0; t < TJ; ++t) d[t] = acc[t][i];
#pragma unroll 1
                    for (int g = 0; g < groups; ++g) {
                        const uint8_t* pu = pairs + g * (BT * kPairBytes) + row * kPairBytes;
                        const uint8_t* pb = ups + (x * groups + g) * (BT * kUpBytes);
                        const bf16x8 hi = *reinterpret_cast<const bf16x8*>(
                            pu + slot_pair(row, 2 * lhalf) * 16);
                        const bf16x8 lo = *reinterpret_cast<const bf16x8*>(
                            pu + slot_pair(row, 2 * lhalf + 1) * 16);
#pragma unroll
                        for (int t = 0; t < TJ; ++t) {
                            const int brow = (wn * TJ + t) * 32 + lrow;
                            const bf16x8 b = *reinterpret_cast<const bf16x8*>(
                                pb + brow * kUpBytes + slot_up(brow, lhalf) * 16);
                            d[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, hi, d[t], 0, 0, 0);
                            d[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, lo, d[t], 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < TJ; ++t)
#pragma unroll
                        for (int v = 0; v < 16; ++v) acc[t][i][v] = hit ? d[t][v] : acc[t][i][v];
                }
            }
            __syncthreads();  // the up rows (and, behind the last round, the pairs) are read
        }
    }
}

}  // namespace engram
