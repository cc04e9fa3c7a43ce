// Low-rank adapters beside the shared projection: what the projection's
// kernels need to add one to their output tiles.
//
//   kv[m][n] = bf16( sum_k a[m][k] w[n][k] + sum_r up[j][n][r] * u[m][r] ),
//   u[m][r]  = scale[j] * sum_k down[j][r][k] a[m][k],   j = ids[m / seg],
//
// with u in fp32 (adapters.hip) and one rounding to bf16 at the end.
#pragma once

#include "tiles.h"

namespace engram {

// No adapters: the projection alone.
struct NoAdapters {
    static constexpr bool on = false;
};

// The second product of the adapters, added to a wave's 32 x 32 MFMA
// accumulators before they are rounded and stored.
//
// u is taken as a bf16 pair (hi = bf16(u), lo = bf16(u - hi)), which leaves
// 2^-16 of it, so that the product runs on the matrix cores at fp32-like
// accuracy.  One adapter of the wave's 32 positions at a time: its product is
// formed for all 32 positions and added to the lanes (one position each) that
// ask for it, so a position's output never touches another adapter's weights
// (a NaN or an infinity in them stays with the requests that use them).
struct AddAdapters {
    static constexpr bool on = true;
    const uint16_t* up;  // [n][n_out][rank], at this launch's first column
    const float* u;      // [M][rp]
    const int32_t* ids;
    int n, rank, rp, seg;
    int64_t up_stride;  // n_out * rank

    __device__ __forceinline__ int id_of(int64_t m) const {
        const int j = ids[seg == 1 ? m : m / seg];
        return j >= 0 && j < n ? j : -1;
    }

    // acc[jt][it]: output columns n0 + 32 jt .. (of N) and positions
    // m0 + 32 it .. (of M); lane: position m0 + 32 it + lane % 32, columns
    // 8 (v / 4) + 4 (lane / 32) + v % 4
    template <int TI, int TJ>
    __device__ __forceinline__ void add(f32x16 (&acc)[TJ][TI], int64_t m0, int64_t M, int n0, int N,
                                        int lane) const {
        const int lrow = lane & 31, lhalf = lane >> 5;
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            const int64_t m = m0 + i * 32 + lrow;
            const int mine = m < M ? id_of(m) : -1;
            const float* um = u + (m < M ? m : M - 1) * rp + 8 * lhalf;
            uint64_t todo = __ballot(mine >= 0);
            while (todo) {
                const int j = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
                const bool hit = mine == j;
                todo &= ~__ballot(hit);
                const uint16_t* upj = up + j * up_stride;
                f32x16 d[TJ];
#pragma unroll
                for (int t = 0; t < TJ; ++t)
#pragma unroll
                    for (int v = 0; v < 16; ++v) d[t][v] = 0.0f;
                for (int r0 = 0; r0 < rp; r0 += 16) {
                    const float4 f0 = *reinterpret_cast<const float4*>(um + r0);
                    const float4 f1 = *reinterpret_cast<const float4*>(um + r0 + 4);
                    const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
                    bf16x8 hi, lo;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        hi[e] = (__bf16)f[e];
                        const float rest = f[e] - (float)hi[e];
                        lo[e] = (__bf16)(__builtin_fabsf((float)hi[e]) < INFINITY ? rest : 0.0f);
                    }
#pragma unroll
                    for (int t = 0; t < TJ; ++t) {
                        const int col = n0 + t * 32 + lrow;
                        bf16x8 b = {};
                        if (col < N && r0 + 8 * lhalf < rank)
                            b = *reinterpret_cast<const bf16x8*>(upj + (int64_t)col * rank + r0 +
                                                                 8 * lhalf);
                        d[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, hi, d[t], 0, 0, 0);
                        d[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, lo, d[t], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int t = 0; t < TJ; ++t)
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[t][i][v] += hit ? d[t][v] : 0.0f;
            }
        }
    }
};

}  // namespace engram
