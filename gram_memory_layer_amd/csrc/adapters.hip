// Low-rank adapters of many requests beside the shared projection (stage 3
// with a rank-r correction for each request; the Engram block's self.wkv is
// the shared part).  Two kernels: the first product, u = scale * down . a, in
// fp32 (here), then the projection with the second product, up . u, added to
// its accumulators (adapters.h, wkv.hip).
#include "adapters.h"

namespace engram {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// u[m][r] = scale[j] * sum_k down[j][r][k] * a[m][k] for the positions m of
// adapter j; r >= rank (up to rp) is 0, positions without one are left.
//
// One workgroup takes 16 positions and, of their distinct adapters in order
// of first use, numbers blockIdx.y, blockIdx.y + gridDim.y, ...: a batch whose
// positions all differ is spread over gridDim.y workgroups, one request's
// positions are one workgroup's work.  Its four waves split K and meet in LDS.
// v_mfma_f32_16x16x32_bf16 takes down as A (its row r0 + lane % 16) and the
// positions as B (lane % 16), 8 consecutive k a lane; both come straight from
// memory in that order.
template <int RT>  // rank tiles of 16
__global__ void __launch_bounds__(256) adapter_down_kernel(
    const uint16_t* __restrict__ a, const uint16_t* __restrict__ down,
    const float* __restrict__ scale, const int32_t* __restrict__ ids, int64_t M, int K, int n,
    int rank, int seg, float* __restrict__ u, uint32_t* __restrict__ err) {
    __shared__ float part[4][RT * 16][17];
    const int64_t m0 = (int64_t)blockIdx.x * 16;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quad = lane >> 4;
    const int64_t m = m0 + col < M ? m0 + col : M - 1;
    int mine = -1;
    if (m0 + col < M) {
        const int j = ids[seg == 1 ? m : m / seg];
        if (j >= 0 && j < n)
            mine = j;
        else if (j != -1 && err && blockIdx.y == 0 && tid < 16)
            atomicOr(err, ENGRAM_ERRBIT_ADAPTER);
    }
    const int steps = K / 32, per = (steps + 3) / 4;
    const int s0 = wave * per, s1 = min(steps, s0 + per);
    const uint16_t* am = a + m * K + 8 * quad;

    uint32_t todo = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
    for (int turn = 0; todo; ++turn) {
        const int j = __builtin_amdgcn_readlane(mine, __builtin_ctz(todo));
        todo &= ~(uint32_t)__ballot(mine == j);
        if (turn % gridDim.y != blockIdx.y) continue;
        const uint16_t* dj = down + (int64_t)j * rank * K + 8 * quad;
        f32x4 acc[RT];
        const uint16_t* dr[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            acc[t] = f32x4{0, 0, 0, 0};
            dr[t] = dj + (int64_t)min(16 * t + col, rank - 1) * K;
        }
#pragma unroll 4
        for (int s = s0; s < s1; ++s) {
            const bf16x8 fa = *reinterpret_cast<const bf16x8*>(am + 32 * s);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const bf16x8 fd = *reinterpret_cast<const bf16x8*>(dr[t] + 32 * s);
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fd, fa, acc[t], 0, 0, 0);
            }
        }
        // D[r][m]: lane holds m = lane % 16, r = 4 (lane / 16) + v
        __syncthreads();  // the last adapter's sums are read
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) part[wave][16 * t + 4 * quad + v][col] = acc[t][v];
        __syncthreads();
        const float sc = scale ? scale[j] : 1.0f;
        // (mine is the same in every wave and quad: lane % 16 names the position)
        const int rp = (rank + 15) & ~15;
        for (int r = tid >> 4; r < rp; r += 16) {
            const float sum = (part[0][r][col] + part[1][r][col]) +
                              (part[2][r][col] + part[3][r][col]);
            if (mine == j) u[m * rp + r] = r < rank ? sc * sum : 0.0f;
        }
    }
}

template <int RT>
hipError_t run_down(const uint16_t* a, const Adapters& ad, const int32_t* ids, int seg, int64_t M,
                    int K, float* u, uint32_t* err, hipStream_t s) {
    const int64_t tiles = (M + 15) / 16;
    int ny = ad.n < 16 ? ad.n : 16;
    if (ny > M) ny = (int)M;
    adapter_down_kernel<RT><<<dim3((uint32_t)tiles, ny), dim3(256), 0, s>>>(
        a, ad.down, ad.scale, ids, M, K, ad.n, ad.rank, seg, u, err);
    return hipGetLastError();
}

}  // namespace

size_t adapters_scratch_bytes(int rank, int64_t M) {
    return (size_t)M * ((rank + 15) / 16 * 16) * sizeof(float);
}

hipError_t launch_wkv_adapters(const uint16_t* a, const uint16_t* w, const Adapters& ad,
                               const int32_t* ids, int seg, int64_t M, int N, int K, uint16_t* kv,
                               void* scratch, uint32_t* err, hipStream_t s) {
    if (M == 0) return hipSuccess;
    float* u = (float*)scratch;
    const int rt = (ad.rank + 15) / 16;
    hipError_t e = rt <= 1   ? run_down<1>(a, ad, ids, seg, M, K, u, err, s)
                   : rt <= 2 ? run_down<2>(a, ad, ids, seg, M, K, u, err, s)
                   : rt <= 4 ? run_down<4>(a, ad, ids, seg, M, K, u, err, s)
                             : run_down<8>(a, ad, ids, seg, M, K, u, err, s);
    if (e != hipSuccess) return e;
    const AddAdapters add{ad.up, u, ids, ad.n, ad.rank, rt * 16, seg, (int64_t)N * ad.rank};
    return launch_wkv_added(a, w, M, N, K, add, kv, s);
}

}  // namespace engram
