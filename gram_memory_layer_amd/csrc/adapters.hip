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
// adapter j, as bf16 pairs; r >= rank (up to rp) is 0, positions without one
// are left.
//
// One workgroup takes 16 positions and, of their distinct adapters in order
// of first use, numbers blockIdx.y, blockIdx.y + gridDim.y, ...: a batch whose
// positions all differ is spread over gridDim.y workgroups, one request's
// positions are one workgroup's work.  Its eight waves split K and meet in LDS.
// v_mfma_f32_16x16x32_bf16 takes down as A (its row r0 + lane % 16) and the
// positions as B (lane % 16), 8 consecutive k a lane; both come straight from
// memory in that order.
//
// With perm, one workgroup more writes the order in which the projection's
// tiles take the positions: those of one adapter together (a counting sort by
// id mod 1023; within a bucket in any order, on which no output depends), so
// that a tile meets few adapters however the requests are mixed.
constexpr int kDownWaves = 8, kBuckets = 1024;

__device__ __forceinline__ void order_positions(const AddAdapters& ad, int M, int32_t* perm,
                                                int* hist) {
    const int tid = threadIdx.x, nt = blockDim.x;
    auto bucket = [&](int m) {
        const int j = ad.id_of(m);
        return j < 0 ? 0 : 1 + j % (kBuckets - 1);
    };
    for (int i = tid; i < kBuckets; i += nt) hist[i] = 0;
    __syncthreads();
    for (int m = tid; m < M; m += nt) atomicAdd(&hist[bucket(m)], 1);
    __syncthreads();
    // exclusive sums: two buckets a thread (512 threads), doubling steps
    const int a = hist[2 * tid], b = hist[2 * tid + 1];
    int sum = a + b;
    __syncthreads();
    hist[tid] = sum;
    __syncthreads();
    for (int o = 1; o < kBuckets / 2; o <<= 1) {
        const int x = tid >= o ? hist[tid - o] : 0;
        __syncthreads();
        hist[tid] = sum = sum + x;
        __syncthreads();
    }
    __syncthreads();
    hist[2 * tid] = sum - a - b;
    hist[2 * tid + 1] = sum - b;
    __syncthreads();
    for (int m = tid; m < M; m += nt) perm[atomicAdd(&hist[bucket(m)], 1)] = m;
}

template <int RT>  // rank tiles of 16
__global__ void __launch_bounds__(64 * kDownWaves) adapter_down_kernel(
    const uint16_t* __restrict__ a, const uint16_t* __restrict__ down,
    const float* __restrict__ scale, const AddAdapters ad, int M, int K,
    uint16_t* __restrict__ u, int32_t* __restrict__ perm, uint32_t* __restrict__ err) {
    static_assert(2 * 64 * kDownWaves == kBuckets, "two buckets a thread");
    __shared__ union {
        float part[kDownWaves][RT * 16][17];
        int hist[kBuckets];
    } sh;
    const int m0 = blockIdx.x * 16;
    if (m0 >= M) {
        if (blockIdx.y == 0) order_positions(ad, M, perm, sh.hist);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quad = lane >> 4;
    const int rank = ad.rank, rp = ad.rp;
    const int m = min(m0 + col, M - 1);
    int mine = -1;
    if (m0 + col < M) {
        mine = ad.id_of(m);
        const int64_t at = ad.first + m;
        if (mine < 0 && err && blockIdx.y == 0 && tid < 16 &&
            ad.ids[ad.seg == 1 ? at : at / ad.seg] != -1)
            atomicOr(err, ENGRAM_ERRBIT_ADAPTER);
    }
    const int steps = K / 32, per = (steps + kDownWaves - 1) / kDownWaves;
    const int s0 = wave * per, s1 = min(steps, s0 + per);
    const uint16_t* am = a + (int64_t)m * K + 8 * quad;

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
#pragma unroll 3
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
            for (int v = 0; v < 4; ++v) sh.part[wave][16 * t + 4 * quad + v][col] = acc[t][v];
        __syncthreads();
        const float sc = scale ? scale[j] : 1.0f;
        // (mine is the same in every wave and quad: lane % 16 names the position)
        for (int r = tid >> 4; r < rp; r += 4 * kDownWaves) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kDownWaves; ++w) sum += sh.part[w][r][col];
            const float f = r < rank ? sc * sum : 0.0f;
            const __bf16 hi = (__bf16)f;
            // (an infinite value has no rest)
            const __bf16 lo =
                (__bf16)(__builtin_fabsf((float)hi) < INFINITY ? f - (float)hi : 0.0f);
            if (mine == j) {
                uint16_t* to = u + ((int64_t)m * rp + (r & ~7)) * 2 + (r & 7);
                to[0] = __builtin_bit_cast(uint16_t, hi);
                to[8] = __builtin_bit_cast(uint16_t, lo);
            }
        }
    }
}

template <int RT>
hipError_t run_down(const uint16_t* a, const Adapters& ad, const AddAdapters& add, int M, int K,
                    uint16_t* u, int32_t* perm, uint32_t* err, hipStream_t s) {
    const int tiles = (M + 15) / 16 + (perm ? 1 : 0);
    int ny = ad.n < 16 ? ad.n : 16;
    if (ny > M) ny = M;
    adapter_down_kernel<RT><<<dim3(tiles, ny), dim3(64 * kDownWaves), 0, s>>>(
        a, ad.down, ad.scale, add, M, K, u, perm, err);
    return hipGetLastError();
}

// The projection with adapters for a decode batch (M <= 16 MT positions, K a
// multiple of 64): W is read once and bounds it.  A workgroup takes 64 columns
// and all positions; its four waves (16 columns each) share the positions' tile
// in LDS.  Both operands' k-tiles of 64 arrive by DMA in a ring of NS stages,
// NS - 1 of them on their way, with one barrier a k-tile.  (With the fragments
// straight from memory, each wave of 32 columns fetching its own quarter of
// K, the positions' loads - 16 rows a load, twice W's bytes - bound it: 44 us
// at 64 positions of 1536 -> 25600 against 19 for the ring.)
template <int LATER>
__device__ __forceinline__ void arrived() {
    static_assert(LATER >= 0 && LATER < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt(0x0070 | (LATER & 15) | ((LATER >> 4) << 14));  // lgkmcnt(0) too
    asm volatile("s_barrier" ::: "memory");
}

template <int MT, int NS>
__device__ __forceinline__ void adapter_rows(const uint16_t* __restrict__ a,
                                             const uint16_t* __restrict__ w, const AddAdapters& ad,
                                             int M, int N, int K, uint16_t* __restrict__ kv,
                                             uint8_t* smem) {
    constexpr int ROWS = 16 * MT, STAGE = (ROWS + 64) * 128;
    constexpr int NA = MT == 4 ? 2 : 1, NLOAD = NA + 2;  // DMA of a wave and k-tile
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quad = lane >> 4;
    const int n0 = blockIdx.x * 64;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a, (uint32_t)(M * K * 2));
    const __amdgpu_buffer_rsrc_t rw =
        make_rsrc(w + (int64_t)n0 * K, (uint32_t)(min(64, N - n0) * K * 2));
    // instruction i of a wave fills 8 rows of 128 bytes (rows past M or N read
    // as zeros; 16 positions are two instructions, which waves 2 and 3 repeat)
    uint32_t ao[NA], wo[2];
    int as[NA], ws[2];
    const int r8 = lane >> 3;
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        const int seg = MT == 1 ? wave & 1 : NA * wave + i, row = seg * 8 + r8;
        ao[i] = (uint32_t)(row * K * 2 + slot128(row, lane & 7) * 16);
        as[i] = seg * 1024;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int seg = 2 * wave + i, row = seg * 8 + r8;
        wo[i] = (uint32_t)(row * K * 2 + slot128(row, lane & 7) * 16);
        ws[i] = ROWS * 128 + seg * 1024;
    }
    auto issue = [&](int kt, int stage) {
        uint8_t* st = smem + stage * STAGE;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(st + ws[i]), 16, wo[i],
                                                     kt * 128, 0, 0);
#pragma unroll
        for (int i = 0; i < NA; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(st + as[i]), 16, ao[i],
                                                     kt * 128, 0, 0);
    };
    const int nk = K / 64;
#pragma unroll
    for (int p = 0; p < NS - 1; ++p)
        if (p < nk) issue(p, p);

    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    const int wrow = 16 * wave + col;
    int stage = 0;
    for (int kt = 0; kt < nk; ++kt) {
        // k-tile kt has landed once at most the NS - 2 issued after it are on
        // their way (near the end: none); behind the barrier it has for
        // everyone, and k-tile kt - 1's stage is free.  (A barrier without a
        // fence, which would wait for all of them.)
        if (kt + NS - 2 < nk)
            arrived<(NS - 2) * NLOAD>();
        else
            arrived<0>();
        if (kt + NS - 1 < nk) issue(kt + NS - 1, stage == 0 ? NS - 1 : stage - 1);
        const uint8_t* st = smem + stage * STAGE;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int c = 4 * ks + quad;
            const bf16x8 fw = *reinterpret_cast<const bf16x8*>(st + ROWS * 128 + wrow * 128 +
                                                               slot128(wrow, c) * 16);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int row = 16 * t + col;
                const bf16x8 fa =
                    *reinterpret_cast<const bf16x8*>(st + row * 128 + slot128(row, c) * 16);
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw, fa, acc[t], 0, 0, 0);
            }
        }
        stage = stage + 1 == NS ? 0 : stage + 1;
    }

    // D[n][m]: lane holds m = 16 t + lane % 16, n = 16 wave + 4 (lane / 16) + v.
    // The second product takes 16 ranks in one v_mfma_f32_16x16x32_bf16: quads 0
    // and 1 hold u's hi, quads 2 and 3 its lo, and up's ranks twice.
    const int mine = lane < M ? ad.id_of(lane) : -1;  // of position `lane`
    const int n = n0 + 16 * wave + col;
    for (int r0 = 0; r0 < ad.rp; r0 += 16) {
        const int r = r0 + 8 * (quad & 1);
        bf16x8 fu[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
            fu[t] = *reinterpret_cast<const bf16x8*>(
                ad.pair(min(16 * t + col, M - 1), r, quad >> 1));
        uint64_t todo = __ballot(mine >= 0);
        while (todo) {
            constexpr int AT = 8;  // adapters on their way
            bf16x8 b[AT];
            uint64_t has[AT];
#pragma unroll
            for (int x = 0; x < AT; ++x) {
                b[x] = bf16x8{};
                has[x] = 0;
                if (todo) {
                    const int j = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
                    has[x] = __ballot(mine == j);
                    todo &= ~has[x];
                    if (n < N && r < ad.rank)
                        b[x] = *reinterpret_cast<const bf16x8*>(ad.up + j * ad.up_stride +
                                                                (int64_t)n * ad.rank + r);
                }
            }
#pragma unroll
            for (int x = 0; x < AT; ++x)
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const uint32_t mask = (uint32_t)(has[x] >> (16 * t)) & 0xFFFFu;
                    if (mask == 0) continue;
                    const f32x4 d =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[x], fu[t], acc[t], 0, 0, 0);
                    const bool hit = (mask >> col) & 1;
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[t][v] = hit ? d[v] : acc[t][v];
                }
        }
    }

    // rows of 64 columns through LDS, so that a position's 128 bytes go out together
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int row = 16 * t + col, byte = (16 * wave + 4 * quad) * 2;
        *reinterpret_cast<uint2*>(smem + row * 128 + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 8)) =
            make_uint2(pack_bf16(acc[t][0], acc[t][1]), pack_bf16(acc[t][2], acc[t][3]));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (ROWS * 8 + 255) / 256; ++i) {
        const int at = i * 256 + tid, row = at >> 3, c = at & 7;
        if (row < M && row < ROWS && n0 + 8 * c < N)
            *reinterpret_cast<uint4*>(kv + (int64_t)row * N + n0 + 8 * c) =
                *reinterpret_cast<const uint4*>(smem + row * 128 + ((c ^ (row & 7)) << 4));
    }
}

template <int MT, int NS>
__global__ void __launch_bounds__(256) adapter_rows_kernel(const uint16_t* __restrict__ a,
                                                           const uint16_t* __restrict__ w,
                                                           const AddAdapters ad, int M, int N, int K,
                                                           uint16_t* __restrict__ kv) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * (16 * MT + 64) * 128];
    adapter_rows<MT, NS>(a, w, ad, M, N, K, kv, smem);
}

template <int MT, int NS>
hipError_t run_rows(const uint16_t* a, const uint16_t* w, const AddAdapters& ad, int M, int N,
                    int K, uint16_t* kv, hipStream_t s) {
    adapter_rows_kernel<MT, NS><<<dim3((N + 63) / 64), dim3(256), 0, s>>>(a, w, ad, M, N, K, kv);
    return hipGetLastError();
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

constexpr int64_t kRowsMax = 64;  // positions of the decode kernel

// Positions of one launch: the tiles address the positions and the pairs with
// 32 bits.
int64_t launch_positions(int K) {
    const int64_t m = ((int64_t)1 << 31) / (2 * (int64_t)K) / 256 * 256;
    return m < 256 ? 256 : m > 262144 ? 262144 : m;
}

}  // namespace

size_t adapters_scratch_bytes(int rank, int64_t M) {
    return up256((size_t)M * ((rank + 15) / 16 * 16) * 2 * sizeof(uint16_t)) +
           up256((size_t)M * sizeof(int32_t));
}

hipError_t launch_wkv_adapters(const uint16_t* a, const uint16_t* w, const Adapters& ad,
                               const int32_t* ids, int seg, int64_t M, int N, int K, uint16_t* kv,
                               void* scratch, uint32_t* err, hipStream_t s) {
    const int rt = (ad.rank + 15) / 16, rp = 16 * rt;
    uint16_t* u = (uint16_t*)scratch;
    int32_t* perm = (int32_t*)((char*)scratch + up256((size_t)M * rp * 2 * sizeof(uint16_t)));
    const int64_t most = launch_positions(K);
    for (int64_t m0 = 0; m0 < M; m0 += most) {
        const int m = (int)(M - m0 < most ? M - m0 : most);
        const uint16_t* am = a + m0 * K;
        uint16_t *um = u + m0 * rp * 2, *kvm = kv + m0 * N;
        const bool rows = m <= kRowsMax && K % 64 == 0 && (int64_t)K * 2 * 64 < (1ll << 31);
        int32_t* order = rows ? nullptr : perm + m0;
        const AddAdapters add{ad.up, um, ids, order, m0, ad.n, ad.rank, rp, seg,
                              (int64_t)N * ad.rank};
        auto down = rt <= 1 ? run_down<1> : rt <= 2 ? run_down<2> : rt <= 4 ? run_down<4> : run_down<8>;
        hipError_t e = down(am, ad, add, m, K, um, order, err, s);
        if (e != hipSuccess) return e;
        if (!rows)
            e = launch_wkv_added(am, w, m, N, K, add, kvm, s);
        else if (m <= 16)
            e = run_rows<1, 6>(am, w, add, m, N, K, kvm, s);
        else if (m <= 32)
            e = run_rows<2, 6>(am, w, add, m, N, K, kvm, s);
        else
            e = run_rows<4, 4>(am, w, add, m, N, K, kvm, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace engram
