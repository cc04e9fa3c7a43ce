// Low-rank adapters of many requests beside the shared projection (stage 3
// with a rank-r correction for each request; the Engram block's self.wkv is
// the shared part).  Two kernels: the first product, u = scale * down . a, in
// fp32 (here), then the projection with the second product, up . u, added to
// its accumulators (adapters.h, wkv.hip).
#include <type_traits>

#include "adapters.h"

namespace engram {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// The order in which the projection's tiles (and the first product) take the
// positions: those of one adapter together, so that a tile meets few adapters
// however the requests are mixed.  A counting sort by id mod 1023, positions
// without an adapter first; within a bucket in any order, on which no output
// depends.  One workgroup of NT threads.  A wave whose 64 positions are of one
// bucket (a prompt) counts them at once: 64 additions to one LDS word go one by
// one.
constexpr int kBuckets = 1024;
template <int NT>
__device__ __forceinline__ void order_positions(const AddAdapters& ad, int M, int2* tile,
                                                uint32_t* err, int (&hist)[kBuckets],
                                                int (&wave_sum)[16]) {
    constexpr int PER = kBuckets / NT;  // buckets a thread
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    bool bad = false;
    auto adapter = [&](int m) {  // -2: no position
        const int j = ad.raw(min(m, M - 1));
        bad |= j < -1 || j >= ad.n;
        return m >= M ? -2 : j >= 0 && j < ad.n ? j : -1;
    };
    auto bucket_of = [&](int j) { return j < 0 ? j + 1 : 1 + j % (kBuckets - 1); };
    // the place of a lane's position in its bucket, counted on from hist
    auto count = [&](int j) {
        const int bucket = bucket_of(j);
        const int first = __builtin_amdgcn_readfirstlane(bucket);
        if (__all(bucket == first)) {
            int at = 0;
            if (first >= 0 && lane == 0) at = atomicAdd(&hist[first], 64);
            return __builtin_amdgcn_readfirstlane(at) + lane;
        }
        return bucket >= 0 ? atomicAdd(&hist[bucket], 1) : 0;
    };
    constexpr int AT = 4;  // positions of a thread on their way
    const int end = (M + 63) / 64 * 64;  // (whole waves count)
    int j[AT], at[AT];
    for (int i = tid; i < kBuckets; i += NT) hist[i] = 0;
    __syncthreads();
    for (int m = tid; m < end; m += AT * NT) {
#pragma unroll
        for (int x = 0; x < AT; ++x) j[x] = adapter(m + x * NT);
#pragma unroll
        for (int x = 0; x < AT; ++x) at[x] = count(j[x]);
    }
    if (bad && err) atomicOr(err, ENGRAM_ERRBIT_ADAPTER);
    __syncthreads();
    // exclusive sums over the buckets
    int own[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += own[i] = hist[tid * PER + i];
    const int mine = sum;
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(sum, o, 64);
        if (lane >= o) sum += x;
    }
    if (lane == 63) wave_sum[wave] = sum;
    __syncthreads();
    int before = sum - mine;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) before += w < wave ? wave_sum[w] : 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        hist[tid * PER + i] = before;
        before += own[i];
    }
    __syncthreads();
    if (end <= AT * NT) {  // all of them still in registers
#pragma unroll
        for (int x = 0; x < AT; ++x) {
            const int m = tid + x * NT;
            if (m < M) tile[hist[bucket_of(j[x])] + at[x]] = make_int2(m, j[x]);
        }
    } else {
        for (int m = tid; m < end; m += AT * NT) {
#pragma unroll
            for (int x = 0; x < AT; ++x) j[x] = adapter(m + x * NT);
#pragma unroll
            for (int x = 0; x < AT; ++x) {
                const int to = count(j[x]);
                if (m + x * NT < M) tile[to] = make_int2(m + x * NT, j[x]);
            }
        }
    }
    for (int p = M + tid; p < (M + 255) / 256 * 256; p += NT) tile[p] = make_int2(M - 1, -1);
}

__global__ void __launch_bounds__(kBuckets) adapter_order_kernel(const AddAdapters ad, int M,
                                                                 int2* __restrict__ tile,
                                                                 uint32_t* __restrict__ err) {
    __shared__ int hist[kBuckets];
    __shared__ int wave_sum[16];
    order_positions<kBuckets>(ad, M, tile, err, hist, wave_sum);
}

constexpr int kDownWaves = 8;

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
// With `order`, one workgroup more writes the order of the positions.
template <int RT>  // rank tiles of 16
__global__ void __launch_bounds__(64 * kDownWaves) adapter_down_kernel(
    const uint16_t* __restrict__ a, const uint16_t* __restrict__ down,
    const float* __restrict__ scale, const AddAdapters ad, int M, int K,
    uint16_t* __restrict__ u, int2* __restrict__ order, uint32_t* __restrict__ err) {
    __shared__ union {
        float part[kDownWaves][RT * 16][17];
        struct {
            int hist[kBuckets], wave_sum[16];
        } sort;
    } sh;
    auto& part = sh.part;
    const int m0 = blockIdx.x * 16;
    if (m0 >= M) {  // one workgroup more, with `order`
        if (blockIdx.y == 0 && blockIdx.z == 0)
            order_positions<64 * kDownWaves>(ad, M, order, nullptr, sh.sort.hist,
                                             sh.sort.wave_sum);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quad = lane >> 4;
    // ranks of this workgroup
    const int first_r = 16 * RT * blockIdx.z, rank = ad.rank, rp = ad.rp;
    int m = min(m0 + col, M - 1), mine = -1;
    if (ad.tile) {
        const int2 own = ad.tile[m0 + col];
        m = own.x;
        mine = own.y;
    } else if (m0 + col < M) {
        mine = ad.id_of(m);
        if (mine < 0 && err && blockIdx.y == 0 && blockIdx.z == 0 && tid < 16 && ad.bad(m))
            atomicOr(err, ENGRAM_ERRBIT_ADAPTER);
    }
    const int steps = K / 32, per = (steps + kDownWaves - 1) / kDownWaves;
    const int s0 = wave * per, s1 = min(steps, s0 + per);
    const uint16_t* am = a + (int64_t)m * K + 8 * quad;
    // AT k-steps on their way (behind the last: that one again, unused); where
    // they are all of this wave's, the workgroup of the first adapter fetches
    // the positions' once, ahead of the ids
    constexpr int AT = RT <= 4 ? 6 : 3;
    bf16x8 fa[AT];
    auto load_a = [&](int s) {
#pragma unroll
        for (int x = 0; x < AT; ++x)
            fa[x] = *reinterpret_cast<const bf16x8*>(am + 32 * max(min(s + x, s1 - 1), 0));
    };
    const bool ahead = s1 - s0 <= AT && blockIdx.y == 0;
    if (ahead) load_a(s0);

    uint32_t todo = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
    for (int turn = 0; todo; ++turn) {
        const int j = __builtin_amdgcn_readlane(mine, __builtin_ctz(todo));
        todo &= ~(uint32_t)__ballot(mine == j);
        if (turn % gridDim.y != blockIdx.y) continue;
        const float sc = scale ? scale[j] : 1.0f;
        const uint16_t* dj = down + (int64_t)j * rank * K + 8 * quad;
        f32x4 acc[RT];
        const uint16_t* dr[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            acc[t] = f32x4{0, 0, 0, 0};
            dr[t] = dj + (int64_t)min(first_r + 16 * t + col, rank - 1) * K;
        }
        for (int s = s0; s < s1; s += AT) {
            bf16x8 fd[AT][RT];
            if (!ahead) load_a(s);
#pragma unroll
            for (int x = 0; x < AT; ++x) {
                const int k = 32 * min(s + x, s1 - 1);
#pragma unroll
                for (int t = 0; t < RT; ++t) fd[x][t] = *reinterpret_cast<const bf16x8*>(dr[t] + k);
            }
#pragma unroll
            for (int x = 0; x < AT; ++x)
                if (s + x < s1)
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fd[x][t], fa[x], acc[t], 0,
                                                                         0, 0);
        }
        // D[r][m]: lane holds m = lane % 16, r = 4 (lane / 16) + v
        __syncthreads();  // the last adapter's sums are read
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) part[wave][16 * t + 4 * quad + v][col] = acc[t][v];
        __syncthreads();
        // (mine is the same in every wave and quad: lane % 16 names the position)
        for (int l = tid >> 4; l < 16 * RT && first_r + l < rp; l += 4 * kDownWaves) {
            const int r = first_r + l;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kDownWaves; ++w) sum += part[w][l][col];
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

// The first product, and with `order` the order of the positions too.
hipError_t run_down(const uint16_t* a, const Adapters& ad, AddAdapters add, int M, int K,
                    uint16_t* u, int2* order, uint32_t* err, hipStream_t s) {
    const int rt = add.rp / 16;
    // Few positions: both in one launch, and the first product takes the positions
    // as they come (613 positions of rank 8: 29.6 us the whole call against 33.9).
    // Many, or of a high rank: in their order, which mixed ones need (1000
    // positions of rank 64, 8 adapters in turn, -> 10240: 67 us against 80).
    const bool first = order && (int64_t)M * rt > 1536;
    if (first) {
        adapter_order_kernel<<<dim3(1), dim3(kBuckets), 0, s>>>(add, M, order, err);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        add.tile = order;
        order = nullptr;
    }
    // positions in order of their adapters meet one or two in 16; others up to 16
    int ny = first ? 2 : 16;
    if (ny > ad.n) ny = ad.n;
    if (ny > M) ny = M;
    const int tiles = (M + 15) / 16 + (order ? 1 : 0);
    auto go = [&](auto kern, int each) {
        kern<<<dim3(tiles, ny, (rt + each - 1) / each), dim3(64 * kDownWaves), 0, s>>>(
            a, ad.down, ad.scale, add, M, K, u, order, err);
        return hipGetLastError();
    };
    // few positions: a workgroup for each 16 ranks (rank 64 at 64 positions: 6.5 us
    // against 10.6 with all in one); many: the positions are fetched once for 64
    // (rank 64 at 4096 positions: 11.9 us against 17.3)
    if (rt == 1 || M <= 1024) return go(adapter_down_kernel<1>, 1);
    if (rt == 2) return go(adapter_down_kernel<2>, 2);
    return go(adapter_down_kernel<4>, 4);
}

// The projection with adapters for a decode batch (16 MT positions a workgroup, K
// a multiple of 64): W is read once and bounds it.  A workgroup takes 64 columns
// and, up to 64, all positions; its four waves (16 columns each) share the
// positions' tile in LDS.  Both operands' k-tiles of 64 arrive by DMA in a ring
// of NS stages, NS - 1 of them on their way, with one barrier a k-tile.  (With
// the fragments straight from memory, each wave of 32 columns fetching its own
// quarter of K, the positions' loads - 16 rows a load, twice W's bytes - bound
// it: 44 us at 64 positions of 1536 -> 25600 without adapters against 17 for
// the ring, 4.6 TB/s of W.)
//
// LDS of a workgroup: the ring, or the up rows (80 KiB less the sums, so that
// two workgroups fit a compute unit) and the sums behind them.
constexpr int kSumsRow = 68;  // floats of a position's 64 columns
constexpr int rows_sums(int mt) { return 16 * mt * kSumsRow * 4; }
constexpr int rows_ups(int mt) { return 81920 - rows_sums(mt); }

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
                                             int tiles_m, int tiles_n, int per_xcd,
                                             uint8_t* smem) {
    constexpr int ROWS = 16 * MT, STAGE = (ROWS + 64) * 128;
    constexpr int NA = MT == 4 ? 2 : 1, NLOAD = NA + 2;  // DMA of a wave and k-tile
    constexpr int RING = NS * STAGE, UPS = rows_ups(MT), SROW = kSumsRow;
    static_assert(rows_sums(MT) <= RING, "the sums fit the ring");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quad = lane >> 4;
    int mt, nt;
    if (!tile_of<2>(blockIdx.x, per_xcd, tiles_m, tiles_n, &mt, &nt)) return;
    const int n0 = nt * 64, m0 = mt * ROWS;
    const int rows = min(ROWS, M - m0);
    a += (int64_t)m0 * K;
    kv += (int64_t)m0 * N;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a, (uint32_t)(rows * K * 2));
    const __amdgpu_buffer_rsrc_t rw =
        make_rsrc(w + (int64_t)n0 * K, (uint32_t)(min(64, N - n0) * K * 2));
    // instruction i of a wave fills 8 rows of 128 bytes (rows past M or N read
    // as zeros; 16 positions are two instructions, which waves 2 and 3 repeat)
    uint32_t ao[NA], wo[2];
    int as[NA], ws[2];
    const int r8 = lane >> 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int seg = 2 * wave + i, row = seg * 8 + r8;
        wo[i] = (uint32_t)(row * K * 2 + slot128(row, lane & 7) * 16);
        ws[i] = ROWS * 128 + seg * 1024;
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        const int seg = MT == 1 ? wave & 1 : NA * wave + i, row = seg * 8 + r8;
        ao[i] = (uint32_t)(row * K * 2 + slot128(row, lane & 7) * 16);
        as[i] = seg * 1024;
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
    // This lane's position: its pairs (the first 64 ranks) are on their way
    // before the ring starts.
    const int lm = lane & (ROWS - 1);
    bf16x8 hi[8], lo[8];
    auto load_pairs = [&](int r0) {
        const uint16_t* from = ad.pair(m0 + min(lm, rows - 1), r0, 0);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (r0 + 8 * k < ad.rank) {
                hi[k] = *reinterpret_cast<const bf16x8*>(from + 16 * k);
                lo[k] = *reinterpret_cast<const bf16x8*>(from + 16 * k + 8);
            }
    };
    const int own = lm < rows ? ad.id_of(m0 + lm) : -1;
    load_pairs(0);
    const int nk = K / 64;
#pragma unroll
    for (int p = 0; p < NS - 1; ++p)
        if (p < nk) issue(p, p);

    // The adapters of this workgroup's positions, each once: lane x holds the
    // x-th in `list`, and a lane's position (lane mod the positions) has its
    // adapter as the `which`-th.
    int list = 0, which = -1, distinct = 0;
    {
        uint64_t todo = __ballot(own >= 0);
        while (todo) {
            const int j = __builtin_amdgcn_readlane(own, __builtin_ctzll(todo));
            const bool same = own == j;
            todo &= ~__ballot(same);
            which = same ? distinct : which;
            list = lane == distinct ? j : list;
            ++distinct;
        }
    }
    // The distinct adapters' up rows of columns n0 + c0 .. and ranks r0 .. (8
    // `chunks` of them) to `to`, one after the other with 16 bytes between two;
    // a wave takes every fourth adapter.  (Columns past N read as zeros.)
    auto load_ups = [&](uint8_t* to, int r0, int chunks, int c0, int nc) {
        const int pieces = nc * chunks, slab = pieces * 16 + 16;
        const int inv = 65536 / chunks + 1;  // L / chunks = L * inv >> 16 for L < 512
        const uint32_t bytes = (uint32_t)(min(nc, N - n0 - c0) * ad.rank * 2);
        const uint16_t* from = ad.up + (int64_t)(n0 + c0) * ad.rank + r0;
        for (int i = 0; i < pieces; i += 64) {
            const int L = i + lane, row = L * inv >> 16, c = L - row * chunks;
            const uint32_t off = L < pieces ? (uint32_t)(row * ad.rank + c * 8) * 2u : 0xF0000000u;
            if (L < pieces)
                for (int x = wave; x < distinct; x += 4) {
                    const int j = __builtin_amdgcn_readlane(list, x);
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(
                        make_rsrc(from + j * ad.up_stride, bytes - (uint32_t)(r0 * 2)),
                        (lds_void*)(to + x * slab + i * 16), 16, off, 0, 0, 0);
                }
        }
    };
    // few adapters fit the LDS behind the ring: their rows come beside it
    const bool early = ad.rank <= 64 && distinct * (128 * ad.rank + 16) <= 81920 - RING;
    if (early) load_ups(smem + RING, 0, ad.rank / 8, 0, 64);

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

    // The second product on the vector units: with an adapter for each position
    // the matrix cores have nothing to share, and going through the adapters one
    // by one costs 0.4 us each in scalar work (32 adapters of rank 16 at 64
    // positions: 17 us beside the projection's 17, against 11 this way).  Here a
    // lane takes one position and a few columns, whatever the other positions
    // have: its pairs are in registers, its adapter's up rows come from LDS, and
    // v_dot2_f32_bf16 adds two products in fp32.  The up rows of all distinct
    // adapters arrive by DMA in the ring's memory, as many of the 64 columns a
    // round as fit (the four waves split them); 16 bytes between two adapters
    // spread equal rows over the banks.
    if (distinct) {
        // [position][SROW]
        float* sums = reinterpret_cast<float*>(smem + (early ? 0 : UPS));
        for (int r0 = 0; r0 < ad.rank; r0 += 64) {
            const int ranks = min(64, ad.rank - r0), chunks = ranks / 8;
            if (r0) load_pairs(r0);
            int nc = 64;
            while (distinct * (nc * chunks * 16 + 16) > UPS) nc >>= 1;
            const int slab = nc * chunks * 16 + 16;
            const int per = nc * MT / 16;  // columns a lane
            const int first = (wave * (4 / MT) + lane / ROWS) * per;
            for (int c0 = 0; c0 < 64 && n0 + c0 < N; c0 += nc) {
                __syncthreads();  // the memory is free: the ring, or the round before, is read
                if (!early) {
                    load_ups(smem, r0, chunks, c0, nc);
                    arrived<0>();
                }
                const uint8_t* up = smem + (early ? RING : 0) + max(which, 0) * slab +
                                    first * (chunks * 16);
                float* to = sums + lm * SROW + c0 + first;
                auto columns = [&](auto count) {
                    constexpr int P = decltype(count)::value;
                    float o[P];
#pragma unroll
                    for (int i = 0; i < P; ++i) o[i] = r0 ? to[i] : 0.0f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (k >= chunks) break;
#pragma unroll
                        for (int i = 0; i < P; ++i) {
                            const bf16x8 b = *reinterpret_cast<const bf16x8*>(
                                up + (i * chunks + k) * 16);
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                const bf16x2 bb = {b[e], b[e + 1]};
                                o[i] = __builtin_amdgcn_fdot2_f32_bf16(
                                    bb, bf16x2{hi[k][e], hi[k][e + 1]}, o[i], false);
                                o[i] = __builtin_amdgcn_fdot2_f32_bf16(
                                    bb, bf16x2{lo[k][e], lo[k][e + 1]}, o[i], false);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < P; ++i) to[i] = which >= 0 ? o[i] : 0.0f;
                };
                if constexpr (MT == 4)
                    if (per == 16) columns(std::integral_constant<int, 16>{});
                if constexpr (MT >= 2)
                    if (per == 8) columns(std::integral_constant<int, 8>{});
                if (per == 4) columns(std::integral_constant<int, 4>{});
                if (per == 2) columns(std::integral_constant<int, 2>{});
                if (per == 1) columns(std::integral_constant<int, 1>{});
            }
        }
        __syncthreads();
        // D[n][m]: lane holds m = 16 t + lane % 16, n = 16 wave + 4 (lane / 16) + v
#pragma unroll
        for (int t = 0; t < MT; ++t)
            acc[t] += *reinterpret_cast<const f32x4*>(sums + (16 * t + col) * SROW + 16 * wave +
                                                      4 * quad);
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
        if (row < rows && n0 + 8 * c < N)
            *reinterpret_cast<uint4*>(kv + (int64_t)row * N + n0 + 8 * c) =
                *reinterpret_cast<const uint4*>(smem + row * 128 + ((c ^ (row & 7)) << 4));
    }
}

template <int MT, int NS>
__global__ void __launch_bounds__(256, 2) adapter_rows_kernel(const uint16_t* __restrict__ a,
                                                           const uint16_t* __restrict__ w,
                                                           const AddAdapters ad, int M, int N, int K,
                                                           uint16_t* __restrict__ kv, int tiles_m,
                                                           int tiles_n, int per_xcd) {
    static_assert(NS * (16 * MT + 64) * 128 <= 81920, "the ring");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[81920];
    adapter_rows<MT, NS>(a, w, ad, M, N, K, kv, tiles_m, tiles_n, per_xcd, smem);
}

template <int MT, int NS>
hipError_t run_rows(const uint16_t* a, const uint16_t* w, const AddAdapters& ad, int M, int N,
                    int K, uint16_t* kv, hipStream_t s) {
    const int tiles_m = (M + 16 * MT - 1) / (16 * MT), tiles_n = (N + 63) / 64;
    const int per_xcd = (tiles_m * tiles_n + N_XCD - 1) / N_XCD;
    adapter_rows_kernel<MT, NS><<<dim3(per_xcd * N_XCD), dim3(256), 0, s>>>(
        a, w, ad, M, N, K, kv, tiles_m, tiles_n, per_xcd);
    return hipGetLastError();
}

// The projection with adapters for at most one tile a compute unit: 128 x 128
// tiles, eight waves of 64 x 64, four for each half of a k-tile, whose sums meet
// in LDS at the end.  One workgroup a compute unit has nobody to hide its
// loads behind, so its k-tiles arrive in a ring of NS stages, up to NS of them on
// their way, each k-step's fragments are read beside the last one's products
// (the next k-tile's first behind the one barrier of a k-tile), and the pairs
// have LDS of their own and come with the first k-tile.  (613 positions of 1536 ->
// 6168, 245 tiles: 21.3 us with adapters of rank 8, 19.4 without any, of which
// 5.7 are start and end; a k-tile takes 0.57 us for the 32 KB that it brings, 14
// TB/s from the L2s in all.  Four waves for all of K: 22.5 us, the same without
// adapters; its reads not ahead of the products: 25.2; two stages: 25.7.)
constexpr int kTile = 128, kStages = 4;
__device__ __forceinline__ void adapter_tile(const uint16_t* __restrict__ a,
                                             const uint16_t* __restrict__ w, const AddAdapters& ad,
                                             int M, int N, int K, uint16_t* __restrict__ kv,
                                             int tiles_m, int tiles_n, int per_xcd,
                                             uint8_t* smem) {
    constexpr int BT = kTile, NS = kStages, STAGE = 2 * BT * 128, NLD = BT / 8 / 8;
    int mt, nt;
    if (!tile_of(blockIdx.x, per_xcd, tiles_m, tiles_n, &mt, &nt)) return;
    const int m0 = mt * BT, n0 = nt * BT;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave >> 1) & 1, wn = wave & 1, wk = wave >> 2, lrow = lane & 31, lhalf = lane >> 5;
    uint8_t* const pairs = smem + NS * STAGE;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a, (uint32_t)M * (uint32_t)K * 2u);
    const __amdgpu_buffer_rsrc_t rw =
        make_rsrc(w + (int64_t)n0 * K, (uint32_t)(min(BT, N - n0) * K * 2));
    int2 own[2];  // position and adapter of rows m0 + 64 k + lane
#pragma unroll
    for (int k = 0; k < 2; ++k) own[k] = ad.tile[m0 + 64 * k + lane];
    // instruction i of a wave fills rows 8 (4 i + wave) .. of an operand
    uint32_t wo[NLD], ao[NLD];
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
        const int row = (8 * i + wave) * 8 + (lane >> 3);
        wo[i] = (uint32_t)(row * K * 2 + slot128(row, lane & 7) * 16);
    }
    auto issue_w = [&](int kt, int stage) {
        uint8_t* st = smem + stage * STAGE + BT * 128;
#pragma unroll
        for (int i = 0; i < NLD; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(st + (8 * i + wave) * 1024),
                                                     16, wo[i], kt * 128, 0, 0);
    };
    auto issue_a = [&](int kt, int stage) {
        uint8_t* st = smem + stage * STAGE;
#pragma unroll
        for (int i = 0; i < NLD; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(st + (8 * i + wave) * 1024),
                                                     16, ao[i], kt * 128, 0, 0);
    };
    const int nk = K / 64;
    // W first, which needs no positions
#pragma unroll
    for (int p = 0; p < NS; ++p)
        if (p < nk) issue_w(p, p);
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
        const int row = (8 * i + wave) * 8 + (lane >> 3);
        const int lo = __shfl(own[0].x, row & 63, 64), hi = __shfl(own[1].x, row & 63, 64);
        ao[i] = (uint32_t)(row < 64 ? lo : hi) * (uint32_t)(K * 2) +
                (uint32_t)(slot128(row, lane & 7) * 16);
    }
    if (any_adapter(own)) load_pairs<BT, 8>(ad, own, M, wave, lane, 0, pairs);
#pragma unroll
    for (int p = 0; p < NS; ++p)
        if (p < nk) issue_a(p, p);

    f32x16 acc[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.0f;
    bf16x8 fa[2][2], fw[2][2];
    auto read = [&](int stage, int ks, int to) {
        const uint8_t* st = smem + stage * STAGE;
        const int c = 2 * ks + lhalf;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ar = wm * 64 + i * 32 + lrow, wr = wn * 64 + i * 32 + lrow;
            fa[to][i] = *reinterpret_cast<const bf16x8*>(st + ar * 128 + slot128(ar, c) * 16);
            fw[to][i] =
                *reinterpret_cast<const bf16x8*>(st + BT * 128 + wr * 128 + slot128(wr, c) * 16);
        }
    };
    auto multiply = [&](int from) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fw[from][j], fa[from][i],
                                                                    acc[j][i], 0, 0, 0);
        // the next fragments' reads between them
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // A k-tile has landed once only what was issued behind its last load is on
    // its way.  (The first NS had their W ahead of every A.)
    static_assert(NS == 4, "the waits below");
    if (nk >= 4)
        arrived<3 * NLD>();
    else
        arrived<0>();
    read(0, 2 * wk, 0);
    int stage = 0;
    for (int kt = 0; kt < nk; ++kt) {
        const int after = (stage + 1) & (NS - 1);
        read(stage, 2 * wk + 1, 1);
        multiply(0);
        if (kt + 1 < nk) {
            // k-tile kt + 1 is there, behind the barrier for everyone, and this
            // one's stage is free
            if (kt < 2) {
                if (kt == 0 && nk >= 4)
                    arrived<2 * NLD>();
                else if (kt == 1 && nk >= 5)
                    arrived<3 * NLD>();
                else
                    arrived<0>();
            } else if (kt + 3 < nk) {
                arrived<4 * NLD>();
            } else if (kt + 3 == nk) {
                arrived<2 * NLD>();
            } else {
                arrived<0>();
            }
            if (kt + NS < nk) {
                issue_w(kt + NS, stage);
                issue_a(kt + NS, stage);
            }
            read(after, 2 * wk, 0);
        }
        multiply(1);
        stage = after;
    }
    __syncthreads();
    // The two halves of K meet: a wave keeps 32 of its 64 columns, the other half
    // of K's wave the others.
    f32x16 sum[1][2];
    {
        uint8_t* mine = smem + wave * 8192 + lane * 16;
        const uint8_t* other = smem + (wave ^ 4) * 8192 + lane * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4 x;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    x[v] = wk ? acc[0][i][4 * q + v] : acc[1][i][4 * q + v];
                *reinterpret_cast<f32x4*>(mine + (4 * i + q) * 1024) = x;
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(other + (4 * i + q) * 1024);
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    sum[0][i][4 * q + v] =
                        (wk ? acc[1][i][4 * q + v] : acc[0][i][4 * q + v]) + x[v];
            }
    }
    const int wc = 2 * wn + wk;  // its 32 columns
    add_tile<BT, 8, 2, 1>(ad, sum, own, M, n0, N, wm, wc, wave, lane, pairs, smem + 2 * STAGE);

    // a wave's 64 x 32 block as bf16 rows through LDS, so that 4 lanes store a
    // position's 64 bytes
    uint8_t* ep = smem + 3 * STAGE + wave * 4096;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = i * 32 + lrow, ch = q ^ ((r >> 1) & 3);
            *reinterpret_cast<uint2*>(ep + r * 64 + ch * 16 + lhalf * 8) =
                make_uint2(pack_bf16(sum[0][i][4 * q], sum[0][i][4 * q + 1]),
                           pack_bf16(sum[0][i][4 * q + 2], sum[0][i][4 * q + 3]));
        }
    const int rsub = lane >> 2, csub = lane & 3, n = n0 + wc * 32 + csub * 8;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int r = it * 16 + rsub;
        const uint4 v =
            *reinterpret_cast<const uint4*>(ep + r * 64 + ((csub ^ ((r >> 1) & 3)) << 4));
        const int lo = __shfl(own[0].x, r, 64), hi = __shfl(own[1].x, r, 64);
        if (m0 + wm * 64 + r < M && n < N)
            *reinterpret_cast<uint4*>(kv + (int64_t)(wm ? hi : lo) * N + n) = v;
    }
}

__global__ void __launch_bounds__(512, 1) adapter_tile_kernel(const uint16_t* __restrict__ a,
                                                              const uint16_t* __restrict__ w,
                                                              const AddAdapters ad, int M, int N,
                                                              int K, uint16_t* __restrict__ kv,
                                                              int tiles_m, int tiles_n,
                                                              int per_xcd) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kStages * 2 * kTile * 128 + kTile * 256];
    adapter_tile(a, w, ad, M, N, K, kv, tiles_m, tiles_n, per_xcd, smem);
}

hipError_t run_tiles(const uint16_t* a, const uint16_t* w, const AddAdapters& ad, int M, int N,
                     int K, uint16_t* kv, hipStream_t s) {
    const int tiles_m = (M + kTile - 1) / kTile, tiles_n = (N + kTile - 1) / kTile;
    const int per_xcd = (tiles_m * tiles_n + N_XCD - 1) / N_XCD;
    adapter_tile_kernel<<<dim3(per_xcd * N_XCD), dim3(512), 0, s>>>(a, w, ad, M, N, K, kv, tiles_m,
                                                                    tiles_n, per_xcd);
    return hipGetLastError();
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Positions of one launch: the tiles address the positions and the pairs with
// 32 bits.
int64_t launch_positions(int K) {
    const int64_t m = ((int64_t)1 << 31) / (2 * (int64_t)K) / 256 * 256;
    return m < 256 ? 256 : m > 262144 ? 262144 : m;
}

}  // namespace

size_t adapters_scratch_bytes(int rank, int64_t M) {
    return up256((size_t)M * ((rank + 15) / 16 * 16) * 2 * sizeof(uint16_t)) +
           (size_t)((M + 255) / 256 * 256) * sizeof(int2);
}

hipError_t launch_wkv_adapters(const uint16_t* a, const uint16_t* w, const Adapters& ad,
                               const int32_t* ids, int seg, int64_t M, int N, int K, uint16_t* kv,
                               void* scratch, uint32_t* err, hipStream_t s) {
    const int rt = (ad.rank + 15) / 16, rp = 16 * rt;
    uint16_t* u = (uint16_t*)scratch;
    int2* tile = (int2*)((char*)scratch + up256((size_t)M * rp * 2 * sizeof(uint16_t)));
    const int64_t most = launch_positions(K);
    for (int64_t m0 = 0; m0 < M; m0 += most) {
        const int m = (int)(M - m0 < most ? M - m0 : most);
        const uint16_t* am = a + m0 * K;
        uint16_t *um = u + m0 * rp * 2, *kvm = kv + m0 * N;
        // the decode kernel as long as two of its workgroups a compute unit take
        // all at once (128 positions of rank 16 -> 6168: 18 us against 26 with the
        // tiles; 128 of -> 25600, twice too many: 41 against 35), or one, where the
        // products of a high rank on the vector units would take longer than the
        // tiles' on the matrix cores (512 of rank 64 -> 2560: 38 against 30; 384,
        // one workgroup each: 25 against 30)
        const int64_t tn = (N + 63) / 64, blocks = (int64_t)((m + 63) / 64) * tn;
        const bool rows =
            K % 64 == 0 && (int64_t)K * 2 * 64 < (1ll << 31) &&
            (m <= 64 || blocks <= (ad.rank > 32 && m >= 256 ? 1 : 2) * (int64_t)cu_count());
        // the ring of tiles where they all run at once (613 of rank 8 -> 6168: 21.3 us
        // the kernel against 25.7 of the projection's own tiles; 800, two rounds: 42
        // us the call against 33, there two workgroups of the latter share a
        // compute unit)
        const bool ring = K % 64 == 0 && (int64_t)K * 2 * kTile < (1ll << 31) &&
                          (int64_t)((m + kTile - 1) / kTile) * ((N + kTile - 1) / kTile) <=
                              cu_count();
        int2* order = rows ? nullptr : tile + m0;
        AddAdapters add{ad.up, um, ids, nullptr, m0, ad.n, ad.rank, rp, seg,
                        (int64_t)N * ad.rank};
        hipError_t e = run_down(am, ad, add, m, K, um, order, err, s);
        if (e != hipSuccess) return e;
        add.tile = order;
        if (!rows && ring)
            e = run_tiles(am, w, add, m, N, K, kvm, s);
        else if (!rows)
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
