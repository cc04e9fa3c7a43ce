// Stage 3: the wkv projection ("Module engram" docs, stage 3 / linear_bf16;
// the Engram block's self.wkv): kv[m][n] = bf16(sum_k a[m][k] * w[n][k]).
//
// bf16 MFMA GEMM for gfx950.  Both operands are K-contiguous ([M, K] and
// [N, K]), which is exactly the per-lane operand layout of
// v_mfma_f32_32x32x16_bf16 (each lane holds 8 consecutive k of one row), so
// tiles go to LDS unchanged and come back out as one 16-byte read per
// fragment.  Two kernels: the main one (M >= 1024, K % 64 == 0, further
// below) and a general one for small M or ragged K (right here).
//
//  * Macro tile BM x BN x 64, double-buffered in LDS; the next k-tile's global
//    loads are issued before the current tile's MFMAs.
//  * LDS rows are 128 bytes (64 bf16); the 16-byte chunk index is XOR-swizzled
//    with the row so that the 32 rows of a fragment read hit distinct banks.
//  * The MFMA computes the transposed product W.A^T, so each lane ends up with
//    4 consecutive output columns per register group and writes 8-byte bf16
//    runs (instead of 2-byte scatters).
//  * Tiles are numbered so that the tiles one XCD runs are contiguous and, in
//    groups of 4 M-tiles, share A and W panels in that XCD's L2.
//  * Edges (M, N, K not multiples of the tile) are zero-filled on load and
//    masked on store; no access leaves the operands.
#include <type_traits>

#include "adapters.h"

namespace engram {
namespace {

constexpr int BK = 64;      // k per LDS tile: 64 bf16 = 128 bytes per row
constexpr int CH = BK / 8;  // 16-byte chunks per row

__device__ __forceinline__ int swz(int row, int ch) {
    return ch ^ ((row & 7) ^ ((row >> 3) & 1));
}

// D: NoAdapters, or AddAdapters (a low-rank adapter's product added to the
// accumulators before they are rounded).
template <int BM, int BN, int WM, int WN, class D>
__global__ void __launch_bounds__((BM / WM) * (BN / WN) * 64, 1)
wkv_kernel(const uint16_t* __restrict__ A, const uint16_t* __restrict__ W, int64_t M, int N,
           int K, uint16_t* __restrict__ C, int tiles_m, int tiles_n, int per_xcd, const D ad) {
    constexpr int WAVES_N = BN / WN;
    constexpr int NT = (BM / WM) * WAVES_N * 64;
    constexpr int TM = WM / 32, TN = WN / 32;
    constexpr int A_LD = BM * CH / NT;
    constexpr int B_LD = BN * CH / NT;
    static_assert(BM * CH % NT == 0 && BN * CH % NT == 0, "tile/thread mismatch");
    __shared__ uint4 lds[2][(BM + BN) * CH];

    // ---- tile of this workgroup
    int mt, nt;
    if (!tile_of(blockIdx.x, per_xcd, tiles_m, tiles_n, &mt, &nt)) return;
    const int64_t m0 = (int64_t)mt * BM;
    const int n0 = nt * BN;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;

    // ---- global load slots: chunk q = tid + i*NT -> (row q/CH, chunk q%CH)
    const uint16_t* a_src[A_LD];
    const uint16_t* b_src[B_LD];
    int a_dst[A_LD], b_dst[B_LD];
    bool a_ok[A_LD], b_ok[B_LD];
    int a_ch[A_LD], b_ch[B_LD];
#pragma unroll
    for (int i = 0; i < A_LD; ++i) {
        const int q = tid + i * NT, row = q / CH, ch = q % CH;
        a_ok[i] = (m0 + row) < M;
        int64_t src = a_ok[i] ? m0 + row : 0;
        if constexpr (D::on) src = ad.tile[m0 + row].x;
        a_src[i] = A + src * (int64_t)K + ch * 8;
        a_dst[i] = row * CH + swz(row, ch);
        a_ch[i] = ch * 8;
    }
#pragma unroll
    for (int i = 0; i < B_LD; ++i) {
        const int q = tid + i * NT, row = q / CH, ch = q % CH;
        b_ok[i] = (n0 + row) < N;
        b_src[i] = W + (int64_t)(b_ok[i] ? (n0 + row) : 0) * K + ch * 8;
        b_dst[i] = (BM + row) * CH + swz(row, ch);
        b_ch[i] = ch * 8;
    }

    uint4 ra[A_LD], rb[B_LD];
    auto load = [&](int kt) {
        const int k0 = kt * BK;
#pragma unroll
        for (int i = 0; i < A_LD; ++i)
            ra[i] = (a_ok[i] && k0 + a_ch[i] < K)
                        ? *reinterpret_cast<const uint4*>(a_src[i] + k0)
                        : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < B_LD; ++i)
            rb[i] = (b_ok[i] && k0 + b_ch[i] < K)
                        ? *reinterpret_cast<const uint4*>(b_src[i] + k0)
                        : make_uint4(0, 0, 0, 0);
    };
    auto store = [&](int buf) {
#pragma unroll
        for (int i = 0; i < A_LD; ++i) lds[buf][a_dst[i]] = ra[i];
#pragma unroll
        for (int i = 0; i < B_LD; ++i) lds[buf][b_dst[i]] = rb[i];
    };

    f32x16 acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.0f;

    const int nk = (K + BK - 1) / BK;
    load(0);
    store(0);
    __syncthreads();

    const int lrow = lane & 31;
    const int lhalf = lane >> 5;
    for (int kt = 0; kt < nk; ++kt) {
        const int cur = kt & 1;
        if (kt + 1 < nk) load(kt + 1);
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks) {
            const int ch = kchunk(ks, lhalf);
            bf16x8 fa[TM], fw[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int row = wm * WM + i * 32 + lrow;
                uint4 u = lds[cur][row * CH + swz(row, ch)];
                fa[i] = __builtin_bit_cast(bf16x8, u);
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int row = wn * WN + j * 32 + lrow;
                uint4 u = lds[cur][(BM + row) * CH + swz(row, ch)];
                fw[j] = __builtin_bit_cast(bf16x8, u);
            }
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fw[j], fa[i], acc[j][i],
                                                                        0, 0, 0);
        }
        if (kt + 1 < nk) store(cur ^ 1);
        __syncthreads();
    }

    if constexpr (D::on) ad.template add<TM, TN>(acc, m0 + wm * WM, n0 + wn * WN, N, lane);

    // ---- epilogue: D[n][m]; lane holds m = lane%32, n = 8*(v/4) + 4*(lane/32) + v%4
#pragma unroll
    for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t m = m0 + wm * WM + i * 32 + lrow;
            if (m >= M) continue;
#pragma unroll
            for (int g4 = 0; g4 < 4; ++g4) {
                const int n = n0 + wn * WN + j * 32 + 8 * g4 + 4 * lhalf;
                if (n >= N) continue;
                const uint32_t lo = pack_bf16(acc[j][i][4 * g4 + 0], acc[j][i][4 * g4 + 1]);
                const uint32_t hi = pack_bf16(acc[j][i][4 * g4 + 2], acc[j][i][4 * g4 + 3]);
                int64_t to = m;
                if constexpr (D::on) to = ad.tile[m].x;
                *reinterpret_cast<uint2*>(C + to * N + n) = make_uint2(lo, hi);
            }
        }
    }
}

template <int BM, int BN, int WM, int WN, class D>
hipError_t run(const uint16_t* a, const uint16_t* w, int64_t M, int N, int K, uint16_t* kv,
               const D& ad, hipStream_t s) {
    constexpr int NT = (BM / WM) * (BN / WN) * 64;
    const int tiles_m = (int)((M + BM - 1) / BM);
    const int tiles_n = (N + BN - 1) / BN;
    const int total = tiles_m * tiles_n;
    const int per_xcd = (total + N_XCD - 1) / N_XCD;
    wkv_kernel<BM, BN, WM, WN, D><<<dim3(per_xcd * N_XCD), dim3(NT), 0, s>>>(
        a, w, M, N, K, kv, tiles_m, tiles_n, per_xcd, ad);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Main kernel for K % 64 == 0: 256 x 256 output tiles, 4 waves of 128 x 128,
// k-tiles of 64 double-buffered in LDS (2 x 64 KiB).
//
// Tiles move global -> LDS with buffer_load_dwordx4 ... lds (no register
// staging): one instruction writes 1 KiB = 8 LDS rows of 128 bytes, lane l
// landing at byte 16*l, so lane l fetches the logical 16-byte chunk that the
// swizzle places at that slot.  Rows past M (or N) lie past the buffer
// descriptor's extent and read as zero.  While k-tile kt is multiplied the
// loads of k-tile kt+1 are in flight; one barrier per k-tile hands the next
// stage over.  (Touching k-tile kt+2 into L2 one tile early, or a 4-stage
// ring of 32-wide k-tiles, measured slower on this shape.)  Within a k-tile the
// fragments of the next 16-wide k-step are read from LDS while the current
// k-step's 16 MFMAs issue.
constexpr int F_NT = 256;  // 4 waves in a 2 x 2 arrangement (the 8-wave variant: 512)
constexpr bool WAVES8 = true;

// BT x BT output tiles (BT = 256: 128 x 128 per wave; BT = 128: 64 x 64 per
// wave).  Columns [0, N) of this launch start at W row 0 and C column 0; C
// rows are `ldc` elements apart.
template <int BT, int WMV, int WNV, class D>
__device__ __forceinline__ void wkv_tile(const uint16_t* __restrict__ A,
                                         const uint16_t* __restrict__ W, int64_t M, int N, int K,
                                         uint16_t* __restrict__ C, int64_t ldc, int tiles_m,
                                         int tiles_n, int per_xcd, const D& ad, uint8_t* smem) {
    constexpr int NW = WMV * WNV;              // waves: WMV along m, WNV along n
    constexpr int BM = BT, BN = BT, WM = BT / WMV, WN = BT / WNV;
    constexpr int TI = WM / 32, TJ = WN / 32;  // 32 x 32 MFMA tiles per wave
    constexpr int NLD = BT / 8 / NW;           // LDS-bound loads per wave per operand
    constexpr int STAGE = (BM + BN) * 128;     // bytes per LDS stage

    int mt, nt;
    if (!tile_of(blockIdx.x, per_xcd, tiles_m, tiles_n, &mt, &nt)) return;
    const int64_t m0 = (int64_t)mt * BM;
    const int n0 = nt * BN;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int wm = wave / WNV, wn = wave % WNV;

    const int64_t rows_a = min((int64_t)BM, M - m0);
    const int rows_w = min(BN, N - n0);
    // with adapters the tile's rows may be any positions (M * K * 2 < 2^31)
    const __amdgpu_buffer_rsrc_t ra = D::on ? make_rsrc(A, (uint32_t)(M * K * 2))
                                            : make_rsrc(A + m0 * K, (uint32_t)(rows_a * K * 2));
    int2 own[BT / 64];  // position and adapter of rows m0 + 64 k + lane
    if constexpr (D::on)
#pragma unroll
        for (int k = 0; k < BT / 64; ++k) own[k] = ad.tile[m0 + 64 * k + lane];
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(W + (int64_t)n0 * K, (uint32_t)(rows_w * K * 2));

    // load slots: instruction i of this wave fills LDS segment
    // seg = NW*i + wave = rows 8*seg .. 8*seg+7 of the A rows (then the W rows)
    uint32_t voff[NLD];
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
        const int row = (NW * i + wave) * 8 + (lane >> 3);
        voff[i] = (uint32_t)(row * K * 2 + slot128(row, lane & 7) * 16);
    }
    uint32_t aoff[NLD];
    auto place_a = [&]() {
#pragma unroll
        for (int i = 0; i < NLD; ++i) {
            aoff[i] = voff[i];
            if constexpr (D::on) {
                const int row = (NW * i + wave) * 8 + (lane >> 3);
                int m = 0;
#pragma unroll
                for (int k = 0; k < BT / 64; ++k) {
                    const int x = __shfl(own[k].x, row & 63, 64);
                    m = (row >> 6) == k ? x : m;
                }
                aoff[i] = (uint32_t)m * (uint32_t)(K * 2) +
                          (uint32_t)(slot128(row, lane & 7) * 16);
            }
        }
    };
    auto issue_a = [&](int kt, int stage) {
        uint8_t* st = smem + stage * STAGE;
#pragma unroll
        for (int i = 0; i < NLD; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra, (lds_void*)(st + (NW * i + wave) * 1024), 16, aoff[i], kt * 128, 0, 0);
    };
    auto issue_w = [&](int kt, int stage) {
        uint8_t* st = smem + stage * STAGE;
#pragma unroll
        for (int i = 0; i < NLD; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rw, (lds_void*)(st + BM * 128 + (NW * i + wave) * 1024), 16, voff[i], kt * 128, 0,
                0);
    };
    auto issue_loads = [&](int kt, int stage) {
        issue_a(kt, stage);
        issue_w(kt, stage);
    };

    const int lrow = lane & 31, lhalf = lane >> 5;
    bf16x8 fa[2][TI], fw[2][TJ];
    auto read_frags = [&](int stage, int ks, int buf) {
        const uint8_t* st = smem + stage * STAGE;
        const int c = kchunk(ks, lhalf);
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            const int row = wm * WM + i * 32 + lrow;
            fa[buf][i] = *reinterpret_cast<const bf16x8*>(st + row * 128 + slot128(row, c) * 16);
        }
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int row = wn * WN + j * 32 + lrow;
            fw[buf][j] = *reinterpret_cast<const bf16x8*>(st + BM * 128 + row * 128 +
                                                          slot128(row, c) * 16);
        }
    };

    f32x16 acc[TJ][TI];
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.0f;

    auto mfma_half = [&](int cur, int half) {
#pragma unroll
        for (int j = half * (TJ / 2); j < (half + 1) * (TJ / 2); ++j)
#pragma unroll
            for (int i = 0; i < TI; ++i)
                acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fw[cur][j], fa[cur][i],
                                                                    acc[j][i], 0, 0, 0);
    };
    // One k-tile = 4 k-steps of TI*TJ MFMAs, each k-step its own scheduling
    // region (sched_barrier fences stop the compiler from regrouping MFMAs by
    // accumulator across k-steps, which would chain dependent MFMAs).  The
    // next k-step's TI+TJ fragment reads are interleaved with the current
    // MFMAs; the next k-tile's LDS-bound buffer loads go out during k-step 0.
    // The last k-step is split around the barrier so that the next k-tile's
    // first fragment reads overlap its second half.
    //   LOADS: k-tile kt+1 exists (its loads are issued here)
    constexpr int NRD = TI + TJ, NMF = TI * TJ;
    auto k_tile = [&](int kt, auto with_loads) {
        constexpr bool LOADS = decltype(with_loads)::value;
        const int stage = kt & 1;
#pragma unroll
        for (int ks = 0; ks < 3; ++ks) {
            const int cur = ks & 1;
            if (LOADS && ks == 0) issue_loads(kt + 1, stage ^ 1);
            read_frags(stage, ks + 1, cur ^ 1);
            mfma_half(cur, 0);
            mfma_half(cur, 1);
            if constexpr ((2 * NLD) % NRD == 0) {
#pragma unroll
                for (int r = 0; r < NRD; ++r) {
                    if (LOADS && ks == 0)
                        __builtin_amdgcn_sched_group_barrier(0x020, 2 * NLD / NRD, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                }
                if (NMF > NRD) __builtin_amdgcn_sched_group_barrier(0x008, NMF - NRD, 0);
            } else if (LOADS && ks == 0) {
                constexpr int RR = 2 * NLD > NRD ? 2 * NLD : NRD;
#pragma unroll
                for (int r = 0; r < RR; ++r) {
                    if (r < 2 * NLD) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                    if (r < NMF) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    if (r < NRD) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                }
                if constexpr (NMF > RR) __builtin_amdgcn_sched_group_barrier(0x008, NMF - RR, 0);
            } else {
#pragma unroll
                for (int r = 0; r < NRD; ++r) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                }
                if constexpr (NMF > NRD) __builtin_amdgcn_sched_group_barrier(0x008, NMF - NRD, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        mfma_half(1, 0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (LOADS) {
            __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's loads landed
            __syncthreads();  // everyone's loads landed; tile kt fully consumed
            __builtin_amdgcn_sched_barrier(0);
            read_frags(stage ^ 1, 0, 0);
        }
        mfma_half(1, 1);
        if constexpr (LOADS) {
#pragma unroll
            for (int r = 0; r < NRD; ++r) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                if (r < NMF / 2) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    using T = std::true_type;
    using F = std::false_type;

    const int nk = K / BK;
    if constexpr (D::on) {  // W needs no positions
        issue_w(0, 0);
        place_a();
        issue_a(0, 0);
    } else {
        place_a();
        issue_loads(0, 0);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    __syncthreads();
    read_frags(0, 0, 0);
    for (int kt = 0; kt + 1 < nk; ++kt) k_tile(kt, T{});
    // the last k-tile leaves the other stage free
    uint8_t* const free_stage = smem + (nk & 1) * STAGE;
    if constexpr (D::on)
        if (any_adapter(own)) load_pairs<BT, NW>(ad, own, M, wave, lane, 0, free_stage);
    k_tile(nk - 1, F{});
    __syncthreads();  // every wave is done with the operand stages
    if constexpr (D::on)
        add_tile<BT, NW, TI, TJ>(ad, acc, own, M, n0, N, wm, wn, wave, lane, free_stage,
                                 smem + ((nk + 1) & 1) * STAGE);

    // ---- epilogue through LDS.  D[n][m]: lane holds m = lane%32 (+32 i) and
    // n = 32 j + 8 (v/4) + 4 (lane/32) + v%4.  Each wave writes its WM x WN
    // block as bf16 rows [m][n] into its own part of LDS (16-byte chunks
    // XOR-swizzled by row), then reads it back so that consecutive lanes store
    // one WN*2-byte row run with 16-byte stores.
    constexpr int RB = WN * 2;            // bytes per epilogue row
    constexpr int CHW = RB / 16;          // 16-byte chunks per row
    constexpr int RPI = 64 / CHW;         // rows per store instruction
    uint8_t* ep = smem + wave * (WM * RB);
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int g4 = 0; g4 < 4; ++g4) {
                const int r = i * 32 + lrow;
                const int nn = j * 32 + 8 * g4 + 4 * lhalf;  // multiple of 4
                const int ch = (nn >> 3) ^ (r & (CHW - 1));
                const uint32_t lo = pack_bf16(acc[j][i][4 * g4 + 0], acc[j][i][4 * g4 + 1]);
                const uint32_t hi = pack_bf16(acc[j][i][4 * g4 + 2], acc[j][i][4 * g4 + 3]);
                *reinterpret_cast<uint2*>(ep + r * RB + ch * 16 + (nn & 4) * 2) =
                    make_uint2(lo, hi);
            }
    const int rsub = lane / CHW, csub = lane % CHW;
#pragma unroll 4
    for (int it = 0; it < WM / RPI; ++it) {
        const int r = it * RPI + rsub;
        const uint4 v =
            *reinterpret_cast<const uint4*>(ep + r * RB + ((csub ^ (r & (CHW - 1))) << 4));
        const int64_t m = m0 + wm * WM + r;
        const int n = n0 + wn * WN + csub * 8;
        int64_t to = m;
        if constexpr (D::on) {
            const int row = wm * WM + r;  // its position is lane row % 64's
#pragma unroll
            for (int k = 0; k < BT / 64; ++k) {
                const int x = __shfl(own[k].x, row & 63, 64);
                to = (row >> 6) == k ? x : to;
            }
        }
        if (m < M && n < N) *reinterpret_cast<uint4*>(C + to * ldc + n) = v;
    }
}

template <class D>
__global__ void __launch_bounds__(F_NT, 1)
wkv_fast_256(const uint16_t* __restrict__ A, const uint16_t* __restrict__ W, int64_t M, int N,
             int K, uint16_t* __restrict__ C, int64_t ldc, int tiles_m, int tiles_n, int per_xcd,
             const D ad) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * (256 + 256) * 128];
    wkv_tile<256, 2, 2>(A, W, M, N, K, C, ldc, tiles_m, tiles_n, per_xcd, ad, smem);
}

template <class D>
__global__ void __launch_bounds__(2 * F_NT, 1)
wkv_fast_256w8(const uint16_t* __restrict__ A, const uint16_t* __restrict__ W, int64_t M, int N,
               int K, uint16_t* __restrict__ C, int64_t ldc, int tiles_m, int tiles_n,
               int per_xcd, const D ad) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * (256 + 256) * 128];
    wkv_tile<256, 2, 4>(A, W, M, N, K, C, ldc, tiles_m, tiles_n, per_xcd, ad, smem);
}

template <class D>
__global__ void __launch_bounds__(F_NT, 1)
wkv_fast_128(const uint16_t* __restrict__ A, const uint16_t* __restrict__ W, int64_t M, int N,
             int K, uint16_t* __restrict__ C, int64_t ldc, int tiles_m, int tiles_n, int per_xcd,
             const D ad) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * (128 + 128) * 128];
    wkv_tile<128, 2, 2>(A, W, M, N, K, C, ldc, tiles_m, tiles_n, per_xcd, ad, smem);
}

template <int BT, class D>
hipError_t run_fast(const uint16_t* a, const uint16_t* w, int64_t M, int N, int K, uint16_t* c,
                    int64_t ldc, const D& ad, hipStream_t s) {
    const int tiles_m = (int)((M + BT - 1) / BT);
    const int tiles_n = (N + BT - 1) / BT;
    const int total = tiles_m * tiles_n;
    const int per_xcd = (total + N_XCD - 1) / N_XCD;
    if constexpr (BT == 256 && WAVES8) {
        wkv_fast_256w8<D><<<dim3(per_xcd * N_XCD), dim3(2 * F_NT), 0, s>>>(
            a, w, M, N, K, c, ldc, tiles_m, tiles_n, per_xcd, ad);
    } else {
        auto launch = [&](auto kern) {
            kern<<<dim3(per_xcd * N_XCD), dim3(F_NT), 0, s>>>(a, w, M, N, K, c, ldc, tiles_m,
                                                              tiles_n, per_xcd, ad);
        };
        if constexpr (BT == 256)
            launch(wkv_fast_256<D>);
        else
            launch(wkv_fast_128<D>);
    }
    return hipGetLastError();
}


// Main path: 256 x 256 tiles over the widest column range whose tile count
// fills whole rounds of the machine, and the remaining columns in 128 x 128
// tiles when those fit in one round (T=4096, N=25600: 1536 big tiles = 6
// rounds, then 256 small tiles, instead of 7 rounds with the last one a
// quarter full).
template <class D>
hipError_t run_main(const uint16_t* a, const uint16_t* w, int64_t M, int N, int K, uint16_t* kv,
                    const D& ad, hipStream_t s) {
    const int cus = cu_count();
    const int tiles_m = (int)((M + 255) / 256);
    const int tiles_n = (N + 255) / 256;
    int nb = tiles_n;
    if ((int64_t)tiles_m * tiles_n % cus != 0) {
        int cand = tiles_n - 1;
        while (cand > 0 && (int64_t)tiles_m * cand % cus != 0) --cand;
        if (cand > 0) {
            const int64_t small = ((M + 127) / 128) * ((N - cand * 256 + 127) / 128);
            if (small <= cus) nb = cand;
        }
    }
    hipError_t e = run_fast<256>(a, w, M, nb * 256 < N ? nb * 256 : N, K, kv, N, ad, s);
    if (e != hipSuccess || nb * 256 >= N) return e;
    D rest = ad;  // the adapters' columns from nb * 256 on
    if constexpr (D::on) rest.up += (int64_t)nb * 256 * ad.rank;
    return run_fast<128>(a, w + (int64_t)nb * 256 * K, M, N - nb * 256, K, kv + (int64_t)nb * 256, N,
                         rest, s);
}

template <class D>
hipError_t project(const uint16_t* a, const uint16_t* w, int64_t M, int N, int K, uint16_t* kv,
                   const D& ad, hipStream_t s) {
    if (M == 0) return hipSuccess;
    if constexpr (D::on) {
        // Two workgroups of 128 x 128 tiles share a compute unit: as many of them as
        // compute units take 20 us (K = 1536), as many 256 x 256 tiles 50 us.  (1536
        // -> 25600, rank 16: 500 positions 77 us with the small ones, 61 with the
        // large, 600 78 and 102, 1000 129 and 106; -> 6168: 1024 positions 34 and 46.)
        auto rounds = [&](int64_t t) {
            const int64_t tiles = ((M + t - 1) / t) * ((N + t - 1) / t), cus = cu_count();
            return (tiles + cus - 1) / cus;
        };
        if (K % BK == 0 && (int64_t)K * 2 * 256 < (1ll << 31)) {
            if (2 * rounds(128) <= 5 * rounds(256))
                return run_fast<128>(a, w, M, N, K, kv, N, ad, s);
            return run_main(a, w, M, N, K, kv, ad, s);
        }
    }
    if (M >= 1024 && K % BK == 0 && (int64_t)K * 2 * 256 < (1ll << 31))
        return run_main(a, w, M, N, K, kv, ad, s);
    if (M >= 1024) return run<256, 256, 128, 64>(a, w, M, N, K, kv, ad, s);
    return run<64, 64, 32, 32>(a, w, M, N, K, kv, ad, s);
}

}  // namespace

int cu_count() {
    static int n = 0;
    if (n == 0) {
        int dev = 0, v = 0;
        if (hipGetDevice(&dev) == hipSuccess &&
            hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess &&
            v > 0)
            n = v;
        else
            n = 256;
    }
    return n;
}

hipError_t launch_wkv(const uint16_t* a, const uint16_t* w, int64_t M, int N, int K,
                      uint16_t* kv, hipStream_t s) {
    return project(a, w, M, N, K, kv, NoAdapters{}, s);
}

hipError_t launch_wkv_added(const uint16_t* a, const uint16_t* w, int64_t M, int N, int K,
                            const AddAdapters& ad, uint16_t* kv, hipStream_t s) {
    return project(a, w, M, N, K, kv, ad, s);
}

}  // namespace engram
