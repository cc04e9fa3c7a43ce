// Embedding rows by id with a scale, copied to a layer's streams, and the
// gradient of that lookup:
//
//   out[i][s] = scale * table[ids[i]],                             s < streams;
//   dtable[v] = (dtable[v]) + scale * sum_{i: ids[i] = v} sum_s dout[i][s].
//
// The gradient's positions are sorted by id (stable, so a row's positions are
// in order), and each row's sum is taken in fp32 in an order that the sizes
// and the ids alone decide: the same on every run, and no atomics on values.
//
// All of it is bound by memory, or by the latencies of the launches where there is
// little.  Measured: 4096 rows of 5120 to four streams 28 us, 185 MB, 6.5 TB/s (it writes
// much more than it reads); the gradient of 4096 positions of four streams to 129,280
// fp32 rows of 5120 430 us, of which 374 are the 2.65 GB of zeros and rows (7.1 TB/s) and 49
// the sums (168 MB read, 4.7 TB/s with what they write); 32,768 positions of 2056, added to what is
// there, 95-102 us: 23 the sort, 64 the sums (274 MB, 4.3 TB/s), 15.5 the rows that
// reach over tiles; 98,304 positions of 64 46 us: 28 the sort, whose four launches on 48
// workgroups are chains of latencies, 16 the sums, 4 the joining.  Elementary
// torch operations (index_add_ in fp32): 186, 670, 610 and 61.
#include <algorithm>
#include <type_traits>

#include "lanes.h"

namespace engram {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
    const bf16x2_t v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// Eight values of a row: 16 bytes of bf16 or 32 of fp32.
template <class T>
struct Eight;
template <>
struct Eight<float> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const f32x4*>(p);
        b = *reinterpret_cast<const f32x4*>(p + 4);
    }
    __device__ __forceinline__ void load_once(const float* p) {
        a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
        b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + 4));
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = a[e], x[e + 4] = b[e];
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = x[e], b[e] = x[e + 4];
    }
    __device__ __forceinline__ void store(float* p) const {
        __builtin_nontemporal_store(a, reinterpret_cast<f32x4*>(p));
        __builtin_nontemporal_store(b, reinterpret_cast<f32x4*>(p + 4));
    }
};
template <>
struct Eight<uint16_t> {
    u32x4 a;
    __device__ __forceinline__ void load(const uint16_t* p) {
        a = *reinterpret_cast<const u32x4*>(p);
    }
    __device__ __forceinline__ void load_once(const uint16_t* p) {
        a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(a[e] << 16);
            x[2 * e + 1] = __uint_as_float(a[e] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = pack2_bf16(x[2 * e], x[2 * e + 1]);
    }
    __device__ __forceinline__ void store(uint16_t* p) const {
        __builtin_nontemporal_store(a, reinterpret_cast<u32x4*>(p));
    }
};

// ---------------------------------------------------------------- lookup
// A thread eight values of a position: read once, stored for every stream, past the
// caches (what is written is larger than they are, or read by another kernel much later).
template <class T, class O>
__global__ void __launch_bounds__(256) embed_kernel(const T* __restrict__ table, int64_t rows,
                                                    int dim, const int32_t* __restrict__ ids,
                                                    uint32_t items, float scale, int streams,
                                                    O* __restrict__ out,
                                                    uint32_t* __restrict__ err) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x, per_row = (uint32_t)dim / 8;
    if (i >= items) return;
    const uint32_t m = i / per_row, c = (i - m * per_row) * 8;
    const int64_t id = ids[m];
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (id >= 0 && id < rows) {
        Eight<T> in;
        in.load(table + id * dim + c);
        in.values(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= scale;
    } else if (err && c == 0) {
        atomicOr(err, ENGRAM_ERRBIT_ROW);
    }
    Eight<O> o;
    o.set(x);
    O* to = out + (int64_t)m * streams * dim + c;
    for (int s = 0; s < streams; ++s) o.store(to + (int64_t)s * dim);
}

template <class T, class O>
hipError_t run_embed(const void* table, int64_t rows, int dim, const int32_t* ids, int64_t n,
                     float scale, int streams, void* out, uint32_t* err, hipStream_t s) {
    const int64_t most = ((int64_t)1 << 31) / (dim / 8) - 1;  // positions a launch
    for (int64_t at = 0; at < n; at += most) {
        const int64_t m = n - at < most ? n - at : most;
        const uint32_t items = (uint32_t)(m * (dim / 8));
        embed_kernel<T, O><<<dim3((items + 255) / 256), dim3(256), 0, s>>>(
            (const T*)table, rows, dim, ids + at, items, scale, streams,
            (O*)out + at * streams * dim, err);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// ---------------------------------------------------------------- positions by id
// Sorted pairs (key, position): a key is the id, or `rows` for a position that
// adds nothing (a pad, a bad id); these come last.  A radix sort from the low
// digit up, each pass stable, in as few digits of at most 11 bits as the keys need
// (two up to four million rows): a pass costs two launches, 11-17 us.
constexpr int kChunk = 2048;        // positions a workgroup sorts
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kEach = kChunk / kSortThreads;
constexpr int kMaxDigit = 11;
constexpr int kMaxBins = 1 << kMaxDigit;
constexpr int kFewChunks = 62;      // up to here each workgroup sums the counts before its own (a thread
                                    // at most 31 of them, in 16 bits; 98,304 positions 46.8 us, with a
                                    // kernel for the sums 49.2)

struct __attribute__((aligned(8))) Pair {
    uint32_t key, pos;
};

// the wave's lanes that hold the same digit as this one
__device__ __forceinline__ uint64_t same_digit(uint32_t digit) {
    uint64_t other = 0;
#pragma unroll
    for (int b = 0; b < kMaxDigit; ++b) {
        const uint64_t vote = __ballot((digit >> b) & 1);
        const uint32_t own = (uint32_t)((int32_t)(digit << (31 - b)) >> 31);
        other |= (uint64_t)((uint32_t)(vote >> 32) ^ own) << 32 | ((uint32_t)vote ^ own);
    }
    return ~other;
}

// Where each of the chunk's pairs goes, counting from its digit's first place:
// the pairs of a wave are kEach rows of 64, in order.  Leaves in count[bin] the
// chunk's number of pairs of that digit, in wave_count[w][bin] those of the
// waves before w.  wave_count holds zeros on entry.
__device__ __forceinline__ void rank_chunk(const uint32_t (&digit)[kEach], int bits,
                                           uint16_t (&rank)[kEach],
                                           uint16_t (*wave_count)[kMaxBins],
                                           uint32_t* count) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const uint64_t mask = same_digit(digit[e]);
        const uint32_t before = wave_count[wave][digit[e]];
        rank[e] = (uint16_t)(before + __builtin_popcountll(mask & ((1ull << lane) - 1)));
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if ((mask >> lane) == 1)  // the last lane of its digit
            wave_count[wave][digit[e]] = (uint16_t)(rank[e] + 1);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    for (int b = threadIdx.x; b < (1 << bits); b += kSortThreads) {
        uint32_t sum = 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t x = wave_count[w][b];
            wave_count[w][b] = (uint16_t)sum;
            sum += x;
        }
        count[b] = sum;
    }
    __syncthreads();
}

// value[0 .. bins) -> the sums before each; all threads of the workgroup
__device__ __forceinline__ void scan_bins(uint32_t* value, int bins, uint32_t* wave_sum) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int PER = kMaxBins / kSortThreads;
    uint32_t x[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = threadIdx.x * PER + i;
        x[i] = b < bins ? value[b] : 0;
        sum += x[i];
    }
    const uint32_t upto = sum_upto(sum);
    if (lane == 63) wave_sum[wave] = upto;
    __syncthreads();
    uint32_t before = upto - sum;
    for (int w = 0; w < wave; ++w) before += wave_sum[w];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = threadIdx.x * PER + i;
        if (b < bins) value[b] = before;
        before += x[i];
    }
    __syncthreads();
}

__device__ __forceinline__ uint32_t key_of(int32_t id, int64_t rows, int32_t pad_id, bool* bad) {
    const bool in = id >= 0 && id < rows;
    *bad |= !in;
    return in && id != pad_id ? (uint32_t)id : (uint32_t)rows;
}

// Zeros over a whole gradient, by workgroups beside the first sorting kernel's: 16 bytes a
// thread, so that all that are running write next to each other, and small workgroups for
// large ones (2.65 GB: 256 threads 385 us, 6.9 TB/s, 1024 threads 425; runs of 64 KiB
// a workgroup 480, with the nontemporal hint 520).
struct Fill {
    u32x4* to;        // null: none
    int64_t units;    // of 16 bytes
    uint32_t first;   // the first workgroup that fills
    int rounds;
};
template <int THREADS>
__device__ __forceinline__ void fill(const Fill& f) {
    const int64_t hop = (int64_t)(gridDim.x - f.first) * THREADS;
    int64_t i = (int64_t)(blockIdx.x - f.first) * THREADS + threadIdx.x;
    for (int r = 0; r < f.rounds; ++r, i += hop)
        if (i < f.units) f.to[i] = u32x4{0, 0, 0, 0};
}

struct SortArgs {
    const int32_t* ids;
    int64_t n, padded;       // positions; places of the sorted arrays (whole tiles, one more)
    int64_t rows;
    int32_t pad_id;
    Pair* pair;              // [padded] out, sorted; keys behind the n-th are `rows`
    uint32_t* owners;        // two counters that a later kernel uses: set to 0
    uint32_t* err;
};

// Up to kRankMost positions: a position's place is the number of pairs before it,
// counted by a wave, the keys of all in LDS.  (A whole gradient of 4096 positions of 64 15
// us, of 8192 24.5; by the passes below 28 and 29.)
constexpr int kRankMost = 8192;
template <int THREADS>
__global__ void __launch_bounds__(THREADS) sort_rank_kernel(const SortArgs a,
                                                                 const Fill zeros) {
    if (blockIdx.x >= zeros.first) return fill<THREADS>(zeros);
    constexpr int EACH = 4096 / THREADS;
    __shared__ u32x4 keys[kRankMost / 4];
    uint32_t* key = reinterpret_cast<uint32_t*>(keys);
    const int tid = threadIdx.x, lane = tid & 63, n = (int)a.n, fours = (n + 3) / 4;
    bool bad = false;
    for (int i0 = tid; i0 < fours * 4; i0 += THREADS * EACH) {
        int32_t id[EACH];  // (all on their way at once)
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
            const int i = i0 + THREADS * j;
            id[j] = i < n ? a.ids[i] : 0;
        }
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
            const int i = i0 + THREADS * j;
            if (i < fours * 4) key[i] = i < n ? key_of(id[j], a.rows, a.pad_id, &bad) : ~0u;
        }
    }
    if (blockIdx.x == 0) {
        if (bad && a.err) atomicOr(a.err, ENGRAM_ERRBIT_ROW);
        if (tid < 2) a.owners[tid] = 0;
        for (int i = n + tid; i < (int)a.padded; i += THREADS)
            a.pair[i] = Pair{(uint32_t)a.rows, 0};
    }
    __syncthreads();
    const int i = __builtin_amdgcn_readfirstlane(blockIdx.x * (THREADS / 64) + (tid >> 6));
    if (i >= n) return;
    const uint32_t own = key[i];
    int before = 0;
#pragma unroll 4
    for (int q = lane; q < fours; q += 64) {
        const u32x4 k = keys[q];
#pragma unroll
        for (int e = 0; e < 4; ++e)  // equal keys in the order of their positions
            before += k[e] < own + (q * 4 + e < i ? 1u : 0u) ? 1 : 0;
    }
    for (int o = 1; o < 64; o <<= 1) before += __shfl_xor(before, o, 64);
    if (lane == 0) a.pair[before] = Pair{own, (uint32_t)i};
}

// More of them: per pass, each chunk's digits counted ...
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortArgs a,
                                                                  const Pair* from, int shift,
                                                                  int d, uint16_t* counts,
                                                                  const Fill zeros) {
    if (blockIdx.x >= zeros.first) return fill<kSortThreads>(zeros);
    __shared__ uint32_t count[kMaxBins];
    const int tid = threadIdx.x, bins = 1 << d;
    for (int b = tid; b < bins; b += kSortThreads) count[b] = 0;
    __syncthreads();
    bool bad = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int64_t i = (int64_t)blockIdx.x * kChunk + e * kSortThreads + tid;
        if (i < a.n) {
            const uint32_t k = FIRST ? key_of(a.ids[i], a.rows, a.pad_id, &bad) : from[i].key;
            atomicAdd(&count[(k >> shift) & (bins - 1)], 1u);
        }
    }
    if (FIRST) {
        if (bad && a.err) atomicOr(a.err, ENGRAM_ERRBIT_ROW);
        if (blockIdx.x == 0 && tid < 2) a.owners[tid] = 0;
    }
    __syncthreads();
    for (int b = tid; b < bins; b += kSortThreads)
        counts[(int64_t)blockIdx.x * bins + b] = (uint16_t)count[b];
}

// ... (many chunks: the counts of the chunks before each, and the totals) ...
__global__ void __launch_bounds__(256) sort_scan_kernel(const uint16_t* counts, int chunks,
                                                        int bins, uint32_t* before,
                                                        uint32_t* totals) {
    const int b = blockIdx.x * 256 + threadIdx.x;
    if (b >= bins) return;
    uint32_t sum = 0;
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) {
        const uint32_t x = counts[(int64_t)c * bins + b];
        before[(int64_t)c * bins + b] = sum;
        sum += x;
    }
    totals[b] = sum;
}

// ... and its pairs put in their places.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(
    const SortArgs a, const Pair* __restrict__ from, int shift, int d,
    const uint16_t* __restrict__ counts, const uint32_t* __restrict__ before,
    const uint32_t* __restrict__ totals, int chunks, Pair* __restrict__ to, int last) {
    __shared__ uint16_t wave_count[kSortWaves][kMaxBins];
    __shared__ uint32_t count[kMaxBins], place[kMaxBins], wave_sum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, bins = 1 << d;
    const int chunk = blockIdx.x;
    const int64_t first = (int64_t)chunk * kChunk + wave * (64 * kEach) + lane;
    uint32_t k[kEach], p[kEach], digit[kEach];
    uint16_t rank[kEach];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int64_t i = first + 64 * e;
        // (places behind the last position sort behind it: every digit of its key is set)
        k[e] = ~0u;
        p[e] = 0;
        if (i < a.n) {
            const Pair x = FIRST ? Pair{key_of(a.ids[i], a.rows, a.pad_id, &bad), (uint32_t)i} : from[i];
            k[e] = x.key;
            p[e] = x.pos;
        }
        digit[e] = (k[e] >> shift) & (bins - 1);
    }
    // the first place of each digit, less the pairs of earlier chunks, and those: a
    // thread eight digits of some of the chunks
    for (int b = tid; b < bins; b += kSortThreads) {
        place[b] = totals ? totals[b] : 0;
        count[b] = totals ? before[(int64_t)chunk * bins + b] : 0;
    }
    if (!totals) {
        __syncthreads();
        const int groups = bins / 8, hop = kSortThreads / groups, g = tid % groups;
        u32x4 earlier = {0, 0, 0, 0}, all = {0, 0, 0, 0};  // two digits a word
        for (int c0 = tid / groups; c0 < chunks; c0 += 16 * hop) {
            u32x4 x[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int c = c0 + j * hop;
                x[j] = u32x4{0, 0, 0, 0};
                if (c < chunks) x[j] = reinterpret_cast<const u32x4*>(counts)[c * groups + g];
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                all += x[j];
                if (c0 + j * hop < chunk) earlier += x[j];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t x = all[e / 2] >> (e & 1 ? 16 : 0) & 0xFFFFu;
            const uint32_t y = earlier[e / 2] >> (e & 1 ? 16 : 0) & 0xFFFFu;
            if (x) atomicAdd(&place[g * 8 + e], x);
            if (y) atomicAdd(&count[g * 8 + e], y);
        }
        __syncthreads();
    }
    uint32_t mine[kMaxBins / kSortThreads];  // pairs of the digit in earlier chunks
#pragma unroll
    for (int i = 0; i < kMaxBins / kSortThreads; ++i) {
        const int b = tid + i * kSortThreads;
        mine[i] = b < bins ? count[b] : 0;
    }
    for (int b = lane; b < bins / 2; b += 64)
        reinterpret_cast<uint32_t*>(wave_count[wave])[b] = 0;
    __syncthreads();
    scan_bins(place, bins, wave_sum);
    rank_chunk(digit, d, rank, wave_count, count);
#pragma unroll
    for (int i = 0; i < kMaxBins / kSortThreads; ++i) {
        const int b = tid + i * kSortThreads;
        if (b < bins) place[b] += mine[i];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        if (first + 64 * e < a.n) {
            const uint32_t at = place[digit[e]] + wave_count[wave][digit[e]] + rank[e];
            to[at] = Pair{k[e], p[e]};
        }
    }
    if (last && chunk == 0)
        for (int64_t i = a.n + tid; i < a.padded; i += kSortThreads)
            to[i] = Pair{(uint32_t)a.rows, 0};
}

// ---------------------------------------------------------------- sums
// A tile is `tile` places of the sorted pairs (equal work whatever the ids); a thread
// takes eight columns of one, adds the positions up in order and stores a row's sum where the row
// ends.  A row that reaches over the tile's ends leaves a part instead: in
// part[t][0] where it began in an earlier tile, in part[t][1] where it begins
// here and goes on; the latter tile is listed, and a second kernel adds the
// parts up in order.
constexpr int kBatch = 4;      // positions whose rows are on their way at once,
constexpr int kBatchOne = 8;   // with one stream
constexpr int kJoined = 16;    // and parts
// tiles that a row reaches into behind its first: that many take the joining kernel's
// workgroups (3, 5, 9: 98,304 positions of 64 columns 48.3, 49.1, 50.5 us; 32,768 of 2056 by
// frequency 96.6, 95.7, 95.3)
constexpr int kMany = 3;

template <class D, class W>
struct SumArgs {
    const Pair* pair;
    const D* dout;
    W* dtable;
    float* part;         // [tiles][2][dim]
    uint32_t* owners;    // the listed tiles' numbers, of few parts and of many, then each and
                         // its last key: those of few from the front, of many from the end
    uint32_t rows;
    uint32_t tiles;
    int dim, streams, tile;
    float scale;
    int accumulate;
};

template <class W>
__device__ __forceinline__ void put_row(W* to, float (&sum)[8], float scale, const Eight<W>& old,
                                        bool accumulate) {
    float x[8];
    old.values(x);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = accumulate ? __builtin_fmaf(scale, sum[e], x[e]) : scale * sum[e];
    Eight<W> o;
    o.set(x);
    o.store(to);
}

__device__ __forceinline__ void put_part(float* to, const float (&sum)[8]) {
    *reinterpret_cast<f32x4*>(to) = f32x4{sum[0], sum[1], sum[2], sum[3]};
    *reinterpret_cast<f32x4*>(to + 4) = f32x4{sum[4], sum[5], sum[6], sum[7]};
}

// The tile's sums.  Where a row begins in it that goes on, one of its threads gives 1 (0
// otherwise), or 2 where that reaches kMany tiles further; t, key: the tile, the row.
template <class D, class W, int STREAMS, bool ONCE>
__device__ __forceinline__ int sum_tile(const SumArgs<D, W>& a, uint32_t& t, uint32_t& key) {
    const uint32_t per_row = (uint32_t)a.dim / 8;
    const uint32_t item = blockIdx.x * 256 + threadIdx.x;
    t = item / per_row;
    if (t >= a.tiles) return 0;
    const int c = (int)(item - t * per_row) * 8;
    constexpr int BATCH = STREAMS == 1 ? kBatchOne : kBatch;
    const int streams = STREAMS ? STREAMS : a.streams;
    const int64_t start = (int64_t)t * a.tile;
    key = a.pair[start].key;
    bool begun = t == 0 || a.pair[start - 1].key != key;  // the row begins in this tile
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < a.tile; j0 += BATCH) {
        if (key == a.rows) break;
        uint32_t k[BATCH + 1], p[BATCH];
        k[0] = key;
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            k[j + 1] = a.pair[start + j0 + j + 1].key;
            p[j] = a.pair[start + j0 + j].pos;
        }
        bool ends[BATCH], whole[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            ends[j] = k[j] != a.rows && k[j + 1] != k[j];
            whole[j] = ends[j] && begun;
            begun |= ends[j];
        }
        Eight<D> in[BATCH][STREAMS ? STREAMS : 1];
        Eight<W> old[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            if (STREAMS && k[j] != a.rows)
#pragma unroll
                for (int s = 0; s < (STREAMS ? STREAMS : 1); ++s) {
                    const D* from = a.dout + ((int64_t)p[j] * streams + s) * a.dim + c;
                    if (ONCE)
                        in[j][s].load_once(from);
                    else
                        in[j][s].load(from);
                }
            if (whole[j] && a.accumulate) old[j].load(a.dtable + (int64_t)k[j] * a.dim + c);
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            if (k[j] == a.rows) continue;
            if (STREAMS) {
#pragma unroll
                for (int s = 0; s < (STREAMS ? STREAMS : 1); ++s) {
                    float x[8];
                    in[j][s].values(x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[e] += x[e];
                }
            } else {
                for (int s = 0; s < streams; ++s) {
                    Eight<D> more;
                    more.load(a.dout + ((int64_t)p[j] * streams + s) * a.dim + c);
                    float x[8];
                    more.values(x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[e] += x[e];
                }
            }
            if (!ends[j]) continue;
            if (whole[j])
                put_row(a.dtable + (int64_t)k[j] * a.dim + c, sum, a.scale, old[j], a.accumulate);
            else
                put_part(a.part + (int64_t)t * 2 * a.dim + c, sum);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
        }
        key = k[BATCH];
    }
    key = a.pair[start + a.tile - 1].key;
    if (key == a.rows || a.pair[start + a.tile].key != key) return 0;
    put_part(a.part + ((int64_t)t * 2 + (begun ? 1 : 0)) * a.dim + c, sum);
    if (!begun || c != 0) return 0;
    return t + kMany < a.tiles && a.pair[start + (int64_t)kMany * a.tile].key == key ? 2 : 1;
}

// The workgroup's tiles into the lists, by one addition to each counter.  (One a tile: 429 us where
// 786,432 positions of 64 columns fill 98,304 tiles, one a workgroup 158.)
template <class D, class W>
__device__ __forceinline__ void list_tiles(const SumArgs<D, W>& a, int kind, uint32_t t, uint32_t key) {
    __shared__ uint32_t number[2], first[2];
    const int tid = threadIdx.x;
    if (tid < 2) number[tid] = 0;
    if (!__syncthreads_or(kind)) return;
    uint32_t at = 0;
    if (kind) at = atomicAdd(&number[kind - 1], 1u);
    __syncthreads();
    if (tid < 2 && number[tid]) first[tid] = atomicAdd(a.owners + tid, number[tid]);
    __syncthreads();
    if (!kind) return;
    at += first[kind - 1];
    if (kind == 2) at = a.tiles - 1 - at;
    a.owners[2 + 2 * at] = t;
    a.owners[3 + 2 * at] = key;
}

// the first place in pair[lo, hi) whose key is at least k
__device__ __forceinline__ int64_t first_at_least(const Pair* pair, int64_t lo, int64_t hi,
                                                  uint32_t k) {
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (pair[mid].key < k)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// the last tile that begins with the row that tile t ends with, 64 looked at together
template <class D, class W>
__device__ __forceinline__ uint32_t last_tile(const SumArgs<D, W>& a, uint32_t t, uint32_t key) {
    const uint32_t lane = threadIdx.x & 63;
    uint32_t lo = t + 1, hi = a.tiles;  // lo does; hi does not, or is none
    while (lo + 1 < hi) {
        const uint32_t step = (hi - lo + 63) / 64, q = lo + lane * step;
        const bool in = q < hi && a.pair[(int64_t)q * a.tile].key == key;
        const uint32_t yes = (uint32_t)__builtin_popcountll(__ballot(in));
        hi = lo + yes * step < hi ? lo + yes * step : hi;
        lo += (yes - 1) * step;
    }
    return lo;
}

// Four columns of share i of n of a row's parts: that of tile t, where it begins, then one
// of each tile behind it.
template <class D, class W>
__device__ __forceinline__ f32x4 sum_parts(const SumArgs<D, W>& a, uint32_t t, uint32_t last, int c,
                                           int i, int n) {
    const int64_t parts = last - t, each = (parts + n - 1) / n;  // behind the first one
    const int64_t from = 1 + i * each, to = min(from + each, parts + 1);
    f32x4 sum = {0, 0, 0, 0};
    if (c >= a.dim) return sum;
    if (i == 0) sum = *reinterpret_cast<const f32x4*>(a.part + ((int64_t)t * 2 + 1) * a.dim + c);
    for (int64_t q0 = from; q0 < to; q0 += kJoined) {
        f32x4 x[kJoined];  // (on their way at once; behind the share's last one that one again)
#pragma unroll
        for (int j = 0; j < kJoined; ++j)
            x[j] = *reinterpret_cast<const f32x4*>(a.part + (t + min(q0 + j, to - 1)) * 2 * a.dim + c);
#pragma unroll
        for (int j = 0; j < kJoined; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = q0 + j < to ? sum[e] + x[j][e] : sum[e];
    }
    return sum;
}

// Four columns of a row that reaches over tiles, by its parts' sum.
template <class D, class W>
__device__ __forceinline__ void put_four(const SumArgs<D, W>& a, uint32_t key, int c, const f32x4& sum) {
    W* to = a.dtable + (int64_t)key * a.dim + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(W) == 4)
            to[e] = a.accumulate ? __builtin_fmaf(a.scale, sum[e], to[e]) : a.scale * sum[e];
        else
            to[e] = (W)f32_to_bf16(a.accumulate ? __builtin_fmaf(a.scale, sum[e], bf16_to_f32(to[e]))
                                                : a.scale * sum[e]);
    }
}

// The rows that reach over tiles.  One of many parts takes a workgroup for 64 columns, 16
// lanes four each of a sixteenth of the parts, the shares joined in order; of the others a
// thread takes four columns.
template <class D, class W>
__global__ void __launch_bounds__(256) grad_join_kernel(const SumArgs<D, W> a) {
    __shared__ f32x4 shares[16][16];
    const uint32_t blocks = (uint32_t)(a.dim + 63) / 64, many = a.owners[1] * blocks;
    const int tid = threadIdx.x;
    for (uint32_t w = blockIdx.x; w < many; w += gridDim.x) {
        const uint32_t at = a.tiles - 1 - w / blocks, t = a.owners[2 + 2 * at], key = a.owners[3 + 2 * at];
        const int c = (int)(w % blocks) * 64 + (tid & 15) * 4;
        shares[tid >> 4][tid & 15] = sum_parts(a, t, last_tile(a, t, key), c, tid >> 4, 16);
        __syncthreads();
        if (tid < 16 && c < a.dim) {
            f32x4 sum = shares[0][tid];
#pragma unroll
            for (int i = 1; i < 16; ++i) {
                const f32x4 x = shares[i][tid];
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += x[e];
            }
            put_four(a, key, c, sum);
        }
        __syncthreads();
    }
    const uint32_t per_row = (uint32_t)a.dim / 4;
    const uint64_t few = (uint64_t)a.owners[0] * per_row;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + tid; i < few; i += (uint64_t)gridDim.x * 256) {
        const uint32_t at = (uint32_t)(i / per_row), t = a.owners[2 + 2 * at], key = a.owners[3 + 2 * at];
        const int c = (int)(i - (uint64_t)at * per_row) * 4;
        bool goes_on[kMany];  // the row reaches into the j-th tile behind its first
#pragma unroll
        for (int j = 1; j < kMany; ++j)
            goes_on[j] = t + j < a.tiles && a.pair[(int64_t)(t + j) * a.tile].key == key;
        f32x4 sum = *reinterpret_cast<const f32x4*>(a.part + ((int64_t)t * 2 + 1) * a.dim + c);
        f32x4 x[kMany];
#pragma unroll
        for (int j = 1; j < kMany; ++j)
            if (goes_on[j]) x[j] = *reinterpret_cast<const f32x4*>(a.part + (int64_t)(t + j) * 2 * a.dim + c);
#pragma unroll
        for (int j = 1; j < kMany; ++j)
            if (goes_on[j])
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += x[j][e];
        put_four(a, key, c, sum);
    }
}

// Rows that no position names are set to zero, a workgroup a run of rows.  The run's
// keys are found by narrowing the sorted keys down by 256 at a time.
constexpr int kFillRows = 256;
template <class W>
__device__ __forceinline__ void fill_run(const Pair* pair, int64_t n, int64_t rows, int each,
                                         int64_t r0, int dim, W* dtable) {
    __shared__ uint8_t named[kFillRows];
    const int tid = threadIdx.x;
    const int here = (int)(rows - r0 < each ? rows - r0 : each);
    named[tid] = 0;
    int64_t lo = 0, hi = n;  // the run's first key lies in [lo, hi]
    while (lo < hi) {
        const int64_t step = (hi - lo + 255) / 256, at = lo + tid * step;
        const int less = __syncthreads_count(at < hi && pair[at].key < (uint32_t)r0);
        const int64_t next = lo + less * step;
        hi = next < hi ? next : hi;
        lo = less ? lo + (less - 1) * step + 1 : lo;
    }
    for (int left = 4; left > 0; --left, lo += 256) {
        const uint32_t k = lo + tid < n ? pair[lo + tid].key : (uint32_t)rows;
        const bool in = k < (uint32_t)(r0 + here);
        if (in) named[k - (uint32_t)r0] = 1;
        if (__syncthreads_count(in) < 256) break;
        // many more: each row looks for itself
        if (left == 1 && tid < here) {
            const uint32_t own = (uint32_t)(r0 + tid);
            const int64_t first = first_at_least(pair, lo + 256, n, own);
            if (first < n && pair[first].key == own) named[tid] = 1;
        }
    }
    __syncthreads();
    const u32x4 zero = {0, 0, 0, 0};
    const uint32_t units = (uint32_t)(dim * sizeof(W) / 16), all = (uint32_t)here * units;
    u32x4* to = reinterpret_cast<u32x4*>(dtable + r0 * dim);
    for (uint32_t i = tid; i < all; i += 256)
        if (!named[i / units]) __builtin_nontemporal_store(zero, to + i);
}

// The first workgroups take tiles, those behind them runs of rows.
template <class D, class W, int STREAMS, bool ONCE>
__global__ void __launch_bounds__(256) grad_sum_kernel(const SumArgs<D, W> a, uint32_t sum_blocks,
                                                       int64_t n, int64_t row0, int each) {
    if (blockIdx.x < sum_blocks) {
        uint32_t t, key;
        const int kind = sum_tile<D, W, STREAMS, ONCE>(a, t, key);
        list_tiles(a, kind, t, key);
    } else
        fill_run<W>(a.pair, n, a.rows, each, row0 + (int64_t)(blockIdx.x - sum_blocks) * each,
                    a.dim, a.dtable);
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) fill_kernel(const Fill zeros) {
    fill<THREADS>(zeros);
}

// Up to 64 positions: one kernel (64 of 4 x 256 to 1000 rows 7.6 us, by three 12.5).  A
// workgroup takes a run of rows, zeros and sums, or, where only rows that ids name are
// written (each = 0), 256 (row, eight columns) pairs.
constexpr int kFewMost = 64;
constexpr int64_t kMuchBytes = 256 << 20;  // zeros by small workgroups
constexpr int64_t kFewBytes = 64 << 20;    // a gradient that one launch fills and sums (32 positions, rows of 1024:
                                           // 49 MB 11.2 us, by two launches 13.6; 82 MB 17.3 both; 164 MB 33 and 27)
template <class D, class W>
__global__ void __launch_bounds__(256) grad_few_kernel(
    const D* __restrict__ dout, const int32_t* __restrict__ ids, int n, int streams, int64_t rows,
    int dim, float scale, int32_t pad_id, int accumulate, int each, int64_t row0,
    W* __restrict__ dtable, uint32_t* __restrict__ err) {
    __shared__ uint32_t key[kFewMost];
    __shared__ int next[kFewMost + 1];  // the next position of the same id; n: none
    __shared__ int list[kFewMost];      // where the ids summed here come first
    __shared__ int lists;
    __shared__ uint8_t named[kFillRows];
    const int tid = threadIdx.x;
    const int64_t r0 = row0 + (int64_t)blockIdx.x * each;
    const int here = (int)(rows - r0 < each ? rows - r0 : each);
    bool bad = false;
    const uint32_t own = tid < n ? key_of(ids[tid], rows, pad_id, &bad) : (uint32_t)rows;
    if (bad && err && r0 == 0) atomicOr(err, ENGRAM_ERRBIT_ROW);
    const bool mine = own < (uint32_t)rows &&
                      (each == 0 || (own >= (uint32_t)r0 && own - (uint32_t)r0 < (uint32_t)here));
    if (tid < kFewMost) key[tid] = own;
    named[tid] = 0;
    if (__syncthreads_or(mine)) {
        if (tid < kFewMost) {  // (one wave)
            bool first = mine;
            int after = n;
#pragma unroll 8
            for (int j = kFewMost - 1; j >= 0; --j) {
                const bool same = key[j] == own;
                first &= !(same && j < tid);
                after = same && j > tid ? j : after;
            }
            next[tid] = tid < n ? after : n;
            const uint64_t firsts = __ballot(first);
            if (first) list[__builtin_popcountll(firsts & ((1ull << tid) - 1))] = tid;
            if (mine && each) named[own - (uint32_t)r0] = 1;
            if (tid == 0) {
                lists = __builtin_popcountll(firsts);
                next[kFewMost] = n;
            }
        }
        __syncthreads();
        const uint32_t per_row = (uint32_t)dim / 8, items = (uint32_t)lists * per_row;
        const uint32_t from = each ? tid : blockIdx.x * 256 + tid;
        const uint32_t hop = each ? 256 : gridDim.x * 256;
        for (uint32_t item = from; item < items; item += hop) {
            const uint32_t at = item / per_row, c = (item - at * per_row) * 8;
            const int first = list[at];
            W* to = dtable + (int64_t)key[first] * dim + c;
            Eight<W> old;
            if (accumulate) old.load(to);
            float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            for (int p = first; p < n;) {
                int q[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    q[j] = p;
                    p = next[p];
                }
                for (int s = 0; s < streams; ++s) {
                    Eight<D> d[kBatch];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j)
                        if (q[j] < n) d[j].load(dout + ((int64_t)q[j] * streams + s) * dim + c);
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        float x[8];
                        d[j].values(x);
                        if (q[j] < n)
#pragma unroll
                            for (int e = 0; e < 8; ++e) sum[e] += x[e];
                    }
                }
            }
            put_row(to, sum, scale, old, accumulate);
        }
    }
    const u32x4 zero = {0, 0, 0, 0};
    const uint32_t units = (uint32_t)(dim * sizeof(W) / 16), all = (uint32_t)here * units;
    u32x4* to = reinterpret_cast<u32x4*>(dtable + r0 * dim);
    for (uint32_t i = tid; i < all; i += 256)
        if (!named[i / units]) __builtin_nontemporal_store(zero, to + i);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Places a tile: enough tiles that the threads fill the machine twice (256 compute
// units of 2048 threads), few enough that rows of many positions leave few parts.  (32,768 positions
// of 2056 by frequency: 95 us, with half or twice the threads 102 and 101.)
constexpr int kMostTile = 64, kLeastTile = kBatchOne;
constexpr int64_t kSumThreads = 512 * 1024;
constexpr int64_t kOnceBytes = 64 << 20;
int tile_of(int64_t n, int dim) {
    int tile = kMostTile;
    while (tile > kLeastTile && n / tile * (dim / 8) < kSumThreads) tile /= 2;
    return tile;
}
// what any number of positions up to n has tiles (scratch for n does for fewer)
int64_t tiles_room(int64_t n, int dim) {
    const int64_t fewest = (n + kMostTile - 1) / kMostTile, most = (n + kLeastTile - 1) / kLeastTile;
    const int64_t filled = 2 * kSumThreads / (dim / 8) + 2;
    return std::min(most, std::max(fewest, filled));
}

struct GradScratch {
    int64_t padded, tiles, chunks;
    int bits, digit_bits, tile;
    size_t pair[2], counts, before, totals, owners, part, bytes;
};

GradScratch grad_layout(int64_t n, int64_t rows, int dim) {
    GradScratch g;
    g.tile = tile_of(n, dim);
    g.tiles = (n + g.tile - 1) / g.tile;
    g.padded = g.tiles * g.tile + kLeastTile;  // (a tile's last batch looks one key ahead)
    const int64_t room = tiles_room(n, dim);
    const size_t places = (size_t)((n + kMostTile - 1) / kMostTile * kMostTile + kLeastTile) * sizeof(Pair);
    g.chunks = (n + kChunk - 1) / kChunk;
    g.bits = 3;  // (eight digits a thread)
    while (((int64_t)1 << g.bits) <= rows) ++g.bits;  // the key `rows` as well
    const int passes = (g.bits + kMaxDigit - 1) / kMaxDigit;
    g.digit_bits = (g.bits + passes - 1) / passes;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += up256(bytes);
        return here;
    };
    const bool radix = n > kRankMost;
    for (int i = 0; i < 2; ++i) {
        g.pair[i] = take(i == 0 || radix ? places : 0);
    }
    g.counts = take(radix ? ((size_t)g.chunks << g.digit_bits) * 2 : 0);
    g.before = take(g.chunks > kFewChunks ? ((size_t)g.chunks << g.digit_bits) * 4 : 0);
    g.totals = take(g.chunks > kFewChunks ? ((size_t)4 << g.digit_bits) : 0);
    g.owners = take((size_t)(room + 1) * 8);
    g.part = take((size_t)room * 2 * dim * sizeof(float));
    g.bytes = at;
    return g;
}

template <class D, class W>
hipError_t run_grad(const void* dout, const int32_t* ids, int64_t n, int streams, int64_t rows,
                    int dim, float scale, int32_t pad_id, bool accumulate, void* dtable,
                    void* scratch, uint32_t* err, hipStream_t s) {
    // Zeros: over everything before the sums where these write few of the rows once
    // more, otherwise by workgroups that leave out the rows that ids name, runs of 64
    // KiB (fp32 rows of 1032: 6000 positions of 32,003 38.7 against 54.5 us, 64,640 of 129,280
    // 229 against 210).
    const int64_t units = accumulate ? 0 : rows * dim * (int64_t)sizeof(W) / 16;
    const bool over = n <= kFewMost ? units * 16 > kFewBytes : n <= rows / 4;
    const int64_t by_size = 65536 / (dim * (int64_t)sizeof(W));
    const int each = (int)(by_size < 1 ? 1 : by_size > kFillRows ? kFillRows : by_size);
    const int64_t most = (int64_t)each << 22;  // rows a launch
    auto zeros = [&](uint32_t first, int threads, uint32_t* grid) {
        Fill f{(u32x4*)dtable, units, first, 1};
        *grid = first;
        if (!over || units == 0) return f;
        const int64_t blocks = (units + threads - 1) / threads, launch = (int64_t)1 << 21;
        f.rounds = (int)((blocks + launch - 1) / launch);
        *grid = first + (uint32_t)(blocks < launch ? blocks : launch);
        return f;
    };
    const bool much = over && units * 16 > kMuchBytes;
    const bool named_only = accumulate || over;  // the sums' kernel writes no zeros
    uint32_t grid = 0;
    hipError_t e = hipSuccess;
    if (n <= kFewMost) {
        const Fill f = zeros(0, 256, &grid);
        if (grid > 0) {
            fill_kernel<256><<<dim3(grid), dim3(256), 0, s>>>(f);
            if ((e = hipGetLastError()) != hipSuccess || n == 0) return e;
        }
        for (int64_t r0 = 0; r0 < (named_only ? 1 : rows); r0 += most) {
            const int64_t m = rows - r0 < most ? rows - r0 : most;
            const int64_t blocks = named_only ? (n * (dim / 8) + 255) / 256 : (m + each - 1) / each;
            grad_few_kernel<D, W><<<dim3((uint32_t)blocks), dim3(256), 0, s>>>(
                (const D*)dout, ids, (int)n, streams, rows, dim, scale, pad_id, accumulate ? 1 : 0,
                named_only ? 0 : each, r0, (W*)dtable, err);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        return e;
    }
    const GradScratch g = grad_layout(n, rows, dim);
    char* base = (char*)scratch;
    Pair* pair[2] = {(Pair*)(base + g.pair[0]), (Pair*)(base + g.pair[1])};
    uint32_t* owners = (uint32_t*)(base + g.owners);
    int now = 0;
    SortArgs a{ids, n, g.padded, rows, pad_id, pair[0], owners, err};
    if (n <= kRankMost) {
        const int threads = much ? 256 : 1024, per = threads / 64;
        const Fill f = zeros((uint32_t)((n + per - 1) / per), threads, &grid);
        if (much)
            sort_rank_kernel<256><<<dim3(grid), dim3(256), 0, s>>>(a, f);
        else
            sort_rank_kernel<1024><<<dim3(grid), dim3(1024), 0, s>>>(a, f);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    } else {
        uint16_t* counts = (uint16_t*)(base + g.counts);
        uint32_t* totals = g.chunks > kFewChunks ? (uint32_t*)(base + g.totals) : nullptr;
        uint32_t* before = totals ? (uint32_t*)(base + g.before) : nullptr;
        const dim3 chunks((uint32_t)g.chunks), threads(kSortThreads);
        for (int shift = 0; shift < g.bits; shift += g.digit_bits) {
            const int d = g.bits - shift < g.digit_bits ? g.bits - shift : g.digit_bits;
            const int last = shift + d >= g.bits;
            Fill f{nullptr, 0, (uint32_t)g.chunks, 0};
            if (shift == 0 && much) {
                f = zeros(0, 256, &grid);
                fill_kernel<256><<<dim3(grid), dim3(256), 0, s>>>(f);
                if ((e = hipGetLastError()) != hipSuccess) return e;
                f = Fill{nullptr, 0, (uint32_t)g.chunks, 0};
                grid = (uint32_t)g.chunks;
                sort_count_kernel<true><<<chunks, threads, 0, s>>>(a, nullptr, shift, d, counts, f);
            } else if (shift == 0) {
                f = zeros((uint32_t)g.chunks, kSortThreads, &grid);
                sort_count_kernel<true><<<dim3(grid), threads, 0, s>>>(a, nullptr, shift, d, counts, f);
            } else {
                sort_count_kernel<false><<<chunks, threads, 0, s>>>(a, pair[now], shift, d, counts, f);
            }
            if ((e = hipGetLastError()) != hipSuccess) return e;
            if (totals) {
                sort_scan_kernel<<<dim3(((1u << d) + 255) / 256), dim3(256), 0, s>>>(
                    counts, (int)g.chunks, 1 << d, before, totals);
                if ((e = hipGetLastError()) != hipSuccess) return e;
            }
            if (shift == 0)
                sort_place_kernel<true><<<chunks, threads, 0, s>>>(
                    a, nullptr, shift, d, counts, before, totals, (int)g.chunks, pair[0], last);
            else
                sort_place_kernel<false><<<chunks, threads, 0, s>>>(a, pair[now], shift, d, counts,
                                                                  before, totals, (int)g.chunks,
                                                                  pair[1 - now], last);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            now = shift == 0 ? 0 : 1 - now;
        }
    }
    SumArgs<D, W> b{pair[now], (const D*)dout, (W*)dtable, (float*)(base + g.part), owners,
                    (uint32_t)rows, (uint32_t)g.tiles, dim, streams, g.tile, scale,
                    accumulate ? 1 : 0};
    // (large gradients are read past the caches: 32,768 positions of 2056 in bf16, 135 MB,
    // 113 -> 99 us a call; 20,000 of 1024, 41 MB, 62 -> 66)
    const bool once = n * streams * dim * (int64_t)sizeof(D) >= kOnceBytes;
    auto kernel = [&](auto streams_) {
        constexpr int S = decltype(streams_)::value;
        return once ? grad_sum_kernel<D, W, S, true> : grad_sum_kernel<D, W, S, false>;
    };
    // (3 and 5 to 8 streams by one kernel, a load at a time and through the caches: 4096
    // positions of 5120 in bf16, added to fp32 rows, 62, 73 and 113 us with 3, 5 and 8; 53, 60 and
    // 70 with 1, 2 and 4.  Of 1024: 25, 30 and 38; 19, 19 and 24)
    auto k = streams == 1   ? kernel(std::integral_constant<int, 1>())
             : streams == 2 ? kernel(std::integral_constant<int, 2>())
             : streams == 4 ? kernel(std::integral_constant<int, 4>())
                            : grad_sum_kernel<D, W, 0, false>;
    uint32_t sum_blocks = (uint32_t)((g.tiles * (dim / 8) + 255) / 256);
    for (int64_t r0 = 0; r0 == 0 || r0 < (named_only ? 0 : rows); r0 += most) {
        const int64_t m = rows - r0 < most ? rows - r0 : most;
        const uint32_t blocks = named_only ? 0 : (uint32_t)((m + each - 1) / each);
        k<<<dim3(sum_blocks + blocks), dim3(256), 0, s>>>(b, sum_blocks, n, r0, each);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        sum_blocks = 0;
    }
    if (g.tiles > 1) {
        const int64_t items = (g.tiles - 1) * (dim / 4);  // at most: a thread each
        grad_join_kernel<D, W><<<dim3((uint32_t)std::min<int64_t>((items + 255) / 256, 2048)), dim3(256), 0, s>>>(b);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace

hipError_t launch_embed(const void* table, bool table_f32, int64_t rows, int dim,
                        const int32_t* ids, int64_t n, float scale, int streams, void* out,
                        bool out_f32, uint32_t* err, hipStream_t s) {
    auto k = table_f32 ? (out_f32 ? run_embed<float, float> : run_embed<float, uint16_t>)
                       : (out_f32 ? run_embed<uint16_t, float> : run_embed<uint16_t, uint16_t>);
    return k(table, rows, dim, ids, n, scale, streams, out, err, s);
}

bool embed_grad_supported(int64_t n, int64_t rows, int dim) {
    return grad_layout(n, rows, dim).tiles * (dim / 8) < ((int64_t)1 << 31);
}

size_t embed_grad_scratch_bytes(int64_t n, int64_t rows, int dim) {
    return grad_layout(n, rows, dim).bytes;
}

hipError_t launch_embed_grad(const void* dout, bool dout_f32, const int32_t* ids, int64_t n,
                             int streams, int64_t rows, int dim, float scale, int32_t pad_id,
                             bool accumulate, void* dtable, bool dtable_f32, void* scratch,
                             uint32_t* err, hipStream_t s) {
    auto k = dout_f32 ? (dtable_f32 ? run_grad<float, float> : run_grad<float, uint16_t>)
                      : (dtable_f32 ? run_grad<uint16_t, float> : run_grad<uint16_t, uint16_t>);
    return k(dout, ids, n, streams, rows, dim, scale, pad_id, accumulate, dtable, scratch, err, s);
}

}  // namespace engram
