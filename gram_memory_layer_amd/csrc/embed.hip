// Embedding rows by id with a scale, copied to a layer's streams, and the
// gradient of that lookup:
//
//   out[i][s] = scale * table[ids[i]],                             s < streams;
//   dtable[v] = (dtable[v]) + scale * sum_{i: ids[i] = v} sum_s dout[i][s].
//
// The gradient's positions are sorted by id (stable, so a row's positions are
// in order), and each row's sum is taken in fp32 in an order that the sizes
// and the ids alone decide: the same on every run, and no atomics on values.
#include "internal.h"

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
// A thread eight values of a position: read once, stored for every stream.
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
// digit up, each pass stable.
constexpr int kChunk = 4096;        // positions a workgroup sorts
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kEach = kChunk / kSortThreads;
constexpr int kMaxDigit = 11;
constexpr int kMaxBins = 1 << kMaxDigit;
constexpr int kFewChunks = 64;      // up to here each workgroup sums the counts before its own

// the wave's lanes that hold the same digit as this one
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits) {
    uint64_t mask = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const bool set = (digit >> b) & 1;
        const uint64_t vote = __ballot(set);
        mask &= set ? vote : ~vote;
    }
    return mask;
}

// Where each of the chunk's pairs goes, counting from its digit's first place:
// the pairs of a wave are kEach rows of 64, in order.  Leaves in count[bin] the
// chunk's number of pairs of that digit, in wave_count[w][bin] those of the
// waves before w.  count and wave_count hold zeros on entry.
__device__ __forceinline__ void rank_chunk(const uint32_t (&digit)[kEach], int bits,
                                           uint16_t (&rank)[kEach],
                                           uint16_t (*wave_count)[kMaxBins],
                                           uint32_t* count) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const uint64_t mask = same_digit(digit[e], bits);
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
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t y = __shfl_up(upto, o, 64);
        if (lane >= o) upto += y;
    }
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

struct SortArgs {
    const int32_t* ids;
    int64_t n, padded;       // positions; places of the sorted arrays (whole tiles, one more)
    int64_t rows;
    int32_t pad_id;
    uint32_t* key;           // [padded] out, sorted; keys behind the n-th are `rows`
    uint32_t* pos;           // [padded] out
    uint32_t* owners;        // a counter that a later kernel uses: set to 0
    uint32_t* err;
};

// Up to kChunk positions: one workgroup, all passes in LDS.
__global__ void __launch_bounds__(kSortThreads) sort_few_kernel(const SortArgs a, int bits,
                                                                int digit_bits) {
    __shared__ uint32_t key[kChunk];
    __shared__ uint16_t pos[kChunk], wave_count[kSortWaves][kMaxBins];
    __shared__ uint32_t count[kMaxBins];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int first = wave * (64 * kEach) + lane;
    uint32_t k[kEach], p[kEach], digit[kEach];
    uint16_t rank[kEach];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int i = first + 64 * e;
        k[e] = i < a.n ? key_of(a.ids[i], a.rows, a.pad_id, &bad) : (uint32_t)a.rows;
        p[e] = i;
    }
    if (bad && a.err) atomicOr(a.err, ENGRAM_ERRBIT_ROW);
    if (tid == 0) *a.owners = 0;
    for (int shift = 0; shift < bits; shift += digit_bits) {
        const int d = bits - shift < digit_bits ? bits - shift : digit_bits, bins = 1 << d;
        for (int b = lane; b < bins; b += 64) wave_count[wave][b] = 0;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int e = 0; e < kEach; ++e) digit[e] = (k[e] >> shift) & (bins - 1);
        rank_chunk(digit, d, rank, wave_count, count);
        scan_bins(count, bins, key);  // (the last pass's keys have been read)
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const uint32_t at = count[digit[e]] + wave_count[wave][digit[e]] + rank[e];
            key[at] = k[e];
            pos[at] = (uint16_t)p[e];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            k[e] = key[first + 64 * e];
            p[e] = pos[first + 64 * e];
        }
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int i = first + 64 * e;
        if (i < a.padded) {
            a.key[i] = k[e];
            a.pos[i] = p[e];
        }
    }
    // (a place behind a full chunk)
    if (tid == 0 && a.padded > kChunk) a.key[kChunk] = (uint32_t)a.rows;
}

// More of them: per pass, each chunk's digits counted ...
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortArgs a,
                                                                  const uint32_t* from_key,
                                                                  int shift, int d,
                                                                  uint32_t* counts) {
    __shared__ uint32_t count[kMaxBins];
    const int tid = threadIdx.x, bins = 1 << d;
    for (int b = tid; b < bins; b += kSortThreads) count[b] = 0;
    __syncthreads();
    bool bad = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int64_t i = (int64_t)blockIdx.x * kChunk + e * kSortThreads + tid;
        if (i < a.n) {
            const uint32_t k = FIRST ? key_of(a.ids[i], a.rows, a.pad_id, &bad) : from_key[i];
            atomicAdd(&count[(k >> shift) & (bins - 1)], 1u);
        }
    }
    if (FIRST) {
        if (bad && a.err) atomicOr(a.err, ENGRAM_ERRBIT_ROW);
        if (blockIdx.x == 0 && tid == 0) *a.owners = 0;
    }
    __syncthreads();
    for (int b = tid; b < bins; b += kSortThreads) counts[(int64_t)blockIdx.x * bins + b] = count[b];
}

// ... (many chunks: the counts of the chunks before each, and the totals) ...
__global__ void __launch_bounds__(256) sort_scan_kernel(uint32_t* counts, int chunks, int bins,
                                                        uint32_t* totals) {
    const int b = blockIdx.x * 256 + threadIdx.x;
    if (b >= bins) return;
    uint32_t sum = 0;
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) {
        const uint32_t x = counts[(int64_t)c * bins + b];
        counts[(int64_t)c * bins + b] = sum;
        sum += x;
    }
    totals[b] = sum;
}

// ... and its pairs put in their places.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(
    const SortArgs a, const uint32_t* __restrict__ from_key, const uint32_t* __restrict__ from_pos,
    int shift, int d, const uint32_t* __restrict__ counts, const uint32_t* __restrict__ totals,
    int chunks, uint32_t* __restrict__ to_key, uint32_t* __restrict__ to_pos, int last) {
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
            k[e] = FIRST ? key_of(a.ids[i], a.rows, a.pad_id, &bad) : from_key[i];
            p[e] = FIRST ? (uint32_t)i : from_pos[i];
        }
        digit[e] = (k[e] >> shift) & (bins - 1);
    }
    // the first place of each digit, less the pairs of earlier chunks, and those
    constexpr int PER = kMaxBins / kSortThreads;
    uint32_t before[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = i * kSortThreads + tid;
        before[i] = 0;
        if (b < bins) {
            uint32_t all = 0;
            if (totals) {
                before[i] = counts[(int64_t)chunk * bins + b];
                all = totals[b];
            } else {
#pragma unroll 4
                for (int c = 0; c < chunks; ++c) {
                    const uint32_t x = counts[c * bins + b];
                    before[i] += c < chunk ? x : 0;
                    all += x;
                }
            }
            place[b] = all;
        }
    }
    for (int b = lane; b < bins; b += 64) wave_count[wave][b] = 0;
    __syncthreads();
    scan_bins(place, bins, wave_sum);
    rank_chunk(digit, d, rank, wave_count, count);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = i * kSortThreads + tid;
        if (b < bins) place[b] += before[i];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        if (first + 64 * e < a.n) {
            const uint32_t at = place[digit[e]] + wave_count[wave][digit[e]] + rank[e];
            to_key[at] = k[e];
            to_pos[at] = p[e];
        }
    }
    if (last && chunk == 0)
        for (int64_t i = a.n + tid; i < a.padded; i += kSortThreads) to_key[i] = (uint32_t)a.rows;
}

// ---------------------------------------------------------------- sums
// A tile is `tile` places of the sorted pairs; a thread takes eight columns of
// one, adds the positions up in order and stores a row's sum where the row
// ends.  A row that reaches over the tile's ends leaves a part instead: in
// part[t][0] where it began in an earlier tile, in part[t][1] where it begins
// here and goes on; the latter tile is listed, and a second kernel adds the
// parts up in order.
constexpr int kBatch = 4;  // positions whose rows are on their way at once

template <class D, class W>
struct SumArgs {
    const uint32_t* key;
    const uint32_t* pos;
    const D* dout;
    W* dtable;
    float* part;         // [tiles][2][dim]
    uint32_t* owners;    // the number of listed tiles, then the tiles
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

template <class D, class W, int STREAMS>
__global__ void __launch_bounds__(256) grad_sum_kernel(const SumArgs<D, W> a) {
    const uint32_t per_row = (uint32_t)a.dim / 8;
    const uint32_t item = blockIdx.x * 256 + threadIdx.x;
    const uint32_t t = item / per_row;
    if (t >= a.tiles) return;
    const int c = (int)(item - t * per_row) * 8;
    const int streams = STREAMS ? STREAMS : a.streams;
    const int64_t start = (int64_t)t * a.tile;
    uint32_t key = a.key[start];
    bool begun = t == 0 || a.key[start - 1] != key;  // the row begins in this tile
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < a.tile; j0 += kBatch) {
        if (key == a.rows) break;
        uint32_t k[kBatch + 1], p[kBatch];
        k[0] = key;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            k[j + 1] = a.key[start + j0 + j + 1];
            p[j] = a.pos[start + j0 + j];
        }
        bool ends[kBatch], whole[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            ends[j] = k[j] != a.rows && k[j + 1] != k[j];
            whole[j] = ends[j] && begun;
            begun |= ends[j];
        }
        Eight<D> in[kBatch][STREAMS ? STREAMS : 1];
        Eight<W> old[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (STREAMS && k[j] != a.rows)
#pragma unroll
                for (int s = 0; s < (STREAMS ? STREAMS : 1); ++s)
                    in[j][s].load(a.dout + ((int64_t)p[j] * streams + s) * a.dim + c);
            if (whole[j] && a.accumulate) old[j].load(a.dtable + (int64_t)k[j] * a.dim + c);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
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
        key = k[kBatch];
    }
    const uint32_t at_end = a.key[start + a.tile - 1];
    if (at_end == a.rows || a.key[start + a.tile] != at_end) return;
    put_part(a.part + ((int64_t)t * 2 + (begun ? 1 : 0)) * a.dim + c, sum);
    if (begun && c == 0) a.owners[1 + atomicAdd(a.owners, 1u)] = t;
}

// the first place in key[lo, hi) whose key is at least k
__device__ __forceinline__ int64_t first_at_least(const uint32_t* key, int64_t lo, int64_t hi,
                                                  uint32_t k) {
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (key[mid] < k)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// The rows that reach over tiles: 16 threads 64 columns, 16 groups of them an
// equal share of the parts each, joined in order.
constexpr int kJoinGroups = 16;
template <class D, class W>
__global__ void __launch_bounds__(256) grad_join_kernel(const SumArgs<D, W> a, int64_t n) {
    __shared__ f32x4 sums[kJoinGroups][17];
    const uint32_t blocks = (uint32_t)(a.dim + 63) / 64;
    const uint32_t total = a.owners[0] * blocks;
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
    for (uint32_t w = blockIdx.x; w < total; w += gridDim.x) {
        const uint32_t at = w / blocks;
        const int64_t t = a.owners[1 + at];
        const int c = (int)(w - at * blocks) * 64 + lane * 4;
        const uint32_t key = a.key[(t + 1) * a.tile - 1];
        const int64_t end = first_at_least(a.key, (t + 1) * a.tile, n, key + 1);
        const int64_t parts = (end - 1) / a.tile - t;  // behind the first one
        f32x4 sum = {0, 0, 0, 0};
        if (c < a.dim) {
            if (group == 0) sum = *reinterpret_cast<const f32x4*>(a.part + (t * 2 + 1) * a.dim + c);
            const int64_t each = (parts + kJoinGroups - 1) / kJoinGroups;
            const int64_t from = 1 + group * each;
            const int64_t to = from + each < parts + 1 ? from + each : parts + 1;
#pragma unroll 8
            for (int64_t q = from; q < to; ++q) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(a.part + (t + q) * 2 * a.dim + c);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += x[e];
            }
        }
        sums[group][lane] = sum;
        __syncthreads();
        if (group == 0 && c < a.dim) {
            for (int g = 1; g < kJoinGroups; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += sums[g][lane][e];
            W* to = a.dtable + (int64_t)key * a.dim + c;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (sizeof(W) == 4)
                    to[e] = a.accumulate ? __builtin_fmaf(a.scale, sum[e], to[e]) : a.scale * sum[e];
                else
                    to[e] = (W)f32_to_bf16(a.accumulate
                                               ? __builtin_fmaf(a.scale, sum[e], bf16_to_f32(to[e]))
                                               : a.scale * sum[e]);
            }
        }
        __syncthreads();
    }
}

// Rows that no position names are set to zero: a workgroup a run of rows, a
// thread of it each row's search among the sorted keys.
constexpr int kFillRows = 256;
__global__ void __launch_bounds__(256) grad_fill_kernel(const uint32_t* __restrict__ key,
                                                        int64_t n, int64_t rows, int each,
                                                        int64_t row0, uint32_t units,
                                                        u32x4* __restrict__ dtable) {
    __shared__ uint8_t named[kFillRows];
    const int64_t r0 = row0 + (int64_t)blockIdx.x * each;
    const int here = (int)(rows - r0 < each ? rows - r0 : each);
    if ((int)threadIdx.x < here) {
        const uint32_t k = (uint32_t)(r0 + threadIdx.x);
        const int64_t at = first_at_least(key, 0, n, k);
        named[threadIdx.x] = at < n && key[at] == k;
    }
    __syncthreads();
    const u32x4 zero = {0, 0, 0, 0};
    u32x4* to = dtable + r0 * units;
    const uint32_t all = (uint32_t)here * units;
    for (uint32_t i = threadIdx.x; i < all; i += 256)
        if (!named[i / units]) __builtin_nontemporal_store(zero, to + i);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Places a tile: enough tiles that the threads fill the machine (256 compute
// units of 1024 threads), few enough that rows of many positions leave few parts.
int tile_of(int64_t n, int dim) {
    int tile = 64;
    while (tile > 8 && n / tile * (dim / 8) < 256 * 1024) tile /= 2;
    return tile;
}

struct GradScratch {
    int64_t padded, tiles, chunks;
    int bits, digit_bits, tile;
    size_t key[2], pos[2], counts, totals, owners, part, bytes;
};

GradScratch grad_layout(int64_t n, int64_t rows, int dim) {
    GradScratch g;
    g.tile = tile_of(n, dim);
    g.tiles = (n + g.tile - 1) / g.tile;
    g.padded = g.tiles * g.tile + kBatch;  // (a tile's last batch looks one key ahead)
    g.chunks = (n + kChunk - 1) / kChunk;
    g.bits = 1;
    while (((int64_t)1 << g.bits) <= rows) ++g.bits;  // the key `rows` as well
    const int passes = (g.bits + kMaxDigit - 1) / kMaxDigit;
    g.digit_bits = (g.bits + passes - 1) / passes;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += up256(bytes);
        return here;
    };
    for (int i = 0; i < 2; ++i) {
        const bool used = i == 0 || g.chunks > 1;
        g.key[i] = take(used ? (size_t)g.padded * 4 : 0);
        g.pos[i] = take(used ? (size_t)g.padded * 4 : 0);
    }
    g.counts = take(g.chunks > 1 ? ((size_t)g.chunks << g.digit_bits) * 4 : 0);
    g.totals = take(g.chunks > kFewChunks ? ((size_t)4 << g.digit_bits) : 0);
    g.owners = take((size_t)(g.tiles + 1) * 4);
    g.part = take((size_t)g.tiles * 2 * dim * sizeof(float));
    g.bytes = at;
    return g;
}

template <class D, class W>
hipError_t run_grad(const void* dout, const int32_t* ids, int64_t n, int streams, int64_t rows,
                    int dim, float scale, int32_t pad_id, bool accumulate, void* dtable,
                    void* scratch, uint32_t* err, hipStream_t s) {
    const GradScratch g = grad_layout(n, rows, dim);
    char* base = (char*)scratch;
    uint32_t* key[2] = {(uint32_t*)(base + g.key[0]), (uint32_t*)(base + g.key[1])};
    uint32_t* pos[2] = {(uint32_t*)(base + g.pos[0]), (uint32_t*)(base + g.pos[1])};
    uint32_t* owners = (uint32_t*)(base + g.owners);
    hipError_t e = hipSuccess;
    int now = 0;
    SortArgs a{ids, n, g.padded, rows, pad_id, key[0], pos[0], owners, err};
    if (n > 0 && g.chunks == 1) {
        sort_few_kernel<<<dim3(1), dim3(kSortThreads), 0, s>>>(a, g.bits, g.digit_bits);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    } else if (n > 0) {
        uint32_t* counts = (uint32_t*)(base + g.counts);
        uint32_t* totals = g.chunks > kFewChunks ? (uint32_t*)(base + g.totals) : nullptr;
        const dim3 grid((uint32_t)g.chunks), threads(kSortThreads);
        for (int shift = 0; shift < g.bits; shift += g.digit_bits) {
            const int d = g.bits - shift < g.digit_bits ? g.bits - shift : g.digit_bits;
            const int last = shift + d >= g.bits;
            if (shift == 0)
                sort_count_kernel<true><<<grid, threads, 0, s>>>(a, nullptr, shift, d, counts);
            else
                sort_count_kernel<false><<<grid, threads, 0, s>>>(a, key[now], shift, d, counts);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            if (totals) {
                sort_scan_kernel<<<dim3(((1u << d) + 255) / 256), dim3(256), 0, s>>>(
                    counts, (int)g.chunks, 1 << d, totals);
                if ((e = hipGetLastError()) != hipSuccess) return e;
            }
            if (shift == 0)
                sort_place_kernel<true><<<grid, threads, 0, s>>>(a, nullptr, nullptr, shift, d,
                                                                 counts, totals, (int)g.chunks,
                                                                 key[0], pos[0], last);
            else
                sort_place_kernel<false><<<grid, threads, 0, s>>>(
                    a, key[now], pos[now], shift, d, counts, totals, (int)g.chunks, key[1 - now],
                    pos[1 - now], last);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            now = shift == 0 ? 0 : 1 - now;
        }
    }
    if (!accumulate) {
        const uint32_t units = (uint32_t)(dim * sizeof(W) / 16);
        const int64_t by_size = 4096 / units;  // 64 KiB a workgroup
        const int each = (int)(by_size < 1 ? 1 : by_size > kFillRows ? kFillRows : by_size);
        const int64_t most = (int64_t)each << 22;  // rows a launch
        for (int64_t r0 = 0; r0 < rows; r0 += most) {
            const int64_t m = rows - r0 < most ? rows - r0 : most;
            grad_fill_kernel<<<dim3((uint32_t)((m + each - 1) / each)), dim3(256), 0, s>>>(
                key[now], n, rows, each, r0, units, (u32x4*)dtable);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    if (n == 0) return hipSuccess;
    SumArgs<D, W> b{key[now], pos[now], (const D*)dout, (W*)dtable, (float*)(base + g.part), owners,
                    (uint32_t)rows, (uint32_t)g.tiles, dim, streams, g.tile, scale,
                    accumulate ? 1 : 0};
    const uint32_t items = (uint32_t)(g.tiles * (dim / 8));
    auto k = streams == 1   ? grad_sum_kernel<D, W, 1>
             : streams == 2 ? grad_sum_kernel<D, W, 2>
             : streams == 4 ? grad_sum_kernel<D, W, 4>
                            : grad_sum_kernel<D, W, 0>;
    k<<<dim3((items + 255) / 256), dim3(256), 0, s>>>(b);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (g.tiles > 1) {
        const int64_t most = (g.tiles - 1) * ((dim + 63) / 64);
        grad_join_kernel<D, W><<<dim3((uint32_t)(most < 2048 ? most : 2048)), dim3(256), 0, s>>>(b, n);
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
