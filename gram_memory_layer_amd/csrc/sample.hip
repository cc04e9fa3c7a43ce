// The next token of a row of logits from a given random number, under
// temperature, top-k, top-p and min-p:
//
//   w(v) = exp((x(v) - max x) / T)         (T = 0: the first largest x alone)
//   in the order of falling x, equal ones by rising v:
//     top-k: the first k stay;  top-p: of these, one stays whose predecessors' w sum
//     to less than p times the sum of them all;  min-p: of these, one stays with w >= m
//   token = the first v of those that stay, v rising, whose sum of w up to it
//   exceeds u times the sum of all that stay.
//
// The sums of weights decide which tokens come out, so weights and sums are held
// in 64 bits, or in whole numbers where additions come in any order.
//
// Two kernels, none of which sorts.  The first reads the logits once, many
// workgroups a row, and leaves per part of 2048 its largest logit and sum of
// weights, and, for rows with a filter, per block of 8192 a histogram of its
// weights (top-k: numbers) over buckets of the logits.  The second, a workgroup
// a row, joins these: the cut of top-k or top-p lies in one bucket, and only what
// may stay before it, or where that is much the bucket and the block that holds
// the random number, is read again.
//
// Measured (129,280 logits a row): one row with top-k 50 and top-p 0.95 6.1 + 11.7
// us, a chain of latencies; 64 fp32 rows with top-p 0.9 17.8 + 35 us, the first one bound
// by the 64-bit exponentials and the histogram (its bytes take 7), the second one by
// the flat rows, whose 517 KB one compute unit reads; 512 bf16
// rows without a filter 55 + 9 us, bound by the exponentials (21 instructions a logit, the
// vector units busy 80% of the time; their bytes take 28).  Elementary torch
// operations, with a sort in 64 bits: 350, 2100 and 3050 us.
#include <type_traits>

#include "lanes.h"
#include "logits.h"

namespace engram {
namespace {

constexpr int kEach = 32;                     // logits a thread of a part
constexpr int kPart = 64 * kEach;             // logits a wave: a part
constexpr int kBlockWaves = 4;
constexpr int kBlock = kBlockWaves * kPart;   // logits a workgroup
constexpr int kBuckets = 512;                 // of 1/24 of exp's argument (of 1/8 where logits are only
                                              // counted), from a block's largest logit down;
constexpr int kRest = kBuckets - 1;           // the last one takes all below, too
constexpr int kXcds = 8;                      // workgroups go to these in turn: a row's all to one, where
                                              // its second kernel's workgroup finds them in the cache
constexpr int kCopies = 4;                    // of the buckets in LDS: lanes that meet in one wait for each other
                                              // (64 rows with top-p 0.5, and equal ones with min-p: 29 and 45
                                              // us; one copy: 34 and 62)
constexpr int kGroup = 4;                     // lanes whose largest logit is kept
constexpr int kRowThreads = 512;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kBinBits = 9, kBins = 1 << kBinBits;  // a thread each
constexpr int kList = 8192;                   // candidates in LDS,
constexpr int kManyBefore = 1024;             // logits before the cut's bucket that are listed with it (64
                                              // fp32 rows with top-p 0.5 and 0.9: 29 and 48 us; 64 of them:
                                              // 41 and 48; as many as the list holds: 29 and 59)
constexpr int kSome = 64, kRanked = 256;      // that are ranked by counting, by a wave or all (top-k 150:
                                              // 27 us, found by narrowing down 36; one row with top-p
                                              // 0.9: 18.7, ranked by all 20.2)
constexpr int kHits = 16 * kRowThreads;       // groups of a row looked at together
constexpr int kMostBlocks = 256;              // of a row whose buckets are joined: longer ones' filters go by passes
                                              // (2 fp32 rows with top-k 50: of 2^21 - 8 logits 99 us, of 2^22
                                              // 6.2 ms)

// exp(d / T) for d <= 0, by c = log2(e) / T: 2^n * 2^f, f in [-1/2, 1/2], 2^f by a
// polynomial of degree eight with the least relative error (1.1e-12, by Remez'
// exchange); 0 gives exactly 1.  Below 2^-999 it is 2^-1000: no weight.
constexpr double kLog2e = 1.4426950408889634074;
constexpr double kRound = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to a whole number
constexpr double kNoWeight = 0x1p-999;
// (for d * c >= -1000)
__device__ __forceinline__ double weight(double d, double c) {
    const double r = __builtin_fma(d, c, kRound);
    const double f = __builtin_fma(d, c, -(r - kRound));
    double p = 1.3344183691340562e-06;
    asm("" : "+v"(p));  // (in registers: an instruction takes one constant)
    p = __builtin_fma(p, f, 1.531420923292218e-05);
    p = __builtin_fma(p, f, 0.00015403098285512635);
    p = __builtin_fma(p, f, 0.0013333434157515403);
    p = __builtin_fma(p, f, 0.009618129558840595);
    p = __builtin_fma(p, f, 0.055504109592288714);
    p = __builtin_fma(p, f, 0.24022650694742584);
    p = __builtin_fma(p, f, 0.6931471805412327);
    p = __builtin_fma(p, f, 1.0);
    return __hiloint2double(__double2hiint(p) + (__double2loint(r) << 20), __double2loint(p));
}

// whole numbers in the order of the logits; both zeros are one
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
constexpr uint32_t kLeastKey = 0x00800000u;  // of the lowest finite logit

struct Request {
    const float* u;
    const float* temperature;  // null: 1
    const int32_t* top_k;      // null: none
    const float* top_p;
    const float* min_p;
};

// A row's own values, checked
struct Want {
    double c;      // log2(e) / temperature; 0: greedy
    double least;  // the difference of logits that weighs 2^-1000
    float s;       // buckets a unit of the logits
    double p, m, u;
    int k;         // 0: no top-k
    bool bad;
    __device__ __forceinline__ Want(const Request& q, int64_t row, int V) {
        const float t = q.temperature ? q.temperature[row] : 1.0f;
        const float pp = q.top_p ? q.top_p[row] : 1.0f;
        const float mm = q.min_p ? q.min_p[row] : 0.0f;
        const float uu = q.u[row];
        const int kk = q.top_k ? q.top_k[row] : 0;
        bad = !(t >= 0.0f && t < INFINITY) || !(pp >= 0.0f && pp <= 1.0f) ||
              !(mm >= 0.0f && mm <= 1.0f) || !(uu >= 0.0f && uu < 1.0f);
        c = t > 0.0f ? kLog2e / (double)t : 0.0;
        least = -1000.0 / c;
        p = pp;
        m = mm;
        u = uu;
        k = kk > 0 && kk < V ? kk : 0;
        s = (k ? 8.0f : 24.0f) / t;
    }
    __device__ __forceinline__ bool greedy() const { return c == 0.0; }
    __device__ __forceinline__ bool filtered() const { return !greedy() && (k > 0 || p < 1.0 || m > 0.0); }
    // whether the weights of the whole row are summed, or only logits counted
    __device__ __forceinline__ bool whole_sum() const { return !greedy() && k == 0; }
    __device__ __forceinline__ double weigh(float x, float top) const {
        return weight(fmax((double)x - (double)top, least), c);
    }
    // A whole number that does not fall as x rises.  (s may be infinite: then
    // zero goes with the negative ones.)
    __device__ __forceinline__ int bucket(float x) const {
        return (int)floorf(fminf(fmaxf(x * s, -0x1p29f), 0x1p29f));
    }
};

// What the blocks leave for the row
struct Found {
    float* tops;       // [parts] a part's largest logit; NaN: a NaN or +infinity is in it
    double* sums;      // [parts] its weights' sum, relative to its largest logit (rows with a
                       // filter: to the block's; where no sum is needed, the number of
                       // logits above -infinity)
    float* groups;     // [blocks * kBlock / (kGroup * VEC)] the largest of a group
    double* buckets;   // [blocks][kBuckets] the sum of weights in the bucket, relative to the block's
                       // largest logit, where the row's sum is needed, otherwise the number of logits
    int blocks;
};

__device__ __forceinline__ double last_lane(double x) {
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(x), 63),
                            __builtin_amdgcn_readlane(__double2loint(x), 63));
}
__device__ __forceinline__ uint64_t last_lane(uint64_t x) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), 63) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
// the largest of four lanes, and of 16, in all of them
__device__ __forceinline__ float largest_of_4(float x) {
    x = fmaxf(x, __uint_as_float(moved<0xB1>(__float_as_uint(x))));
    return fmaxf(x, __uint_as_float(moved<0x4E>(__float_as_uint(x))));
}
__device__ __forceinline__ float largest_of_16(float x) {
    x = fmaxf(x, __uint_as_float(moved<0x128>(__float_as_uint(x))));  // (rotations: no lane goes without)
    x = fmaxf(x, __uint_as_float(moved<0x124>(__float_as_uint(x))));
    x = fmaxf(x, __uint_as_float(moved<0x122>(__float_as_uint(x))));
    return fmaxf(x, __uint_as_float(moved<0x121>(__float_as_uint(x))));
}
// of the wave, in all lanes
__device__ __forceinline__ float largest(float x) {
    x = largest_of_16(x);
    const int u = __float_as_int(x);
    return fmaxf(fmaxf(__int_as_float(__builtin_amdgcn_readlane(u, 0)), __int_as_float(__builtin_amdgcn_readlane(u, 16))),
                 fmaxf(__int_as_float(__builtin_amdgcn_readlane(u, 32)), __int_as_float(__builtin_amdgcn_readlane(u, 48))));
}

// One wave a part, four of them a block.  Rows without a filter need a part's largest
// logit and its sum of weights; rows with one also how much weight, or where that is
// not asked for how many logits, lie in each bucket.  A wave's 2048 logits are all on
// their way at once and stay in registers, as the weights need the block's largest first;
// a block's histogram (fixed point, so that the order of the additions does not
// matter) is small against its logits (4 KB a block of 16 or 32).
template <class T, bool FILTERS>
__global__ void __launch_bounds__(64 * kBlockWaves) sample_part_kernel(
    const T* __restrict__ logits, int64_t ld, const Request q, int64_t rows, int V, const Found out) {
    constexpr int VEC = Row<T>::VEC, NL = kEach / VEC, NT = 64 * kBlockWaves;
    __shared__ unsigned long long bucket[FILTERS ? kBuckets * kCopies : 1];
    uint32_t* const number = reinterpret_cast<uint32_t*>(bucket);
    __shared__ float wave_top[kBlockWaves];
    const uint32_t along = blockIdx.x / kXcds, at = along % out.blocks;
    const int64_t row = (int64_t)(along / out.blocks) * kXcds + blockIdx.x % kXcds;
    if (row >= rows) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t block = row * out.blocks + at;
    const int part = at * kBlockWaves + wave;
    const Row<T> r(logits + row * ld);
    const int64_t from = (int64_t)part * NL * 64;
    const bool inside = r.column(from) >= 0 && r.column(from + NL * 64) <= V;
    float v[NL][VEC];
    {
        uint4 raw[NL];
        if (inside) {
            const uint4* p = reinterpret_cast<const uint4*>(r.src + r.column(from + lane));
#pragma unroll
            for (int i = 0; i < NL; ++i) raw[i] = p[64 * i];
#pragma unroll
            for (int i = 0; i < NL; ++i) r.values(raw[i], v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NL; ++i) raw[i] = r.fetch(from + lane + 64 * i, V);
#pragma unroll
            for (int i = 0; i < NL; ++i) r.unpack(raw[i], from + lane + 64 * i, V, v[i]);
        }
    }
    const Want want(q, row, V);
    float own[NL], top = -INFINITY, low = INFINITY;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        own[i] = v[i][0];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            own[i] = fmaxf(own[i], v[i][e]);
            low = fminf(low, v[i][e]);
        }
        top = fmaxf(top, own[i]);
    }
    top = largest(top);
    const bool filtered = FILTERS && want.filtered();
    auto sum_all = [&] {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < NL; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += weight((double)v[i][e] - (double)top, want.c);
        return s;
    };
    if constexpr (!FILTERS) {
        // (no logit weighs nothing; a NaN, which neither bound shows, makes the sum one)
        if (want.whole_sum() && fabsf(top) < INFINITY && __all((double)low - (double)top >= want.least)) {
            const double s = last_lane(sum_upto(sum_all()));
            if (lane == 0) {
                out.tops[row * out.blocks * kBlockWaves + part] = s == s ? top : (float)s;
                out.sums[row * out.blocks * kBlockWaves + part] = s;
            }
            return;
        }
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NL; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) bad |= !(v[i][e] < INFINITY);
    bad = __any(bad);
    if (lane == 0)
        out.tops[row * out.blocks * kBlockWaves + part] = bad ? __uint_as_float(0x7FC00000u) : top;
    if (filtered) {
        for (int b = tid; b < kBuckets * kCopies; b += NT) bucket[b] = 0;
        if (lane == 0) wave_top[wave] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kBlockWaves; ++w) top = fmaxf(top, wave_top[w]);
        // (the one thing that is read of blocks without a logit above -infinity, too)
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const float g = largest_of_4(own[i]);
            if ((lane & (kGroup - 1)) == 0)
                out.groups[row * out.blocks * (NT * NL / kGroup) + (from + lane + 64 * i) / kGroup] = g;
        }
    }
    if (top == -INFINITY) return;  // (the whole block, where it has a barrier ahead)
    double s = 0.0;
    if (!filtered) {
        if (!want.whole_sum() || bad) return;
        if (FILTERS && __all((double)low - (double)top >= want.least)) {
            s = sum_all();
        } else {
#pragma unroll
            for (int i = 0; i < NL; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s += want.weigh(v[i][e], top);
        }
    } else {
        const int most = want.bucket(top), copy = lane & (kCopies - 1);
        const bool weights = want.whole_sum();
        if (weights) {
#pragma unroll
            for (int i = 0; i < NL; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float x = v[i][e];
                    const double w = want.weigh(x, top);
                    s += w;
                    // whole numbers of 2^-50, in any order: 2^13 of them at most, and off by 2^-38 of
                    // the block's largest together
                    if (x > -INFINITY)
                        atomicAdd(&bucket[min(most - want.bucket(x), kRest) * kCopies + copy],
                                  (unsigned long long)(__double_as_longlong(w + 4.0) -
                                                       __double_as_longlong(4.0)));
                }
        } else {
#pragma unroll
            for (int i = 0; i < NL; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float x = v[i][e];
                    if (x > -INFINITY) {
                        s += 1.0;
                        atomicAdd(&number[min(most - want.bucket(x), kRest) * kCopies + copy], 1u);
                    }
                }
        }
        __syncthreads();
        for (int b = tid; b < kBuckets; b += NT) {
            uint64_t all = 0;
#pragma unroll
            for (int j = 0; j < kCopies; ++j)
                all += weights ? bucket[b * kCopies + j] : number[b * kCopies + j];
            out.buckets[block * kBuckets + b] = (double)all * (weights ? 0x1p-50 : 1.0);
        }
    }
    s = last_lane(sum_upto(s));
    if (lane == 0) out.sums[row * out.blocks * kBlockWaves + part] = s;
}

// Sums of weights, of 1 at most each, in whole numbers, the same in any order, and how many
// there are.  Of up to 2^13 of them (WIDE = false) in one word, units 2^-50: off by 2^-38 at most
// together, where the row's largest weighs 1.
template <bool WIDE>
struct Sum {
    uint64_t upper = 0, lower = 0;
    static __device__ __forceinline__ uint64_t units_of(double w) {
        return (uint64_t)(__double_as_longlong(w + 4.0) - __double_as_longlong(4.0));
    }
    static __device__ __forceinline__ uint64_t upper_of(uint64_t units) { return units; }
    static __device__ __forceinline__ uint64_t lower_of(uint64_t) { return 1; }
    __device__ __forceinline__ uint64_t number() const { return lower; }
    __device__ __forceinline__ double value() const { return (double)upper * 0x1p-50; }
    __device__ __forceinline__ bool reaches(double target) const { return (double)upper >= target * 0x1p50; }
};
// Of up to 2^22 in two words, units 2^-60, what is below cut off (2^-38 together, too): upper
// parts of 2^-41, and lower ones of 19 bits, whose sums take 41 below the number.  (In one word
// the unit would be 2^-41, and a row's weights below it, which count as nothing then, can be
// 2^-19 together.)
template <>
struct Sum<true> {
    static constexpr int kLow = 19, kNumber = 41;
    static constexpr uint64_t kLowMask = (1ull << kLow) - 1, kSumMask = (1ull << kNumber) - 1;
    uint64_t upper = 0, lower = 0;
    static __device__ __forceinline__ uint64_t units_of(double w) {
        const uint64_t b = (uint64_t)__double_as_longlong(w);
        const uint32_t e = 1023u - (uint32_t)(b >> 52);
        return e < 64 ? ((b & 0xFFFFFFFFFFFFFull) | 1ull << 52) << 8 >> e : 0;
    }
    static __device__ __forceinline__ uint64_t upper_of(uint64_t units) { return units >> kLow; }
    static __device__ __forceinline__ uint64_t lower_of(uint64_t units) {
        return (units & kLowMask) | 1ull << kNumber;
    }
    __device__ __forceinline__ uint64_t number() const { return lower >> kNumber; }
    // the lower parts' carry on to the upper ones
    __device__ __forceinline__ uint64_t high() const { return upper + ((lower & kSumMask) >> kLow); }
    __device__ __forceinline__ double low() const { return (double)(uint32_t)(lower & kLowMask); }
    __device__ __forceinline__ double value() const { return (double)high() * 0x1p-41 + low() * 0x1p-60; }
    // compared exactly, so that what holds of a sum holds of larger ones
    __device__ __forceinline__ bool reaches(double target) const {
        if (!(target > 0.0)) return true;
        const double t = target * 0x1p41, whole = floor(t);
        const uint64_t h = high(), w = (uint64_t)whole;
        return h > w || (h == w && low() >= (t - whole) * 0x1p19);
    }
};

// What the threads of a row's workgroup exchange
struct Shared {
    double sum[kRowWaves];
    uint64_t whole[2][kRowWaves];
    uint64_t count[kBins];     // Sums' lower words,
    uint64_t mass[kBins + 1];  // and upper ones (a row's blocks are at most that many)
    int first, last, hits, listed, at[kRowWaves];
    uint32_t range[2];
    bool none;
    uint64_t above[3];
    double found[3];
    double factor[kMostBlocks], blocks[kMostBlocks];
    int offset[kMostBlocks];
    int list[kList];
    __align__(8) uint16_t hit[kHits];
};

// sum over the workgroup, and this thread's share of it: what lies before it
__device__ __forceinline__ double scan(double own, Shared& sh, double* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const double upto = sum_upto(own);
    __syncthreads();
    if (lane == 63) sh.sum[wave] = upto;
    __syncthreads();
    double before = 0.0, all = 0.0;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) {
        const double x = sh.sum[w];
        if (w < wave) before += x;
        all += x;
    }
    *total = all;
    return before + moved<0x138>(upto);  // (the lane before; 0 for the first)
}
// two at once: what lies before this thread's n and m
__device__ __forceinline__ void scan(uint64_t& n, uint64_t& m, Shared& sh) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t upto_n = sum_upto(n), upto_m = sum_upto(m);
    if (lane == 63) {
        sh.whole[0][wave] = upto_n;
        sh.whole[1][wave] = upto_m;
    }
    __syncthreads();
    n = upto_n - n;
    m = upto_m - m;
#pragma unroll
    for (int w = 0; w < kRowWaves - 1; ++w) {
        const uint64_t a = sh.whole[0][w], b = sh.whole[1][w];
        n += w < wave ? a : 0;
        m += w < wave ? b : 0;
    }
}
__device__ __forceinline__ uint64_t total_of(uint64_t own, Shared& sh) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    own = sum_upto(own);
    __syncthreads();
    if (lane == 63) sh.whole[0][wave] = own;
    __syncthreads();
    uint64_t all = 0;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) all += sh.whole[0][w];
    return all;
}

// the lowest thread for which `is` holds, kRowThreads if none; all threads call
__device__ __forceinline__ int lowest(bool is, Shared& sh) {
    const uint64_t set = __ballot(is);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh.at[threadIdx.x >> 6] = set ? (int)threadIdx.x + __builtin_ctzll(set) : kRowThreads;
    __syncthreads();
    int first = kRowThreads;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) first = min(first, sh.at[w]);
    return first;
}
// the highest one, -1 if none
__device__ __forceinline__ int highest(bool is, Shared& sh) {
    const uint64_t set = __ballot(is);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh.at[threadIdx.x >> 6] = set ? (int)threadIdx.x + 63 - __builtin_clzll(set) : -1;
    __syncthreads();
    int last = -1;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) last = max(last, sh.at[w]);
    return last;
}

// The thread whose share of the sums holds `target`: the first whose end lies behind
// it (by roundings there may be none: then the last that holds anything).
__device__ __forceinline__ int holder(double before, double own, double target, Shared& sh) {
    const int t = lowest(own > 0.0 && before + own > target, sh);
    return t < kRowThreads ? t : highest(own > 0.0, sh);
}

// Where the order is cut: an element stays if its key is larger, or the same and
// its index at most idx.
struct Cut {
    uint32_t key = 0;
    uint32_t idx = 0xFFFFFFFFu;
    __device__ bool keeps(float x, int i) const {
        const uint32_t k = key_of(x);
        return k > key || (k == key && (uint32_t)i <= idx);
    }
};

// Logits and their weights in whole numbers, so that they add up to the same
// in any order.  Each: each(f) calls f(logit, index, units) for its logits above -infinity,
// spread over the workgroup's threads; units() are the weight.
// RUNS: neighbours are often equal, and there may be a whole row of them.  T: what the
// logits were (bf16: half of a key says which).
template <class T, bool RUNS, class Each>
struct Narrow {
    using Sums = Sum<RUNS>;
    using Lower = std::conditional_t<RUNS, uint64_t, uint32_t>;  // a lower word in LDS
    static constexpr int DROP = sizeof(T) == 2 ? 16 : 0;
    const Each& each;
    const Want& want;
    const float top;
    Shared& sh;

    // The first place (of those in [lo, hi], what place(logit, index) is; ~0: no candidate) up
    // to which reached(sum) holds of the candidates; passes over them narrow it
    // down by a factor of kBins each.  False where it is never reached.  before: what
    // lies before the place, ties: the candidates at it.
    // WEIGHTS: they are summed, otherwise candidates are only counted (known when run, both
    // take longer: equal fp32 logits with top-p 231 us for 211, with top-k 178 for 141).
    template <bool WEIGHTS, class Place, class Reached>
    __device__ __forceinline__ bool find(uint32_t& lo, uint32_t hi, Place place, Reached reached,
                         Sums& before, uint64_t& ties) const {
        const int tid = threadIdx.x;
        Lower* const count = reinterpret_cast<Lower*>(sh.count);
        before = Sums();
        while (true) {
            const int shift = lo < hi ? max(0, 32 - kBinBits - __builtin_clz(hi - lo)) : 0;
            __syncthreads();
            count[tid] = 0;
            sh.mass[tid] = 0;
            if (tid == 0) sh.none = true;
            __syncthreads();
            each([&](float x, int i, auto units) {
                const uint32_t at = place(x, i);
                if (at < lo || at > hi) return;
                const uint32_t bin = (at - lo) >> shift;
                const uint64_t w = WEIGHTS ? units() : 0;
                if constexpr (RUNS) {  // equal logits, or near indices: the wave's together
                    const uint64_t here = __ballot(1);
                    const uint32_t one = __builtin_amdgcn_readfirstlane(bin);
                    const uint64_t w_one = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(w >> 32)) << 32 |
                                           (uint32_t)__builtin_amdgcn_readfirstlane((int)w);
                    if (__ballot(bin == one && w == w_one) == here) {
                        if ((uint32_t)__builtin_ctzll(here) == (tid & 63))
                            add<WEIGHTS>(one, w_one, __builtin_popcountll(here));
                        return;
                    }
                }
                add<WEIGHTS>(bin, w, 1);
            });
            __syncthreads();
            const uint64_t own_u = sh.mass[tid], own_l = count[tid];
            uint64_t u = own_u, l = own_l;
            scan(u, l, sh);
            const Sums from{before.upper + u, before.lower + l}, to{from.upper + own_u, from.lower + own_l};
            // (one thread's share is the first that reaches)
            if (own_l > 0 && reached(to) && !(l > 0 && reached(from))) {
                sh.above[0] = from.upper;
                sh.above[1] = from.lower;
                sh.above[2] = own_l;
                sh.first = tid;
                sh.none = false;
            }
            __syncthreads();
            if (sh.none) return false;
            const int at = sh.first;
            before = Sums{sh.above[0], sh.above[1]};
            ties = Sums{0, sh.above[2]}.number();
            lo += (uint32_t)at << shift;
            if (shift == 0) return true;
            hi = min(hi, lo + ((1u << shift) - 1));
        }
    }
    // a weight, so many times
    template <bool WEIGHTS>
    __device__ __forceinline__ void add(uint32_t bin, uint64_t units, uint32_t number) const {
        uint32_t* const numbers = reinterpret_cast<uint32_t*>(sh.count);
        if constexpr (!WEIGHTS) {  // (a number alone lies in the word's upper half)
            atomicAdd(numbers + (RUNS ? 2 * bin + 1 : bin), number << (RUNS ? 9 : 0));
            return;
        }
        const uint64_t u = Sums::upper_of(units) * number, l = Sums::lower_of(units) * number;
        if constexpr (RUNS)
            atomicAdd((unsigned long long*)&sh.count[bin], (unsigned long long)l);
        else
            atomicAdd(numbers + bin, (uint32_t)l);
        atomicAdd((unsigned long long*)&sh.mass[bin], (unsigned long long)u);
    }
    // the index of the r-th of the logits with this key that `in` keeps
    __device__ __forceinline__ uint32_t index_of(uint32_t key, const Cut in, uint64_t r, int V) const {
        uint32_t idx = 0;
        Sums before;
        uint64_t ties;
        return find<false>(idx, (uint32_t)V - 1,
                    [&](float x, int i) { return key_of(x) == key && in.keeps(x, i) ? (uint32_t)i : ~0u; },
                    [&](const Sums& upto) { return upto.number() >= r; }, before, ties)
                   ? idx
                   : ~0u;
    }
    // The cut that keeps the first k of those that `in` keeps (k > 0), or those before
    // which less than target lies; all of them lie in [least, most].  index: as index_of.
    template <class Index>
    __device__ __forceinline__ Cut cut(const Cut in, int k, double target, float most, float least, int V,
                                       Index index) const {
        uint32_t at = ~key_of(most) >> DROP;
        Sums before;
        uint64_t ties;
        const uint32_t last = ~max(in.key, key_of(least)) >> DROP;
        auto place = [&](float x, int i) { return in.keeps(x, i) ? ~key_of(x) >> DROP : ~0u; };
        if (!(k ? find<false>(at, last, place, [&](const Sums& upto) { return upto.number() >= (uint64_t)k; },
                              before, ties)
                : find<true>(at, last, place, [&](const Sums& upto) { return upto.reaches(target); }, before,
                             ties))) {
            // all of them do not reach it (by a rounding, or there are fewer)
            Cut all = in;
            if (key_of(least) > in.key) all.key = key_of(least), all.idx = ~0u;
            return all;
        }
        Cut out;
        out.key = ~(at << DROP);
        if (DROP && (out.key & 0x80000000u)) out.key &= ~0xFFFFu;  // (the lower half is clear from zero on)
        out.idx = in.key == out.key ? in.idx : ~0u;
        // how many of the equal ones at the cut stay, and the last of these
        double stay = (double)k - (double)before.number();
        if (k == 0) stay = ceil((target - before.value()) / want.weigh(value_of(out.key), top));
        const uint64_t r = stay < 1.0 ? 1 : stay > 0x1p31 ? (uint64_t)1 << 31 : (uint64_t)stay;
        if (r < ties) out.idx = index(out.key, in, r);
        return out;
    }
};
template <class T, bool RUNS, class Each>
__device__ __forceinline__ Narrow<T, RUNS, Each> narrow(const Each& each, const Want& want, float top, Shared& sh) {
    return Narrow<T, RUNS, Each>{each, want, top, sh};
}

// One workgroup a row.
template <class T>
struct Sampler {
    static constexpr int VEC = Row<T>::VEC, NL = kEach / VEC, kPieces = kBlock / VEC;
    const Row<T> r;
    const int V, pieces;
    const Want& want;
    const float top;
    Shared& sh;
    int32_t* token;
    float* logprob;  // or null
    float floor;     // the least logit that min-p lets stay

    __device__ __forceinline__ void emit(int i, double lp) const {
        *token = i;
        if (logprob) *logprob = (float)lp;
    }
    template <class F>
    __device__ __forceinline__ void some(int i, F f) const {
        float x[VEC];
        r.unpack(r.fetch(i, V), i, V, x);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (x[e] > -INFINITY) f(x[e], (int)r.column(i) + e);
    }
    // f for the row's logits but those at -infinity, pieces in turn
    template <class F>
    __device__ __forceinline__ void every(F f) const {
        constexpr int AT = 4;
        for (int i0 = threadIdx.x; i0 < pieces; i0 += AT * kRowThreads) {
            uint4 raw[AT];
#pragma unroll
            for (int j = 0; j < AT; ++j) raw[j] = r.fetch(i0 + j * kRowThreads, V);
#pragma unroll
            for (int j = 0; j < AT; ++j) {
                float x[VEC];
                r.unpack(raw[j], i0 + j * kRowThreads, V, x);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (x[e] > -INFINITY) f(x[e], (int)r.column(i0 + j * kRowThreads) + e);
            }
        }
    }
    // The token among logits whose weights w (0: does not stay) the threads hold, those of
    // pieces from begin on: the first whose sum exceeds target.
    template <int E>
    __device__ __forceinline__ void choose(const double (&w)[E][VEC], int begin, double target, double total) const {
        double own = 0.0, here;
#pragma unroll
        for (int j = 0; j < E; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) own += w[j][e];
        double sum = scan(own, sh, &here), w_token = 0.0;
        if ((int)threadIdx.x != holder(sum, own, target, sh)) return;
        int at = -1;
        bool done = false;
#pragma unroll
        for (int j = 0; j < E; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if (done || !(w[j][e] > 0.0)) continue;
                sum += w[j][e];
                at = (int)r.column(begin + j) + e;
                w_token = w[j][e];
                done = sum > target;
            }
        emit(at, log(w_token / total));
    }

    // The token among the logits of a part, all of which stay.
    __device__ __forceinline__ void pick_near(int part, double target, double total) const {
        constexpr int PER = NL * 64, E = (PER + kRowThreads - 1) / kRowThreads;
        const int begin = part * PER + threadIdx.x * E;
        double w[E][VEC];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int i = threadIdx.x * E + j < PER ? begin + j : pieces;
            float x[VEC];
            r.unpack(r.fetch(i, V), i, V, x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                w[j][e] = want.weigh(x[e], top);
                if (!(w[j][e] > kNoWeight && x[e] > -INFINITY)) w[j][e] = 0.0;
            }
        }
        choose(w, begin, target, total);
    }

    // A block's logits that stay: 16 neighbours x a thread, a bit each; their places in
    // order into the list, where they are at most `most`; how many there are.
    static constexpr int NEAR = kPieces / kRowThreads;
    template <class Stays>
    __device__ __forceinline__ int list_block(int block, int most, float (&x)[NEAR][VEC], uint32_t& stay,
                                              Stays stays) const {
        const int tid = threadIdx.x, begin = block * kPieces + tid * NEAR;
        uint4 raw[NEAR];
#pragma unroll
        for (int j = 0; j < NEAR; ++j) raw[j] = r.fetch(begin + j, V);
        stay = 0;
#pragma unroll
        for (int j = 0; j < NEAR; ++j) {
            r.unpack(raw[j], begin + j, V, x[j]);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (x[j][e] > -INFINITY && stays(x[j][e], (int)r.column(begin + j) + e)) stay |= 1u << (j * VEC + e);
        }
        const int own = __builtin_popcount(stay), upto = (int)sum_upto((uint32_t)own);
        if ((tid & 63) == 63) sh.at[tid >> 6] = upto;
        __syncthreads();
        int at = upto - own, n = 0;
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w) {
            at += w < (tid >> 6) ? sh.at[w] : 0;
            n += sh.at[w];
        }
        if (n > most) return n;
        for (uint32_t left = stay; left; left &= left - 1, ++at)
            sh.list[at] = (int)r.column(begin) + __builtin_ctz(left);
        __syncthreads();
        return n;
    }

    // The same among a block's that stay.  Where these are few, their places in order
    // first, so that few weights are taken (one row, normal, top-p 0.5: 34.2 us, all
    // weighed 35.4).
    template <class Stays>
    __device__ __forceinline__ void pick_listed(int block, double target, double total, Stays stays) const {
        constexpr int FEW = 4;  // a thread
        const int tid = threadIdx.x;
        float x[NEAR][VEC];
        uint32_t stay;
        const int n = list_block(block, FEW * kRowThreads, x, stay, stays);
        if (n > FEW * kRowThreads) {
            double w[NEAR][VEC];
#pragma unroll
            for (int j = 0; j < NEAR; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    w[j][e] = want.weigh(x[j][e], top);
                    if (!(stay >> (j * VEC + e) & 1) || !(w[j][e] > kNoWeight)) w[j][e] = 0.0;
                }
            return choose(w, block * kPieces + tid * NEAR, target, total);
        }
        const int each = (n + kRowThreads - 1) / kRowThreads, from = tid * each, to = min(from + each, n);
        int places[FEW];
        double w[FEW], own_sum = 0.0, here;
#pragma unroll
        for (int j = 0; j < FEW; ++j) places[j] = from + j < to ? sh.list[from + j] : 0;
        float y[FEW];
#pragma unroll
        for (int j = 0; j < FEW; ++j) y[j] = value(places[j]);
#pragma unroll
        for (int j = 0; j < FEW; ++j) {
            w[j] = 0.0;
            if (j >= each) break;
            w[j] = want.weigh(y[j], top);
            if (!(from + j < to && w[j] > kNoWeight)) w[j] = 0.0;
            own_sum += w[j];
        }
        double sum = scan(own_sum, sh, &here), w_token = 0.0;
        if (tid != holder(sum, own_sum, target, sh)) return;
        int token_at = -1;
        bool done = false;
#pragma unroll
        for (int j = 0; j < FEW; ++j) {
            if (done || !(w[j] > 0.0)) continue;
            sum += w[j];
            token_at = places[j];
            w_token = w[j];
            done = sum > target;
        }
        emit(token_at, log(w_token / total));
    }

    // Numbers of the row's logits summed by block, a wave each in turn; total: all of them.
    // The block that holds the share-th part of it (at >= 0: that holds `at`), and what lies before.
    template <class Of>
    __device__ __forceinline__ int sum_blocks(Of of, double share, double at, double& before, double& total) const {
        constexpr int AT = 4;
        const int tid = threadIdx.x, lane = tid & 63, blocks = (pieces + kPieces - 1) / kPieces;
        double* by = reinterpret_cast<double*>(sh.mass);
        __syncthreads();
        for (int g = tid >> 6; g < blocks; g += kRowWaves) {
            double s = 0.0;
            for (int i0 = g * kPieces + lane; i0 < (g + 1) * kPieces; i0 += AT * 64) {
                uint4 raw[AT];
#pragma unroll
                for (int j = 0; j < AT; ++j) raw[j] = r.fetch(i0 + 64 * j, V);
#pragma unroll
                for (int j = 0; j < AT; ++j) {
                    float x[VEC];
                    r.unpack(raw[j], i0 + 64 * j, V, x);
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (x[e] > -INFINITY) s += of(x[e], (int)r.column(i0 + 64 * j) + e);
                }
            }
            s = last_lane(sum_upto(s));
            if (lane == 0) by[g] = s;
        }
        __syncthreads();
        const int each = (blocks + kRowThreads - 1) / kRowThreads, from = tid * each, to = min(from + each, blocks);
        double own = 0.0;
        for (int g = from; g < to; ++g) own += by[g];
        double sum = scan(own, sh, &total);
        const double target = at >= 0.0 ? at : share * total;
        if (tid == holder(sum, own, target, sh)) {
            for (int g = from; g < to; ++g) {
                if (!(by[g] > 0.0)) continue;
                sh.found[0] = sum;
                sh.hits = g;
                sum += by[g];
                if (sum > target) break;
            }
        }
        __syncthreads();
        before = sh.found[0];
        return sh.hits;
    }
    // (for it: the weight of a logit that stays)
    template <class Stays>
    __device__ __forceinline__ auto weight_of(Stays stays) const {
        return [=, this](float x, int i) {
            if (!stays(x, i)) return 0.0;
            const double w = want.weigh(x, top);
            return w > kNoWeight ? w : 0.0;
        };
    }

    // The token among the row's logits that stay: the first whose sum exceeds u times the
    // sum of all.
    template <class Stays>
    __device__ __forceinline__ void pick(Stays stays) const {
        double before, total;
        const int block = sum_blocks(weight_of(stays), want.u, -1.0, before, total);
        pick_listed(block, want.u * total - before, total, stays);
    }

    // the first of the largest: its part, then its place
    __device__ __forceinline__ void greedy(const float* tops, int parts) const {
        __syncthreads();
        if (threadIdx.x == 0) {
            sh.first = parts;
            sh.last = V;
        }
        __syncthreads();
        for (int p = threadIdx.x; p < parts; p += kRowThreads)
            if (tops[p] == top) atomicMin(&sh.first, p);
        __syncthreads();
        const int from = sh.first * (NL * 64);
        for (int i = from + threadIdx.x; i < min(from + NL * 64, pieces); i += kRowThreads)
            some(i, [&](float x, int at) {
                if (x == top) atomicMin(&sh.last, at);
            });
        __syncthreads();
        if (threadIdx.x == 0) emit(sh.last, 0.0);
    }

    // No filter: the part that holds the number, then the logit.
    __device__ __forceinline__ void all(const float* tops, const double* sums, int parts) const {
        const int each = (parts + kRowThreads - 1) / kRowThreads;
        const int from = threadIdx.x * each, to = min(from + each, parts);
        auto sum_of = [&](int p) {
            const double w = want.weigh(tops[p], top);
            return w > kNoWeight ? sums[p] * w : 0.0;
        };
        double own = 0.0, total;
        for (int p = from; p < to; ++p) own += sum_of(p);
        const double before = scan(own, sh, &total), target = want.u * total;
        const int t = holder(before, own, target, sh);
        if ((int)threadIdx.x == t) {
            double sum = before;
            int part = from;
            for (int p = from; p < to; ++p) {
                const double x = sum_of(p);
                if (!(x > 0.0)) continue;
                sh.found[0] = sum;
                part = p;
                sum += x;
                if (sum > target) break;
            }
            sh.hits = part;
        }
        __syncthreads();
        pick_near(sh.hits, target - sh.found[0], total);
    }

    // Any filters on any row, by passes over it: the cut's key, the last of the equal ones, and
    // the weights by block.  The first cut lies in [least, over), with `above` (logits for
    // top-k, else weight) before these.  (64 rows: bf16 with top-p 0.9 at temperature 2 187
    // us, equal fp32 ones 211; narrowing by whole keys and indices, in an earlier form, 362 and 289.)
    __device__ __forceinline__ void by_passes(double total, float least, float over, double above) const {
        float most = fminf(below(over), top);
        if constexpr (sizeof(T) == 4) {  // (bf16 has few keys: a pass less, or none more)
            uint32_t lo = ~0u, hi = 0;
            every([&](float x, int) {
                if (x < least || x >= over) return;
                lo = min(lo, key_of(x));
                hi = max(hi, key_of(x));
            });
            __syncthreads();
            if (threadIdx.x == 0) {
                sh.range[0] = ~0u;
                sh.range[1] = 0;
            }
            __syncthreads();
            atomicMin(&sh.range[0], lo);
            atomicMax(&sh.range[1], hi);
            __syncthreads();
            least = value_of(sh.range[0]);
            most = value_of(sh.range[1]);
        }
        auto each = [&](auto f) {
            every([&](float x, int i) {
                if (x >= least && x <= most) f(x, i, [&] { return Sum<true>::units_of(want.weigh(x, top)); });
            });
        };
        const auto row = narrow<T, true>(each, want, top, sh);
        Cut keep;
        for (int again = 0; again < 2; ++again) {  // top-k, then top-p
            if (again ? want.p == 1.0 : want.k == 0) continue;
            if (again && want.k) {
                double before;
                sum_blocks(weight_of([=](float x, int i) { return keep.keeps(x, i); }), 0.0, -1.0, before, total);
                above = 0.0;
                least = value_of(keep.key);
                most = top;
            }
            keep = row.cut(keep, again ? 0 : want.k - (int)above, again ? want.p * total - above : 0.0,
                           most, least, V, [&](uint32_t key, const Cut in, uint64_t number) {
                               const float v = value_of(key);  // by blocks: the one that holds it, then there
                               auto equal = [=](float x, int i) {
                                   return x == v && (in.key < key || (uint32_t)i <= in.idx);
                               };
                               double before, ties;
                               const int block = sum_blocks([=](float x, int i) { return equal(x, i) ? 1.0 : 0.0; },
                                                            0.0, (double)number - 0.5, before, ties);
                               float x[NEAR][VEC];
                               uint32_t stay;
                               list_block(block, kList, x, stay, equal);
                               const uint32_t idx = (uint32_t)sh.list[(int)((double)number - before) - 1];
                               __syncthreads();  // (before the list is written again)
                               return idx;
                           });
        }
        const float lowest = floor;
        pick([=](float x, int i) { return keep.keeps(x, i) && x >= lowest; });
    }

    // Up to 64 candidates, the first of the order, in LDS: one wave, a candidate a lane.
    // (total: the sum of all weights of the row, where there is no top-k)
    __device__ __forceinline__ void few(int n, double total) const {
        const int lane = threadIdx.x;
        if (lane >= 64) return;
        const int idx = lane < n ? sh.list[lane] : 0;
        const uint32_t key = lane < n ? key_of(value(idx)) : 0;
        const double w = lane < n ? want.weigh(value_of(key), top) : 0.0;
        uint2* all = reinterpret_cast<uint2*>(sh.hit);
        all[lane] = make_uint2(key, (uint32_t)idx);
        wave_fence();
        int rank = 0, place = 0;  // in the order, by the index
#pragma unroll 8
        for (int l = 0; l < n; ++l) {
            const uint2 o = all[l];
            const bool less = (int)o.y < idx;
            rank += (o.x > key || (o.x == key && less)) ? 1 : 0;
            place += less ? 1 : 0;
        }
        double* by = reinterpret_cast<double*>(sh.mass);
        int* at = reinterpret_cast<int*>(sh.count);
        if (lane < n) by[rank] = w;
        wave_fence();
        const int most = want.k > 0 && want.k < n ? want.k : n;
        const double sorted = lane < most ? by[lane] : 0.0;
        wave_fence();
        double upto = sum_upto(sorted);
        if (want.k > 0) total = last_lane(upto);
        const double before = moved<0x138>(upto);  // (the lane before's)
        const bool stays = lane < most && (lane == 0 || ((want.p == 1.0 || before < want.p * total) &&
                                                         sorted > kNoWeight));
        // (the first ones, by each filter)
        const int kept = min(__builtin_popcountll(__ballot(stays)),
                             __builtin_popcountll(__ballot(lane < n && value_of(key) >= floor)));
        if (lane < n) {
            by[place] = rank < kept ? w : 0.0;
            at[place] = idx;
        }
        wave_fence();
        const double own = lane < n ? by[lane] : 0.0;
        upto = sum_upto(own);
        const double sum = last_lane(upto), target = want.u * sum;
        const uint64_t behind = __ballot(own > 0.0 && upto > target), any = __ballot(own > 0.0);
        const int chosen = behind ? __builtin_ctzll(behind) : 63 - __builtin_clzll(any);
        if (lane == chosen) emit(at[lane], log(own / sum));
    }

    // Up to kRanked of them: two threads a candidate count those before it in the order
    // and by the index.
    __device__ __forceinline__ void ranked(int n, double total) const {
        static_assert(2 * kRanked <= kRowThreads && kRanked * sizeof(uint2) <= sizeof(sh.hit), "");
        const int tid = threadIdx.x, j = tid >> 1;
        const bool there = j < n;
        const int idx = there ? sh.list[j] : 0;
        const float x = value(idx);
        const uint32_t key = key_of(x);
        const double w = want.weigh(x, top);
        uint2* all = reinterpret_cast<uint2*>(sh.hit);
        if (there && !(tid & 1)) all[j] = make_uint2(key, (uint32_t)idx);
        __syncthreads();
        int rank = 0, place = 0;
#pragma unroll 8
        for (int l = tid & 1; l < n; l += 2) {
            const uint2 o = all[l];
            const bool less = (int)o.y < idx;
            rank += (o.x > key || (o.x == key && less)) ? 1 : 0;
            place += less ? 1 : 0;
        }
        rank += __shfl_xor(rank, 1, 64);
        place += __shfl_xor(place, 1, 64);
        const bool writes = there && !(tid & 1);
        double* by = reinterpret_cast<double*>(sh.mass);
        int* at = reinterpret_cast<int*>(sh.count);
        if (writes) by[rank] = w;
        __syncthreads();
        const int most = want.k > 0 && want.k < n ? want.k : n;
        const double sorted = tid < most ? by[tid] : 0.0;
        double sum;
        const double before = scan(sorted, sh, &sum);
        if (want.k > 0) total = sum;
        const int kept = min(
            __syncthreads_count(tid < most && (tid == 0 || ((want.p == 1.0 || before < want.p * total) &&
                                                            sorted > kNoWeight))),
            __syncthreads_count(writes && x >= floor));
        if (writes) {
            by[place] = rank < kept ? w : 0.0;
            at[place] = idx;
        }
        __syncthreads();
        const double own = tid < n ? by[tid] : 0.0;
        const double upto = scan(own, sh, &sum);
        if (tid == holder(upto, own, want.u * sum, sh)) emit(at[tid], log(own / sum));
    }

    // The least logit for which `is` holds (it does for the largest, and for those above one
    // that it holds for): 64 lanes narrow its key down.
    template <class Is>
    __device__ __forceinline__ float least_such(Is is) const {
        uint32_t lo = kLeastKey, hi = key_of(top);
        const uint32_t lane = threadIdx.x & 63;
        while (lo < hi) {
            const uint32_t step = (hi - lo) / 64 + 1, at = min(lo + lane * step, hi);
            const uint64_t yes = __ballot(is(value_of(at)));
            const uint32_t first = yes ? __builtin_ctzll(yes) : 64;
            hi = min(hi, lo + first * step);
            lo = first ? min(lo + (first - 1) * step + 1, hi) : lo;
        }
        return value_of(hi);
    }
    __device__ __forceinline__ float least_of(int q) const {
        return least_such([&](float x) { return want.bucket(x) >= q; });
    }

    __device__ __forceinline__ float value(int i) const {
        if constexpr (sizeof(T) == 4)
            return r.src[i];
        else
            return bf16_to_f32(r.src[i]);
    }

    static constexpr int AT = 32 / VEC;  // pieces of 32 logits

    // The wave's logits that are found, a bit each of a lane's 32, into the list;
    // place_of(bit): where it is in the row.
    template <class PlaceOf>
    __device__ __forceinline__ void list(uint32_t found, PlaceOf place_of) const {
        const uint32_t own = __builtin_popcount(found), upto = sum_upto(own);
        const uint32_t all = __builtin_amdgcn_readlane(upto, 63);
        if (all == 0) return;
        uint32_t at = 0;
        if ((threadIdx.x & 63) == 0) at = atomicAdd((uint32_t*)&sh.listed, all);
        at = __builtin_amdgcn_readfirstlane(at) + upto - own;
        for (; found; found &= found - 1, ++at)
            if (at < kList) sh.list[at] = place_of(__builtin_ctz(found));
    }
    // A piece's logits above low and not above high, a bit each below found's: a
    // difference's sign (four instructions a logit).
    __device__ __forceinline__ uint32_t found_in(uint32_t found, const uint4& raw, float low, float high) const {
        float v[VEC];
        r.values(raw, v);
        if (low == -INFINITY) {  // (a difference would be none)
            found <<= VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) found |= v[e] > low && v[e] <= high ? 1u << e : 0u;
        } else {
#pragma unroll
            for (int e = VEC - 1; e >= 0; --e)
                found = __builtin_amdgcn_alignbit(
                    found, __float_as_uint(low - v[e]) ^ __float_as_uint(high - v[e]), 31);
        }
        return found;
    }
    // the next logit below x, which is above -infinity
    __device__ __forceinline__ float below(float x) const {
        const float y = value_of(key_of(x) - 1);
        return y == 0.0f && !(x > 0.0f) ? -0x1p-149f : y;  // (below both zeros)
    }

    // The places of the logits in [least, most) into the list, the row's pieces in turn, the
    // next ones on their way; its ends, which are no whole pieces, first.
    __device__ __forceinline__ int in_turn(float least, float most) const {
        const int tid = threadIdx.x;
        const int begin = r.before ? 1 : 0, end = max((r.before + V) / VEC, begin);
        if (tid < 2 * VEC) {
            const int i = tid < VEC ? tid : end * VEC - r.before + tid - VEC;
            if (i < (tid < VEC ? min(begin * VEC - r.before, V) : V) && value(i) >= least && value(i) < most) {
                const int at = atomicAdd(&sh.listed, 1);
                if (at < kList) sh.list[at] = i;
            }
        }
        const float low = below(least), high = below(most);
        const char* const base = reinterpret_cast<const char*>(r.src - r.before);
        auto piece = [&](int i) {
            return *reinterpret_cast<const uint4*>(base + (uint32_t)min(i, end - 1) * 16u);
        };
        if (end > begin) {
            uint4 raw[AT];
#pragma unroll
            for (int j = 0; j < AT; ++j) raw[j] = piece(begin + tid + j * kRowThreads);
            for (int i0 = begin + tid; __any(i0 < end); i0 += AT * kRowThreads) {
                uint32_t found = 0;
#pragma unroll
                for (int j = AT - 1; j >= 0; --j) {  // (a load after each piece: eight at once hold the waves up)
                    found = found_in(found, raw[j], low, high);
                    raw[j] = piece(i0 + (AT + j) * kRowThreads);
                    __builtin_amdgcn_sched_barrier(0);
                }
                const int there = i0 < end ? (end - i0 + kRowThreads - 1) / kRowThreads : 0;
                if (there < AT) found &= (1u << there * VEC) - 1;
                list(found, [&](int bit) {
                    return (i0 + bit / VEC * kRowThreads) * VEC - r.before + bit % VEC;
                });
            }
        }
        __syncthreads();
        return sh.listed;
    }

    // The same by the groups whose largest logit is one, where these are not most.
    // (tops: the first kHits groups')
    __device__ __forceinline__ int gather(const float* groups, int n_groups,
                                          const float (&tops)[kHits / kRowThreads], float least,
                                          float most) const {
        const int tid = threadIdx.x, lane = tid & (kGroup - 1);
        const float low = below(least), high = below(most);
        __syncthreads();
        if (tid == 0) sh.listed = sh.hits = 0;
        __syncthreads();
        for (int g0 = 0; g0 < n_groups; g0 += kHits) {
            uint32_t hit = 0;
#pragma unroll
            for (int j = 0; j < kHits / kRowThreads; ++j) {
                const int g = g0 + j * kRowThreads + tid;
                const float x = g0 == 0 ? tops[j] : g < n_groups ? groups[g] : -INFINITY;
                hit |= x >= least ? 1u << j : 0u;
            }
            const uint32_t own = __builtin_popcount(hit), upto = sum_upto(own);
            uint32_t at = 0;
            if ((tid & 63) == 63) at = atomicAdd((uint32_t*)&sh.hits, upto);
            at = __builtin_amdgcn_readlane(at, 63) + upto - own;
            for (; hit; hit &= hit - 1, ++at)
                sh.hit[at] = (uint16_t)(__builtin_ctz(hit) * kRowThreads + tid);
            __syncthreads();
            const int hits = sh.hits;
            // (64 rows, normal, top-p 0.9: 51 us, by groups 56)
            if (g0 == 0 && 2 * hits > min(n_groups, kHits)) return in_turn(least, most);
            // where the row's ends or no group are a piece is all -infinity until its
            // logits are looked at one by one
            constexpr int HOP = kRowThreads / kGroup;
            constexpr uint32_t NONE = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
            for (int h0 = tid / kGroup; __any(h0 < hits); h0 += AT * HOP) {
                uint4 raw[AT];
                uint32_t part = 0;
#pragma unroll
                for (int j = 0; j < AT; ++j) {
                    raw[j] = make_uint4(NONE, NONE, NONE, NONE);
                    if (h0 + j * HOP < hits) {
                        const int col = ((g0 + sh.hit[h0 + j * HOP]) * kGroup + lane) * VEC - r.before;
                        if (col >= 0 && col <= V - VEC)
                            raw[j] = *reinterpret_cast<const uint4*>(r.src + col);
                        else
                            part |= 1u << j;
                    }
                }
                uint32_t found = 0;
#pragma unroll
                for (int j = AT - 1; j >= 0; --j) found = found_in(found, raw[j], low, high);
                while (part) {
                    const int j = __builtin_ctz(part);
                    const int col = ((g0 + sh.hit[h0 + j * HOP]) * kGroup + lane) * VEC - r.before;
                    part &= part - 1;
                    for (int e = 0; e < VEC; ++e)
                        if (col + e >= 0 && col + e < V && value(col + e) >= least && value(col + e) < most)
                            found |= 1u << (j * VEC + e);
                }
                list(found, [&](int bit) {
                    return ((g0 + sh.hit[h0 + bit / VEC * HOP]) * kGroup + lane) * VEC - r.before + bit % VEC;
                });
            }
            __syncthreads();
            if (g0 + kHits < n_groups) {
                if (tid == 0) sh.hits = 0;
                __syncthreads();
            }
        }
        return sh.listed;
    }

    // Filters: the blocks' buckets joined say in which bucket the order is cut.  False
    // where they do not, or it holds too many logits; total: the sum of the row's
    // weights, where top-p asks for it, or the number of its logits.
    __device__ __forceinline__ bool by_buckets(const float* tops, const double* sums, const float* groups,
                                               const double* buckets, int blocks, double& total,
                                               float& least, float& over, double& above) const {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
        const bool weights = want.whole_sum();
        double own = 0.0;
        total = above = 0.0;
        least = value_of(kLeastKey);
        over = INFINITY;
        if (blocks > kMostBlocks) {
            if (weights) {
                double own = 0.0;
                for (int g = tid; g < blocks; g += kRowThreads) {
                    const float4 t = reinterpret_cast<const float4*>(tops)[g];
                    const float x = fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w));
                    if (!(x > -INFINITY)) continue;
                    double s = 0.0;
                    for (int w = 0; w < kBlockWaves; ++w) s += sums[g * kBlockWaves + w];
                    own += s * want.weigh(x, top);
                }
                scan(own, sh, &total);
            }
            return false;
        }
        // (on their way ahead)
        const int n_groups = blocks * (kPieces / kGroup);
        float group_tops[kHits / kRowThreads];
#pragma unroll
        for (int j = 0; j < kHits / kRowThreads; ++j) {
            const int g = j * kRowThreads + tid;
            group_tops[j] = g < n_groups ? groups[g] : -INFINITY;
        }
        const int most = want.bucket(top);
        if (tid < blocks) {
            const float4 t = reinterpret_cast<const float4*>(tops)[tid];
            const float x = fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w));
            const bool live = x > -INFINITY;
            const double factor = live ? want.weigh(x, top) : 0.0;
            sh.offset[tid] = live ? min(most - want.bucket(x), kBuckets) : kBuckets + 1;
            sh.factor[tid] = weights ? factor : 1.0;
            if (live) {
                for (int w = 0; w < kBlockWaves; ++w) own += sums[tid * kBlockWaves + w];
                if (weights) own *= factor;
            }
        }
        scan(own, sh, &total);  // (and the barriers for offset and factor)
        static_assert(kBuckets == kRowThreads && kBins == kRowThreads && kMostBlocks <= kBins, "");
        // a thread a bucket; the row's last one takes what is left (of weights: nothing
        // is cut there)
        double in = 0.0, all;
        for (int g0 = 0; g0 < blocks; g0 += 16) {
            double x[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {  // (on their way at once)
                const int g = min(g0 + j, blocks - 1), i = max(tid - sh.offset[g], 0);
                x[j] = buckets[g * kBuckets + i];
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int g = min(g0 + j, blocks - 1);
                if (g0 + j < blocks && tid >= sh.offset[g]) in += x[j] * sh.factor[g];
            }
        }
        if (tid == kRest) in = 0.0;
        const double before = scan(in, sh, &all);
        if (tid == kRest) in = weights ? 0.0 : total - all;
        // the bucket that holds the cut: top-k's or top-p's, or min-p's where that is higher
        int last = kRest;
        if (want.k || want.p < 1.0)
            last = min(last, lowest(in > 0.0 && before + in >= (want.k ? (double)want.k : want.p * total), sh));
        bool cut_here = last < kRest;
        if (want.m > 0.0 && !(want.k && want.p < 1.0)) {  // (the sum of top-k's has to be whole)
            const int bound = most - want.bucket(floor);
            cut_here &= last <= bound;
            last = min(last, bound);
        }
        // how many logits there are up to it, and in it: where weights were summed at most
        // as many as if each had its bucket's least
        double n = in;
        if (weights) n = tid == kRest ? 2.0 * kList : in * exp2f((float)(tid + 1) * (1.4427f / 24.0f)) + 1.0;
        const double n_before = weights ? scan(n, sh, &all) : before;
        __syncthreads();
        if (tid == last) {
            sh.found[0] = before;
            sh.found[1] = n_before;
            sh.found[2] = n;
        }
        __syncthreads();
        const double n_above = sh.found[1], here = sh.found[2];
        // The logits up to the cut's bucket, where the list holds them; without top-k those of
        // the bucket, as the blocks' buckets say what lies before it.
        const bool few_before = n_above + here <= (weights && last < kRest && here <= kList ? kManyBefore : kList);
        if (last < kRest) least = least_of(most - last);
        if (!few_before) {
            if (last == kRest) return false;
            if (last > 0) over = least_of(most - last + 1);
            above = sh.found[0];
            if (want.k || here > kList) {
                if (cut_here) return false;
                least = value_of(kLeastKey);
                over = INFINITY;
                above = 0.0;
                return false;
            }
        }
        const int listed = gather(groups, n_groups, group_tops, least, over);
        if (listed > kList) return false;
        if (few_before && listed <= kSome) {
            few(listed, total);
            return true;
        }
        if (few_before && listed <= kRanked) {
            ranked(listed, total);
            return true;
        }
        constexpr int E = kList / kRowThreads;
        float x[E];
        int idx[E];
        uint64_t w[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            idx[j] = tid + j * kRowThreads < listed ? sh.list[tid + j * kRowThreads] : 0;
            x[j] = value(idx[j]);
        }
#pragma unroll
        for (int j = 0; j < E; ++j) w[j] = Sum<false>::units_of(want.weigh(x[j], top));
        auto each = [&](auto f) {
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (tid + j * kRowThreads < listed) f(x[j], idx[j], [&] { return w[j]; });
        };
        const auto list = narrow<T, false>(each, want, top, sh);
        auto sum_of = [&](auto stays) {
            Sum<false> sum;
            each([&](float v, int i, auto units) { sum.upper += stays(v, i) ? units() : 0; });
            sum.upper = total_of(sum.upper, sh);
            return sum.value();
        };
        auto index = [&](uint32_t key, const Cut in, uint64_t number) { return list.index_of(key, in, number, V); };
        Cut keep;
        double target = want.p * total - above;
        if (want.k) {
            keep = list.cut(keep, want.k, 0.0, top, least, V, index);
            if (want.p < 1.0) target = want.p * sum_of([&](float v, int i) { return keep.keeps(v, i); });
        }
        if (want.p < 1.0 && (few_before || cut_here)) keep = list.cut(keep, 0, target, fminf(over, top), least, V, index);
        if (few_before) {
            auto stays = [&](float v, int i) {
                return keep.keeps(v, i) && v >= floor && want.weigh(v, top) > kNoWeight;
            };
            const double sum = sum_of(stays);
            const double number = want.u * sum;
            uint32_t first = 0;
            Sum<false> before_first;
            uint64_t ties;
            // (a number of 0 takes the first one, however little it weighs)
            list.template find<true>(first, (uint32_t)V - 1,
                      [&](float v, int i) { return stays(v, i) ? (uint32_t)i : ~0u; },
                      [&](const Sum<false>& upto) { return number == 0.0 || upto.value() > number; },
                      before_first, ties);
            each([&](float v, int i, auto) {
                if ((uint32_t)i == first) emit(i, log(want.weigh(v, top) / sum));
            });
            return true;
        }
        // which block holds the number: its buckets before the cut's, and what stays of that
        __syncthreads();
        sh.mass[tid] = 0;
        __syncthreads();
        each([&](float v, int i, auto units) {
            if (v >= floor && keep.keeps(v, i))
                atomicAdd((unsigned long long*)&sh.mass[(i + r.before) / kBlock], (unsigned long long)units());
        });
        for (int g = wave; g < blocks; g += kRowWaves) {
            double s = 0.0;
#pragma unroll
            for (int j = 0; j < kBuckets / 64; ++j) {
                const int i = lane + 64 * j;
                const double y = buckets[g * kBuckets + i];
                if (i + sh.offset[g] < last) s += y;
            }
            s = last_lane(sum_upto(s));
            if (lane == 0) sh.blocks[g] = s * sh.factor[g];
        }
        __syncthreads();
        own = tid < blocks ? sh.blocks[tid] + Sum<false>{sh.mass[tid], 0}.value() : 0.0;
        double stay;
        const double at = scan(own, sh, &stay);
        target = want.u * stay;
        const int block = holder(at, own, target, sh);
        if (tid == block) sh.found[0] = at;
        __syncthreads();
        pick_listed(block, target - sh.found[0], stay,
                    [&](float v, int i) { return v >= over || (v >= least && v >= floor && keep.keeps(v, i)); });
        return true;
    }
};

// A workgroup a row: of 35 us for 64 flat rows 12 go into reading a row's logits again, 4 into the
// cut, 6 into the token's block, and 7 into joining the histograms.
template <class T, bool FILTERS>
__global__ void __launch_bounds__(kRowThreads) sample_row_kernel(
    const T* __restrict__ logits, int64_t ld, const Request q, int V, const Found in,
    int32_t* __restrict__ tokens, float* __restrict__ logprobs, uint32_t* __restrict__ err) {
    __shared__ Shared sh;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, parts = in.blocks * kBlockWaves;
    const float* tops = in.tops + row * parts;
    float top = -INFINITY;
    bool nan = false;
    for (int p = tid; p < parts; p += kRowThreads) {
        const float t = tops[p];
        nan |= t != t;
        top = fmaxf(top, t);
    }
    const Want want(q, row, V);
    top = largest(top);
    if ((tid & 63) == 0) sh.sum[tid >> 6] = top;
    nan = __syncthreads_or(nan);
    for (int w = 0; w < kRowWaves; ++w) top = fmaxf(top, (float)sh.sum[w]);
    const Row<T> r(logits + row * ld);
    Sampler<T> s{r, V, (r.before + V + Row<T>::VEC - 1) / Row<T>::VEC, want, top, sh,
                       tokens + row, logprobs ? logprobs + row : nullptr, value_of(kLeastKey)};
    if (want.bad || nan || top == -INFINITY) {
        if (tid == 0) {
            s.emit(-1, -INFINITY);
            if (err && (want.bad || nan))
                atomicOr(err, (want.bad ? ENGRAM_ERRBIT_SAMPLE : 0) | (nan ? ENGRAM_ERRBIT_LOGIT : 0));
        }
        return;
    }
    const double* sums = in.sums + row * parts;
    if (want.greedy()) return s.greedy(tops, parts);
    if (!FILTERS || !want.filtered()) return s.all(tops, sums, parts);
    if constexpr (FILTERS) {
        if (want.m > 0.0) s.floor = s.least_such([&](float x) { return want.weigh(x, top) >= want.m; });
        const int64_t blocks = row * in.blocks;
        double total, above;
        float least, over;  // where the cut lies
        if (!s.by_buckets(tops, sums, in.groups + blocks * (kBlock / Row<T>::VEC / kGroup),
                          in.buckets + blocks * kBuckets, in.blocks, total, least, over, above))
            s.by_passes(total, least, over, above);
    }
}

int blocks_of(int V) { return (int)(((int64_t)V + 7 + kBlock - 1) / kBlock); }

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

size_t layout(int64_t B, int V, void* base, Found* f) {
    const size_t blocks = (size_t)B * blocks_of(V);
    char* at = (char*)base;
    auto take = [&](size_t bytes) {
        char* here = at;
        at += up256(bytes);
        return here;
    };
    f->blocks = blocks_of(V);
    f->sums = (double*)take(blocks * kBlockWaves * sizeof(double));
    f->buckets = (double*)take(blocks * kBuckets * sizeof(double));
    f->tops = (float*)take(blocks * kBlockWaves * sizeof(float));
    f->groups = (float*)take(blocks * (kBlock / Row<float>::VEC / kGroup) * sizeof(float));
    return (size_t)(at - (char*)base);
}

template <class T>
hipError_t run_sample(const void* logits, int64_t ld, const Request& q, int64_t B, int V,
                      int32_t* tokens, float* logprobs, void* scratch, uint32_t* err,
                      hipStream_t s) {
    Found f;
    layout(B, V, scratch, &f);
    // (without any filter kernels that hold fewer registers: 512 rows 59 -> 55 us)
    const bool filters = q.top_k || q.top_p || q.min_p;
    auto part = filters ? sample_part_kernel<T, true> : sample_part_kernel<T, false>;
    part<<<dim3((uint32_t)((B + kXcds - 1) / kXcds * kXcds * f.blocks)), dim3(64 * kBlockWaves), 0, s>>>(
        (const T*)logits, ld, q, B, V, f);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    auto whole = filters ? sample_row_kernel<T, true> : sample_row_kernel<T, false>;
    whole<<<dim3((uint32_t)B), dim3(kRowThreads), 0, s>>>((const T*)logits, ld, q, V, f, tokens,
                                                        logprobs, err);
    return hipGetLastError();
}

}  // namespace

bool sample_supported(int64_t B, int V) {
    return (B + kXcds - 1) / kXcds * kXcds * blocks_of(V) * (64 * kBlockWaves) < ((int64_t)1 << 32);
}

size_t sample_scratch_bytes(int64_t B, int V) {
    Found f;
    return layout(B, V, nullptr, &f);
}

hipError_t launch_sample(const void* logits, bool f32, int64_t ld, const float* u,
                         const float* temperature, const int32_t* top_k, const float* top_p,
                         const float* min_p, int64_t B, int V, int32_t* tokens, float* logprobs,
                         void* scratch, uint32_t* err, hipStream_t s) {
    const Request q{u, temperature, top_k, top_p, min_p};
    return f32 ? run_sample<float>(logits, ld, q, B, V, tokens, logprobs, scratch, err, s)
               : run_sample<uint16_t>(logits, ld, q, B, V, tokens, logprobs, scratch, err, s);
}

}  // namespace engram
