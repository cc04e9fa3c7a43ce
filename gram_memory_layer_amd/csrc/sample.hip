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
// in 64 bits.
#include "logits.h"

namespace engram {
namespace {

constexpr int kPartThreads = 256;
constexpr int kEach = 32;                       // logits a thread of a part
constexpr int kPart = kPartThreads * kEach;     // logits a part
constexpr int kRowThreads = 1024;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kBins = 1024;

// exp(d / T) for d <= 0, by c = log2(e) / T: 2^n * 2^f, f in [-1/2, 1/2], 2^f by a
// polynomial of degree eight with the least relative error (1.1e-12, by Remez'
// exchange); 0 gives exactly 1.  Below 2^-999 it is 2^-1000: no weight.
constexpr double kLog2e = 1.4426950408889634074;
constexpr double kRound = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to a whole number
constexpr double kNoWeight = 0x1p-999;
__device__ __forceinline__ double weight(double d, double c) {
    const double t = fmax(d * c, -1000.0);
    const double r = t + kRound;
    const double f = t - (r - kRound);
    double p = 1.3344183691340562e-06;
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
    double p, m, u;
    int k;         // 0: no top-k
    bool bad;
    __device__ Want(const Request& q, int64_t row, int V) {
        const float t = q.temperature ? q.temperature[row] : 1.0f;
        const float pp = q.top_p ? q.top_p[row] : 1.0f;
        const float mm = q.min_p ? q.min_p[row] : 0.0f;
        const float uu = q.u[row];
        const int kk = q.top_k ? q.top_k[row] : 0;
        bad = !(t >= 0.0f && t < INFINITY) || !(pp >= 0.0f && pp <= 1.0f) ||
              !(mm >= 0.0f && mm <= 1.0f) || !(uu >= 0.0f && uu < 1.0f);
        c = t > 0.0f ? kLog2e / (double)t : 0.0;
        p = pp;
        m = mm;
        u = uu;
        k = kk > 0 && kk < V ? kk : 0;
    }
    __device__ bool greedy() const { return c == 0.0; }
    __device__ bool filtered() const { return k > 0 || p < 1.0 || m > 0.0; }
    // whether the weights of the whole row are summed
    __device__ bool whole_sum() const { return !greedy() && k == 0 && (p < 1.0 || m == 0.0); }
};

// One workgroup a part of a row: its largest logit (NaN: a NaN or +infinity is in
// it) and, where the row needs it, the sum of its weights relative to that.
template <class T>
__global__ void __launch_bounds__(kPartThreads) sample_part_kernel(
    const T* __restrict__ logits, int64_t ld, const Request q, int V, int parts,
    float* __restrict__ tops, double* __restrict__ sums) {
    constexpr int VEC = Row<T>::VEC, NL = kEach / VEC, NW = kPartThreads / 64;
    __shared__ float wave_top[NW];
    __shared__ double wave_sum[NW];
    __shared__ int wave_bad[NW];
    const int64_t row = blockIdx.y;
    const int part = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Row<T> r(logits + row * ld);
    const int64_t first = (int64_t)part * NL * kPartThreads + tid;
    uint4 raw[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) raw[i] = r.fetch(first + i * kPartThreads, V);
    const Want want(q, row, V);
    float v[NL][VEC], top = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        r.unpack(raw[i], first + i * kPartThreads, V, v[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            bad |= !(v[i][e] < INFINITY);
            top = fmaxf(top, v[i][e]);
        }
    }
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    bad = __any(bad);
    if (lane == 0) {
        wave_top[wave] = top;
        wave_bad[wave] = bad;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        top = fmaxf(top, wave_top[w]);
        bad |= wave_bad[w] != 0;
    }
    if (tid == 0) tops[row * parts + part] = bad ? __uint_as_float(0x7FC00000u) : top;
    if (!want.whole_sum() || bad || top == -INFINITY) return;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < NL; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += weight((double)v[i][e] - (double)top, want.c);
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
    if (lane == 0) wave_sum[wave] = s;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < NW; ++w) s += wave_sum[w];
        sums[row * parts + part] = s;
    }
}

// What the threads of a row's workgroup exchange
struct Shared {
    double sum[kRowWaves];
    uint64_t whole[kRowWaves];
    uint32_t count[kBins];
    uint64_t mass[kBins];
    int first, last;
    double below;
    int32_t token;
    double token_weight;
};

// sum over the workgroup, and this thread's share of it: what lies before it
__device__ __forceinline__ double scan(double own, Shared& sh, double* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double upto = own;
    for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(upto, o, 64);
        if (lane >= o) upto += y;
    }
    __syncthreads();
    if (lane == 63) sh.sum[wave] = upto;
    __syncthreads();
    double before = 0.0, all = 0.0;
    for (int w = 0; w < kRowWaves; ++w) {
        if (w < wave) before += sh.sum[w];
        all += sh.sum[w];
    }
    *total = all;
    const double prev = __shfl_up(upto, 1, 64);
    return before + (lane ? prev : 0.0);
}
__device__ __forceinline__ uint64_t scan(uint64_t own, Shared& sh) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t upto = own;
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t y = __shfl_up(upto, o, 64);
        if (lane >= o) upto += y;
    }
    __syncthreads();
    if (lane == 63) sh.whole[wave] = upto;
    __syncthreads();
    uint64_t before = upto - own;
    for (int w = 0; w < wave; ++w) before += sh.whole[w];
    return before;
}

// the lowest thread for which `is` holds, kRowThreads if none; all threads call
__device__ __forceinline__ int lowest(bool is, Shared& sh) {
    __syncthreads();
    if (threadIdx.x == 0) sh.first = kRowThreads;
    __syncthreads();
    if (is) atomicMin(&sh.first, (int)threadIdx.x);
    __syncthreads();
    return sh.first;
}
__device__ __forceinline__ int highest(bool is, Shared& sh) {
    __syncthreads();
    if (threadIdx.x == 0) sh.last = -1;
    __syncthreads();
    if (is) atomicMax(&sh.last, (int)threadIdx.x);
    __syncthreads();
    return sh.last;
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
    int idx = 0x7FFFFFFF;
    __device__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= idx); }
};

// A row, its weights, and passes over it by the workgroup
template <class T>
struct Whole {
    static constexpr int VEC = Row<T>::VEC;
    const Row<T> r;
    const int V;
    const double c;
    const float top;
    const int pieces;
    __device__ Whole(const T* row, int V_, double c_, float top_)
        : r(row), V(V_), c(c_), top(top_), pieces((r.before + V_ + VEC - 1) / VEC) {}
    __device__ double weight_of(float x) const { return weight((double)x - (double)top, c); }

    // f(x, index) for all logits but those at -infinity, pieces in turn
    template <class F>
    __device__ __forceinline__ void every(F f) const {
        for (int i = threadIdx.x; i < pieces; i += kRowThreads) some(i, f);
    }
    // the same with a run of neighbouring pieces for each thread
    template <class F>
    __device__ __forceinline__ void in_order(F f) const {
        const int each = (pieces + kRowThreads - 1) / kRowThreads;
        const int from = threadIdx.x * each, to = min(from + each, pieces);
        for (int i = from; i < to; ++i) some(i, f);
    }
    template <class F>
    __device__ __forceinline__ void some(int i, F f) const {
        float x[VEC];
        r.unpack(r.fetch(i, V), i, V, x);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (x[e] > -INFINITY) f(x[e], (int)r.column(i) + e);
    }

    // The cut that keeps the first k elements of `in`, or (k = 0) those whose
    // predecessors weigh less than target.  Passes over the row narrow the keys
    // down by a factor of kBins each; weights add up as whole numbers of 2^-scale, in
    // any order.
    __device__ Cut cut(const Cut in, int k, double target, Shared& sh) const {
        const int scale = min(50, 62 - (32 - __builtin_clz(V)));
        const double magic = ldexp(1.0, 52 - scale), unit = ldexp(1.0, -scale);
        uint32_t lo = max(in.key, kLeastKey), hi = key_of(top);
        uint64_t above = 0, mass = 0;
        const int tid = threadIdx.x;
        while (lo < hi) {
            const int shift = max(0, 22 - __builtin_clz(hi - lo));
            const uint32_t bins = ((hi - lo) >> shift) + 1;
            __syncthreads();
            sh.count[tid] = 0;
            sh.mass[tid] = 0;
            __syncthreads();
            every([&](float x, int i) {
                const uint32_t key = key_of(x);
                if (key < lo || key > hi || !in.keeps(key, i)) return;
                const uint32_t at = bins - 1 - ((key - lo) >> shift);  // the largest first
                atomicAdd(&sh.count[at], 1u);
                if (k == 0) {
                    const double w = weight_of(x) + magic;
                    atomicAdd((unsigned long long*)&sh.mass[at],
                              (unsigned long long)(__double_as_longlong(w) - __double_as_longlong(magic)));
                }
            });
            __syncthreads();
            const uint64_t own_n = sh.count[tid], own_m = sh.mass[tid];
            const uint64_t n = above + scan(own_n, sh), m = mass + scan(own_m, sh);
            const int at = lowest(k ? n + own_n >= (uint64_t)k : (double)(m + own_m) * unit >= target, sh);
            if (at == kRowThreads) return in;  // all of them do not reach it
            __syncthreads();
            if (tid == at) {
                sh.whole[0] = n;
                sh.whole[1] = m;
            }
            __syncthreads();
            above = sh.whole[0];
            mass = sh.whole[1];
            lo += (bins - 1 - (uint32_t)at) << shift;
            hi = min(hi, lo + ((1u << shift) - 1));
        }
        // how many of the equal ones at the cut stay, and the last of these
        double stay = (double)k - (double)above;
        if (k == 0) {
            const double w = weight_of(value_of(lo));
            stay = ceil((target - (double)mass * unit) / w);
        }
        const uint64_t r = stay < 1.0 ? 1 : stay > 0x1p31 ? (uint64_t)1 << 31 : (uint64_t)stay;
        uint64_t ties = 0;
        in_order([&](float x, int i) { ties += key_of(x) == lo && in.keeps(lo, i); });
        const uint64_t before = scan(ties, sh);
        Cut out;
        out.key = lo;
        const int at = lowest(before < r && before + ties >= r, sh);
        if (at == kRowThreads) {  // all of them
            out.idx = in.key == lo ? in.idx : 0x7FFFFFFF;
            return out;
        }
        __syncthreads();
        if (tid == at) {
            uint64_t seen = before;
            in_order([&](float x, int i) {
                if (key_of(x) == lo && in.keeps(lo, i) && ++seen == r) sh.last = i;
            });
        }
        __syncthreads();
        out.idx = sh.last;
        return out;
    }
};

// One workgroup a row.
template <class T>
__global__ void __launch_bounds__(kRowThreads) sample_row_kernel(
    const T* __restrict__ logits, int64_t ld, const Request q, int V, int parts,
    const float* __restrict__ tops, const double* __restrict__ sums, int32_t* __restrict__ tokens,
    float* __restrict__ logprobs, uint32_t* __restrict__ err) {
    constexpr int VEC = Row<T>::VEC;
    __shared__ Shared sh;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const Want want(q, row, V);
    auto emit = [&](int token, double logprob) {
        tokens[row] = token;
        if (logprobs) logprobs[row] = (float)logprob;
    };
    // (a part a thread: parts <= kRowThreads)
    const float own_top = tid < parts ? tops[row * parts + tid] : -INFINITY;
    float top = own_top;
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    const bool nan = __syncthreads_or(own_top != own_top);
    if ((tid & 63) == 0) sh.sum[tid >> 6] = top;
    __syncthreads();
    for (int w = 0; w < kRowWaves; ++w) top = fmaxf(top, (float)sh.sum[w]);
    if (want.bad || nan || top == -INFINITY) {
        if (tid == 0) {
            emit(-1, -INFINITY);
            if (err && (want.bad || nan))
                atomicOr(err, (want.bad ? ENGRAM_ERRBIT_SAMPLE : 0) | (nan ? ENGRAM_ERRBIT_LOGIT : 0));
        }
        return;
    }
    const Whole<T> x(logits + row * ld, V, want.c, top);
    if (want.greedy()) {
        // the first part with the largest logit, and its first place there
        const int part = lowest(own_top == top, sh);
        __syncthreads();
        if (tid == 0) sh.last = V;
        __syncthreads();
        constexpr int pieces = kPart / VEC;
        for (int i = part * pieces + tid; i < min((part + 1) * pieces, x.pieces); i += kRowThreads)
            x.some(i, [&](float v, int at) {
                if (v == top) atomicMin(&sh.last, at);
            });
        __syncthreads();
        if (tid == 0) emit(sh.last, 0.0);
        return;
    }
    double own = 0.0, total = 0.0, before = 0.0;
    if (want.whole_sum()) {
        const double w = weight((double)own_top - (double)top, want.c);
        if (w > kNoWeight) own = sums[row * parts + tid] * w;
        before = scan(own, sh, &total);
    }
    // f(thread's run of pieces): the pick among the run's elements that stay
    auto pick = [&](double target, double at, auto stays, auto run) {
        double sum = at;
        int token = -1;
        double w_token = 0.0;
        bool done = false;
        run([&](float v, int i) {
            const double w = x.weight_of(v);
            if (done || !(w > kNoWeight) || !stays(v, i, w)) return;
            sum += w;
            token = i;
            w_token = w;
            done = sum > target;
        });
        emit(token, log(w_token / total));
    };
    if (!want.filtered()) {
        // the part that holds the number, then the piece
        double target = want.u * total;
        const int part = holder(before, own, target, sh);
        __syncthreads();
        if (tid == part) sh.below = before;
        __syncthreads();
        target -= sh.below;
        constexpr int pieces = kPart / VEC, each = (pieces + kRowThreads - 1) / kRowThreads;
        const int from = part * pieces + tid * each, to = min(from + each, x.pieces);
        auto run = [&](auto f) {
            for (int i = from; i < to; ++i) x.some(i, f);
        };
        own = 0.0;
        run([&](float v, int) {
            const double w = x.weight_of(v);
            own += w > kNoWeight ? w : 0.0;
        });
        double here;
        before = scan(own, sh, &here);
        if (tid == holder(before, own, target, sh))
            pick(target, before, [](float, int, double) { return true; }, run);
        return;
    }
    Cut keep;
    if (want.k) {
        keep = x.cut(keep, want.k, 0.0, sh);
        if (want.p < 1.0) {
            own = 0.0;
            x.in_order([&](float v, int i) {
                if (keep.keeps(key_of(v), i)) own += x.weight_of(v);
            });
            scan(own, sh, &total);
        }
    }
    if (want.p < 1.0) keep = x.cut(keep, 0, want.p * total, sh);
    auto stays = [&](float v, int i, double w) { return keep.keeps(key_of(v), i) && w >= want.m; };
    own = 0.0;
    x.in_order([&](float v, int i) {
        const double w = x.weight_of(v);
        if (w > kNoWeight && stays(v, i, w)) own += w;
    });
    before = scan(own, sh, &total);
    const double target = want.u * total;
    if (tid == holder(before, own, target, sh))
        pick(target, before, stays, [&](auto f) { x.in_order(f); });
}

int parts_of(int V) { return (int)(((int64_t)V + 7 + kPart - 1) / kPart); }

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

template <class T>
hipError_t run_sample(const void* logits, int64_t ld, const Request& q, int64_t B, int V,
                      int32_t* tokens, float* logprobs, void* scratch, uint32_t* err,
                      hipStream_t s) {
    const int parts = parts_of(V);
    double* sums = (double*)scratch;
    float* tops = (float*)((char*)scratch + up256((size_t)B * parts * sizeof(double)));
    sample_part_kernel<T><<<dim3(parts, (uint32_t)B), dim3(kPartThreads), 0, s>>>(
        (const T*)logits, ld, q, V, parts, tops, sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    sample_row_kernel<T><<<dim3((uint32_t)B), dim3(kRowThreads), 0, s>>>(
        (const T*)logits, ld, q, V, parts, tops, sums, tokens, logprobs, err);
    return hipGetLastError();
}

}  // namespace

size_t sample_scratch_bytes(int64_t B, int V) {
    const size_t n = (size_t)B * parts_of(V);
    return up256(n * sizeof(double)) + up256(n * sizeof(float));
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
