// Beam search around the hash: the choice of the next tokens over beams and
// vocabulary, and the reordering of the carried states after it.
//
//   score(w, v) = cum[w] + logits[w][v] - log sum_v' exp(logits[w][v'])
//
// per sequence, and the W best (beam, token) pairs of the W * V, in order of
// falling score, ties to the lowest beam * V + token.
//
// The logits are read once.  Scores that lie next to each other decide which
// tokens come out, so the sums of exponentials, their logarithm and the
// scores are held in 64 bits.
#include "internal.h"

namespace engram {
namespace {

constexpr int kWaves = 4;  // waves of a workgroup that takes parts

// LDS written by lanes of this wave is read by others of it afterwards (LDS
// accesses of a wave are performed in order; this keeps the compiler to it)
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// exp(x) 2^-N in 64 bits, to 5e-11 relative, for -700 <= x - N ln 2 <= 1 and |x| <=
// 5000, with `round` = 1.5 * 2^52 - N; a NaN stays one.  2^t = 2^n * 2^f with n the
// nearest whole number, f in [-1/2, 1/2] and 2^f = 1 + f P(f), P of degree six with
// the least relative error (4.7e-11, by Remez' exchange).  Adding `round` rounds t
// to n and leaves n - N in the sum's low word, from where it goes into the
// exponent.
constexpr double kLog2e = 1.4426950408889634074, kLn2 = 0.69314718055994530942;
constexpr double kRound = 6755399441055744.0;
__device__ __forceinline__ double exp2_near(double x, double round) {
    const double r = __builtin_fma(x, kLog2e, round);
    const double f = __builtin_fma(x, kLog2e, -(r - round));
    double p = 1.5196156674707408e-05;
    p = __builtin_fma(p, f, 0.0001546675631744836);
    p = __builtin_fma(p, f, 0.0013333935054995816);
    p = __builtin_fma(p, f, 0.009618038132061645);
    p = __builtin_fma(p, f, 0.05550410365992162);
    p = __builtin_fma(p, f, 0.24022651066561068);
    p = __builtin_fma(p, f, 0.693147180704532);
    p = __builtin_fma(p, f, 1.0);
    return __hiloint2double(__double2hiint(p) + (__double2loint(r) << 20), __double2loint(p));
}

// exp(x) for any x <= 1: below -700 it is below 1e-304.
__device__ __forceinline__ double exp_neg(double x) { return exp2_near(fmax(x, -700.0), kRound); }

// What a sum of exponentials of logits up to `top` is relative to: 2^whole_of(top),
// a power of two next to exp(top), so that a logit's term has the same bits
// wherever its part begins and sums go from one power to another exactly; for
// tops too large for exp2_near, exp(top).
__device__ __forceinline__ bool has_whole(float top) { return fabsf(top) <= 4096.0f; }
__device__ __forceinline__ double whole_of(float top) { return rint((double)top * kLog2e); }
// its logarithm less top
__device__ __forceinline__ double base_over(float top) {
    return has_whole(top) ? __builtin_fma(whole_of(top), kLn2, -(double)top) : 0.0;
}
// a sum relative to `from`'s, relative to that of `to` >= from
__device__ __forceinline__ double rebase(double sum, float from, float to) {
    if (has_whole(from) && has_whole(to))
        return ldexp(sum, (int)(whole_of(from) - whole_of(to)));
    return sum * exp_neg(((double)from - (double)to) + (base_over(from) - base_over(to)));
}

// What one wave finds in its part of a row of logits.
struct Partials {
    double* sum;  // [parts] sum exp(logit), relative to top's power of two
    float* top;   // [parts] the part's largest logit; NaN: a NaN or +inf in it
};

// The W best of a wave's values, key falling, then index rising: lane i < W
// returns the i-th in *out_key, *out_idx (key -inf where fewer are there; the
// index is then unspecified).  Each lane holds E keys in registers; a key of
// -inf is no candidate.  Indices are distinct.
//
// W groups of lanes each have a largest key, and the smallest of these W keys
// bounds the W-th best from below: usually only a few more than W keys reach
// it.  They are gathered in LDS (64 places a wave), one a lane, and ranked by
// counting.  Where more than 64 reach it (long runs of equal keys), W rounds
// each look for the best key behind the last one.
template <int E>
__device__ __forceinline__ void wave_top(const double (&key)[E], const int32_t (&idx)[E], int W,
                                         int group_lanes, int lane, double* lds_key,
                                         int32_t* lds_idx, double* out_key, int32_t* out_idx) {
    const double none = -INFINITY;
    double t = none;
#pragma unroll
    for (int e = 0; e < E; ++e) t = key[e] > t ? key[e] : t;
    for (int o = 1; o < group_lanes; o <<= 1) {
        const double x = __shfl_xor(t, o, 64);
        t = x > t ? x : t;
    }
    for (int o = group_lanes; o < 64; o <<= 1) {
        const double x = __shfl_xor(t, o, 64);
        t = x < t ? x : t;
    }
    int count = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint64_t hit = __ballot(key[e] >= t && key[e] > none);
        const int at = count + __builtin_popcountll(hit & ((1ull << lane) - 1));
        if (((hit >> lane) & 1) && at < 64) {
            lds_key[at] = key[e];
            lds_idx[at] = idx[e];
        }
        count += __builtin_popcountll(hit);
    }
    wave_fence();
    if (count <= 64) {
        const double k = lane < count ? lds_key[lane] : none;
        const int32_t i = lane < count ? lds_idx[lane] : 0x7FFFFFFF;
        const int32_t hi = __double2hiint(k), lo = __double2loint(k);
        int rank = 0;
        for (int l = 0; l < count; ++l) {
            const double ok = __hiloint2double(__builtin_amdgcn_readlane(hi, l),
                                               __builtin_amdgcn_readlane(lo, l));
            const int32_t oi = __builtin_amdgcn_readlane(i, l);
            rank += (ok > k || (ok == k && oi < i)) ? 1 : 0;
        }
        wave_fence();
        if (lane < count) {
            lds_key[rank] = k;
            lds_idx[rank] = i;
        }
        wave_fence();
        *out_key = lane < count ? lds_key[lane] : none;
        *out_idx = lane < count ? lds_idx[lane] : 0;
        wave_fence();
        return;
    }
    double last = INFINITY;
    int32_t last_i = -1;
    *out_key = none;
    *out_idx = 0;
    for (int r = 0; r < W; ++r) {
        double b = none;
        int32_t bi = 0x7FFFFFFF;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const bool behind = key[e] < last || (key[e] == last && idx[e] > last_i);
            if (behind && (key[e] > b || (key[e] == b && idx[e] < bi))) {
                b = key[e];
                bi = idx[e];
            }
        }
        for (int o = 1; o < 64; o <<= 1) {
            const double xb = __shfl_xor(b, o, 64);
            const int32_t xi = __shfl_xor(bi, o, 64);
            if (xb > b || (xb == b && xi < bi)) {
                b = xb;
                bi = xi;
            }
        }
        if (!(b > none)) break;
        if (lane == r) {
            *out_key = b;
            *out_idx = bi;
        }
        last = b;
        last_i = bi;
    }
}

// A row of logits in 16-byte pieces.  It may start at any element: pieces are
// laid out from the 16-byte boundary before it, and a piece that reaches out
// of the row is read by elements (-inf outside).
template <class T>
struct Row {
    static constexpr int VEC = 16 / sizeof(T);
    const T* src;
    int before;  // elements between the boundary and the row

    __device__ explicit Row(const T* row)
        : src(row), before((int)(((uintptr_t)row & 15) / sizeof(T))) {}
    // the column of piece i's first element
    __device__ int64_t column(int64_t i) const { return i * VEC - before; }
    __device__ bool whole(int64_t i, int V) const {
        return column(i) >= 0 && column(i) + VEC <= V;
    }
    // in two steps, so that several pieces can be on their way
    __device__ uint4 fetch(int64_t i, int V) const {
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (whole(i, V)) raw = *reinterpret_cast<const uint4*>(src + column(i));
        return raw;
    }
    __device__ void values(const uint4& raw, float (&x)[VEC]) const {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if constexpr (sizeof(T) == 4)
                x[e] = __uint_as_float(w[e]);
            else
                x[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
        }
    }
    __device__ void unpack(const uint4& raw, int64_t i, int V, float (&x)[VEC]) const {
        values(raw, x);
        if (whole(i, V)) return;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int64_t c = column(i) + e;
            x[e] = -INFINITY;
            if (c >= 0 && c < V) {
                if constexpr (sizeof(T) == 4)
                    x[e] = src[c];
                else
                    x[e] = bf16_to_f32(src[c]);
            }
        }
    }
};

// One wave a part: 64 lanes of E logits, E / VEC pieces of 64 lanes.  (512 rows of
// 129,280: fp32 46-50 us, 5.3-5.8 TB/s, bound by memory; bf16 49 us, bound by the
// 64-bit instructions of the exponentials, 13 a logit.  Parts of twice the length,
// or a wave that goes through several with the next one's loads ahead, gain
// nothing: 55 and 57 us a bf16 call against 54.)
template <class T, int E>
__global__ void __launch_bounds__(64 * kWaves) beam_part_kernel(
    const T* __restrict__ logits, int64_t ld, const float* __restrict__ cum,
    const uint8_t* __restrict__ finished, int V, int parts, Partials out,
    uint32_t* __restrict__ err) {
    constexpr int VEC = Row<T>::VEC, NL = E / VEC;
    const int64_t row = blockIdx.y;
    // (both on their way at once)
    const uint8_t fin = finished ? finished[row] : 0;
    const float c = cum[row];
    if (fin || !(c > -INFINITY && c < INFINITY)) return;  // offers nothing
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = blockIdx.x * kWaves + wave;
    const Row<T> r(logits + row * ld);
    const int64_t first = (int64_t)part * NL * 64 + lane;
    float v[NL][VEC];
    if (r.column((int64_t)part * NL * 64) >= 0 && r.column((int64_t)(part + 1) * NL * 64) <= V) {
        // all of it inside the row
        const uint4* from = reinterpret_cast<const uint4*>(r.src + r.column(first));
        uint4 raw[NL];
#pragma unroll
        for (int i = 0; i < NL; ++i) raw[i] = from[64 * i];
#pragma unroll
        for (int i = 0; i < NL; ++i) r.values(raw[i], v[i]);
    } else {
        uint4 raw[NL];
#pragma unroll
        for (int i = 0; i < NL; ++i) raw[i] = r.fetch(first + 64 * i, V);
#pragma unroll
        for (int i = 0; i < NL; ++i) r.unpack(raw[i], first + 64 * i, V, v[i]);
    }
    float m = -INFINITY, least = INFINITY;  // (both pass a NaN over)
#pragma unroll
    for (int i = 0; i < NL; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            m = fmaxf(m, v[i][e]);
            least = fminf(least, v[i][e]);
        }
    float top = m;
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    double s = 0.0;
    bool bad = false;
    if (has_whole(top)) {
        const double round = kRound - whole_of(top);
        if (__all(least - top >= -600.0f)) {
            // the common case: nothing masked, nothing to clamp; a NaN comes through
#pragma unroll
            for (int i = 0; i < NL; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s += exp2_near((double)v[i][e], round);
            bad = s != s;
        } else {
#pragma unroll
            for (int i = 0; i < NL; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    bad |= !(v[i][e] < INFINITY);
                    s += exp2_near((double)fmaxf(v[i][e], top - 700.0f), round);
                }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NL; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                bad |= !(v[i][e] < INFINITY);
                if (top > -INFINITY) s += exp_neg((double)v[i][e] - (double)top);
            }
    }
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
    bad = __any(bad);
    if (lane == 0) {
        out.top[row * parts + part] = bad ? __uint_as_float(0x7FC00000u) : top;
        out.sum[row * parts + part] = s;
        if (bad && err) atomicOr(err, ENGRAM_ERRBIT_LOGIT);
    }
}

// One workgroup of 16 waves a sequence:
//  1. a wave a beam: its log sum, and the largest scores of at least W groups
//     of its parts;
//  2. the W-th largest of all groups' scores: at least W parts reach it, so
//     what the selection takes reaches it too (and little else does);
//  3. the parts that reach it, listed; where a long run of equal scores makes
//     that more than the list holds, exactly the W best parts instead (ties to
//     the lowest), in which the selection lies as well;
//  4. these parts' logits once more: what reaches the bound is gathered and
//     ranked by counting.
constexpr int kMaxBeams = 32;
constexpr int kJoinWaves = 16;
constexpr int kParts = 64;  // listed parts
constexpr int kList = 512;  // gathered candidates

template <class T, int E>
__global__ void __launch_bounds__(64 * kJoinWaves) beam_join_kernel(
    const T* __restrict__ logits, int64_t ld, const float* cum, const uint8_t* finished, int W,
    int V, int parts, int group_lanes, const Partials in, int32_t eos_id, int32_t pad_id,
    int32_t* __restrict__ tokens, int32_t* __restrict__ parents, float* new_cum,
    uint8_t* new_finished, uint32_t* __restrict__ err) {
    constexpr int VEC = Row<T>::VEC, NL = E / VEC, NT = 64 * kJoinWaves;
    // score = own + ((logit - top) - low): the difference first, which keeps it
    // whole also where logits are masked by the type's lowest value
    __shared__ double low[kMaxBeams];  // log sum exp(logit - top); NaN: offers nothing
    __shared__ float top[kMaxBeams], own[kMaxBeams];
    __shared__ uint8_t done[kMaxBeams];
    __shared__ double group_key[kJoinWaves * kMaxBeams], list_key[kList];
    __shared__ double win_key[kJoinWaves];
    __shared__ int32_t list_idx[kList], win_idx[kJoinWaves];
    __shared__ int32_t listed[kParts];  // parts as beam * parts + part
    __shared__ double reach;
    __shared__ int part_count, count;
    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const double none = -INFINITY;
    const float* tops = in.top + b * W * parts;
    const double* sums = in.sum + b * W * parts;
    if (tid == 0) count = part_count = 0;
    auto score_of = [](float c, float m, double lo, float x) {
        return (double)c + (((double)x - (double)m) - lo);
    };
    auto score = [&](int w, float x) { return score_of(own[w], top[w], low[w], x); };

    double group = none;  // the largest score of this lane's group of parts
    for (int w = wave; w < W; w += kJoinWaves) {
        // the first parts are on their way before it is known whether they count
        // (a dead or finished beam's are not written: they are not looked at)
        constexpr int AT = 4;
        float t[AT];
        double x[AT];
        auto load = [&](int p0) {
#pragma unroll
            for (int i = 0; i < AT; ++i) {
                const int p = p0 + 64 * i;
                t[i] = p < parts ? tops[w * parts + p] : -INFINITY;
                x[i] = p < parts ? sums[w * parts + p] : 0.0;
            }
        };
        load(lane);
        const float c = cum[b * W + w];
        const bool fin = finished && finished[b * W + w];
        const bool live = c > -INFINITY && c < INFINITY;
        double lo = __longlong_as_double(0x7FF8000000000000ll);
        float all = -INFINITY;
        if (live && !fin) {
            double s = 0.0;
            float m = -INFINITY;
            bool bad = false;
            for (int p0 = lane;;) {
                float nm = m;
#pragma unroll
                for (int i = 0; i < AT; ++i) {
                    bad |= t[i] != t[i];
                    nm = fmaxf(nm, t[i]);
                }
                if (m > -INFINITY) s = rebase(s, m, nm);
#pragma unroll
                for (int i = 0; i < AT; ++i)
                    if (t[i] > -INFINITY) s += rebase(x[i], t[i], nm);
                m = nm;
                p0 += 64 * AT;
                if (p0 - lane >= parts) break;
                load(p0);
            }
            all = m;
            for (int o = 1; o < 64; o <<= 1) all = fmaxf(all, __shfl_xor(all, o, 64));
            if (m > -INFINITY) s = rebase(s, m, all);
            for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
            if (!__any(bad) && all > -INFINITY) {
                // in steps of 2^-36: rows of the same logits that lie differently
                // are summed in another order, and are to tie all the same
                lo = rint((log(s) + base_over(all)) * 0x1p36) * 0x1p-36;
                if (m > -INFINITY) group = fmax(group, score_of(c, all, lo, m));
            }
        }
        if (lane == 0) {
            low[w] = lo;
            top[w] = all;
            own[w] = c;
            done[w] = fin;
            if (!live && c != -INFINITY && err) atomicOr(err, ENGRAM_ERRBIT_LOGIT);
        }
    }
    // (lanes equal modulo the groups of a wave, so that few parts spread over them)
    const int per_wave = 64 / group_lanes;
    for (int o = per_wave; o < 64; o <<= 1) group = fmax(group, __shfl_xor(group, o, 64));
    const int waves = W < kJoinWaves ? W : kJoinWaves;
    const int groups = waves * per_wave;
    if (lane < per_wave && wave < waves) group_key[wave * per_wave + lane] = group;
    __syncthreads();
    // (sixteen lanes count for one)
    const int one = tid >> 4, part16 = tid & 15;
    for (int i = one; i < groups; i += NT / 16) {
        const double k = group_key[i];
        int rank = 0;
#pragma unroll 8
        for (int l = part16; l < groups; l += 16) {
            const double x = group_key[l];
            rank += (x > k || (x == k && l < i)) ? 1 : 0;
        }
        for (int o = 1; o < 16; o <<= 1) rank += __shfl_xor(rank, o, 64);
        if (rank == W - 1) reach = k;  // -inf: fewer than W parts
    }
    __syncthreads();
    const double t = reach;
    for (int w = wave; w < W; w += kJoinWaves) {
        if (low[w] != low[w]) continue;
        for (int p = lane; p < parts; p += 64) {
            const float x = tops[w * parts + p];
            if (x > -INFINITY && score(w, x) >= t) {
                const int at = atomicAdd(&part_count, 1);
                if (at < kParts) listed[at] = w * parts + p;
            }
        }
    }
    __syncthreads();
    int n_listed = part_count;
    if (n_listed > kParts) {
        __syncthreads();  // everyone has seen the count
        if (wave == 0) {
            // the wave keeps its best so far in its lanes and takes four more a
            // lane with them
            constexpr int kTake = 4;
            double best = none;
            int32_t best_i = 0;
            for (int c0 = 0; c0 < W * parts; c0 += 64 * kTake) {
                double key[kTake + 1];
                int32_t idx[kTake + 1];
#pragma unroll
                for (int e = 0; e < kTake; ++e) {
                    idx[e] = c0 + e * 64 + lane;
                    key[e] = none;
                    if (idx[e] < W * parts) {
                        const float x = tops[idx[e]];
                        const int w = idx[e] / parts;
                        if (low[w] == low[w] && x > -INFINITY) key[e] = score(w, x);
                    }
                }
                key[kTake] = lane < W ? best : none;
                idx[kTake] = best_i;
                wave_top<kTake + 1>(key, idx, W, group_lanes, lane, list_key, list_idx, &best,
                                    &best_i);
            }
            if (lane < W) listed[lane] = best_i;  // (more than W parts reach the bound)
        }
        n_listed = W;
        __syncthreads();
    }

    // the listed parts' logits that may reach the bound, a wave a part:
    // f(score, beam * V + token).  Nearly all fail a comparison with the logit at
    // the bound, lowered by more than its roundings: 2^-22 for the one to fp32,
    // 2^-49 of every term for those in 64 bits, which are what counts where the
    // logits are near 0 and the terms cancel (a row of zeros).
    auto scan = [&](auto f) {
        for (int q = wave; q < n_listed; q += kJoinWaves) {
            const int at = __builtin_amdgcn_readfirstlane(listed[q]);
            const int w = at / parts;
            const int64_t first = (int64_t)(at - w * parts) * (NL * 64) + lane;
            const Row<T> r(logits + (b * W + w) * ld);
            uint4 raw[NL];
#pragma unroll
            for (int i = 0; i < NL; ++i) raw[i] = r.fetch(first + 64 * i, V);
            const float c = own[w], m = top[w];
            const double lo = low[w];
            const double at_t = (double)m + ((t - (double)c) + lo);
            const float edge = (float)(at_t - (fabs(at_t) + fabs((double)m)) * 0x1p-22 -
                                       (fabs(t) + fabs((double)c) + fabs(lo)) * 0x1p-49);
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                float x[VEC];
                r.unpack(raw[i], first + 64 * i, V, x);
                float most = x[0];
#pragma unroll
                for (int e = 1; e < VEC; ++e) most = fmaxf(most, x[e]);
                if (!(most >= edge)) continue;
                const int base = w * V + (int)r.column(first + 64 * i);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (x[e] >= edge && x[e] > -INFINITY) f(score_of(c, m, lo, x[e]), base + e);
            }
        }
        if (tid < W && done[tid] && own[tid] > -INFINITY && own[tid] < INFINITY)
            f((double)own[tid], tid * V + pad_id);  // a finished beam's one candidate
    };
    auto emit = [&](int slot, double key, int32_t i) {
        const int parent = i / V, token = i - parent * V;
        const int64_t row = b * W + slot;
        tokens[row] = token;
        parents[row] = parent;
        new_cum[row] = (float)key;
        if (new_finished) new_finished[row] = done[parent] || token == eos_id;
    };
    scan([&](double key, int32_t i) {
        if (key >= t) {
            const int at = atomicAdd(&count, 1);
            if (at < kList) {
                list_key[at] = key;
                list_idx[at] = i;
            }
        }
    });
    __syncthreads();
    int found = count;
    if (found <= kList) {
        // (the list's order is not the same on every run; the ranks are)
        for (int j = one; j < found; j += NT / 16) {
            const double k = list_key[j];
            const int32_t i = list_idx[j];
            int rank = 0;
#pragma unroll 4
            for (int l = part16; l < found; l += 16)
                rank += (list_key[l] > k || (list_key[l] == k && list_idx[l] < i)) ? 1 : 0;
            for (int o = 1; o < 16; o <<= 1) rank += __shfl_xor(rank, o, 64);
            if (part16 == 0 && rank < W) emit(rank, k, i);
        }
    } else {
        // long runs of equal scores: W rounds, each for the best behind the last
        double last = INFINITY;
        int32_t last_i = -1;
        found = W;
        for (int r = 0; r < W; ++r) {
            double k = none;
            int32_t ki = 0x7FFFFFFF;
            scan([&](double key, int32_t i) {
                if ((key < last || (key == last && i > last_i)) && (key > k || (key == k && i < ki))) {
                    k = key;
                    ki = i;
                }
            });
            for (int o = 1; o < 64; o <<= 1) {
                const double xk = __shfl_xor(k, o, 64);
                const int32_t xi = __shfl_xor(ki, o, 64);
                if (xk > k || (xk == k && xi < ki)) {
                    k = xk;
                    ki = xi;
                }
            }
            __syncthreads();  // the last round's winners are read
            if (lane == 0) {
                win_key[wave] = k;
                win_idx[wave] = ki;
            }
            __syncthreads();
            k = none;
            ki = 0x7FFFFFFF;
            for (int x = 0; x < kJoinWaves; ++x)
                if (win_key[x] > k || (win_key[x] == k && win_idx[x] < ki)) {
                    k = win_key[x];
                    ki = win_idx[x];
                }
            if (tid == 0) emit(r, k, ki);
            last = k;
            last_i = ki;
        }
    }
    if (tid >= found && tid < W) {  // fewer than W are offered
        const int64_t row = b * W + tid;
        tokens[row] = pad_id;
        parents[row] = tid;
        new_cum[row] = -INFINITY;
        if (new_finished) new_finished[row] = 0;
    }
}

// Elements a lane holds (a part is 64 of these), by the rows there are: many
// rows fill the machine with long parts (fewer partial sums to join), few rows
// are cut short so that one row spreads over many compute units.  (64 rows of
// 129,280 in bf16: 16 elements 15.0 us a call, 8 16.2; 512 rows: 32 elements 54,
// 8 65.)
int elements_of(int64_t rows, int V) {
    const int64_t n = rows * ((V + 8191) / 8192);
    return n >= 2048 ? 32 : n >= 256 ? 16 : 8;
}

int parts_of(int64_t rows, int V) {
    const int e = elements_of(rows, V);
    // rows start up to 7 elements after a 16-byte boundary
    return (int)(((int64_t)V + 7 + 64 * e * kWaves - 1) / (64 * e * kWaves)) * kWaves;
}

// lanes of each of at least W groups
int group_lanes_of(int W) {
    int lanes = 64;
    while (64 / lanes < W) lanes /= 2;
    return lanes;
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

template <class T, int E>
hipError_t run_select(const T* logits, int64_t ld, const float* cum, const uint8_t* finished,
                      int64_t B, int W, int V, int parts, const Partials& p, int32_t eos_id,
                      int32_t pad_id, int32_t* tokens, int32_t* parents, float* new_cum,
                      uint8_t* new_finished, uint32_t* err, hipStream_t s) {
    beam_part_kernel<T, E><<<dim3(parts / kWaves, (uint32_t)(B * W)), dim3(64 * kWaves), 0, s>>>(
        logits, ld, cum, finished, V, parts, p, err);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    beam_join_kernel<T, E><<<dim3((uint32_t)B), dim3(64 * kJoinWaves), 0, s>>>(
        logits, ld, cum, finished, W, V, parts, group_lanes_of(W), p, eos_id, pad_id, tokens,
        parents, new_cum, new_finished, err);
    return hipGetLastError();
}

// ---------------------------------------------------------------- reordering
// A workgroup's 256 threads take 256 columns (units of 4, 8 or 16 bytes) of one
// state: of one sequence where a row has more than 128 columns, otherwise
// columns of consecutive sequences.
struct ReorderArgs {
    uint32_t* base[kMaxStates];
    int64_t words[kMaxStates];         // 4-byte words of a row
    int64_t first[kMaxStates + 1];     // first workgroup of each state
    int32_t per_seq[kMaxStates];       // workgroups a sequence (0: sequences share them)
    int64_t start;                     // first workgroup of this launch
    int n;
};

template <int UNIT>
struct Column;
template <>
struct Column<1> {
    typedef uint32_t type;
};
template <>
struct Column<2> {
    typedef uint32_t type __attribute__((ext_vector_type(2)));
};
template <>
struct Column<4> {
    typedef uint32_t type __attribute__((ext_vector_type(4)));
};

// state[b][w] = state[b][parents[b][w]], in place: a thread owns one column of
// all W rows of a sequence, reads every row's parent, then writes the rows
// that change.  No other thread touches its column.  Memory bounds it (two states
// of 8 x 8 rows of 4 MiB: 151 us, 5.3 TB/s read and written); stores with the
// nontemporal hint (64 x 8 rows of 40 KiB, 8 states: 52.8 -> 43.0 us).  Loading
// only the rows that move, behind a branch each, serialises the loads and
// doubles the time.
template <int UNIT, int WMAX>
__global__ void __launch_bounds__(256) beam_reorder_kernel(const ReorderArgs a,
                                                           const int32_t* __restrict__ parents,
                                                           int B, int W,
                                                           uint32_t* __restrict__ err) {
    typedef typename Column<UNIT>::type vec;
    const int64_t at = a.start + blockIdx.x;
    int st = 0;
    while (at >= a.first[st + 1]) ++st;
    const int64_t words = a.words[st], cols = words / UNIT;
    const int64_t block = at - a.first[st];
    int64_t col;
    int b;
    if (a.per_seq[st]) {
        b = (int)(block / a.per_seq[st]);
        col = (block - (int64_t)b * a.per_seq[st]) * 256 + threadIdx.x;
        if (col >= cols) return;
    } else {  // at most 65535 * 128 columns in all
        const uint32_t item = (uint32_t)block * 256 + threadIdx.x;
        b = (int)(item / (uint32_t)cols);
        col = item - (uint32_t)b * (uint32_t)cols;
        if (b >= B) return;
    }
    const int32_t* par = parents + (int64_t)b * W;
    vec* base = reinterpret_cast<vec*>(a.base[st] + b * W * words) + col;
    vec v[WMAX];
    int32_t from[WMAX];
    bool bad = false;
#pragma unroll
    for (int w = 0; w < WMAX; ++w) {
        // (slots behind the last beam read that beam's row again and write none)
        const int own = w < W ? w : W - 1;
        const int32_t p = par[own];
        const bool in = p >= 0 && p < W;
        bad |= !in;
        from[w] = in ? p : own;
        v[w] = base[from[w] * cols];
    }
#pragma unroll
    for (int w = 0; w < WMAX; ++w)
        if (w < W && from[w] != w) __builtin_nontemporal_store(v[w], base + w * cols);
    if (bad && err && st == 0 && col == 0) atomicOr(err, ENGRAM_ERRBIT_PARENT);
}

template <int UNIT>
hipError_t run_reorder(ReorderArgs& a, const int32_t* parents, int64_t B, int W, uint32_t* err,
                       hipStream_t s) {
    a.first[0] = 0;
    for (int i = 0; i < a.n; ++i) {
        const int64_t cols = a.words[i] / UNIT;
        a.per_seq[i] = cols > 128 ? (int32_t)((cols + 255) / 256) : 0;
        a.first[i + 1] = a.first[i] + (cols > 128 ? B * a.per_seq[i] : (B * cols + 255) / 256);
    }
    auto k = W <= 4    ? beam_reorder_kernel<UNIT, 4>
             : W <= 8  ? beam_reorder_kernel<UNIT, 8>
             : W <= 16 ? beam_reorder_kernel<UNIT, 16>
                       : beam_reorder_kernel<UNIT, 32>;
    constexpr int64_t most = ((int64_t)1 << 31) / 256;  // a launch has fewer than 2^32 threads
    for (a.start = 0; a.start < a.first[a.n]; a.start += most) {
        const int64_t blocks = a.first[a.n] - a.start < most ? a.first[a.n] - a.start : most;
        k<<<dim3((uint32_t)blocks), dim3(256), 0, s>>>(a, parents, (int)B, W, err);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t beam_scratch_bytes(int64_t rows, int W, int V) {
    const size_t n = (size_t)rows * parts_of(rows, V);
    return up256(n * sizeof(double)) + up256(n * sizeof(float));
}

hipError_t launch_beam_select(const void* logits, bool f32, int64_t ld, const float* cum,
                              const uint8_t* finished, int64_t B, int W, int V, int32_t eos_id,
                              int32_t pad_id, int32_t* tokens, int32_t* parents, float* new_cum,
                              uint8_t* new_finished, void* scratch, uint32_t* err,
                              hipStream_t s) {
    const int64_t rows = B * W;
    const int parts = parts_of(rows, V);
    const int each = elements_of(rows, V);
    Partials p;
    p.sum = (double*)scratch;
    p.top = (float*)((char*)scratch + up256((size_t)rows * parts * sizeof(double)));
    auto go = [&](auto run, auto* x) {
        return run(x, ld, cum, finished, B, W, V, parts, p, eos_id, pad_id, tokens, parents,
                   new_cum, new_finished, err, s);
    };
    if (f32)
        return go(each == 32   ? run_select<float, 32>
                  : each == 16 ? run_select<float, 16>
                               : run_select<float, 8>,
                  (const float*)logits);
    return go(each == 32   ? run_select<uint16_t, 32>
              : each == 16 ? run_select<uint16_t, 16>
                           : run_select<uint16_t, 8>,
              (const uint16_t*)logits);
}

hipError_t launch_beam_reorder(void* const* states, const int64_t* row_bytes, int n,
                               const int32_t* parents, int64_t B, int W, uint32_t* err,
                               hipStream_t s) {
    ReorderArgs a;
    a.n = n;
    uintptr_t low = 0;  // the rows' and the pointers' common alignment
    for (int i = 0; i < n; ++i) {
        a.base[i] = (uint32_t*)states[i];
        a.words[i] = row_bytes[i] / 4;
        low |= (uintptr_t)states[i] | (uintptr_t)row_bytes[i];
    }
    if (low % 16 == 0) return run_reorder<4>(a, parents, B, W, err, s);
    if (low % 8 == 0) return run_reorder<2>(a, parents, B, W, err, s);
    return run_reorder<1>(a, parents, B, W, err, s);
}

}  // namespace engram
