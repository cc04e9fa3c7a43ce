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

constexpr int kWaves = 4;  // waves of a workgroup

// LDS written by lanes of this wave is read by others of it afterwards (LDS
// accesses of a wave are performed in order; this keeps the compiler to it)
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// exp(x) for x <= 0 in 64 bits, to 3e-11 relative; below -700 it is 0.
// 2^t = 2^n * 2^f with n the nearest whole number and f in [-1/2, 1/2]; 2^f by
// its Taylor series in f ln 2 up to the 9th power (the rest is below
// (ln 2 / 2)^10 / 10! = 7e-12).
__device__ __forceinline__ double exp_neg(double x) {
    const double t = fmax(x, -700.0) * 1.4426950408889634074;
    const double n = __builtin_rint(t);
    const double f = (t - n) * 0.69314718055994530942;
    double p = 1.0 / 362880;
    p = __builtin_fma(p, f, 1.0 / 40320);
    p = __builtin_fma(p, f, 1.0 / 5040);
    p = __builtin_fma(p, f, 1.0 / 720);
    p = __builtin_fma(p, f, 1.0 / 120);
    p = __builtin_fma(p, f, 1.0 / 24);
    p = __builtin_fma(p, f, 1.0 / 6);
    p = __builtin_fma(p, f, 0.5);
    p = __builtin_fma(p, f, 1.0);
    p = __builtin_fma(p, f, 1.0);
    return ldexp(p, (int)n);
}

// What one wave finds in its part of a row of logits.
struct Partials {
    float* top;    // [parts] the part's largest logit; NaN: a NaN or +inf in it
    double* sum;   // [parts] sum exp(logit - top)
    float* value;  // [parts][W] its W largest logits, falling (-inf: none left)
    int32_t* index;  // [parts][W] their tokens
};

// The W best of a wave's values, key falling, then index rising: lane i < W
// returns the i-th in *out_key, *out_idx (key -inf where fewer are there; the
// index is then unspecified).  Each lane holds E keys in registers; a key of
// -inf is no candidate.  Indices are distinct.
//
// W groups of lanes each have a largest key, and the smallest of these W keys
// bounds the W-th best from below: usually only a few more than W keys reach
// it.  They are gathered in LDS (64 places a wave) and ranked by counting.
// Where more than 64 reach it (long runs of equal keys), W rounds each look
// for the best key behind the last one.
template <int E, class Key>
__device__ __forceinline__ void wave_top(const Key (&key)[E], const int32_t (&idx)[E], int W,
                                         int group_lanes, int lane, Key* lds_key, int32_t* lds_idx,
                                         Key* out_key, int32_t* out_idx) {
    const Key none = -INFINITY;
    Key t = none;
#pragma unroll
    for (int e = 0; e < E; ++e) t = key[e] > t ? key[e] : t;
    for (int o = 1; o < group_lanes; o <<= 1) {
        const Key x = __shfl_xor(t, o, 64);
        t = x > t ? x : t;
    }
    for (int o = group_lanes; o < 64; o <<= 1) {
        const Key x = __shfl_xor(t, o, 64);
        t = x < t ? x : t;
    }
    int count = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint64_t hit = __ballot(key[e] >= t && key[e] > none);
        if (hit) {
            const int at = count + __builtin_popcountll(hit & ((1ull << lane) - 1));
            if (((hit >> lane) & 1) && at < 64) {
                lds_key[at] = key[e];
                lds_idx[at] = idx[e];
            }
            count += __builtin_popcountll(hit);
        }
    }
    if (count <= 64) {
        wave_fence();
        const Key k = lane < count ? lds_key[lane] : none;
        const int32_t i = lane < count ? lds_idx[lane] : 0x7FFFFFFF;
        int rank = 0;
        for (int l = 0; l < count; ++l) {
            const Key ok = lds_key[l];
            const int32_t oi = lds_idx[l];
            rank += (ok > k || (ok == k && oi < i)) ? 1 : 0;
        }
        wave_fence();
        if (lane < count && rank < 64) {
            lds_key[rank] = k;
            lds_idx[rank] = i;
        }
        wave_fence();
        *out_key = lane < count ? lds_key[lane] : none;
        *out_idx = lane < count ? lds_idx[lane] : 0;
        wave_fence();
        return;
    }
    Key last = INFINITY;
    int32_t last_i = -1;
    *out_key = none;
    *out_idx = 0;
    for (int r = 0; r < W; ++r) {
        Key b = none;
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
            const Key xb = __shfl_xor(b, o, 64);
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

template <class T>
struct Logit;
template <>
struct Logit<float> {
    static constexpr int VEC = 4;
    __device__ static float get(const uint4& v, int e) {
        return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
    }
    __device__ static float one(const float* p) { return *p; }
};
template <>
struct Logit<uint16_t> {
    static constexpr int VEC = 8;
    __device__ static float get(const uint4& v, int e) {
        const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
        return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
    }
    __device__ static float one(const uint16_t* p) { return bf16_to_f32(*p); }
};

// One wave a part: E logits a lane, 16-byte pieces of 64 lanes in a row.  A row
// may start at any element: pieces are laid out from the 16-byte boundary
// before it, and a piece that reaches out of the row is read by elements.
template <class T, int E>
__global__ void __launch_bounds__(64 * kWaves) beam_part_kernel(
    const T* __restrict__ logits, int64_t ld, const float* __restrict__ cum,
    const uint8_t* __restrict__ finished, int W, int V, int parts, int group_lanes, Partials out,
    uint32_t* __restrict__ err) {
    constexpr int VEC = Logit<T>::VEC, NL = E / VEC;
    __shared__ float lds_key[kWaves][64];
    __shared__ int32_t lds_idx[kWaves][64];
    const int64_t row = blockIdx.y;
    if (finished && finished[row]) return;
    const float c = cum[row];
    if (!(c > -INFINITY && c < INFINITY)) return;  // offers nothing
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int part = blockIdx.x * kWaves + wave;
    const T* src = logits + row * ld;
    const int before = (int)(((uintptr_t)src & 15) / sizeof(T));  // elements after the boundary
    float v[E];
    int32_t idx[E];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int64_t e0 = ((int64_t)part * NL + i) * (64 * VEC) + lane * VEC - before;
        uint4 raw;
        const bool whole = e0 >= 0 && e0 + VEC <= V;
        if (whole) raw = *reinterpret_cast<const uint4*>(src + e0);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float x = -INFINITY;
            if (whole)
                x = Logit<T>::get(raw, e);
            else if (e0 + e >= 0 && e0 + e < V)
                x = Logit<T>::one(src + e0 + e);
            bad |= !(x < INFINITY);
            v[i * VEC + e] = x;
            idx[i * VEC + e] = (int32_t)(e0 + e);
        }
    }
    bad = __any(bad);
    if (bad && lane == 0 && err) atomicOr(err, ENGRAM_ERRBIT_LOGIT);
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, v[e]);
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    double s = 0.0;
    if (m > -INFINITY && !bad) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            s += v[e] > -INFINITY ? exp_neg((double)v[e] - (double)m) : 0.0;
    }
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
    const int64_t at = row * parts + part;
    if (lane == 0) {
        out.top[at] = bad ? __uint_as_float(0x7FC00000u) : m;
        out.sum[at] = s;
    }
    if (bad) return;
    float k;
    int32_t i;
    wave_top<E, float>(v, idx, W, group_lanes, lane, lds_key[wave], lds_idx[wave], &k, &i);
    if (lane < W) {
        out.value[at * W + lane] = k;
        out.index[at * W + lane] = i;
    }
}

// One workgroup a sequence: each beam's log sum, then the W best of all
// parts' candidates.
constexpr int kMaxBeams = 32;
constexpr int kJoin = 16;  // candidates a lane takes at a time

__global__ void __launch_bounds__(64 * kWaves) beam_join_kernel(
    const float* cum, const uint8_t* finished, int W, int V, int parts, int group_lanes,
    const Partials in, int32_t eos_id, int32_t pad_id, int32_t* __restrict__ tokens,
    int32_t* __restrict__ parents, float* new_cum, uint8_t* new_finished,
    uint32_t* __restrict__ err) {
    // score = own + ((logit - top) - low): the difference first, which keeps it
    // whole also where logits are masked by the type's lowest value
    __shared__ double low[kMaxBeams];  // log sum exp(logit - top); NaN: offers nothing
    __shared__ float top[kMaxBeams];
    __shared__ float own[kMaxBeams];
    __shared__ uint8_t done[kMaxBeams];
    __shared__ double lds_key[kWaves][64];
    __shared__ int32_t lds_idx[kWaves][64];
    __shared__ double win_key[kWaves][kMaxBeams];
    __shared__ int32_t win_idx[kWaves][kMaxBeams];
    const int64_t b = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const double none = -INFINITY;
    for (int w = wave; w < W; w += kWaves) {
        const int64_t row = b * W + w;
        const float c = cum[row];
        const bool fin = finished && finished[row];
        double lo = __longlong_as_double(0x7FF8000000000000ll);
        float m = -INFINITY;
        const bool live = c > -INFINITY && c < INFINITY;
        if (!live && !(c == -INFINITY) && lane == 0 && err) atomicOr(err, ENGRAM_ERRBIT_LOGIT);
        if (live && !fin) {
            bool bad = false;
            for (int p = lane; p < parts; p += 64) {
                const float t = in.top[row * parts + p];
                bad |= t != t;
                m = fmaxf(m, t);
            }
            for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x, 64));
            if (!__any(bad) && m > -INFINITY) {
                double s = 0.0;
                for (int p = lane; p < parts; p += 64) {
                    const float t = in.top[row * parts + p];
                    if (t > -INFINITY) s += in.sum[row * parts + p] * exp_neg((double)t - (double)m);
                }
                for (int x = 1; x < 64; x <<= 1) s += __shfl_xor(s, x, 64);
                lo = log(s);
            }
        }
        if (lane == 0) {
            low[w] = lo;
            top[w] = m;
            own[w] = c;
            done[w] = fin;
        }
    }
    __syncthreads();

    // each wave keeps its W best so far in its lanes and takes kJoin more
    // candidates a lane with them
    double best = none;
    int32_t best_i = 0;
    const uint32_t per_beam = (uint32_t)parts * W, total = per_beam * W;  // [beam][part][W]
    const float* values = in.value + b * total;
    const int32_t* indices = in.index + b * total;
    for (uint32_t c0 = wave * 64 * kJoin; c0 < total; c0 += kWaves * 64 * kJoin) {
        double key[kJoin + 1];
        int32_t idx[kJoin + 1];
#pragma unroll
        for (int e = 0; e < kJoin; ++e) {
            const uint32_t i = c0 + e * 64 + lane;
            key[e] = none;
            idx[e] = 0x7FFFFFFF - e * 64 - lane;
            if (i < total) {
                const int w = (int)(i / per_beam);
                const double lo = low[w];
                if (lo == lo) {
                    const float x = values[i];
                    if (x > -INFINITY) {
                        key[e] = (double)own[w] + (((double)x - (double)top[w]) - lo);
                        idx[e] = w * V + indices[i];
                    }
                }
            }
        }
        key[kJoin] = best;
        idx[kJoin] = best > none ? best_i : 0x7FFFFFFF - kJoin * 64 - lane;
        if (lane >= W) key[kJoin] = none;
        wave_top<kJoin + 1, double>(key, idx, W, group_lanes, lane, lds_key[wave], lds_idx[wave],
                                    &best, &best_i);
    }
    if (lane < W) {
        win_key[wave][lane] = best;
        win_idx[wave][lane] = best_i;
    }
    __syncthreads();
    if (wave != 0) return;
    // the waves' winners and the finished beams' one candidate each
    double key[3];
    int32_t idx[3];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = e * 64 + lane;  // [wave][W]
        key[e] = none;
        idx[e] = 0;
        if (i < kWaves * W) {
            key[e] = win_key[i / W][i % W];
            idx[e] = win_idx[i / W][i % W];
        }
    }
    key[2] = none;
    idx[2] = 0;
    if (lane < W && done[lane] && own[lane] > -INFINITY && own[lane] < INFINITY) {
        key[2] = own[lane];
        idx[2] = lane * V + pad_id;
    }
    wave_top<3, double>(key, idx, W, group_lanes, lane, lds_key[0], lds_idx[0], &best, &best_i);
    if (lane < W) {
        const int64_t row = b * W + lane;
        const bool some = best > none;
        const int parent = some ? best_i / V : lane;
        const int token = some ? best_i % V : pad_id;
        tokens[row] = token;
        parents[row] = parent;
        new_cum[row] = (float)best;
        if (new_finished) new_finished[row] = some && (done[parent] || token == eos_id);
    }
}

// Elements a lane holds (a part is 64 of these), by the rows there are: many
// rows fill the machine with long parts (fewer candidates to join), few rows
// are cut short so that one row spreads over many compute units.
int elements_of(int64_t rows, int V) {
    return rows * ((V + 8191) / 8192) >= 1024 ? 32 : 8;
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

Partials carve(int64_t rows, int W, int parts, void* scratch) {
    Partials p;
    char* at = (char*)scratch;
    const size_t n = (size_t)rows * parts;
    p.sum = (double*)at;
    at += up256(n * sizeof(double));
    p.top = (float*)at;
    at += up256(n * sizeof(float));
    p.value = (float*)at;
    at += up256(n * W * sizeof(float));
    p.index = (int32_t*)at;
    return p;
}

template <class T, int E>
void run_part(const T* logits, int64_t ld, const float* cum, const uint8_t* finished, int64_t rows,
              int W, int V, int parts, const Partials& p, uint32_t* err, hipStream_t s) {
    beam_part_kernel<T, E><<<dim3(parts / kWaves, (uint32_t)rows), dim3(64 * kWaves), 0, s>>>(
        logits, ld, cum, finished, W, V, parts, group_lanes_of(W), p, err);
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
// that change.  No other thread touches its column.
template <int UNIT, int WMAX>
__global__ void __launch_bounds__(256) beam_reorder_kernel(const ReorderArgs a,
                                                           const int32_t* __restrict__ parents,
                                                           int B, int W,
                                                           uint32_t* __restrict__ err) {
    typedef typename Column<UNIT>::type vec;
    int st = 0;
    while ((int64_t)blockIdx.x >= a.first[st + 1]) ++st;
    const int64_t words = a.words[st], cols = words / UNIT;
    const int64_t block = blockIdx.x - a.first[st];
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
        if (w < W && from[w] != w) base[w * cols] = v[w];
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
    if (a.first[a.n] > INT32_MAX) return hipErrorInvalidValue;
    auto k = W <= 4    ? beam_reorder_kernel<UNIT, 4>
             : W <= 8  ? beam_reorder_kernel<UNIT, 8>
             : W <= 16 ? beam_reorder_kernel<UNIT, 16>
                       : beam_reorder_kernel<UNIT, 32>;
    k<<<dim3((uint32_t)a.first[a.n]), dim3(256), 0, s>>>(a, parents, (int)B, W, err);
    return hipGetLastError();
}

}  // namespace

size_t beam_scratch_bytes(int64_t rows, int W, int V) {
    const size_t n = (size_t)rows * parts_of(rows, V);
    return up256(n * sizeof(double)) + up256(n * sizeof(float)) + 2 * up256(n * W * sizeof(float));
}

hipError_t launch_beam_select(const void* logits, bool f32, int64_t ld, const float* cum,
                              const uint8_t* finished, int64_t B, int W, int V, int32_t eos_id,
                              int32_t pad_id, int32_t* tokens, int32_t* parents, float* new_cum,
                              uint8_t* new_finished, void* scratch, uint32_t* err,
                              hipStream_t s) {
    const int64_t rows = B * W;
    const int parts = parts_of(rows, V);
    const bool wide = elements_of(rows, V) == 32;
    const Partials p = carve(rows, W, parts, scratch);
    if (f32) {
        auto f = wide ? run_part<float, 32> : run_part<float, 8>;
        f((const float*)logits, ld, cum, finished, rows, W, V, parts, p, err, s);
    } else {
        auto f = wide ? run_part<uint16_t, 32> : run_part<uint16_t, 8>;
        f((const uint16_t*)logits, ld, cum, finished, rows, W, V, parts, p, err, s);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    beam_join_kernel<<<dim3((uint32_t)B), dim3(64 * kWaves), 0, s>>>(
        cum, finished, W, V, parts, group_lanes_of(W), p, eos_id, pad_id, tokens, parents, new_cum,
        new_finished, err);
    return hipGetLastError();
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
