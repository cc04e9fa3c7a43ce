// Root-mean-square norm of a residual stream with the residual's addition and
// an 8-bit output, for the fp8 product that follows a layer:
//
//   h = x + r,  total = bf16(h),  y = h * rsqrt(mean(h^2) + eps) * weight,
//   per group of 32 or 128 values, or per row:  amax = max |y|,
//   e8m0 (groups of 32): scale = the smallest 2^(c-127), c >= 0, with
//     amax <= 448 * scale (the embedding table's own format);
//   fp32 (groups of 128, or the row): scale = amax / 448;
//   code = e4m3(y / scale), round to nearest even.
//
// h, the squares, y and the scale are fp32, in the order written; the norm is
// taken of h before it is rounded for `total` (one rounding for each output).  An e8m0 scale is a step of
// two: where fp32's roundings could decide it, 64 bits do.
#include "internal.h"

namespace engram {
namespace {

__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

enum { SCALE_E8M0_32 = 0, SCALE_F32_128 = 1, SCALE_F32_ROW = 2 };

// the smallest e8m0 code c with amax <= 448 * 2^(c-127); 448 = 1.75 * 2^8.
// Zero takes 0.  (A subnormal amax is below 448 * 2^-127: code 0 holds it.)
__device__ __forceinline__ uint32_t e8m0_code(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127;
    const int k = (b & 0x7FFFFFu) > 0x600000u ? e - 7 : e - 8;  // amax = 1.m * 2^e
    return (uint32_t)max(k + 127, 0);
}

// 2^(127-c): the inverse of code c's scale (c is at most 247)
__device__ __forceinline__ float e8m0_inverse(uint32_t c) {
    return __uint_as_float((254u - c) << 23);
}

// Four values as e4m3 codes, nearest even.  |v| is at most 448 up to rounding, or
// a NaN or an infinity, which the convert makes a NaN code of either sign: 0x7F
// here, by clearing the sign of every byte whose other bits are all set.
__device__ __forceinline__ uint32_t e4m3_codes(float a, float b, float c, float d) {
    uint32_t o = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    o = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, (int)o, true);
    return o & ~(((o & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
    const bf16x2_t v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

constexpr uint32_t kNear = 24;  // fp32 steps from an e8m0 step that 64 bits decide

// One workgroup a row; thread t holds the 8-value chunks t, t + nthr, ... from
// the loads to the codes, so every byte is moved once: memory bounds it (16384
// rows of 5120 with a residual, 587 MB: 100 us, 5.9 TB/s), next to the vector
// instructions, about ten a value.  y is formed in the formula's order, so that
// nothing leaves fp32's range that y does not leave, and y / scale is that
// quotient, rounded as a division rounds it: a product with the inverse and a
// correction, two more instructions a value (a power of two needs neither).  In
// another order, or with the inverse alone, one of 10^4 values gets another
// code: bf16 products put that many quotients halfway between two codes.  The
// outputs are stored with the nontemporal hint (4096 rows: 32.2 -> 25.4 us); the
// same hint on the loads, and a wave a row instead of a workgroup (no barrier,
// ten chunks a lane: 160 us), were slower.
template <int NCH, int SC>
__global__ void __launch_bounds__(1024) norm_quant_kernel(
    const uint16_t* x, const uint16_t* res, const uint16_t* __restrict__ weight, int dim,
    float eps, uint16_t* total, uint8_t* __restrict__ codes, void* __restrict__ scales,
    int64_t row0, double per_dim, int kept) {
    extern __shared__ u32x4 keep[];  // [dim / 8] of the input that total replaces
    __shared__ double sums[16];
    __shared__ float tops[16];
    const int tid = threadIdx.x, nthr = blockDim.x, d8 = dim / 8;
    const int lane = tid & 63, wave = tid >> 6, nw = nthr >> 6;
    const int64_t row = row0 + blockIdx.x;
    u32x4 hx[NCH], hr[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = tid + i * nthr;
        hx[i] = hr[i] = u32x4{0, 0, 0, 0};
        if (c < d8) {
            hx[i] = *reinterpret_cast<const u32x4*>(x + row * dim + c * 8);
            if (res) hr[i] = *reinterpret_cast<const u32x4*>(res + row * dim + c * 8);
            if (kept) keep[c] = kept & 1 ? hx[i] : hr[i];
        }
    }
    float y[NCH][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = tid + i * nthr;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[i][2 * e] = lo_f(hx[i][e]);
            y[i][2 * e + 1] = hi_f(hx[i][e]);
        }
        if (res)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[i][2 * e] += lo_f(hr[i][e]);
                y[i][2 * e + 1] += hi_f(hr[i][e]);
            }
        if (total && c < d8) {
            u32x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = pack2_bf16(y[i][2 * e], y[i][2 * e + 1]);
            __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(total + row * dim + c * 8));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += y[i][e] * y[i][e];
    }
    u32x4 ww[NCH];
    if (weight)
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = tid + i * nthr;
            ww[i] = u32x4{0, 0, 0, 0};
            if (c < d8) ww[i] = *reinterpret_cast<const u32x4*>(weight + c * 8);
        }
    // (the threads' sums meet in 64 bits)
    double all = ss;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) all += __shfl_xor(all, o, 64);
    if (lane == 0) sums[wave] = all;
    __syncthreads();
    all = 0;
    for (int w = 0; w < nw; ++w) all += sums[w];
    const double var = all * per_dim + (double)eps;
    // rounded once: a step of Newton's from the approximate root, in 64 bits
    float rstd = rsqrtf((float)var);
    const bool usual = rstd > 0.0f && rstd < INFINITY;  // no NaN or infinity in h, not all 0 / 0
    if (usual) rstd = (float)(rstd * (1.5 - 0.5 * var * rstd * rstd));

    // y and its largest magnitude (a group's, or the row's; a NaN is passed over)
    float amax[NCH], top = 0.0f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] *= rstd;
        if (weight)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[i][2 * e] *= lo_f(ww[i][e]);
                y[i][2 * e + 1] *= hi_f(ww[i][e]);
            }
        amax[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax[i] = fmaxf(amax[i], fabsf(y[i][e]));
        if (!usual)  // a NaN here is h's: its group's scale is one too (below)
#pragma unroll
            for (int e = 0; e < 8; ++e) amax[i] = y[i][e] == y[i][e] ? amax[i] : INFINITY;
        // a group is 4 or 16 consecutive chunks, so as many consecutive lanes
        if constexpr (SC != SCALE_F32_ROW)
#pragma unroll
            for (int o = 1; o < (SC == SCALE_E8M0_32 ? 4 : 16); o <<= 1)
                amax[i] = fmaxf(amax[i], __shfl_xor(amax[i], o, 64));
        top = fmaxf(top, amax[i]);
    }
    if constexpr (SC == SCALE_F32_ROW) {
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
        if (lane == 0) tops[wave] = top;
        __syncthreads();
        for (int w = 0; w < nw; ++w) top = fmaxf(top, tops[w]);
    }

    const int groups = SC == SCALE_E8M0_32 ? (dim + 31) / 32 : SC == SCALE_F32_128 ? (dim + 127) / 128 : 1;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = tid + i * nthr;
        const bool there = c < d8;  // (lanes past a short group's end go along)
        float most = SC == SCALE_F32_ROW ? top : amax[i];
        if (!usual) most *= 0.0f;  // (an infinity: NaN)
        if constexpr (SC == SCALE_E8M0_32) {
            uint32_t code = e8m0_code(most);
            // A maximum near 448 times a power of two: which side of it, in 64 bits, the
            // row's squares too (a wave with such a group sums them once more).  fp32
            // has the mean within 34 * 2^-24 (a thread's 32 squares, h's rounding) and
            // the maximum within 21 * 2^-24: 19 of its steps here.
            const uint32_t bits = __float_as_uint(most);
            const bool near = (bits & 0x7FFFFFu) - (0x600000u - kNear) <= 2 * kNear;
            if (__any(near)) {
                // x and the residual once more, from LDS where total is in their place
                auto wide_h = [&](int at, double (&hh)[8]) {
                    u32x4 rr = {0, 0, 0, 0};
                    const u32x4 xx = kept & 1 ? keep[at] : *reinterpret_cast<const u32x4*>(x + row * dim + at * 8);
                    if (kept & 2)
                        rr = keep[at];
                    else if (res)
                        rr = *reinterpret_cast<const u32x4*>(res + row * dim + at * 8);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        hh[2 * e] = (double)lo_f(xx[e]) + (double)lo_f(rr[e]);
                        hh[2 * e + 1] = (double)hi_f(xx[e]) + (double)hi_f(rr[e]);
                    }
                };
                double hh[8], squares = 0.0, wide = 0.0;
#pragma unroll 1
                for (int at = lane; at < d8; at += 64) {
                    wide_h(at, hh);
#pragma unroll
                    for (int e = 0; e < 8; ++e) squares += hh[e] * hh[e];
                }
#pragma unroll
                for (int o = 32; o >= 1; o >>= 1) squares += __shfl_xor(squares, o, 64);
                if (there) {
                    wide_h(c, hh);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const double lo = weight ? (double)lo_f(ww[i][e]) : 1.0;
                        const double hi = weight ? (double)hi_f(ww[i][e]) : 1.0;
                        wide = fmax(wide, fmax(fabs(hh[2 * e] * lo), fabs(hh[2 * e + 1] * hi)));
                    }
                }
                wide = fmax(wide, __shfl_xor(wide, 1, 64));
                wide = fmax(wide, __shfl_xor(wide, 2, 64));
                const uint32_t edge = (bits & 0xFF800000u) | 0x600000u;
                const double lim = (double)__uint_as_float(edge);
                const bool in = wide * wide <= lim * lim * (squares / dim + (double)eps);
                if (near) code = e8m0_code(__uint_as_float(in ? edge : edge + 1));
            }
            const float inverse = e8m0_inverse(code);
            if (there && c % 4 == 0)
                ((uint8_t*)scales)[row * groups + c / 4] = (uint8_t)(most == most ? code : 255u);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][e] *= inverse;
        } else {
            const float scale = most / 448.0f;
            if (there && (SC == SCALE_F32_128 ? c % 16 == 0 : c == 0))
                ((float*)scales)[row * groups + (SC == SCALE_F32_128 ? c / 16 : 0)] = scale;
            if (most >= 0x1p-100f || !(most > 0.0f)) {
                // y / scale as a product with the inverse and one correction (by zeros
                // where there is no scale: a finite y becomes 0)
                const bool some = most > 0.0f && most < INFINITY;
                const float by = some ? scale : 0.0f;
                float inverse = __builtin_amdgcn_rcpf(scale);
                inverse = some ? __builtin_fmaf(__builtin_fmaf(-scale, inverse, 1.0f), inverse, inverse) : 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float q = y[i][e] * inverse;
                    y[i][e] = __builtin_fmaf(__builtin_fmaf(-q, by, y[i][e]), inverse, q);
                }
            } else {
                // the scale may be subnormal, and by rounding short of most / 448
                const float by = scale * 0x1p100f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float q = by > 0.0f ? y[i][e] * 0x1p100f / by : y[i][e] * 0.0f;
                    y[i][e] = q > 448.0f ? 448.0f : q < -448.0f ? -448.0f : q;
                }
            }
        }
        const u32x2 o = {e4m3_codes(y[i][0], y[i][1], y[i][2], y[i][3]),
                         e4m3_codes(y[i][4], y[i][5], y[i][6], y[i][7])};
        if (there) __builtin_nontemporal_store(o, reinterpret_cast<u32x2*>(codes + row * dim + c * 8));
    }
}

template <int SC>
hipError_t run(const uint16_t* x, const uint16_t* res, const uint16_t* weight, int64_t rows,
               int dim, float eps, uint16_t* total, uint8_t* codes, void* scales, hipStream_t s) {
    const int d8 = dim / 8;
    // up to 4 chunks a thread: dim 32768 is 1024 threads of 4
    const int nch = d8 <= 256 ? 1 : d8 <= 2048 ? 2 : 4;
    const int nthr = ((d8 + nch - 1) / nch + 63) / 64 * 64;
    auto k = nch == 1   ? norm_quant_kernel<1, SC>
             : nch == 2 ? norm_quant_kernel<2, SC>
                        : norm_quant_kernel<4, SC>;
    const int kept = SC != SCALE_E8M0_32 || !total ? 0 : (total == x ? 1 : 0) | (total == res ? 2 : 0);
    const int64_t most = ((int64_t)1 << 31) / nthr;  // a launch has fewer than 2^32 threads
    for (int64_t r0 = 0; r0 < rows; r0 += most) {
        const int64_t n = rows - r0 < most ? rows - r0 : most;
        k<<<dim3((uint32_t)n), dim3(nthr), kept ? dim * 2 : 0, s>>>(x, res, weight, dim, eps, total, codes, scales,
                                                   r0, 1.0 / dim, kept);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_norm_quant(const uint16_t* x, const uint16_t* res, const uint16_t* weight,
                             int64_t rows, int dim, float eps, int scale_format, uint16_t* total,
                             uint8_t* codes, void* scales, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    auto f = scale_format == SCALE_E8M0_32   ? run<SCALE_E8M0_32>
             : scale_format == SCALE_F32_128 ? run<SCALE_F32_128>
                                             : run<SCALE_F32_ROW>;
    return f(x, res, weight, rows, dim, eps, total, codes, scales, s);
}

}  // namespace engram
