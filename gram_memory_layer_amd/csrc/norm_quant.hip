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
// h, the sum of squares, y and the scale are fp32; the norm is taken of h
// before it is rounded for `total` (one rounding for each output).
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

// y * inv as e4m3 codes, nearest even; |y * inv| <= 448 up to rounding, NaN
// and infinity give the NaN code 0x7F
__device__ __forceinline__ uint32_t e4m3_code(float v) {
    const uint32_t nan = !(__builtin_fabsf(v) < INFINITY);
    const float c = __builtin_fminf(__builtin_fmaxf(v, -448.0f), 448.0f);
    const uint32_t u = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, c, 0, false) & 0xFFu;
    return nan ? 0x7Fu : u;
}

// One workgroup a row; thread t holds the 8-value chunks t, t + nthr, ...
template <int NCH, int SC>
__global__ void __launch_bounds__(1024) norm_quant_kernel(
    const uint16_t* x, const uint16_t* res, const uint16_t* __restrict__ weight, int dim,
    float eps, uint16_t* total, uint8_t* __restrict__ codes, void* __restrict__ scales) {
    __shared__ float red[2][16];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, nthr = blockDim.x, d8 = dim / 8;
    const int lane = tid & 63, wave = tid >> 6, nw = nthr >> 6;
    float y[NCH][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = tid + i * nthr;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] = 0.0f;
        if (c < d8) {
            const uint4 h = *reinterpret_cast<const uint4*>(x + row * dim + c * 8);
            const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[i][2 * e] = lo_f(hw[e]);
                y[i][2 * e + 1] = hi_f(hw[e]);
            }
            if (res) {
                const uint4 r = *reinterpret_cast<const uint4*>(res + row * dim + c * 8);
                const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[i][2 * e] += lo_f(rw[e]);
                    y[i][2 * e + 1] += hi_f(rw[e]);
                }
            }
            if (total) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[e] = f32_to_bf16(y[i][2 * e]) | (f32_to_bf16(y[i][2 * e + 1]) << 16);
                *reinterpret_cast<uint4*>(total + row * dim + c * 8) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += y[i][e] * y[i][e];
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) ss += __shfl_xor(ss, o, 64);
    if (lane == 0) red[0][wave] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int w = 0; w < nw; ++w) ss += red[0][w];
    const float rstd = rsqrtf(ss / (float)dim + eps);

    float amax[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = tid + i * nthr;
        amax[i] = 0.0f;
        if (c < d8) {
            const uint4 w4 = weight ? *reinterpret_cast<const uint4*>(weight + c * 8)
                                    : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
            const uint32_t ww[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[i][2 * e] = y[i][2 * e] * rstd * lo_f(ww[e]);
                y[i][2 * e + 1] = y[i][2 * e + 1] * rstd * hi_f(ww[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) amax[i] = fmaxf(amax[i], fabsf(y[i][e]));
    }
    if constexpr (SC == SCALE_F32_ROW) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) t = fmaxf(t, amax[i]);
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) t = fmaxf(t, __shfl_xor(t, o, 64));
        if (lane == 0) red[1][wave] = t;
        __syncthreads();
        for (int w = 0; w < nw; ++w) t = fmaxf(t, red[1][w]);
#pragma unroll
        for (int i = 0; i < NCH; ++i) amax[i] = t;
    } else {
        // a group is 4 or 16 consecutive chunks, so as many consecutive lanes
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int o = 1; o < (SC == SCALE_E8M0_32 ? 4 : 16); o <<= 1)
                amax[i] = fmaxf(amax[i], __shfl_xor(amax[i], o, 64));
    }
    const int groups = SC == SCALE_E8M0_32 ? (dim + 31) / 32 : SC == SCALE_F32_128 ? (dim + 127) / 128 : 1;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = tid + i * nthr;
        if (c >= d8) continue;
        float inv, lift = 1.0f;
        if constexpr (SC == SCALE_E8M0_32) {
            const uint32_t code = e8m0_code(amax[i]);
            inv = e8m0_inverse(code);
            if (c % 4 == 0) ((uint8_t*)scales)[row * groups + c / 4] = (uint8_t)code;
        } else {
            // 448 / amax; a tiny maximum is lifted first, with its values (exact),
            // since its inverse would overflow
            lift = amax[i] < 0x1p-100f ? 0x1p100f : 1.0f;
            inv = amax[i] > 0.0f ? 448.0f / (amax[i] * lift) : 0.0f;
            const float sc = amax[i] / 448.0f;
            if (SC == SCALE_F32_128 ? c % 16 == 0 : c == 0)
                ((float*)scales)[row * groups + (SC == SCALE_F32_128 ? c / 16 : 0)] = sc;
        }
        uint32_t o[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e / 4] |= e4m3_code(y[i][e] * lift * inv) << (8 * (e % 4));
        *reinterpret_cast<uint2*>(codes + row * dim + c * 8) = make_uint2(o[0], o[1]);
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
    k<<<dim3((uint32_t)rows), dim3(nthr), 0, s>>>(x, res, weight, dim, eps, total, codes, scales);
    return hipGetLastError();
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
