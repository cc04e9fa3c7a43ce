// What the kernels that read rows of logits share: beam search's selection and
// sampling.
#pragma once

#include "internal.h"

namespace engram {

// LDS written by lanes of this wave is read by others of it afterwards (LDS
// accesses of a wave are performed in order; this keeps the compiler to it)
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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

}  // namespace engram
