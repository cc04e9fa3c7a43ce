// Sums over a wave's lanes by data-parallel moves (sampling, the sort by id).
#pragma once

#include "internal.h"

namespace engram {

// x of another lane, by a data-parallel move (0 where that gives none)
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t moved(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, true);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double moved(double x) {
    return __hiloint2double((int)moved<CTRL, ROWS>((uint32_t)__double2hiint(x)),
                            (int)moved<CTRL, ROWS>((uint32_t)__double2loint(x)));
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint64_t moved(uint64_t x) {
    return (uint64_t)moved<CTRL, ROWS>((uint32_t)(x >> 32)) << 32 | moved<CTRL, ROWS>((uint32_t)x);
}
// the sum of x up to and with each lane of the wave: shifts within rows of 16 lanes,
// then the rows' last lanes on to the rows behind them
template <class X>
__device__ __forceinline__ X sum_upto(X x) {
    x += moved<0x111>(x);
    x += moved<0x112>(x);
    x += moved<0x114>(x);
    x += moved<0x118>(x);
    x += moved<0x142, 0xA>(x);
    x += moved<0x143, 0xC>(x);
    return x;
}

}  // namespace engram
