// What the kernels that lay rows into pages share (append.hip, rotary.hip).
#pragma once

#include "cache.h"
#include "common.h"

namespace dspark {

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// Eight tokens of eight dims: in, token (bit 5, bit 4, bit 0 of the lane)'s dims 0..7; out,
// dim (the same bits)'s tokens 0..7.
__device__ __forceinline__ uint4 turned(uint4 x) {
    swap32(x.x, x.z);
    swap32(x.y, x.w);
    swap16(x.x, x.y);
    swap16(x.z, x.w);
    // this lane's half of each word and the neighbour's
    const uint32_t pick = threadIdx.x & 1 ? 0x03020706u : 0x05040100u;
    uint32_t* w = &x.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t other = __builtin_amdgcn_mov_dpp(w[i], 0xB1, 0xF, 0xF, true);  // lanes 1, 0, 3, 2
        w[i] = __builtin_amdgcn_perm(other, w[i], pick);
    }
    return x;
}

}  // namespace dspark
