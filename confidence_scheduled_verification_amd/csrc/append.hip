// Appending a step's K and V rows to the paged cache.
//
// Row j of request r goes to position len[r] + j.  A page lies as blocks of 16 tokens, K
// as [D/8][16][8] (eight neighbouring dims of the 16 tokens together) and V as [D][16]
// (the 16 tokens of one dim together), the order in which attention's matrix instructions
// take their operands.
//
// A wave takes eight tokens and 64 dims at a time, 16 bytes of one token's row to a lane:
// eight rows of one whole line each are read, and K's bytes go to eight whole lines as they
// are.  V's eight by eight values are turned over between lanes in registers: token bits 2
// and 1 are lane bits 5 and 4, so two exchanges of half-waves (permlane32_swap) and of
// rows (permlane16_swap) put them into the word's number, and a neighbour's word
// (lane bit 0) gives the other half of each word.  The tokens of a block that the step does
// not fill are written one by one, so that what stands beside them is neither read nor
// written.  A page that another row holds too is not written to either.
//
// Its floor is the bytes, once read, once written.  1145 rows of 8 key heads of 128 (9.4 MB): 9.8
// us, which are the launch and loads that wait for each other (rows, page ids, counts, and behind
// them the data, which does not depend on the last two); eight prompts of 14351 rows (117 MB):
// 36 us, 3.3 TB/s, where a large copy reaches 5.5.  A wave to
// every (block, 64 dims) rather than a workgroup that walks the heads: 36 against 41 us.  V
// turned over through LDS instead of in registers: 82.
#include <algorithm>

#include "cache.h"
#include "common.h"

namespace dspark {

namespace {

constexpr int kT = 256;
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

__global__ __launch_bounds__(kT) void append_kernel(AppendArgs a) {
    const int r = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int o = a.offsets[r], o1 = a.offsets[r + 1], ln = a.len[r];
    const long long n = (long long)o1 - o + a.lead, start = (long long)o + (long long)a.lead * r;
    if (ln < 0) return;
    if (o < 0 || n < 0 || n > a.max_new || start + n > a.rows || (ln + n + a.page - 1) / a.page > a.width) {
        if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) raise_status(a.status, kStatusBadRow);
        return;
    }
    if (n == 0) return;  // (the block that the tokens kept end in is not this step's)
    const int shift = a.page_shift;
    const int row8 = (lane >> 5) * 4 + (lane >> 4 & 1) * 2 + (lane & 1);  // token of the eight; afterwards dim of the eight
    const int c8 = lane >> 1 & 7;                                        // eight dims of the 64
    const int items = a.Hkv * (a.D / 64);                                // (key head, 64 dims)
    const long long end = ln + n;
    for (long long pos = (ln & ~(kBlockTokens - 1)) + (long long)blockIdx.y * kBlockTokens; pos < end;
         pos += (long long)gridDim.y * kBlockTokens) {
        const int page = a.table[(size_t)r * a.width + (pos >> shift)];
        if (page < 0 || page >= a.n_pages || a.ref[page] > 1) {  // not there, or another row's too
            if (blockIdx.z == 0 && threadIdx.x == 0) raise_status(a.status, kStatusBadPage);
            continue;
        }
        const size_t block0 = ((size_t)page * a.Hkv << (shift - 4)) + ((pos & ((1 << shift) - 1)) >> 4);
        const int item = blockIdx.z * 4 + wave;
        if (item < items) {
            const int h = item / (a.D / 64), d0 = item % (a.D / 64) * 64;
            const size_t block = (block0 + ((size_t)h << (shift - 4))) * (size_t)(kBlockTokens * a.D);
            uint4 k[2], v[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const long long p = pos + half * 8 + row8;
                k[half] = v[half] = make_uint4(0, 0, 0, 0);
                if (p >= ln && p < end) {
                    const size_t row = (size_t)(start + p - ln), at = (size_t)h * a.D + d0 + c8 * 8;
                    k[half] = *(const uint4*)(a.k_new + row * a.k_stride + at);
                    v[half] = *(const uint4*)(a.v_new + row * a.v_stride + at);
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const long long p0 = pos + half * 8, p = p0 + row8;
                if (p0 + 8 <= ln || p0 >= end) continue;
                if (p >= ln && p < end)
                    *(uint4*)(a.k + block + (size_t)(d0 / 8 + c8) * (kBlockTokens * 8) + (half * 8 + row8) * 8) = k[half];
                const uint4 x = turned(v[half]);
                uint16_t* to = a.v + block + (size_t)(d0 + c8 * 8 + row8) * kBlockTokens + half * 8;
                if (p0 >= ln && p0 + 8 <= end) {
                    *(uint4*)to = x;
                } else {
                    const uint32_t* w = &x.x;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (p0 + j >= ln && p0 + j < end) to[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
                }
            }
        }
    }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, hipStream_t s) {
    // blocks that max_new tokens can touch, and a wave for every 64 dims of each
    const int blocks = (int)std::min((a.max_new + 2ll * (kBlockTokens - 1)) / kBlockTokens, 4096ll);
    const int items = a.Hkv * (a.D / 64);
    hipLaunchKernelGGL(append_kernel, dim3(a.R, blocks, (items + 3) / 4), dim3(kT), 0, s, a);
    return hipGetLastError();
}

}  // namespace dspark
