// Appending a step's K and V rows to the paged cache.
//
// Row j of request r goes to position len[r] + j.  A page lies as blocks of 16 tokens, K
// as [D/8][16][8] (eight neighbouring dims of the 16 tokens together) and V as [D][16]
// (the 16 tokens of one dim together), the order in which attention's matrix instructions
// take their operands.  One thread takes eight dims of one block's tokens: it reads 16
// bytes of each row, which lie in one line with its neighbours', keeps K as it is and
// transposes V in registers.  A block that the step fills is written 16 bytes at a time,
// 256 bytes of K and 256 of V to a thread; the tokens of a partly filled one are written
// one by one, so that what stands beside them is neither read nor written.
#include "cache.h"
#include "common.h"

namespace dspark {

namespace {

constexpr int kT = 256;

__global__ __launch_bounds__(kT) void append_kernel(AppendArgs a) {
    const int r = blockIdx.x;
    const int o = a.offsets[r];
    const long long n = (long long)a.offsets[r + 1] - o + a.lead;
    const long long start = (long long)o + (long long)a.lead * r;
    const int ln = a.len[r];
    if (ln < 0) return;
    if (o < 0 || n < 0 || n > a.max_new || start + n > a.rows ||
        (ln + n + a.page - 1) / a.page > a.width) {
        if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) raise_status(a.status, kStatusBadRow);
        return;
    }
    const int chunks = a.D / 8;
    const int item = blockIdx.z * kT + threadIdx.x;  // (key head, chunk of eight dims)
    if (item >= a.Hkv * chunks) return;
    const int h = item / chunks, c = item % chunks;
    const long long p0 = ln & ~(kBlockTokens - 1);
    for (long long blk = blockIdx.y;; blk += gridDim.y) {
        const long long pos = p0 + blk * kBlockTokens;
        if (pos >= ln + n) return;
        const int lo = pos < ln ? (int)(ln - pos) : 0;
        const int hi = ln + n - pos < kBlockTokens ? (int)(ln + n - pos) : kBlockTokens;
        const int page = a.table[(size_t)r * a.width + pos / a.page];
        if (page < 0 || page >= a.n_pages) {
            raise_status(a.status, kStatusBadPage);
            continue;
        }
        const size_t block = ((size_t)page * a.Hkv + h) * (a.page / kBlockTokens) + (size_t)(pos % a.page) / kBlockTokens;
        uint16_t* kd = a.k + (block * chunks + c) * (kBlockTokens * 8);
        uint16_t* vd = a.v + (block * a.D + c * 8) * kBlockTokens;
        const uint16_t* ks = a.k_new + (start + pos - ln) * a.k_stride + (size_t)h * a.D + c * 8;
        const uint16_t* vs = a.v_new + (start + pos - ln) * a.v_stride + (size_t)h * a.D + c * 8;
        if (lo == 0 && hi == kBlockTokens) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint4 kr[8], vr[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    kr[j] = *(const uint4*)(ks + (half * 8 + j) * a.k_stride);
                    vr[j] = *(const uint4*)(vs + (half * 8 + j) * a.v_stride);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) *(uint4*)(kd + (half * 8 + j) * 8) = kr[j];
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t x = (&vr[2 * j].x)[d / 2], y = (&vr[2 * j + 1].x)[d / 2];
                        w[j] = d & 1 ? (x >> 16) | (y & 0xFFFF0000u) : (x & 0xFFFFu) | (y << 16);
                    }
                    *(uint4*)(vd + d * kBlockTokens + half * 8) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        } else {
            for (int j = lo; j < hi; ++j) {
                const uint4 x = *(const uint4*)(ks + j * a.k_stride);
                const uint4 y = *(const uint4*)(vs + j * a.v_stride);
                *(uint4*)(kd + j * 8) = x;
#pragma unroll
                for (int d = 0; d < 8; ++d) vd[d * kBlockTokens + j] = (uint16_t)((&y.x)[d / 2] >> (16 * (d & 1)));
            }
        }
    }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, hipStream_t s) {
    const int blocks = (a.max_new + 2 * (kBlockTokens - 1)) / kBlockTokens;  // blocks that max_new tokens can touch
    const int items = a.Hkv * (a.D / 8);
    hipLaunchKernelGGL(append_kernel, dim3(a.R, blocks < 1024 ? blocks : 1024, (items + kT - 1) / kT), dim3(kT), 0, s,
                       a);
    return hipGetLastError();
}

}  // namespace dspark
