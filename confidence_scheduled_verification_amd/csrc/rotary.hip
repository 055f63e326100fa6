// A step's queries and keys turned to their positions, and its keys and values laid into the
// pages (append.hip says how a page lies).
//
// A pair of dims turns by position * frequency.  Positions are whole numbers and whole turns
// say nothing, so the angle is one 64-bit product of the position and the frequency in turns
// as a fraction of 2^64, whose overflow is what would be taken off anyway: the top 32 bits
// are the angle to 2^-32 turns at every position, where a product in fp32 is off by up to 2^-8
// radians at 131072, half a step of bf16.  Sines come from it in fp32.
//
// A workgroup takes the 16 tokens of a block of positions and one of three kinds of work: 64 dims
// of V to a wave, turned over between lanes as in append.hip; some heads of K; or some heads of Q.
// It computes the sines of its tokens once, into LDS, for all of its heads.  Of K and Q a lane takes
// both pieces of eight dims that a pair lies in (in halves; interleaved, two neighbouring ones),
// for K eight tokens side by side, whose pieces make a line of the page, for Q the pieces of a head.
#include <algorithm>

#include "append_dev.h"
#include "tree.h"

namespace dspark {

namespace {

constexpr int kT = 256;
constexpr int kHeads = 16;  // of Q or K, to a workgroup

struct RBf16 {
    static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
    static __device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
};
struct RF16 {
    static __device__ __forceinline__ float half(uint32_t h) { return (float)__builtin_bit_cast(_Float16, (uint16_t)h); }
    static __device__ __forceinline__ float lo(uint32_t w) { return half(w & 0xFFFFu); }
    static __device__ __forceinline__ float hi(uint32_t w) { return half(w >> 16); }
    static __device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
};

// A pair's two values turned by (cosine, sine); the one rounding of each to 16 bits.
template <class E>
__device__ __forceinline__ void turn(float x, float y, float2 cs, uint32_t& a, uint32_t& b) {
    a = E::bits(x * cs.x - y * cs.y);
    b = E::bits(x * cs.y + y * cs.x);
}

// Two pieces of eight dims: in halves, dim i of x pairs with dim i of y (cs[0..7]); interleaved, each
// piece's neighbours pair (x: cs[0..3], y: cs[4..7]).
template <class E>
__device__ __forceinline__ void turn_pieces(uint4& x, uint4& y, const float2* cs, bool interleaved) {
    uint32_t *p = &x.x, *q = &y.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a, b, c, d;
        if (interleaved) {
            turn<E>(E::lo(p[i]), E::hi(p[i]), cs[i], a, b);
            turn<E>(E::lo(q[i]), E::hi(q[i]), cs[4 + i], c, d);
            p[i] = a | b << 16;
            q[i] = c | d << 16;
        } else {
            turn<E>(E::lo(p[i]), E::lo(q[i]), cs[2 * i], a, c);
            turn<E>(E::hi(p[i]), E::hi(q[i]), cs[2 * i + 1], b, d);
            p[i] = a | b << 16;
            q[i] = c | d << 16;
        }
    }
}

// Where item e of a head's D / 16 lies: its two pieces of eight dims, and whether they turn.
struct Pieces {
    int x, y;
    bool turns;
};
__device__ __forceinline__ Pieces pieces(const RotaryArgs& a, int e) {
    const int first = a.first >> 3, n = a.dim >> 4;  // items that turn
    if (e < n) return a.interleaved ? Pieces{first + 2 * e, first + 2 * e + 1, true} : Pieces{first + e, first + n + e, true};
    const int u = 2 * (e - n), v = u + 1;  // pieces that pass, counted without those that turn
    return Pieces{u < first ? u : u + 2 * n, v < first ? v : v + 2 * n, false};
}

template <class E>
__global__ __launch_bounds__(kT) void append_rotary_kernel(RotaryArgs g, int v_parts, int k_parts) {
    extern __shared__ __attribute__((aligned(16))) float2 s_cs[];  // [16][dim / 2]
    const AppendArgs& a = g.a;
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int o = a.offsets[r], o1 = a.offsets[r + 1], ln = a.len[r];
    const long long n = (long long)o1 - o + a.lead, start = (long long)o + (long long)a.lead * r;
    if (ln < 0) return;
    if (o < 0 || n < 0 || n > a.max_new || start + n > a.rows || (ln + n + a.page - 1) / a.page > a.width) {
        if (blockIdx.y == 0 && blockIdx.z == 0 && tid == 0) raise_status(a.status, kStatusBadRow);
        return;
    }
    if (n == 0) return;
    const int shift = a.page_shift, part = blockIdx.z, D = a.D, items = D / 16, pairs = g.dim / 2;
    const bool is_v = part < v_parts, is_k = !is_v && part < v_parts + k_parts;
    const long long end = ln + n;
    for (long long pos = (ln & ~(kBlockTokens - 1)) + (long long)blockIdx.y * kBlockTokens; pos < end;
         pos += (long long)gridDim.y * kBlockTokens) {
        size_t block0 = 0;  // the block in the page's first head
        if (is_v || is_k) {
            const int page = a.table[(size_t)r * a.width + (pos >> shift)];
            if (page < 0 || page >= a.n_pages || a.ref[page] > 1) {  // not there, or another row's too
                if (part == 0 && tid == 0) raise_status(a.status, kStatusBadPage);
                continue;
            }
            block0 = ((size_t)page * a.Hkv << (shift - 4)) + ((pos & ((1 << shift) - 1)) >> 4);
        }
        if (is_v) {
            const int row8 = (lane >> 5) * 4 + (lane >> 4 & 1) * 2 + (lane & 1);  // token of the eight; afterwards dim of the eight
            const int c8 = lane >> 1 & 7, item = part * 4 + wave;                // eight dims of the 64
            if (item >= a.Hkv * (D / 64)) continue;
            const int h = item / (D / 64), d0 = item % (D / 64) * 64;
            const size_t block = (block0 + ((size_t)h << (shift - 4))) * (size_t)(kBlockTokens * D);
            uint4 v[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const long long p = pos + half * 8 + row8;
                v[half] = make_uint4(0, 0, 0, 0);
                if (p >= ln && p < end)
                    v[half] = *(const uint4*)(a.v_new + (size_t)(start + p - ln) * a.v_stride + (size_t)h * D + d0 + c8 * 8);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const long long p0 = pos + half * 8;
                if (p0 + 8 <= ln || p0 >= end) continue;
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
            continue;
        }
        // Tokens [t0, t1) of the block are the step's; their rows begin at row0 + t0.
        const int t0 = (int)max(ln - pos, 0ll), t1 = (int)min(end - pos, (long long)kBlockTokens);
        const long long row0 = start + pos - ln;
        __syncthreads();  // the last block's sines have been read
        for (int i = tid; i < (t1 - t0) * pairs; i += kT) {
            const int t = t0 + i / pairs, f = i % pairs;
            const long long at = g.depth ? (long long)ln + g.depth[row0 + t] : pos + t;
            const int32_t angle = (int32_t)(((uint64_t)at * g.turns[f]) >> 32);  // of 2^32 a turn
            float s, c;
            sincospif((float)angle * 0x1p-31f, &s, &c);
            s_cs[t * pairs + f] = make_float2(c * g.attention, s * g.attention);
        }
        __syncthreads();
        const int h0 = (is_k ? part - v_parts : part - v_parts - k_parts) * kHeads;
        const int heads = min(kHeads, (is_k ? a.Hkv : g.H) - h0);
        const int tokens = t1 - t0;
        for (int i = tid; i < tokens * heads * items; i += kT) {
            int t, e, h;
            if (is_k) {
                t = t0 + i % tokens;
                e = i / tokens % items;
                h = h0 + i / tokens / items;
            } else {
                e = i % items;
                h = h0 + i / items % heads;
                t = t0 + i / items / heads;
            }
            const Pieces p = pieces(g, e);
            const size_t row = (size_t)(row0 + t);
            const uint16_t* from = (is_k ? a.k_new + row * a.k_stride : g.q + row * g.q_stride) + (size_t)h * D;
            uint4 x = *(const uint4*)(from + p.x * 8), y = *(const uint4*)(from + p.y * 8);
            if (p.turns) turn_pieces<E>(x, y, s_cs + t * pairs + e * 8, g.interleaved);
            if (is_k) {
                uint16_t* to = a.k + (block0 + ((size_t)h << (shift - 4))) * (size_t)(kBlockTokens * D) + t * 8;
                *(uint4*)(to + p.x * (kBlockTokens * 8)) = x;
                *(uint4*)(to + p.y * (kBlockTokens * 8)) = y;
            } else {
                uint16_t* to = g.q_out + row * g.q_out_stride + (size_t)h * D;
                *(uint4*)(to + p.x * 8) = x;
                *(uint4*)(to + p.y * 8) = y;
            }
        }
    }
}

}  // namespace

hipError_t launch_append_rotary(const RotaryArgs& g, hipStream_t s) {
    // blocks that max_new tokens can touch
    const int blocks = (int)std::min((g.a.max_new + 2ll * (kBlockTokens - 1)) / kBlockTokens, 4096ll);
    const int v_parts = (g.a.Hkv * (g.a.D / 64) + 3) / 4, k_parts = (g.a.Hkv + kHeads - 1) / kHeads;
    const dim3 grid(g.a.R, blocks, v_parts + k_parts + (g.H + kHeads - 1) / kHeads);
    const size_t lds = kBlockTokens * (g.dim / 2) * sizeof(float2);
    if (g.dtype == DSPARK_F16)
        hipLaunchKernelGGL(append_rotary_kernel<RF16>, grid, dim3(kT), lds, s, g, v_parts, k_parts);
    else
        hipLaunchKernelGGL(append_rotary_kernel<RBf16>, grid, dim3(kT), lds, s, g, v_parts, k_parts);
    return hipGetLastError();
}

}  // namespace dspark
