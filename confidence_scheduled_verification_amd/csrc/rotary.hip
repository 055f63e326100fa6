// A step's queries and keys turned to their positions, and its keys and values laid into the
// pages (append.hip says how a page lies).
//
// A pair of dims turns by position * frequency.  Positions are whole numbers and whole turns
// say nothing, so the angle is one 64-bit product of the position and the frequency in turns
// as a fraction of 2^64, whose overflow is what would be taken off anyway: the top 32 bits
// are the angle to 2^-32 turns at every position, where a product in fp32 is off by up to 2^-8
// radians at 131072, half a step of bf16.  Sines come from it in fp32.
//
// A workgroup takes one of three kinds of work: 16 tokens of a block of positions and 64 dims of V to
// a wave, turned over between lanes as in append.hip; the block's K of a few heads; or the Q of up to
// eight rows.  Of K and Q a lane takes one token and the two pieces of eight dims that hold both of a
// pair (in halves; interleaved, two neighbours), and a few heads one after the other with the same
// sines, the next one's loads under way.  Eight tokens stand side by side in a wave, so that their
// pieces make a line of the page; of rows that are fewer, more heads.  The workgroup computes its
// tokens' sines once, into LDS, while the first loads are under way.  Where no request has more than eight
// rows, they are one such set for K and V too, whichever one or two blocks they go to: by blocks most
// workgroups would have few rows or none.
//
// Bytes bound it, once read, once written.  The workgroups that share rows are neighbours in the grid:
// 14351 fp16 rows of 32 query and 8 key heads of 128 (353 MB) take 76 us a call (4.6 TB/s; a large copy
// reaches 4.9); when it was tried, 108 where a kind's workgroups follow each other through all rows, against 78.
// 1152 rows of 64 and 8 heads (47 MB), of requests of up to eight: 18.5 us a call, 19.0 in a graph (21.6 by
// blocks), of which 6 are the launch and the loads that wait for each other; a copy of as many bytes takes 10,
// for which the waves would have to be resident at once.  An earlier form of both took 78 and 21 us; with eight heads
// a lane instead of two 92 and 22 (fewer waves), one head 22; a request's blocks walked in a loop in place of a
// workgroup each: 97 and 28 (twice the registers, half the waves).
#include <algorithm>

#include "append_dev.h"
#include "tree.h"

namespace dspark {

namespace {

constexpr int kT = 256;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4), may_alias));
constexpr int kPasses = 2;  // heads that a lane takes

struct RBf16 {
    typedef __bf16 two __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
    static __device__ __forceinline__ uint32_t bits(float x, float y) { return __builtin_bit_cast(uint32_t, two{(__bf16)x, (__bf16)y}); }
};
struct RF16 {
    typedef _Float16 two __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(two, w)[0]; }
    static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(two, w)[1]; }
    static __device__ __forceinline__ uint32_t bits(float x, float y) { return __builtin_bit_cast(uint32_t, two{(_Float16)x, (_Float16)y}); }
};

// Two pieces of eight dims turned by cs = (cosine, sine): in halves, dim i of x pairs with dim i of y;
// interleaved, each piece's neighbours pair (x: cs[0..3], y: cs[4..7]).  Each value is rounded to 16 bits once.
template <class E, bool kInterleaved>
__device__ __forceinline__ void turn_pieces(uint4& x, uint4& y, const float2 (&cs)[8]) {
    uint32_t *p = &x.x, *q = &y.x;
    const auto a = [](float x, float y, float2 cs) { return x * cs.x - y * cs.y; };
    const auto b = [](float x, float y, float2 cs) { return x * cs.y + y * cs.x; };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __builtin_amdgcn_sched_barrier(0);  // (all at once would take twice the registers)
        const float x0 = E::lo(p[i]), x1 = E::hi(p[i]), y0 = E::lo(q[i]), y1 = E::hi(q[i]);
        if (kInterleaved) {
            p[i] = E::bits(a(x0, x1, cs[i]), b(x0, x1, cs[i]));
            q[i] = E::bits(a(y0, y1, cs[4 + i]), b(y0, y1, cs[4 + i]));
        } else {
            p[i] = E::bits(a(x0, y0, cs[2 * i]), a(x1, y1, cs[2 * i + 1]));
            q[i] = E::bits(b(x0, y0, cs[2 * i]), b(x1, y1, cs[2 * i + 1]));
        }
    }
}

__device__ __forceinline__ uint4 once(const uint16_t* p) {  // read once
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load((const u32x4*)p));
}

// (cosine, sine) of 2 pi times the 32-bit fraction of a turn, to 2^-23: the nearest quarter taken off, the
// series of both on what is left, |x| <= pi / 4, where the first terms left out are 2e-9 and 3e-8.
__device__ __forceinline__ float2 cos_sin(uint32_t angle, float m) {
    const uint32_t quarter = angle + 0x20000000u;
    const float x = (float)(int32_t)(angle - (quarter & 0xC0000000u)) * 0x1.921fb6p-30f, y = x * x;
    const float s = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
    const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, 1.f / 40320, -1.f / 720), 1.f / 24), -.5f), 1.f);
    const bool odd = quarter & 0x40000000u;
    return make_float2(m * __uint_as_float(__float_as_uint(odd ? s : c) ^ ((quarter + 0x40000000u) & 0x80000000u)),
                       m * __uint_as_float(__float_as_uint(odd ? c : s) ^ (quarter & 0x80000000u)));
}

struct Split {  // of the work on a block of 16 tokens (few: on all) among workgroups
    int shift_t;           // Q (few: K too): 1 << shift_t tokens side by side in a wave
    int q_halves;          // Q: 1 where the other half of the block has workgroups of its own
    int v_parts, k_parts;  // Q has the rest of the grid
    long long first_block;
};

template <class E, bool kInterleaved, bool kFew>
__global__ __launch_bounds__(kT, 8) void append_rotary_kernel(RotaryArgs g, Split sp) {
    extern __shared__ __attribute__((aligned(16))) float2 s_cs[];  // [tokens][dim / 2]
    const AppendArgs& a = g.a;
    const int r = blockIdx.z, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int o = a.offsets[r], o1 = a.offsets[r + 1], ln = a.len[r], shift = a.page_shift;
    const long long rows = (long long)o1 - o + a.lead, start = (long long)o + (long long)a.lead * r;
    if (ln < 0) return;
    if (o < 0 || rows < 0 || rows > a.max_new || start + rows > a.rows || (ln + rows + (1 << shift) - 1) >> shift > a.width) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) raise_status(a.status, kStatusBadRow);
        return;
    }
    const int n = (int)rows, row0 = (int)start, D = a.D;
    const int part = blockIdx.x;
    const bool is_q = part >= sp.v_parts + sp.k_parts, is_v = part < sp.v_parts;
    const int q_part = part - sp.v_parts - sp.k_parts, unit = (is_q ? q_part >> sp.q_halves : is_v ? part : part - sp.v_parts) * 4 + wave;
    // Rows j0 .. of the request: of a block of positions (V, K), or from the first row on (Q).
    const int ahead = ln & (kBlockTokens - 1);  // tokens in front of the first one in its block
    const long long block = sp.first_block + blockIdx.y, j64 = kFew ? 0 : block * kBlockTokens - (is_q ? -((q_part & sp.q_halves) * 8) : ahead);
    if (n == 0 || j64 >= n) return;  // (with n = 0 the block that the kept tokens end in is not this step's)
    const int j0 = (int)j64;
    // The block of row j's position, in its page's first head; -1 where there is no page to write to.
    const auto block_of = [&](int j) -> long long {
        const long long pos = (long long)ln + j;
        const int page = a.table[(size_t)r * a.width + (pos >> shift)];
        if (page < 0 || page >= a.n_pages || a.ref[page] > 1) {  // not there, or another row's too
            if (part == 0 && tid == 0) raise_status(a.status, kStatusBadPage);
            return -1;
        }
        return ((long long)page * a.Hkv << (shift - 4)) + ((int)(pos & ((1 << shift) - 1)) >> 4);
    };
    long long block0 = 0, block1 = 0;  // block1: of the rows behind the first block (few)
    if (!is_q) {
        block0 = block1 = block_of(j0);
        if (kFew && ahead + n > kBlockTokens) block1 = block_of(n - 1);
        if (block0 < 0 && block1 < 0) return;
    }
    if (is_v) {
        const int row8 = (lane >> 5) * 4 + (lane >> 4 & 1) * 2 + (lane & 1);  // token of the eight; afterwards dim of the eight
        const int c8 = lane >> 1 & 7, shift_h = __builtin_ctz(D >> 6);       // eight dims of the 64
        const int h = unit >> shift_h, d0 = (unit & ((D >> 6) - 1)) * 64;
        if (h >= a.Hkv) return;
        const size_t head = (size_t)h << (shift - 4), in = (size_t)(d0 + c8 * 8 + row8) * kBlockTokens;
        if (kFew) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row8 < n) v = once(a.v_new + (size_t)(row0 + row8) * a.v_stride + h * D + d0 + c8 * 8);
            const uint4 x = turned(v);
            const uint32_t* w = &x.x;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const long long b = ahead + i < kBlockTokens ? block0 : block1;
                if (i < n && b >= 0)
                    a.v[((size_t)b + head) * (size_t)(kBlockTokens * D) + in + (ahead + i) % kBlockTokens] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            }
            return;
        }
        uint16_t* block = a.v + ((size_t)block0 + head) * (size_t)(kBlockTokens * D) + in;
        uint4 v[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int j = j0 + half * 8 + row8;
            v[half] = make_uint4(0, 0, 0, 0);
            if (j >= 0 && j < n) v[half] = once(a.v_new + (size_t)(row0 + j) * a.v_stride + h * D + d0 + c8 * 8);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int j = j0 + half * 8;
            if (j + 8 <= 0 || j >= n) continue;
            const uint4 x = turned(v[half]);
            uint16_t* to = block + half * 8;
            if (j >= 0 && j + 8 <= n) {
                *(uint4*)to = x;
            } else {
                const uint32_t* w = &x.x;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (j + i >= 0 && j + i < n) to[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            }
        }
        return;
    }
    // A lane's token, its item of a head (two pieces of eight dims) and its heads.
    const int items = D >> 4, shift_items = __builtin_ctz(items), shift_side = 6 - (is_q || kFew ? sp.shift_t : 3);
    const int halves = is_q || kFew ? 0 : 1, strips = max(shift_items - shift_side, 0), step = 1 << max(shift_side - shift_items, 0);
    const int slot = (lane & ((1 << shift_side) - 1)) + ((unit >> halves & ((1 << strips) - 1)) << shift_side);
    const int e = slot & (items - 1), h0 = (unit >> (halves + strips)) * kPasses * step + (slot >> shift_items);
    const int t = (halves ? (unit & 1) * 8 : 0) + (lane >> shift_side), j = j0 + t;
    int left = min(h0 + kPasses * step, is_q ? g.H : a.Hkv) - h0;  // while > 0
    if (j < 0 || j >= n) left = 0;
    const long long to_block = kFew && ahead + j >= kBlockTokens ? block1 : block0;
    if (kFew && to_block < 0) left = 0;
    // Its two pieces: a pair's, in halves, or two neighbours; behind those that turn, the others.
    const int first = g.first >> 3, turning = g.dim >> 4, pass = 2 * (e - turning);
    const bool turns = e < turning;
    const int px = turns ? first + (kInterleaved ? 2 * e : e) : pass < first ? pass : pass + 2 * turning;
    const int py = turns ? px + (kInterleaved ? 1 : turning) : pass + 1 < first ? pass + 1 : pass + 1 + 2 * turning;
    const size_t row = (size_t)(row0 + j);
    const uint16_t* from = (is_q ? g.q + row * g.q_stride : a.k_new + row * a.k_stride) + h0 * D + px * 8;
    const int from_y = (py - px) * 8;
    uint4 x, y;
    if (left > 0) {
        x = once(from);
        y = once(from + from_y);
    }
    const int pairs = g.dim >> 1;
    for (int i = wave; i < (is_q || kFew ? 1 << sp.shift_t : kBlockTokens); i += kT / 64) {
        if (j0 + i < 0 || j0 + i >= n) continue;
        const long long at = ln + (long long)(g.depth ? g.depth[row0 + j0 + i] : j0 + i);
        for (int f = lane; f < pairs; f += 64)
            s_cs[i * pairs + f] = cos_sin((uint32_t)(((uint64_t)at * g.turns[f]) >> 32), g.attention);
    }
    __syncthreads();
    float2 cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = s_cs[t * pairs + (turns ? e : 0) * 8 + i];
    const int to_piece = is_q ? 8 : kBlockTokens * 8, to_y = (py - px) * to_piece;
    const size_t to_step = is_q ? step * D : (size_t)(step * D) << shift;
    uint16_t* to = (is_q ? g.q_out + row * g.q_out_stride + h0 * D
                         : a.k + (size_t)to_block * (kBlockTokens * D) + ((size_t)(h0 * D) << shift) + (kFew ? (ahead + j) % kBlockTokens : t) * 8) + px * to_piece;
#pragma unroll 1
    while (left > 0) {
        uint4 u = x, v = y;
        left -= step;
        from += step * D;
        if (left > 0) {
            x = once(from);
            y = once(from + from_y);
        }
        if (turns) turn_pieces<E, kInterleaved>(u, v, cs);
        *(uint4*)to = u;
        *(uint4*)(to + to_y) = v;
        to += to_step;
    }
}

}  // namespace

hipError_t launch_append_rotary(const RotaryArgs& g, hipStream_t s) {
    const int items = g.a.D / 16;
    Split sp;
    sp.shift_t = g.a.max_new > 4 ? 3 : g.a.max_new > 2 ? 2 : g.a.max_new > 1 ? 1 : 0;
    sp.q_halves = g.a.max_new > 8;
    const auto parts = [&](int side, int heads, int halves) {  // `side` items side by side in a wave
        const int strips = std::max(items / side, 1), at_once = std::max(side / items, 1) * kPasses;
        return ((heads + at_once - 1) / at_once * strips * halves + 3) / 4;
    };
    sp.v_parts = (g.a.Hkv * (g.a.D / 64) + 3) / 4;
    // Up to eight rows stand side by side whatever the blocks they go to; more are taken by blocks, whose
    // rows of V are then written whole.
    const bool few = g.a.max_new <= 8;
    sp.k_parts = few ? parts(64 >> sp.shift_t, g.a.Hkv, 1) : parts(8, g.a.Hkv, 2);
    const int all = sp.v_parts + sp.k_parts + (parts(64 >> sp.shift_t, g.H, 1) << sp.q_halves);
    const long long blocks = few ? 1 : (std::min(g.a.max_new, g.a.rows) + 2ll * (kBlockTokens - 1)) / kBlockTokens;  // that the tokens can touch
    const size_t lds = (few ? 1 << sp.shift_t : kBlockTokens) * (g.dim / 2) * sizeof(float2);
    const auto pick = [&](auto e) {
        typedef decltype(e) E;
        return g.interleaved ? few ? append_rotary_kernel<E, true, true> : append_rotary_kernel<E, true, false>
               : few         ? append_rotary_kernel<E, false, true>
                             : append_rotary_kernel<E, false, false>;
    };
    const auto kernel = g.dtype == DSPARK_F16 ? pick(RF16{}) : pick(RBf16{});
    for (sp.first_block = 0; sp.first_block < blocks; sp.first_block += 65535)
        hipLaunchKernelGGL(kernel, dim3(all, (unsigned)std::min(blocks - sp.first_block, 65535ll), g.a.R), dim3(kT), lds, s, g, sp);
    return hipGetLastError();
}

}  // namespace dspark
