// Attention of a step's packed rows over the paged cache.
//
// out = softmax(scale q K^T) V for each (row, query head), in one pass over the keys with
// the running maximum and sum of the softmax.  A tile is 32 query rows (row, head of the
// group that shares a key head); a wave takes 32 keys at a time and computes the scores
// transposed, S^T = K Q^T, so that a query is a column: one lane and the one 32 lanes on
// hold a column's 32 scores, its maximum and sum need one exchange, and the column's
// weights are the second product's operand as they stand, O^T += V^T P^T.  For that the
// keys of a block of 16 enter the first product with bits 2 and 3 of their number
// swapped: the accumulator's rows 8a + 4h + b of lane half h are then the keys 8h + 4a + b
// that the second product's operand wants there.  Both operands of the cache are read
// from memory in the order in which they lie (a block's K as [D/8][16][8], its V as
// [D][16]), so neither passes through LDS.
//
// Work: the keys are cut into units of 128 (four waves of 32).  Every workgroup takes the
// same number of consecutive units, in the order request, key head, tile, unit, so few
// long contexts and many short ones fill the device alike; a segment (request, key head,
// tile) that ends inside one workgroup is finished there, and the parts of one that is
// split are joined by a second kernel.  A shared prefix is a first launch of the same
// kernel, whose segments are a group's rows taken together and whose keys are read once a
// tile of 32 of them; the requests' own segments then add its part as they end.
//
// Masks: only blocks that reach past a column's last key are masked.  What lies in masked
// places has no say whatever it is: scores are replaced, V past the end is cleared, and a
// value of V that is not a number in such a block is taken out of the product and handed
// to the columns that see it by counting (see add_special).
#include <algorithm>

#include "cache.h"
#include "common.h"

namespace dspark {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kT = 256;
constexpr float kInf = __builtin_huge_valf();

struct Bf16 {
    static constexpr uint32_t kExp = 0x7F80u, kMant = 0x007Fu, kOne = 0x3F80u;
    static __device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint16_t bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
};
struct F16 {
    static constexpr uint32_t kExp = 0x7C00u, kMant = 0x03FFu, kOne = 0x3C00u;
    static __device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    }
    static __device__ __forceinline__ uint16_t bits(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
};

// One request's rows and keys: 1 rows that see keys [kb, ln + n) of its own; 0 rows that
// see nothing (vacant, or its length does not fit its table or prefix); -1 its rows do not
// lie in the buffer as they should.
struct Request {
    int start, n, ln, kb, group;
};

__device__ int group_of(const AttendArgs& a, int r) {
    int lo = 0, hi = a.n_groups;  // the last group that starts at or before r
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.group_off[mid] <= r) lo = mid + 1; else hi = mid;
    }
    return lo > 0 && r < a.group_off[lo] ? lo - 1 : -1;
}

__device__ int request_of(const AttendArgs& a, int r, Request& q, uint32_t& bad) {
    const int o = a.offsets[r];
    const long long n = (long long)a.offsets[r + 1] - o + a.lead, start = (long long)o + (long long)a.lead * r;
    q.n = 0;
    q.kb = 0;
    q.group = -1;
    if (o < 0 || n < 0 || n > a.max_new || start + n > a.rows) {
        bad = kStatusBadRow;
        return -1;
    }
    q.start = (int)start;
    q.n = (int)n;
    q.ln = a.len[r];
    if (q.ln < 0 || n == 0) return 0;
    if ((q.ln + n + a.page - 1) >> a.page_shift > a.width) {
        bad = kStatusBadRow;
        return 0;
    }
    if (a.n_groups) {
        q.group = group_of(a, r);
        if (q.group >= 0) {
            const int sp = a.shared_pages[q.group];
            if (sp < 0 || sp > a.shared_width || (long long)sp * a.page > q.ln) {
                bad = kStatusBadRow;
                return 0;
            }
            q.kb = sp * a.page;
        }
    }
    return 1;
}

// A group's rows [start, start + n) and the keys [0, ke) that they share; ke = 0 for none.
struct Group {
    int start, n, ke;
};

__device__ Group shared_of(const AttendArgs& a, int g, uint32_t& bad) {
    Group q{0, 0, 0};
    const int r0 = a.group_off[g], r1 = a.group_off[g + 1], sp = a.shared_pages[g];
    if (r0 < 0 || r1 < r0 || r1 > a.R || sp < 0 || sp > a.shared_width) {
        bad = kStatusBadRow;
        return q;
    }
    const long long s0 = (long long)a.offsets[r0] + (long long)a.lead * r0,
                    s1 = (long long)a.offsets[r1] + (long long)a.lead * r1;
    if (s0 < 0 || s1 < s0 || s1 > a.rows) {
        bad = kStatusBadRow;
        return q;
    }
    q.start = (int)s0;
    q.n = (int)(s1 - s0);
    q.ke = sp * a.page;
    return q;
}

// What one item (request or group) brings: its rows, the keys [kb, ke) that this launch
// gives them and the table that these lie in.  The last key that row j sees is ln + j.
struct Work {
    int start, n, kb, ke, ln, group;
    const int32_t* table;
};

template <int kSet>
__device__ Work work_of(const AttendArgs& a, int i) {
    uint32_t bad = 0;
    Work w;
    if (kSet) {
        const Group g = shared_of(a, i, bad);
        w = Work{g.start, g.n, 0, g.ke, 0, -1, a.shared_table + (size_t)i * a.shared_width};
    } else {
        Request q;
        request_of(a, i, q, bad);
        w = Work{q.start, q.n, q.kb, q.ln + q.n, q.ln, q.group, a.table + (size_t)i * a.width};
    }
    // the same in every lane: held in scalar registers
    w.start = __builtin_amdgcn_readfirstlane(w.start);
    w.n = __builtin_amdgcn_readfirstlane(w.n);
    w.kb = __builtin_amdgcn_readfirstlane(w.kb);
    w.ke = __builtin_amdgcn_readfirstlane(w.ke);
    w.ln = __builtin_amdgcn_readfirstlane(w.ln);
    w.group = __builtin_amdgcn_readfirstlane(w.group);
    return w;
}

template <int kTile>
__device__ __forceinline__ int tiles_of(const AttendArgs& a, int n) {
    return (n * a.G + kTile - 1) / kTile;
}
template <int kUnit>
__device__ __forceinline__ int units_of(int keys) {
    return (keys + kUnit - 1) / kUnit;
}
// The same for launch `set`, whose form the host has chosen.
__device__ __forceinline__ int tiles_in(const AttendArgs& a, int set, int n) {
    return (n * a.G + a.tile[set] - 1) / a.tile[set];
}
__device__ __forceinline__ int units_in(const AttendArgs& a, int set, int keys) {
    return (keys + a.unit[set] - 1) / a.unit[set];
}

// Workers that have a unit at all, so that no part between two others is missing.
__device__ __forceinline__ int workers_of(const AttendArgs& a, int set, uint32_t total) {
    return total < (uint32_t)a.workers[set] ? (int)total : a.workers[set];
}
// Worker w's first unit, and the worker of unit u, when `workers` share `total` units.
__device__ __forceinline__ uint32_t first_unit(uint32_t total, int workers, int w) {
    return (uint32_t)((uint64_t)total * (uint32_t)w / (uint32_t)workers);
}
__device__ __forceinline__ int worker_of(uint32_t total, int workers, uint32_t u) {
    return (int)((((uint64_t)u + 1) * (uint32_t)workers - 1) / total);
}

__device__ __forceinline__ float* slot_of(const AttendArgs& a, int set, int worker, int which) {
    return a.slots[set] + (size_t)(worker * 2 + which) * ((size_t)a.tile[set] * (a.D + 2));
}

// Running units (of one key head) of the items in LDS, kept for the second kernel too;
// returns the units of all heads.  One workgroup of 256 threads.
template <int kSet>
__device__ uint32_t plan(const AttendArgs& a, int n, uint32_t* s_cum, uint32_t* s_base) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t base = 0, bad = 0;
    for (int i0 = 0; i0 < n; i0 += kT) {
        const int i = i0 + tid;
        uint32_t x = 0;
        if (i < n) {
            if (kSet) {
                const Group g = shared_of(a, i, bad);
                x = (uint32_t)tiles_in(a, 1, g.n) * units_in(a, 1, g.ke);
            } else {
                Request q;
                if (request_of(a, i, q, bad) == 1) x = (uint32_t)tiles_in(a, 0, q.n) * units_in(a, 0, q.ln + q.n - q.kb);
            }
        }
        uint32_t y = x;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t z = __shfl_up(y, d, 64);
            if (lane >= d) y += z;
        }
        __syncthreads();
        if (lane == 63) s_base[wave] = y;
        __syncthreads();
        for (int w = 0; w < wave; ++w) y += s_base[w];
        if (i < n) s_cum[i] = base + y - x;
        base += s_base[0] + s_base[1] + s_base[2] + s_base[3];
    }
    if (tid == 0) s_cum[n] = base;
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int i = tid; i <= n; i += kT) a.cum[kSet][i] = s_cum[i];
        if (bad) raise_status(a.status, bad);
    }
    return __builtin_amdgcn_readfirstlane(base) * a.Hkv;
}

// The item that unit u belongs to.
__device__ __forceinline__ int item_of(const AttendArgs& a, const uint32_t* s_cum, int n, uint32_t u) {
    int i = 0;
    for (int hi = n; hi - i > 1;) {
        const int mid = (i + hi) >> 1;
        if (__builtin_amdgcn_readfirstlane(s_cum[mid]) * a.Hkv <= u) i = mid; else hi = mid;
    }
    return i;
}

// A request's table has to begin with its group's pages.
__device__ void check_prefix(const AttendArgs& a, const Work& q) {
    bool differs = false;
    const int32_t* shared = a.shared_table + (size_t)q.group * a.shared_width;
    for (int p = threadIdx.x; p < q.kb >> a.page_shift; p += kT) differs |= q.table[p] != shared[p];
    if (differs) raise_status(a.status, kStatusBadPage);
}

// Adds a part (maximum pm and sum pl of one column, o its values) to a running one.
__device__ __forceinline__ void join(float& m, float& l, float (&acc)[8], float pm, float pl, const float* o) {
    if (pm == -kInf) return;
    const float mx = fmaxf(m, pm);
    const float s0 = __builtin_amdgcn_exp2f(m - mx), s1 = __builtin_amdgcn_exp2f(pm - mx);
    m = mx;
    l = l * s0 + pl * s1;
    const float4 x = *(const float4*)o, y = *(const float4*)(o + 4);
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = acc[i] * s0 + v[i] * s1;
}

// Adds the parts of the segment whose units are [u0, u0 + units): column `col` of its tile.
__device__ __forceinline__ void join_parts(const AttendArgs& a, int set, uint32_t total, uint32_t u0, uint32_t units,
                                           int col, int c8, float& m, float& l, float (&acc)[8]) {
    const int workers = workers_of(a, set, total), tile = a.tile[set];
    const int wa = worker_of(total, workers, u0), wb = worker_of(total, workers, u0 + units - 1);
    for (int w = wa; w <= wb; ++w) {
        const float* s = slot_of(a, set, w, w == wa);
        join(m, l, acc, s[(size_t)tile * a.D + col], s[(size_t)tile * (a.D + 1) + col], s + (size_t)col * a.D + c8 * 8);
    }
}

// Adds the shared keys' part of query row f (row G + head of the group) of key head h.
__device__ void join_shared(const AttendArgs& a, int group, int f, int h, int c8, float& m, float& l, float (&acc)[8]) {
    uint32_t bad = 0;
    const Group g = shared_of(a, group, bad);
    const int at = f - g.start * a.G;
    if (g.ke <= 0 || at < 0 || at >= g.n * a.G) return;
    const uint32_t* cum = a.cum[1];
    const uint32_t total = cum[a.n_groups] * a.Hkv, units = units_in(a, 1, g.ke), tiles = tiles_in(a, 1, g.n);
    const uint32_t u0 = cum[group] * a.Hkv + (h * tiles + at / a.tile[1]) * units;
    const int workers = workers_of(a, 1, total);
    if (worker_of(total, workers, u0) == worker_of(total, workers, u0 + units - 1)) {
        const size_t n = (size_t)a.Hkv * a.rows * a.G, i = (size_t)h * a.rows * a.G + f;
        join(m, l, acc, a.dense[n * a.D + i], a.dense[n * (a.D + 1) + i], a.dense + i * a.D + c8 * 8);
    } else {
        join_parts(a, 1, total, u0, units, at % a.tile[1], c8, m, l, acc);
    }
}

template <class E>
__device__ __forceinline__ void store_row(const AttendArgs& a, int f, int h, int c8, float m, float l,
                                          const float (&acc)[8]) {
    const int row = f / a.G, head = h * a.G + f % a.G;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // the one rounding to 16 bits of the result
        const float x = l == 0.f ? 0.f : acc[2 * i] / l, y = l == 0.f ? 0.f : acc[2 * i + 1] / l;
        w[i] = E::bits(x) | (uint32_t)E::bits(y) << 16;
    }
    *(uint4*)(a.out + (size_t)row * a.out_stride + (size_t)head * a.D + c8 * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    if (c8 == 0 && a.lse)
        a.lse[(size_t)row * a.H + head] = l == 0.f ? -kInf : (m + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
}

// Values of V that are not finite, in blocks whose columns do not all see the same keys: the
// product runs without them (see clear_masked), and once the segment's keys are through they
// are given to the columns that see them.  Counting them for each dim and column by the
// same matrix instruction says what they come to: a NaN, or infinities of both signs, make
// NaN, infinities of one sign that infinity.  A NaN counts 4096, +inf 64 and -inf 1, and a
// block's 32 keys stay below 64 of each.
template <class E>
__device__ __forceinline__ void add_special(f32x16& o, s16x8 v0, s16x8 v1, s16x8 sees0, s16x8 sees1) {
    const auto weight = [](short v) -> short {
        const uint32_t y = (uint16_t)v;
        if ((y & E::kExp) != E::kExp) return 0;
        return (short)E::bits(y & E::kMant ? 4096.f : y & 0x8000u ? 1.f : 64.f);
    };
    s16x8 x0, x1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x0[i] = weight(v0[i]);
        x1[i] = weight(v1[i]);
    }
    const f32x16 n = E::mfma(x1, sees1, E::mfma(x0, sees0, f32x16{}));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t c = (uint32_t)n[i], neg = c & 63u, pos = (c >> 6) & 63u;
        if (c >= 4096u || (neg && pos)) o[i] = __builtin_nanf("");
        else if (pos) o[i] += kInf;
        else if (neg) o[i] -= kInf;
    }
}

// Eight values of which the first `valid` belong to the segment: the others are cleared, and
// so are those that are not finite; returns whether there were such.  Two values to a word:
// an exponent of ones carries into its half's top bit.
template <class E>
__device__ __forceinline__ uint32_t clear_masked(s16x8& v, int valid) {
    u32x4 x = __builtin_bit_cast(u32x4, v);
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = x[i] & (valid >= 2 * i + 2 ? 0xFFFFFFFFu : valid == 2 * i + 1 ? 0xFFFFu : 0u);
        const uint32_t top = ((w & (E::kExp * 0x10001u)) + (E::kMant + 1) * 0x10001u) & 0x80008000u;
        any |= top;
        x[i] = w & ~(top | (top - (top >> 15)));
    }
    v = __builtin_bit_cast(s16x8, x);
    return any;
}

// Column c of the tile at f0 is done as far as this workgroup goes: eight dims of it, from
// 8 c8 on.  The result, where the segment ends here and its keys were the requests' own;
// else the part, for whoever joins it.
template <class E, int kSet>
__device__ __forceinline__ void finish(const AttendArgs& a, const Work& q, bool whole, bool begins, int f0, int c, int h,
                                       int c8, float m, float l, float (&acc)[8]) {
    if (whole && kSet == 0) {
        if (q.kb > 0) join_shared(a, q.group, f0 + c, h, c8, m, l, acc);
        store_row<E>(a, f0 + c, h, c8, m, l, acc);
        return;
    }
    float *po, *pm, *pl;
    if (whole) {
        const size_t all = (size_t)a.Hkv * a.rows * a.G, at = (size_t)h * a.rows * a.G + f0 + c;
        po = a.dense + at * a.D;
        pm = a.dense + all * a.D + at;
        pl = a.dense + all * (a.D + 1) + at;
    } else {
        const size_t tile = a.tile[kSet];
        float* slot = slot_of(a, kSet, blockIdx.x, begins);
        po = slot + (size_t)c * a.D;
        pm = slot + tile * a.D + c;
        pl = slot + tile * (a.D + 1) + c;
    }
    *(float4*)(po + c8 * 8) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    *(float4*)(po + c8 * 8 + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
    if (c8 == 0) {
        *pm = m;
        *pl = l;
    }
}

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32, 64); }

// Page ids of a table row, 64 entries at a time in the lanes of a wave: entry i is read
// with readlane, so that the next block's address does not wait for memory.
struct PageIds {
    const int32_t* table;
    int n;     // entries of interest: [0, n)
    int base;  // the entry in lane 0
    int ids;
    __device__ __forceinline__ void start(const int32_t* t, int count, int first, int lane) {
        table = t;
        n = count;
        fetch(first, lane);
    }
    __device__ __forceinline__ void fetch(int first, int lane) {
        base = first;
        const int i = first + lane;
        ids = table[i < n ? i : n - 1];
        asm volatile("" : "+v"(ids));  // waited for here, so that readers need not wait for what else is under way
    }
    __device__ __forceinline__ int at(int i, int lane) {
        if (i - base >= 64) fetch(i, lane);
        return __builtin_amdgcn_readlane(ids, i - base);
    }
};

// The few-rows form.  A workgroup takes kTiles tiles of the segment's columns: its four
// waves are 4 / kTiles groups of keys by kTiles tiles, so that up to 64 columns read the
// keys once.  Each wave streams: the next block's K is requested as soon as the first
// product has used this one's, the next V after the second product, so about 16 KB a wave
// are under way while it computes (kSet 0: the requests' own keys; 1: the groups' shared
// ones).
template <class E, int D, int kSet, int kTiles>
__global__ __launch_bounds__(kT, D <= 128 ? 2 : 1) void attend_kernel(AttendArgs a) {
    constexpr int NT = D / 32, NC = D / 16;
    constexpr int kKeyWaves = 4 / kTiles;
    constexpr int kUnit = 32 * kKeyWaves;
    constexpr int kDims = D <= 128 ? D : 128;  // dims joined over the waves at a time
    constexpr int kPitch = kDims + 4;
    __shared__ float s_o[4][32][kPitch];
    __shared__ float s_m[4][32], s_l[4][32];
    __shared__ uint32_t s_base[8];
    extern __shared__ uint32_t s_cum[];  // running units, n + 1
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int key_wave = wave / kTiles, sub = wave % kTiles;
    const int n = kSet ? a.n_groups : a.R;
    const uint32_t total = plan<kSet>(a, n, s_cum, s_base);
    const int workers = workers_of(a, kSet, total);
    if ((int)blockIdx.x >= workers) return;
    uint32_t u = first_unit(total, workers, blockIdx.x);
    const uint32_t u_end = first_unit(total, workers, blockIdx.x + 1);
    const int shift = a.page_shift - 4, in_page = (1 << shift) - 1;  // blocks of 16 in a page
    const int head_shift = __builtin_ctz(D) + a.page_shift;  // a head's elements in a page

    uint32_t item_u0 = 0, item_u1 = 0;  // units of the item at hand
    Work q{};
    while (u < u_end) {
        if (u >= item_u1) {
            const int i = item_of(a, s_cum, n, u);
            item_u0 = __builtin_amdgcn_readfirstlane(s_cum[i]) * a.Hkv;
            item_u1 = __builtin_amdgcn_readfirstlane(s_cum[i + 1]) * a.Hkv;
            q = work_of<kSet>(a, i);
        }
        const uint32_t units = units_of<kUnit>(q.ke - q.kb), tiles = tiles_of<32 * kTiles>(a, q.n);
        const uint32_t in = u - item_u0, seg = in / units, unit0 = in % units;
        const int h = seg / tiles, tile = seg % tiles;
        const uint32_t unit1 = min(units, unit0 + (u_end - u));
        const int f0 = q.start * a.G + tile * (32 * kTiles);
        const int nf = min(32 * kTiles, q.n * a.G - tile * (32 * kTiles));
        if (kSet == 0 && q.kb > 0 && seg == 0 && unit0 == 0) check_prefix(a, q);

        // Q^T as the first product's second operand: this lane's column, dims 16 c + 8 half + 0..7.
        const int f = f0 + min(sub * 32 + col, nf - 1);
        const uint16_t* qp = a.q + (size_t)(f / a.G) * a.q_stride + (size_t)(h * a.G + f % a.G) * D + half * 8;
        s16x8 qf[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) qf[c] = *(const s16x8*)(qp + c * 16);
        const int last = kSet ? q.ke - 1 : q.ln + f / a.G - q.start;            // the column's last key
        const int first_last = kSet ? q.ke - 1 : q.ln + f0 / a.G - q.start;  // the earliest of them

        f32x16 o[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t] = f32x16{};
        float m = -kInf, l = 0.f;  // m of the raw scores; l this half's share of the sum

        const int swapped = (col & 3) | ((col & 4) << 1) | ((col & 8) >> 1);  // key of this lane in its block of 16
        int pos = q.kb + (int)(unit0 * kUnit) + key_wave * 32;
        const int pos_end = min(q.ke, q.kb + (int)(unit1 * kUnit));
        if (pos < pos_end && sub * 32 < nf) {
            PageIds pages;
            pages.start(q.table, (q.ke + (1 << a.page_shift) - 1) >> a.page_shift, pos >> a.page_shift, lane);
            const uint16_t *kp[2], *vp[2];
            bool have[2], next_have[2], bad_page = false;
            s16x8 kf[NC], vf[NT][2];
            // The two blocks of 16 keys at position p: where K and V lie, and whether they are there.
            const auto locate = [&](int p, bool(&there)[2]) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int blk = (p >> 4) + b;
                    there[b] = p + b * 16 < q.ke;
                    int page = there[b] ? pages.at(blk >> shift, lane) : 0;
                    if ((unsigned)page >= (unsigned)a.n_pages) {
                        page = 0;
                        there[b] = false;
                        bad_page = true;
                    }
                    const size_t at =
                        (((size_t)(unsigned)page * (unsigned)a.Hkv + h) << head_shift) + (size_t)(blk & in_page) * (16 * D);
                    kp[b] = a.k + at;
                    vp[b] = a.v + at;
                }
            };
            const auto load_k = [&]() {
                const uint16_t* kl = (col < 16 ? kp[0] : kp[1]) + half * 128 + swapped * 8;
#pragma unroll
                for (int c = 0; c < NC; ++c) kf[c] = *(const s16x8*)(kl + c * 256);
            };
            const auto load_v = [&]() {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int b = 0; b < 2; ++b) vf[t][b] = *(const s16x8*)(vp[b] + (t * 32 + col) * 16 + half * 8);
            };
            int special_from = -1;  // the first block with values that add_special has to add
            locate(pos, have);
            load_k();
            load_v();
            for (;;) {
                f32x16 s = {};
#pragma unroll
                for (int c = 0; c < NC; ++c) s = E::mfma(kf[c], qf[c], s);
                const int next = pos + kUnit;
                const bool more = next < pos_end;
                if (more) {
                    locate(next, next_have);
                    load_k();
                }
                const bool masked = pos + 31 > first_last || !have[0] || !have[1];
                if (masked) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (pos + (j / 8) * 16 + half * 8 + j % 8 > last || !have[j / 8]) s[j] = -kInf;
                }
                float mx = s[0];
#pragma unroll
                for (int j = 1; j < 16; ++j) mx = fmaxf(mx, s[j]);
                mx = fmaxf(mx, other_half(mx));
                if (__ballot(mx > m)) {  // a larger maximum: what has been summed so far shrinks
                    const float m_new = fmaxf(m, mx);
                    const float alpha = __builtin_amdgcn_exp2f((m - (m_new == -kInf ? 0.f : m_new)) * a.scale_log2);
                    m = m_new;
                    l *= alpha;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[t][j] *= alpha;
                }
                const float mc = m == -kInf ? 0.f : m * a.scale_log2;
                s16x8 pf[2];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j], a.scale_log2, -mc));
                    l += p;
                    pf[j / 8][j % 8] = (short)E::bits(p);  // weights of at most 1, rounded for the matrix instruction
                }
                if (masked) {
                    uint32_t special = 0;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            special |= clear_masked<E>(vf[t][b], have[b] ? q.ke - (pos + b * 16 + half * 8) : 0);
                    if (special_from < 0 && __ballot(special != 0)) special_from = pos;
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) o[t] = E::mfma(vf[t][1], pf[1], E::mfma(vf[t][0], pf[0], o[t]));
                if (!more) break;
                load_v();
                pos = next;
                have[0] = next_have[0];
                have[1] = next_have[1];
            }
            l += other_half(l);
            if (bad_page && lane == 0) raise_status(a.status, kStatusBadPage);
            if (special_from >= 0) {
                pages.fetch(special_from >> a.page_shift, lane);
                for (pos = special_from; pos < pos_end; pos += kUnit) {
                    locate(pos, have);
                    s16x8 sees[2];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        sees[j / 8][j % 8] =
                            pos + (j / 8) * 16 + half * 8 + j % 8 <= last && have[j / 8] ? (short)E::kOne : (short)0;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        add_special<E>(o[t], *(const s16x8*)(vp[0] + (t * 32 + col) * 16 + half * 8),
                                       *(const s16x8*)(vp[1] + (t * 32 + col) * 16 + half * 8), sees[0], sees[1]);
                }
            }
        }
        const float ms = m == -kInf ? -kInf : m * a.scale_log2;

        // The waves' parts joined, column by column, eight dims to a thread.
        const bool whole = unit0 == 0 && unit1 == units;
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += kDims) {
            __syncthreads();
            if (half == 0) {
                s_m[wave][col] = ms;
                s_l[wave][col] = l;
            }
#pragma unroll
            for (int t = 0; t < kDims / 32; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x16& x = o[d0 / 32 + t];
                    *(float4*)&s_o[wave][col][t * 32 + 8 * j + 4 * half] =
                        make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
                }
            __syncthreads();
            for (int e = tid; e < nf * (kDims / 8); e += kT) {
                const int c = e / (kDims / 8), c8 = e % (kDims / 8);
                float jm = -kInf, jl = 0.f, acc[8] = {};
#pragma unroll
                for (int w = 0; w < kKeyWaves; ++w) {
                    const int from = w * kTiles + c / 32;
                    join(jm, jl, acc, s_m[from][c % 32], s_l[from][c % 32], &s_o[from][c % 32][c8 * 8]);
                }
                finish<E, kSet>(a, q, whole, unit0 == 0, f0, c, h, d0 / 8 + c8, jm, jl, acc);
            }
        }
        u += unit1 - unit0;
    }
}

// Joins the parts of the segments that were split, and gives zeros to rows that see nothing.
template <class E>
__global__ __launch_bounds__(kT) void attend_join_kernel(AttendArgs a) {
    const int r = blockIdx.x, h = blockIdx.y, tile = blockIdx.z, width = a.tile[0];
    Request q;
    uint32_t bad = 0;
    const int state = request_of(a, r, q, bad);
    if (state < 0 || tile * width >= q.n * a.G) return;
    const int f0 = q.start * a.G + tile * width, nf = min(width, q.n * a.G - tile * width);
    const uint32_t *cum = a.cum[0], total = cum[a.R] * a.Hkv;
    const uint32_t units = state ? units_in(a, 0, q.ln + q.n - q.kb) : 0;
    const uint32_t u0 = state ? cum[r] * a.Hkv + (h * tiles_in(a, 0, q.n) + tile) * units : 0;
    const int workers = workers_of(a, 0, total);
    if (state && worker_of(total, workers, u0) == worker_of(total, workers, u0 + units - 1)) return;
    for (int e = threadIdx.x; e < nf * (a.D / 8); e += kT) {
        const int c = e / (a.D / 8), c8 = e % (a.D / 8);
        float m = -kInf, l = 0.f, acc[8] = {};
        if (state) {
            join_parts(a, 0, total, u0, units, c, c8, m, l, acc);
            if (q.kb > 0) join_shared(a, q.group, f0 + c, h, c8, m, l, acc);
        }
        store_row<E>(a, f0 + c, h, c8, m, l, acc);
    }
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

template <class E, int D, int kSet>
hipError_t run_set(const AttendArgs& a, hipStream_t s) {
    const size_t lds = ((kSet ? a.n_groups : a.R) + 1) * sizeof(uint32_t);
    if (a.tile[kSet] == 64)
        hipLaunchKernelGGL((attend_kernel<E, D, kSet, 2>), dim3(a.workers[kSet]), dim3(kT), lds, s, a);
    else
        hipLaunchKernelGGL((attend_kernel<E, D, kSet, 1>), dim3(a.workers[kSet]), dim3(kT), lds, s, a);
    return hipGetLastError();
}

template <class E, int D>
hipError_t run(const AttendArgs& a, hipStream_t s) {
    hipError_t e = a.n_groups ? run_set<E, D, 1>(a, s) : hipSuccess;
    if (e == hipSuccess) e = run_set<E, D, 0>(a, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(attend_join_kernel<E>, dim3(a.R, a.Hkv, (a.max_new * a.G + a.tile[0] - 1) / a.tile[0]), dim3(kT),
                       0, s, a);
    return hipGetLastError();
}

template <class E>
hipError_t run_dim(const AttendArgs& a, hipStream_t s) {
    return a.D == 64 ? run<E, 64>(a, s) : a.D == 128 ? run<E, 128>(a, s) : run<E, 256>(a, s);
}

size_t slots_bytes(int D) { return round256((size_t)kAttendMaxWorkers * 2 * kAttendMaxTile * (D + 2) * sizeof(float)); }
size_t dense_bytes(int R, int H, int D, int max_new) {
    return round256((size_t)R * max_new * H * (D + 2) * sizeof(float));
}

}  // namespace

size_t attend_ws_bytes(int R, int H, int D, int max_new, int n_groups) {
    size_t n = slots_bytes(D) + round256((size_t)(R + 1) * 4);
    if (n_groups) n += slots_bytes(D) + round256((size_t)(n_groups + 1) * 4) + dense_bytes(R, H, D, max_new);
    return n;
}

void attend_ws_layout(AttendArgs& a, void* ws) {
    char* p = (char*)ws;
    a.slots[0] = (float*)p;
    p += slots_bytes(a.D);
    a.cum[0] = (uint32_t*)p;
    p += round256((size_t)(a.R + 1) * 4);
    if (!a.n_groups) return;
    a.slots[1] = (float*)p;
    p += slots_bytes(a.D);
    a.cum[1] = (uint32_t*)p;
    p += round256((size_t)(a.n_groups + 1) * 4);
    a.dense = (float*)p;
}

hipError_t launch_attend(AttendArgs a, int cus, hipStream_t s) {
    const int w = std::min(cus * (a.D <= 128 ? 2 : 1), kAttendMaxWorkers);
    // 64 columns to a workgroup where a request (a group) may have more than 32 of them
    for (int set = 0; set < 2; ++set) {
        const long long columns = (long long)(set ? a.rows : a.max_new) * a.G;
        a.tile[set] = columns > 32 ? 64 : 32;
        a.unit[set] = a.tile[set] == 64 ? 64 : 128;
        a.workers[set] = w;
    }
    return a.dtype == DSPARK_F16 ? run_dim<F16>(a, s) : run_dim<Bf16>(a, s);
}

}  // namespace dspark
