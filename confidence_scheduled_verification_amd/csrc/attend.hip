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
constexpr int kWideFrom = 64;  // columns of a request or group beyond which the many-rows form runs
constexpr float kInf = __builtin_huge_valf();

struct Bf16 {
    static constexpr uint32_t kExp = 0x7F80u, kMant = 0x007Fu, kOne = 0x3F80u, k64 = 0x4280u, k4096 = 0x4580u;
    static __device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint16_t bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
};
struct F16 {
    static constexpr uint32_t kExp = 0x7C00u, kMant = 0x03FFu, kOne = 0x3C00u, k64 = 0x5400u, k4096 = 0x6C00u;
    static __device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    }
    static __device__ __forceinline__ uint16_t bits(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
};

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

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
    return (n * a.G + a.tile[set] - 1) >> a.tile_shift[set];
}
__device__ __forceinline__ int units_in(const AttendArgs& a, int set, int keys) {
    return (keys + a.unit[set] - 1) >> a.unit_shift[set];
}

// How `total` units are dealt to the workers: each takes `each` consecutive ones, the first
// `more` one more than that.  Where there are fewer units than workers the others have none.
struct Split {
    uint32_t each, more;
    int workers;
    __device__ __forceinline__ Split(uint32_t total, int most) {
        workers = total < (uint32_t)most ? (int)total : most;
        each = workers ? total / (uint32_t)workers : 0;
        more = workers ? total % (uint32_t)workers : 0;
    }
    __device__ __forceinline__ uint32_t first(uint32_t w) const { return w * each + min(w, more); }
    __device__ __forceinline__ int worker_of(uint32_t u) const {
        const uint32_t big = more * (each + 1);
        return (int)(u < big ? u / (each + 1) : more + (u - big) / each);
    }
};

__device__ __forceinline__ float* slot_of(const AttendArgs& a, int set, int worker, int which) {
    return a.slots[set] + (size_t)(worker * 2 + which) * ((size_t)a.tile[set] * (a.D + 2));
}

// Running units (of one key head) of the items in LDS, and what each of the first kCached
// brings, so that a workgroup looks at the requests once; the groups' running units are kept
// for the next launch too.  Returns the units of all heads.
constexpr int kCached = 384;  // items: LDS for two workgroups a compute unit at head_dim 128

// Rows that see nothing get zeros: those of the requests without units.  Request i is looked
// at by enough workgroups, from number i on, to give each wave about four of its rows.
template <int kThreads>
__device__ void clear_unseen(const AttendArgs& a, int n, const uint32_t* s_cum) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, grid = gridDim.x;
    constexpr int kWaves = kThreads / 64;
    const int takes = min(grid, (a.max_new + 4 * kWaves - 1) / (4 * kWaves));
    for (int i0 = 0; i0 < n; i0 += 64) {
        const int at = i0 + lane;
        const bool mine = at < n && s_cum[at] == s_cum[at + 1] && (blockIdx.x + grid - at % grid) % grid < takes;
        for (uint64_t left = __ballot(mine); left; left &= left - 1) {
            const int i = i0 + (int)__ffsll((unsigned long long)left) - 1;
            Request q;
            uint32_t none = 0;
            if (request_of(a, i, q, none) != 0) continue;
            const int turn = (blockIdx.x + grid - i % grid) % grid;
            for (int j = turn * kWaves + wave; j < q.n; j += takes * kWaves) {
                uint16_t* row = a.out + (size_t)(q.start + j) * a.out_stride;
                for (int e = lane; e < a.H * (a.D / 8); e += 64) *(uint4*)(row + e * 8) = make_uint4(0, 0, 0, 0);
                if (a.lse)
                    for (int e = lane; e < a.H; e += 64) a.lse[(size_t)(q.start + j) * a.H + e] = -kInf;
            }
        }
    }
}

template <int kSet, int kThreads>
__device__ uint32_t plan(const AttendArgs& a, int n, uint32_t* s_cum, uint32_t* s_base) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Request* s_info = (Request*)(s_cum + n + 1);
    uint32_t base = 0, bad = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        uint32_t x = 0;
        if (i < n) {
            if (kSet) {
                const Group g = shared_of(a, i, bad);
                x = (uint32_t)tiles_in(a, 1, g.n) * units_in(a, 1, g.ke);
            } else {
                Request q;
                const int state = request_of(a, i, q, bad);
                if (state == 1) x = (uint32_t)tiles_in(a, 0, q.n) * units_in(a, 0, q.ln + q.n - q.kb);
                if (i < kCached) s_info[i] = q;
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
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) base += s_base[w];
    }
    if (tid == 0) s_cum[n] = base;
    __syncthreads();
    if (blockIdx.x == 0) {
        if (kSet)
            for (int i = tid; i <= n; i += kThreads) a.cum[i] = s_cum[i];
        if (bad) raise_status(a.status, bad);
    }
    if (kSet == 0) clear_unseen<kThreads>(a, n, s_cum);
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

// The units of a group in its launch, as the requests' launch needs them to find the parts:
// those of its tile t with key head h are [u0 + (h tiles + t) units, + units).
struct Shared {
    int start, n;  // the group's rows; n = 0 for none
    uint32_t u0, units, tiles;
};

// What one item (request or group) brings: its rows, the keys [kb, ke) that this launch
// gives them and the table that these lie in.  The last key that row j sees is ln + j.
struct Work {
    int start, n, kb, ke, ln, group;
    const int32_t* table;
    Shared shared;
};

template <int kSet>
__device__ Work work_of(const AttendArgs& a, int i, int n, const uint32_t* s_cum) {
    uint32_t bad = 0;
    Work w{};
    if (kSet) {
        const Group g = shared_of(a, i, bad);
        w.start = uniform(g.start);
        w.n = uniform(g.n);
        w.ke = uniform(g.ke);
        w.group = -1;
        w.table = a.shared_table + (size_t)i * a.shared_width;
        return w;
    }
    Request q;
    if (i < kCached) q = ((const Request*)(s_cum + n + 1))[i];
    else request_of(a, i, q, bad);
    // the same in every lane: held in scalar registers
    w.start = uniform(q.start);
    w.n = uniform(q.n);
    w.kb = uniform(q.kb);
    w.ln = uniform(q.ln);
    w.ke = w.ln + w.n;
    w.group = uniform(q.group);
    w.table = a.table + (size_t)i * a.width;
    if (w.kb > 0) {
        const Group g = shared_of(a, w.group, bad);
        // (rows outside the group's, as offsets that fall would have it, have no part there)
        if (uniform(g.ke) > 0 && w.start >= uniform(g.start) && w.start + w.n <= uniform(g.start + g.n)) {
            w.shared.start = uniform(g.start);
            w.shared.n = uniform(g.n);
            w.shared.units = units_in(a, 1, uniform(g.ke));
            w.shared.tiles = tiles_in(a, 1, w.shared.n);
            w.shared.u0 = uniform(a.cum[w.group]) * a.Hkv;
        }
    }
    return w;
}

// A request's table has to begin with its group's pages.
__device__ void check_prefix(const AttendArgs& a, const Work& q) {
    bool differs = false;
    const int32_t* shared = a.shared_table + (size_t)q.group * a.shared_width;
    for (int p = threadIdx.x; p < q.kb >> a.page_shift; p += blockDim.x) differs |= q.table[p] != shared[p];
    if (differs) raise_status(a.status, kStatusBadPage);
}

// Adds a part (maximum pm and sum pl of one column, x and y eight of its values) to a running one.
__device__ __forceinline__ void join(float& m, float& l, float (&acc)[8], float pm, float pl, float4 x, float4 y) {
    if (pm == -kInf) return;
    const float mx = fmaxf(m, pm);
    const float s0 = __builtin_amdgcn_exp2f(m - mx), s1 = __builtin_amdgcn_exp2f(pm - mx);
    m = mx;
    l = l * s0 + pl * s1;
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = acc[i] * s0 + v[i] * s1;
}

// Adds the parts that workers wa..wb have left of a segment: column `col` of its tile.  Four
// parts are requested at a time, so that a long segment's parts do not wait for each other.
__device__ __forceinline__ void join_parts(const AttendArgs& a, int set, int wa, int wb, int col, int c8, float& m,
                                           float& l, float (&acc)[8]) {
    const size_t tile = a.tile[set];
    for (int w0 = wa; w0 <= wb; w0 += 4) {
        float pm[4], pl[4];
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int w = min(w0 + i, wb);
            const float* s = slot_of(a, set, w, w == wa);
            pm[i] = s[tile * a.D + col];
            pl[i] = s[tile * (a.D + 1) + col];
            x[i] = *(const float4*)(s + (size_t)col * a.D + c8 * 8);
            y[i] = *(const float4*)(s + (size_t)col * a.D + c8 * 8 + 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (w0 + i <= wb) join(m, l, acc, pm[i], pl[i], x[i], y[i]);
    }
}

// The shared keys' parts for the columns from f0 on: they lie in one tile of the group's
// launch, or from column `edge` on in the next one (a tile there is at least as wide).
struct SharedParts {
    int edge, col0;        // the first column of the second tile; f0's column in the first one
    int first[2], last[2];  // the workers that hold parts of the two
};

__device__ SharedParts shared_parts(const AttendArgs& a, const Split& split, const Shared& g, int f0, int h) {
    SharedParts p{};
    const int at = f0 - g.start * a.G, tile = at >> a.tile_shift[1];
    p.col0 = at - (tile << a.tile_shift[1]);
    p.edge = a.tile[1] - p.col0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t u0 = g.u0 + (h * g.tiles + min(tile + i, (int)g.tiles - 1)) * g.units;
        p.first[i] = uniform(split.worker_of(u0));
        p.last[i] = uniform(split.worker_of(u0 + g.units - 1));
    }
    return p;
}

// Adds them for column c of f0's tile, key head h.
__device__ __forceinline__ void join_shared(const AttendArgs& a, const SharedParts& p, int f0, int c, int h, int c8, float& m,
                                            float& l, float (&acc)[8]) {
    const int i = c >= p.edge;
    if (p.first[i] == p.last[i]) {
        const size_t n = (size_t)a.Hkv * a.rows * a.G, f = (size_t)h * a.rows * a.G + f0 + c;
        const float* o = a.dense + f * a.D + c8 * 8;
        join(m, l, acc, a.dense[n * a.D + f], a.dense[n * (a.D + 1) + f], *(const float4*)o, *(const float4*)(o + 4));
    } else {
        join_parts(a, 1, p.first[i], p.last[i], i ? c - p.edge : p.col0 + c, c8, m, l, acc);
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
        const uint32_t inf = y & 0x8000u ? E::kOne : E::k64, w = y & E::kMant ? E::k4096 : inf;
        return (short)((y & E::kExp) == E::kExp ? w : 0u);
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
        const float add = pos ? kInf : neg ? -kInf : 0.f;
        o[i] = c >= 4096u || (neg && pos) ? __builtin_nanf("") : o[i] + add;
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
__device__ __forceinline__ void finish(const AttendArgs& a, const SharedParts& parts, bool shared, bool whole,
                                       bool begins, int f0, int c, int h, int c8, float m, float l, float (&acc)[8]) {
    if (whole && kSet == 0) {
        if (shared) join_shared(a, parts, f0, c, h, c8, m, l, acc);
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
    const uint32_t total = plan<kSet, kT>(a, n, s_cum, s_base);
    const Split split(total, a.workers[kSet]);
    if (kSet == 0 && tid == 0) a.ends[blockIdx.x].units = 0;
    if ((int)blockIdx.x >= split.workers) return;
    const Split split1(kSet == 0 && a.n_groups ? uniform(a.cum[a.n_groups]) * a.Hkv : 0, a.workers[1]);
    uint32_t u = split.first(blockIdx.x);
    const uint32_t u_end = split.first(blockIdx.x + 1);
    const int shift = a.page_shift - 4, in_page = (1 << shift) - 1;  // blocks of 16 in a page
    const int head_shift = __builtin_ctz(D) + a.page_shift;  // a head's elements in a page

    uint32_t item_u0 = 0, item_u1 = 0;  // units of the item at hand
    Work q{};
    while (u < u_end) {
        if (u >= item_u1) {
            const int i = item_of(a, s_cum, n, u);
            item_u0 = __builtin_amdgcn_readfirstlane(s_cum[i]) * a.Hkv;
            item_u1 = __builtin_amdgcn_readfirstlane(s_cum[i + 1]) * a.Hkv;
            q = work_of<kSet>(a, i, n, s_cum);
        }
        const uint32_t units = units_of<kUnit>(q.ke - q.kb), tiles = tiles_of<32 * kTiles>(a, q.n);
        const uint32_t in = u - item_u0, seg = in / units, unit0 = in % units;
        const int h = seg / tiles, tile = seg % tiles;
        const uint32_t unit1 = min(units, unit0 + (u_end - u));
        const int f0 = q.start * a.G + tile * (32 * kTiles);
        const int nf = min(32 * kTiles, q.n * a.G - tile * (32 * kTiles));
        if (kSet == 0 && q.kb > 0 && seg == 0 && unit0 == 0) check_prefix(a, q);
        if (kSet == 0 && unit0 > 0 && tid == 0)  // begun by an earlier worker: for the joining kernel
            a.ends[blockIdx.x] = AttendEnd{units, split.worker_of(u - unit0), split.worker_of(u - unit0 + units - 1), f0,
                                           nf, h, q.shared.start, q.shared.n, q.shared.u0, q.shared.units, q.shared.tiles};

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
        SharedParts parts{};
        if (kSet == 0 && whole && q.shared.n > 0) parts = shared_parts(a, split1, q.shared, f0, h);
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
                    join(jm, jl, acc, s_m[from][c % 32], s_l[from][c % 32], *(const float4*)&s_o[from][c % 32][c8 * 8],
                         *(const float4*)&s_o[from][c % 32][c8 * 8 + 4]);
                }
                finish<E, kSet>(a, parts, q.shared.n > 0, whole, unit0 == 0, f0, c, h, d0 / 8 + c8, jm, jl, acc);
            }
        }
        u += unit1 - unit0;
    }
}

// The many-rows form, for groups and prompts: a wave takes 32 columns, the workgroup eight
// (at head_dim 64 and 256: four) times as many, and all waves read the same 64 keys from LDS, which
// the next 64 are brought to meanwhile (global_load_lds: memory to LDS with no registers
// between).  The lanes of such a load pick their 16 bytes so that what a wave reads later,
// an operand of a matrix instruction, lies in LDS lane after lane.  The running maximum of
// a column follows only when it grows by more than 8 in the exponent of two; until then the
// weights are taken relative to the older one, at most 2^8, and nothing has to be rescaled.
template <int D>
struct Wide {
    static constexpr int kWaves = D == 128 ? 8 : 4;
    static constexpr int kThreads = kWaves * 64, kTile = kWaves * 32, kUnit = 64;
    static constexpr int kPerCu = D == 64 ? 3 : 1;  // workgroups: as many as the registers allow
    static constexpr int kBlock = 16 * D;           // elements of a block's K or V
};

template <class E, int D, int kSet>
__global__ __launch_bounds__(Wide<D>::kThreads, Wide<D>::kWaves / 4 * Wide<D>::kPerCu) void attend_wide_kernel(AttendArgs a) {
    typedef Wide<D> W;
    constexpr int NT = D / 32, NC = D / 16, kPitch = 36;
    constexpr int kStage = 8 * W::kBlock * 2, kJoin = W::kWaves * 32 * kPitch * 4;  // bytes
    __shared__ __attribute__((aligned(16))) char s_mem[2 * kStage > kJoin ? 2 * kStage : kJoin];
    __shared__ int s_have[2][4];
    __shared__ uint32_t s_base[8];
    extern __shared__ uint32_t s_cum[];  // running units, n + 1, then the requests
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int n = kSet ? a.n_groups : a.R;
    const uint32_t total = plan<kSet, W::kThreads>(a, n, s_cum, s_base);
    const Split split(total, a.workers[kSet]);
    if (kSet == 0 && tid == 0) a.ends[blockIdx.x].units = 0;
    if ((int)blockIdx.x >= split.workers) return;
    const Split split1(kSet == 0 && a.n_groups ? uniform(a.cum[a.n_groups]) * a.Hkv : 0, a.workers[1]);
    uint32_t u = split.first(blockIdx.x);
    const uint32_t u_end = split.first(blockIdx.x + 1);
    const int shift = a.page_shift - 4, in_page = (1 << shift) - 1;  // blocks of 16 in a page
    const int head_shift = __builtin_ctz(D) + a.page_shift;          // a head's elements in a page
    // where this lane's 16 bytes of each 1 KB of a block come from: K's keys with bits 2 and 3 of
    // their number swapped, V's halves of 16 tokens one after the other
    const int key = lane & 15, k_from = (lane >> 4) * 128 + ((key & 3) | ((key & 4) << 1) | ((key & 8) >> 1)) * 8;
    const int v_from = col * 16 + half * 8;

    uint32_t item_u0 = 0, item_u1 = 0;  // units of the item at hand
    Work q{};
    while (u < u_end) {
        if (u >= item_u1) {
            const int i = item_of(a, s_cum, n, u);
            item_u0 = uniform(s_cum[i]) * a.Hkv;
            item_u1 = uniform(s_cum[i + 1]) * a.Hkv;
            q = work_of<kSet>(a, i, n, s_cum);
        }
        const uint32_t units = units_of<W::kUnit>(q.ke - q.kb), tiles = tiles_of<W::kTile>(a, q.n);
        const uint32_t in = u - item_u0, seg = in / units, unit0 = in % units;
        const int h = seg / tiles, tile = seg % tiles;
        const uint32_t unit1 = min(units, unit0 + (u_end - u));
        const int f0 = q.start * a.G + tile * W::kTile;
        const int nf = min(W::kTile, q.n * a.G - tile * W::kTile);
        if (kSet == 0 && q.kb > 0 && seg == 0 && unit0 == 0) check_prefix(a, q);
        if (kSet == 0 && unit0 > 0 && tid == 0)  // begun by an earlier worker: for the joining kernel
            a.ends[blockIdx.x] = AttendEnd{units, split.worker_of(u - unit0), split.worker_of(u - unit0 + units - 1), f0,
                                           nf, h, q.shared.start, q.shared.n, q.shared.u0, q.shared.units, q.shared.tiles};

        const int f = f0 + min(wave * 32 + col, nf - 1);
        const uint16_t* qp = a.q + (size_t)(f / a.G) * a.q_stride + (size_t)(h * a.G + f % a.G) * D + half * 8;
        s16x8 qf[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) qf[c] = *(const s16x8*)(qp + c * 16);
        // The column's last key; the wave's earliest and latest of them, and the tile's latest.
        const int last = kSet ? q.ke - 1 : q.ln + f / a.G - q.start;
        const int first_last = kSet ? q.ke - 1 : q.ln + (f0 + min(wave * 32, nf - 1)) / a.G - q.start;
        const int wave_end = wave * 32 >= nf ? 0 : kSet ? q.ke : q.ln + (f0 + min(wave * 32 + 31, nf - 1)) / a.G - q.start + 1;
        const int tile_end = kSet ? q.ke : q.ln + (f0 + nf - 1) / a.G - q.start + 1;

        f32x16 o[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t] = f32x16{};
        float m = -kInf, l = 0.f;  // m of the raw scores; l this half's share of the sum
        int pos = q.kb + (int)(unit0 * W::kUnit);
        const int pos_end = min(tile_end, q.kb + (int)(unit1 * W::kUnit));
        int special_from = -1;
        bool bad_page = false;
        PageIds pages;
        if (pos < pos_end)
            pages.start(q.table, (q.ke + (1 << a.page_shift) - 1) >> a.page_shift,
                        min(pos + (wave & 3) * 16, q.ke - 1) >> a.page_shift, lane);

        // Block b of the 64 keys at p: whether it is there, and its first element of K and V.
        const auto locate = [&](int p, int b, size_t& at) {
            const int blk = (p >> 4) + b;
            bool there = p + b * 16 < q.ke;
            int page = there ? pages.at(blk >> shift, lane) : 0;
            if ((unsigned)page >= (unsigned)a.n_pages) {
                page = 0;
                there = false;
                bad_page = true;
            }
            at = (((size_t)(unsigned)page * (unsigned)a.Hkv + h) << head_shift) + (size_t)(blk & in_page) * W::kBlock;
            return there;
        };
        const auto bring = [&](int p, int buf) {
            const int b = wave & 3;
            size_t at;
            const bool there = locate(p, b, at);
            if (wave < 4 && lane == 0) s_have[buf][b] = there;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                if (W::kWaves == 8 && kv != wave >> 2) continue;  // waves 0-3 bring K, 4-7 V; or each both
                const uint16_t* from = kv ? a.v + at + v_from : a.k + at + k_from;
                char* to = s_mem + buf * kStage + (kv * 4 + b) * (W::kBlock * 2);
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from + j * 512),
                                                     (__attribute__((address_space(3))) void*)(to + j * 1024), 16, 0, 0);
            }
        };

        __syncthreads();  // LDS is free
        if (pos < pos_end) bring(pos, 0);
        for (int buf = 0; pos < pos_end; buf ^= 1, pos += W::kUnit) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's share of the 64 keys has landed
            __syncthreads();                                  // everyone's has, and the other buffer is free
            if (pos + W::kUnit < pos_end) bring(pos + W::kUnit, buf ^ 1);
            if (pos >= wave_end) continue;  // the wave's columns see none of these
            const char* mem = s_mem + buf * kStage;
            f32x16 s[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                s[b] = f32x16{};
                const char* kl = mem + (2 * b + (col >> 4)) * (W::kBlock * 2) + (half * 16 + (col & 15)) * 16;
#pragma unroll
                for (int c = 0; c < NC; ++c) s[b] = E::mfma(*(const s16x8*)(kl + c * 512), qf[c], s[b]);
            }
            const int4 have = *(const int4*)s_have[buf];
            const bool all = uniform(have.x & have.y & have.z & have.w);
            const bool masked = pos + 63 > first_last || !all;
            if (masked) {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int there = j < 8 ? have.x : j < 16 ? have.y : j < 24 ? have.z : have.w;
                    if (pos + (j / 8) * 16 + half * 8 + j % 8 > last || !there) s[j / 16][j % 16] = -kInf;
                }
            }
            float mx = s[0][0];
#pragma unroll
            for (int j = 1; j < 32; ++j) mx = fmaxf(mx, s[j / 16][j % 16]);
            mx = fmaxf(mx, other_half(mx));
            if (__ballot((mx - m) * a.scale_log2 > 8.f)) {
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
            s16x8 pf[4];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j / 16][j % 16], a.scale_log2, -mc));
                l += p;
                pf[j / 8][j % 8] = (short)E::bits(p);  // the weights, rounded for the matrix instruction
            }
            const char* vl = mem + 4 * (W::kBlock * 2) + lane * 16;
            if (!masked) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        o[t] = E::mfma(*(const s16x8*)(vl + b * (W::kBlock * 2) + t * 1024), pf[b], o[t]);
            } else {
                uint32_t special = 0;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        s16x8 v = *(const s16x8*)(vl + b * (W::kBlock * 2) + t * 1024);
                        const int there = b == 0 ? have.x : b == 1 ? have.y : b == 2 ? have.z : have.w;
                        special |= clear_masked<E>(v, there ? q.ke - (pos + b * 16 + half * 8) : 0);
                        o[t] = E::mfma(v, pf[b], o[t]);
                    }
                if (special_from < 0 && __ballot(special != 0)) special_from = pos;
            }
        }
        l += other_half(l);
        if (bad_page && lane == 0) raise_status(a.status, kStatusBadPage);
        if (special_from >= 0) {
            pages.fetch(special_from >> a.page_shift, lane);
            for (pos = special_from; pos < min(pos_end, wave_end); pos += 32) {
                size_t at[2];
                const bool have[2] = {locate(pos, 0, at[0]), locate(pos, 1, at[1])};
                s16x8 sees[2];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    sees[j / 8][j % 8] =
                        pos + (j / 8) * 16 + half * 8 + j % 8 <= last && have[j / 8] ? (short)E::kOne : (short)0;
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    add_special<E>(o[t], *(const s16x8*)(a.v + at[0] + t * 512 + v_from),
                                   *(const s16x8*)(a.v + at[1] + t * 512 + v_from), sees[0], sees[1]);
            }
        }
        const float ms = m == -kInf ? -kInf : m * a.scale_log2;

        // The wave's columns, 32 dims at a time through LDS, eight dims of a column to a lane.
        const bool whole = unit0 == 0 && unit1 == units;
        SharedParts parts{};
        if (kSet == 0 && whole && q.shared.n > 0) parts = shared_parts(a, split1, q.shared, f0, h);
        __syncthreads();
        float* s_o = (float*)s_mem + wave * (32 * kPitch);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *(float4*)&s_o[col * kPitch + 8 * j + 4 * half] =
                    make_float4(o[t][4 * j], o[t][4 * j + 1], o[t][4 * j + 2], o[t][4 * j + 3]);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int e = lane; e < 128; e += 64) {
                const int c = e >> 2, c8 = e & 3;
                const float jm = __shfl(ms, c, 64), jl = __shfl(l, c, 64);
                const float4 x = *(const float4*)&s_o[c * kPitch + c8 * 8], y = *(const float4*)&s_o[c * kPitch + c8 * 8 + 4];
                float acc[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                if (wave * 32 + c < nf)
                    finish<E, kSet>(a, parts, q.shared.n > 0, whole, unit0 == 0, f0, wave * 32 + c, h, t * 4 + c8, jm, jl, acc);
            }
            __builtin_amdgcn_wave_barrier();
        }
        u += unit1 - unit0;
    }
}

// Joins the parts of the segments that were split.  Where worker w goes on with a segment that
// worker w - 1 began, workgroup (w, .) joins it, eight dims of a column to a thread.
template <class E>
__global__ __launch_bounds__(kT) void attend_join_kernel(AttendArgs a) {
    const AttendEnd e = a.ends[blockIdx.x];
    if (e.units == 0 || e.first != (int)blockIdx.x - 1) return;
    const int chunks = a.D / 8, c = blockIdx.y * (kT / chunks) + threadIdx.x / chunks, c8 = threadIdx.x % chunks;
    if (c >= e.nf) return;
    float m = -kInf, l = 0.f, acc[8] = {};
    join_parts(a, 0, e.first, e.last, c, c8, m, l, acc);
    if (e.shared_n > 0) {
        const Split split1(a.cum[a.n_groups] * a.Hkv, a.workers[1]);
        const Shared g{e.shared_start, e.shared_n, e.shared_u0, e.shared_units, e.shared_tiles};
        join_shared(a, shared_parts(a, split1, g, e.f0, e.h), e.f0, c, e.h, c8, m, l, acc);
    }
    store_row<E>(a, e.f0 + c, e.h, c8, m, l, acc);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

template <class E, int D, int kSet>
hipError_t run_set(const AttendArgs& a, hipStream_t s) {
    const size_t lds = kSet ? (a.n_groups + 1) * sizeof(uint32_t)
                            : (a.R + 1) * sizeof(uint32_t) + std::min(a.R, kCached) * sizeof(Request);
    if (a.tile[kSet] == Wide<D>::kTile)
        hipLaunchKernelGGL((attend_wide_kernel<E, D, kSet>), dim3(a.workers[kSet]), dim3(Wide<D>::kThreads), lds, s, a);
    else if (a.tile[kSet] == 64)
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
    hipLaunchKernelGGL(attend_join_kernel<E>, dim3(a.workers[0], a.tile[0] / (kT / (D / 8))), dim3(kT), 0, s, a);
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
    size_t n = slots_bytes(D) + round256(kAttendMaxWorkers * sizeof(AttendEnd));
    if (n_groups) n += slots_bytes(D) + round256((size_t)(n_groups + 1) * 4) + dense_bytes(R, H, D, max_new);
    return n;
}

void attend_ws_layout(AttendArgs& a, void* ws) {
    char* p = (char*)ws;
    a.slots[0] = (float*)p;
    p += slots_bytes(a.D);
    a.ends = (AttendEnd*)p;
    p += round256(kAttendMaxWorkers * sizeof(AttendEnd));
    if (!a.n_groups) return;
    a.slots[1] = (float*)p;
    p += slots_bytes(a.D);
    a.cum = (uint32_t*)p;
    p += round256((size_t)(a.n_groups + 1) * 4);
    a.dense = (float*)p;
}

hipError_t launch_attend(AttendArgs a, int cus, hipStream_t s) {
    // The many-rows form where a request (a group) may have more columns than the other form
    // takes at once; else 64 columns to a workgroup where it may have more than 32.
    const int wide = a.D == 64 ? Wide<64>::kTile : a.D == 128 ? Wide<128>::kTile : Wide<256>::kTile;
    for (int set = 0; set < 2; ++set) {
        const long long columns = (long long)(set ? a.rows : a.max_new) * a.G;
        a.tile[set] = columns > kWideFrom ? wide : columns > 32 ? 64 : 32;
        a.unit[set] = a.tile[set] == 32 ? 128 : 64;
        const int per_cu = a.tile[set] == wide ? (a.D == 64 ? Wide<64>::kPerCu : 1) : a.D <= 128 ? 2 : 1;
        a.workers[set] = std::min(cus * per_cu, kAttendMaxWorkers);
        a.tile_shift[set] = __builtin_ctz(a.tile[set]);
        a.unit_shift[set] = __builtin_ctz(a.unit[set]);
    }
    return a.dtype == DSPARK_F16 ? run_dim<F16>(a, s) : run_dim<Bf16>(a, s);
}

}  // namespace dspark
