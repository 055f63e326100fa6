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
// Work: the keys are cut into units of 64 or 128.  Every workgroup, a worker, takes the same
// number of consecutive units, in the order request, key head, tile, unit, so few long contexts
// and many short ones fill the device alike; a segment (request, key head, tile) that ends
// inside one worker is finished there, and the parts of one that is split are joined by a
// kernel of their own.  Shared prefixes are a launch of their own, whose segments are a group's
// rows taken together, so that its keys are read once for all of them; where there are such,
// the last kernel joins each row's own part and its group's.
//
// Forms: with few columns the keys' bytes are the bound, and every wave streams its keys from
// memory straight into the matrix instruction's registers (attend_kernel).  With many the
// matrix and vector units are, and the keys come to LDS once for all waves
// (attend_wide_kernel).  Each kernel says what it reaches.
//
// Masks: only blocks that reach past a column's last key are masked.  What lies in masked
// places has no say whatever it is: scores are replaced, V past the end is cleared, and a
// value of V that is not a number in such a block is taken out of the product and handed
// to the columns that see it by counting (see add_special).
#include <algorithm>
#include <type_traits>

#include "cache.h"
#include "common.h"

namespace dspark {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kT = 256;
// The form of a launch, by the columns that one request (a group) may have.  Up to 32 fill one
// wave's tile, up to 64 two waves'; beyond them the many-rows form reads the keys once for 128
// or 256 columns.  From 33 on it would be slower where few are filled (256 requests of
// up to 64 columns, 514 tokens each: 177 us against 275), from 129 on the few-rows form would read the
// keys of 65 to 128 columns twice (two requests of up to 131072 tokens and 72 columns: 194 against 200).
constexpr int kWideFrom = 64;
// The units that are worth a workgroup of their own: fewer spread a small call over more of
// the device, more leave fewer parts to join.  Many rows: 1, 4, 8 give 58, 56, 59 us for 16
// requests behind 2048 shared tokens, and 232, 241, 270 where 1145 rows share 64.  Few rows: an
// eighth of what a request brings to a key head on average, at least 1 and at most 8, so that a
// segment has about eight parts: four single tokens after up to 700 take 12.7 us with 1 and 24.7
// with 8, one after 8192 takes 31.6 with 1 and 22.1 with 8; with 2 for both, 14.7 and 25.1.
constexpr int kWideLeast = 4, kFewParts = 8, kFewMost = 8;
constexpr float kInf = __builtin_huge_valf();
// The running maximum follows only when it grows by more than this exponent of two; until
// then the weights are taken relative to the older one, at most 2^8, and nothing that has
// been summed has to be rescaled.  The weights and their sums are besides scaled by 2^kRaise of
// their type: an fp16 weight below half of its smallest number, 2^-24, would be zero in the
// second product and not in the sum, and a long row of such keys would be missing from the
// result (600 keys of 2^-26 each: 38% of it).  With 2^6 that ends at 2^-31, and the largest
// weight, 2^14, stays a factor of four below fp16's largest number.  bf16 has fp32's exponents.
constexpr float kLag = 8.f;
// A weight is exp2 of one fused multiply-add, score times scale minus the scaled maximum, whose
// rounding all weights of a part have in common.  Past this exponent of two that rounding (2^-4
// here) would grow to whole powers of two, at 2^25 past fp16's range and at 2^31 past fp32's; such
// a wave subtracts the maximum from its scores first, which is exact near the maximum.
constexpr float kLarge = 1048576.f;

struct Bf16 {
    static constexpr float kRaise = 0.f;
    static constexpr uint32_t kExp = 0x7F80u, kMant = 0x007Fu, kOne = 0x3F80u, k64 = 0x4280u, k4096 = 0x4580u;
    static __device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint16_t bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
};
struct F16 {
    static constexpr float kRaise = 6.f;
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
    if (a.cum[1][a.n_groups] == 0) return -1;  // no group counts, as their launch has found (see plan)
    int lo = 0, hi = a.n_groups;  // the last group that starts at or before r
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.group_off[mid] <= r) lo = mid + 1; else hi = mid;
    }
    return lo > 0 && r < a.group_off[lo] ? lo - 1 : -1;
}

// A group's rows [start, start + n) and the keys [0, ke) that they share; ke = 0 for none.
// The rows end where the buffer does: a request of the group whose rows pass it is left out
// by itself.
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
    const long long all = a.rows, s0 = (long long)a.offsets[r0] + (long long)a.lead * r0,
                    s1 = (long long)a.offsets[r1] + (long long)a.lead * r1;
    const long long from = min(max(s0, 0ll), all), to = min(max(s1, from), all);
    q.start = (int)from;
    q.n = (int)(to - from);
    q.ke = sp * a.page;
    return q;
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
            // Where the group does not fit, or its rows are not around this request's (as offsets
            // that fall have it), the request reads its own table, which holds those keys too.
            const Group g = shared_of(a, q.group, bad);
            if (q.start >= g.start && q.start + q.n <= g.start + g.n) {
                if (g.ke > q.ln) {
                    bad = kStatusBadRow;
                    return 0;
                }
                q.kb = g.ke;
            }
        }
    }
    return 1;
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

// How a launch's units are dealt to its workers: each takes `each` consecutive ones, the first
// `more` one more than that.  Workers beyond one for every `least` units have none.
struct Split {
    uint32_t each, more;
    int workers;
    __device__ __forceinline__ Split(const AttendArgs& a, int set, uint32_t total) {
        const uint32_t least =
            a.least[set] ? (uint32_t)a.least[set] : min(max(total / a.parts[set], 1u), (uint32_t)kFewMost);
        workers = min((uint32_t)a.workers[set], (total + least - 1) / least);
        each = workers ? total / (uint32_t)workers : 0;
        more = workers ? total % (uint32_t)workers : 0;
    }
    __device__ __forceinline__ uint32_t first(uint32_t w) const { return w * each + min(w, more); }
    __device__ __forceinline__ int worker_of(uint32_t u) const {
        const uint32_t big = more * (each + 1);
        return (int)(u < big ? u / (each + 1) : more + (u - big) / each);
    }
    // Which worker a workgroup is.  Those of one XCD, every eighth workgroup, take units next to
    // each other, so that keys which many columns see come through its L2 (two groups of 4096
    // tokens, 4096 rows: 265 to 257 us).  A segment's worker w is then not workgroup w.
    __device__ __forceinline__ int by_xcd() const {
        const int b = blockIdx.x, xcd = b & 7;
        return b < workers ? xcd * (workers / 8) + min(xcd, workers % 8) + (b >> 3) : b;
    }
};

__device__ __forceinline__ float* slot_of(const AttendArgs& a, int set, int worker, int which) {
    return a.slots[set] + (size_t)(worker * 2 + which) * ((size_t)a.tile[set] * (a.D + 2));
}

// Running units (of one key head) of the items in LDS, and what each of the first kCached
// brings, so that a workgroup looks at the requests once; with shared prefixes the running
// units are kept for the kernel that joins the parts.  Returns the units of all heads.
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
    // More units than 32 bits number can only come from offsets that fall and rise again, so
    // that requests or groups share rows: the sums then stop past the bound, and none are served.
    // So do the groups' where group_off fall: groups may then have requests in common, and each
    // would leave parts of their rows.  Without groups the requests read their own tables.
    const uint32_t most = min(0x7FFFFFFFu / (uint32_t)a.Hkv, 0x7FFFFFFEu);
    uint32_t base = 0, bad = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        uint32_t x = 0;
        if (i < n) {
            if (kSet) {
                const Group g = shared_of(a, i, bad);
                x = (uint32_t)tiles_in(a, 1, g.n) * units_in(a, 1, g.ke);
                if (a.group_off[i + 1] < a.group_off[i]) x = most + 1;
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
            if (lane >= d) y = min(y + z, most + 1);
        }
        __syncthreads();
        if (lane == 63) s_base[wave] = y;
        __syncthreads();
        for (int w = 0; w < wave; ++w) y = min(y + s_base[w], most + 1);
        if (i < n) s_cum[i] = min(base + y, most + 1) - x;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) base = min(base + s_base[w], most + 1);
    }
    if (tid == 0) s_cum[n] = base;
    __syncthreads();
    if (base > most) {
        for (int i = tid; i <= n; i += kThreads) s_cum[i] = 0;
        base = 0;
        bad = kStatusBadRow;
        __syncthreads();
    }
    if (blockIdx.x == 0) {
        if (a.n_groups)
            for (int i = tid; i <= n; i += kThreads) a.cum[kSet][i] = s_cum[i];
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

// What one item (request or group) brings: its rows, the keys [kb, ke) that this launch
// gives them and the table that these lie in.  The last key that row j sees is ln + j.
struct Work {
    int start, n, kb, ke, ln, group;
    const int32_t* table;
};

template <int kSet>
__device__ __forceinline__ void work_of(const AttendArgs& a, int i, int n, const uint32_t* s_cum, Work& w) {
    uint32_t bad = 0;
    if (kSet) {
        const Group g = shared_of(a, i, bad);
        w.start = uniform(g.start);
        w.n = uniform(g.n);
        w.ke = uniform(g.ke);
        w.table = a.shared_table + (size_t)i * a.shared_width;
        return;
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
}

// A request's table has to begin with its group's pages.  One wave.
__device__ void check_prefix(const AttendArgs& a, const Work& q) {
    bool differs = false;
    const int32_t* shared = a.shared_table + (size_t)q.group * a.shared_width;
    for (int p = threadIdx.x & 63; p < q.kb >> a.page_shift; p += 64) differs |= q.table[p] != shared[p];
    if (differs) raise_status(a.status, kStatusBadPage);
}

// Adds a part (maximum pm and sum pl of one column, x and y eight of its values) to a running one.
// A part that saw no key has a sum of zero.  Its maximum does not say so: scores that are all NaN
// leave it at -inf too, and their part has to make the result NaN.
__device__ __forceinline__ void join(float& m, float& l, float (&acc)[8], float pm, float pl, float4 x, float4 y) {
    if (pl == 0.f) return;
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

// Where a launch leaves the part of a column of a segment that it did not split: set 0 where
// the requests' shared keys are still to be joined, set 1 always.
struct Dense {
    float *o, *m, *l;
};
__device__ __forceinline__ Dense dense_of(const AttendArgs& a, int set, int f, int h) {
    const size_t all = (size_t)a.Hkv * a.rows * a.G, at = (size_t)h * a.rows * a.G + f;
    float* p = a.dense[set];
    return Dense{p + at * a.D, p + all * a.D + at, p + all * (a.D + 1) + at};
}

// Adds what launch `set` has of query row f (row G + head of the group) of key head h: column c
// of its item, whose first unit is u0 and whose key heads have `tiles` tiles of `units`.
__device__ __forceinline__ void join_item(const AttendArgs& a, int set, const Split& split, uint32_t u0, int tiles,
                                          uint32_t units, int f, int c, int h, int c8, float& m, float& l, float (&acc)[8]) {
    const uint32_t u = u0 + (h * tiles + (c >> a.tile_shift[set])) * units;
    const int wa = split.worker_of(u), wb = split.worker_of(u + units - 1);
    if (wa == wb) {
        const Dense d = dense_of(a, set, f, h);
        join(m, l, acc, *d.m, *d.l, *(const float4*)(d.o + c8 * 8), *(const float4*)(d.o + c8 * 8 + 4));
    } else {
        join_parts(a, set, wa, wb, c & (a.tile[set] - 1), c8, m, l, acc);
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

// Column c of the tile at f0 is done as far as this worker goes: eight dims of it, from 8 c8
// on.  The result, where the segment ends here and has all of its keys (final); else the
// part, for whoever joins it.
template <class E, int kSet>
__device__ __forceinline__ void finish(const AttendArgs& a, int worker, bool final, bool whole, bool begins, int f0, int c,
                                       int h, int c8, float m, float l, const float (&acc)[8]) {
    if (kSet == 0 && final) {
        store_row<E>(a, f0 + c, h, c8, m, l, acc);
        return;
    }
    Dense d;
    if (whole) {
        d = dense_of(a, kSet, f0 + c, h);
    } else {
        const size_t tile = a.tile[kSet];
        float* slot = slot_of(a, kSet, worker, begins);
        d = Dense{slot + (size_t)c * a.D, slot + tile * a.D + c, slot + tile * (a.D + 1) + c};
    }
    *(float4*)(d.o + c8 * 8) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    *(float4*)(d.o + c8 * 8 + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
    if (c8 == 0) {
        *d.m = m;
        *d.l = l;
    }
}

// A wave's 32 columns done, from c0 of the tile at f0 on: 32 dims at a time through LDS (pitch
// 36: the lanes' 16-byte stores and loads meet no bank twice), eight dims of a column to a
// lane.  m and l are the lanes' columns'.
constexpr int kPitch = 36;

template <class E, int kSet, int NT>
__device__ __forceinline__ void finish_wave(const AttendArgs& a, float* s_o, int worker, bool final, bool whole,
                                            bool begins, int f0, int c0, int nf, int h, float m, float l, const f32x16 (&o)[NT]) {
    const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
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
            const float jm = __shfl(m, c, 64), jl = __shfl(l, c, 64);
            const float4 x = *(const float4*)&s_o[c * kPitch + c8 * 8], y = *(const float4*)&s_o[c * kPitch + c8 * 8 + 4];
            const float acc[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            if (c0 + c < nf) finish<E, kSet>(a, worker, final, whole, begins, f0, c0 + c, h, t * 4 + c8, jm, jl, acc);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Whether a column's maximum m (of the raw scores) is finite and larger than kLarge says.
__device__ __forceinline__ bool any_large(float m, float scale_log2) {
    return __ballot(m != -kInf && fabsf(m) * scale_log2 > kLarge) != 0;
}

// The larger of a lane's value and that of the lane 32 on; and their sum.
__device__ __forceinline__ float max_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

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
    }
    // Waits for the ids here, so that readers need not wait for what else is under way.
    __device__ __forceinline__ void settle() { asm volatile("" : "+v"(ids)); }
    __device__ __forceinline__ int at(int i, int lane) {
        if (i - base >= 64) {
            fetch(i, lane);
            settle();
        }
        return __builtin_amdgcn_readlane(ids, i - base);
    }
};

// A barrier for what the waves leave each other in LDS; loads from memory stay under way.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A worker's way through its units: the segment at hand, and the item it belongs to.
template <int kSet, int kTile, int kUnit>
struct Cursor {
    uint32_t u, u_end;
    uint32_t item_u0 = 0, item_u1 = 0;  // units of the item
    Work q{};
    uint32_t units, unit0, unit1;  // the segment's units; those [unit0, unit1) are the worker's
    int h, f0, nf;                 // its key head and columns

    int worker;
    bool leads;  // this lane speaks for the worker

    __device__ __forceinline__ Cursor(const Split& split, int w, bool lead)
        : u(split.first(w)), u_end(split.first(w + 1)), worker(w), leads(lead) {}
    // The segment of unit u.
    __device__ __forceinline__ void look(const AttendArgs& a, const Split& split, int n, const uint32_t* s_cum) {
        if (u >= item_u1) {
            const int i = item_of(a, s_cum, n, u);
            item_u0 = uniform(s_cum[i]) * a.Hkv;
            item_u1 = uniform(s_cum[i + 1]) * a.Hkv;
            work_of<kSet>(a, i, n, s_cum, q);
        }
        units = units_of<kUnit>(q.ke - q.kb);
        const uint32_t tiles = tiles_of<kTile>(a, q.n), in = u - item_u0, seg = in / units;
        unit0 = in % units;
        unit1 = min(units, unit0 + (u_end - u));
        h = seg / tiles;
        const int tile = seg % tiles;
        f0 = q.start * a.G + tile * kTile;
        nf = min(kTile, q.n * a.G - tile * kTile);
        if (kSet == 0 && q.kb > 0 && seg == 0 && unit0 == 0) check_prefix(a, q);
        if (kSet == 0 && unit0 > 0 && leads)  // begun by an earlier worker: for the joining kernel
            a.ends[worker] = AttendEnd{units, split.worker_of(u - unit0), split.worker_of(u - unit0 + units - 1), f0,
                                           nf, h};
    }
    __device__ __forceinline__ bool whole() const { return unit0 == 0 && unit1 == units; }
    // On to the next segment; false where there is none.
    __device__ __forceinline__ bool step() {
        u += unit1 - unit0;
        return u < u_end;
    }
    // The last key that the columns of query row f / G see.
    __device__ __forceinline__ int last_of(const AttendArgs& a, int f) const {
        return kSet ? q.ke - 1 : q.ln + f / a.G - q.start;
    }
};

// Q^T as the first product's second operand: column f's dims 16 c + 8 half + 0..7.
template <int D>
__device__ __forceinline__ void load_q(const AttendArgs& a, s16x8 (&qf)[D / 16], int f, int h, int half) {
    const uint16_t* qp = a.q + (size_t)(f / a.G) * a.q_stride + (size_t)(h * a.G + f % a.G) * D + half * 8;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) qf[c] = *(const s16x8*)(qp + c * 16);
}

// The few-rows form.  A workgroup takes kTiles tiles of the segment's columns: its four
// waves are 4 / kTiles groups of keys by kTiles tiles, so that up to 64 columns read the
// keys once.  Each wave streams: the next block's K is requested as soon as the first product
// has used this one's, the next V after the second product, so about 16 KB a wave are under way
// while it computes; and the next segment's rows, page ids and first keys are requested before
// this one's waves are joined (kSet 0: the requests' own keys; 1: the groups' shared ones).
//
// 256 requests of 1145 rows, 64 query and 8 key heads of 128, bf16: 176 us for 131500 tokens
// (539 MB, 3.1 TB/s), 512 for four times as many (4.2 TB/s): the loads bound it, and the joining
// of four waves at each of 2048 segments.  Four single tokens, 1750 tokens in all: 9 us, of
// which the bytes would take 1.3; the others are loads that wait for each other, from the
// requests' rows to their page ids, keys, values and the parts.
template <class E, int D, int kSet, int kTiles>
__global__ __launch_bounds__(kT, D <= 128 ? 2 : 1) void attend_kernel(AttendArgs a) {
    constexpr int NT = D / 32, NC = D / 16;
    constexpr int kKeyWaves = 4 / kTiles;
    constexpr int kUnit = 32 * kKeyWaves;
    constexpr int kDims = D <= 128 ? D : 128;  // dims joined over the waves at a time
    constexpr int kRow = kDims + 4;
    __shared__ __attribute__((aligned(16))) float s_o[4][32][kRow];
    static_assert(__alignof__(s_o) == 16 && kRow % 4 == 0, "read as float4");
    __shared__ float s_m[4][32], s_l[4][32];
    __shared__ uint32_t s_base[8];
    extern __shared__ uint32_t s_cum[];  // running units, n + 1, then the requests
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int key_wave = wave / kTiles, sub = wave % kTiles;
    const int n = kSet ? a.n_groups : a.R;
    const uint32_t total = plan<kSet, kT>(a, n, s_cum, s_base);
    const Split split(a, kSet, total);
    if (kSet == 0 && tid == 0) a.ends[blockIdx.x].units = 0;
    if ((int)blockIdx.x >= split.workers) return;
    const int shift = a.page_shift - 4, in_page = (1 << shift) - 1;  // blocks of 16 in a page
    const int head_shift = __builtin_ctz(D) + a.page_shift;          // a head's elements in a page
    const int swapped = (col & 3) | ((col & 4) << 1) | ((col & 8) >> 1);  // key of this lane in its block of 16

    Cursor<kSet, 32 * kTiles, kUnit> cur(split, blockIdx.x, tid == 0);
    s16x8 qf[NC], kf[NC], vf[NT][2];
    f32x16 o[NT];
    PageIds pages;
    const uint16_t *kp[2], *vp[2];
    bool have[2], bad_page = false;
    int pos, pos_end, last, first_last;

    // The two blocks of 16 keys at position p: where K and V lie, and whether they are there.
    const auto locate = [&](int p, bool(&there)[2]) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int blk = (p >> 4) + b;
            there[b] = p + b * 16 < cur.q.ke;
            int page = there[b] ? pages.at(blk >> shift, lane) : 0;
            if ((unsigned)page >= (unsigned)a.n_pages) {
                page = 0;
                there[b] = false;
                bad_page = true;
            }
            const size_t at =
                (((size_t)(unsigned)page * (unsigned)a.Hkv + cur.h) << head_shift) + (size_t)(blk & in_page) * (16 * D);
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
    // A segment's beginning, in two steps: its columns and page ids, then its first keys.
    const auto enter = [&]() {
        const int f = cur.f0 + min(sub * 32 + col, cur.nf - 1);
        load_q<D>(a, qf, f, cur.h, half);
        last = cur.last_of(a, f);               // the column's last key
        first_last = cur.last_of(a, cur.f0);  // the earliest of them
        pos = cur.q.kb + (int)(cur.unit0 * kUnit) + key_wave * 32;
        pos_end = sub * 32 < cur.nf ? min(cur.q.ke, cur.q.kb + (int)(cur.unit1 * kUnit)) : 0;
        if (pos < pos_end)
            pages.start(cur.q.table, (cur.q.ke + (1 << a.page_shift) - 1) >> a.page_shift, pos >> a.page_shift, lane);
    };
    const auto first_keys = [&]() {
        if (pos >= pos_end) return;
        pages.settle();
        locate(pos, have);
        load_k();
        __builtin_amdgcn_sched_barrier(0);  // K first, as in the loop: its waits count on this order
        load_v();
    };

    // What joining a finished segment's waves needs, while the next segment is at hand.
    float ms = -kInf, l = 0.f;
    bool final = false, whole = false, begins = false;
    int f0 = 0, nf = 0, h = 0;
    // The waves' parts joined, column by column, eight dims to a thread, kDims dims at a time.
    const auto put = [&](int d0) {
        lds_barrier();
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
        lds_barrier();
    };
    const auto take = [&](int d0) {
        for (int e = tid; e < nf * (kDims / 8); e += kT) {
            const int c = e / (kDims / 8), c8 = e % (kDims / 8);
            float jm = -kInf, jl = 0.f, acc[8] = {};
#pragma unroll
            for (int w = 0; w < kKeyWaves; ++w) {
                const int from = w * kTiles + c / 32;
                join(jm, jl, acc, s_m[from][c % 32], s_l[from][c % 32], *(const float4*)&s_o[from][c % 32][c8 * 8],
                     *(const float4*)&s_o[from][c % 32][c8 * 8 + 4]);
            }
            finish<E, kSet>(a, blockIdx.x, final, whole, begins, f0, c, h, d0 / 8 + c8, jm, jl, acc);
        }
    };

    bool more = true;
    for (bool first = true;; first = false) {
        if (more) {
            cur.look(a, split, n, s_cum);
            enter();
        }
        if (D <= kDims) {
            if (!first) put(0);
            if (more) first_keys();  // on their way while the last segment is joined
            if (!first) take(0);
        } else {  // (no registers for both)
            if (!first) {
#pragma unroll
                for (int d0 = 0; d0 < D; d0 += kDims) {
                    put(d0);
                    take(d0);
                }
            }
            if (more) first_keys();
        }
        if (!more) break;
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t] = f32x16{};
        float m = -kInf, mc = 0.f;  // of the raw scores, and scaled; l is this half's share of the sum
        bool large = false;
        l = 0.f;
        int special_from = -1;     // the first block with values that add_special has to add
        // One block of 32 keys: scores, weights, and the second product.  kFast: all of its keys
        // are seen by all columns, and another block follows, whose K and V are requested with no
        // condition (a load that may be left out would have every later wait count on its absence).
        const auto block = [&](auto fast) {
            constexpr bool kFast = decltype(fast)::value;
            f32x16 s = {};
#pragma unroll
            for (int c = 0; c < NC; ++c) s = E::mfma(kf[c], qf[c], s);
            const int next = pos + kUnit;
            const bool follows = kFast || next < pos_end;
            bool next_have[2] = {false, false};
            if (follows) {
                locate(next, next_have);
                load_k();
            }
            const bool masked = !kFast && (pos + 31 > first_last || !have[0] || !have[1]);
            if (masked) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (pos + (j / 8) * 16 + half * 8 + j % 8 > last || !have[j / 8]) s[j] = -kInf;
            }
            float mx = s[0];
#pragma unroll
            for (int j = 1; j < 16; ++j) mx = fmaxf(mx, s[j]);
            mx = max_halves(mx);
            if (__ballot((mx - m) * a.scale_log2 > kLag) || large) {
                const float m_new = fmaxf(m, mx);
                const float alpha = __builtin_amdgcn_exp2f((m - (m_new == -kInf ? 0.f : m_new)) * a.scale_log2);
                m = m_new;
                mc = m == -kInf ? 0.f : m * a.scale_log2 - E::kRaise;
                l *= alpha;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[t][j] *= alpha;
                large = any_large(m, a.scale_log2);
                if (large) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] -= m == -kInf ? 0.f : m;
                    mc = -E::kRaise;
                }
            }
            s16x8 pf[2];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j], a.scale_log2, -mc));
                l += p;
                pf[j / 8][j % 8] = (short)E::bits(p);  // the weights, rounded for the matrix instruction
            }
            if (masked) {
                uint32_t special = 0;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        special |= clear_masked<E>(vf[t][b], have[b] ? cur.q.ke - (pos + b * 16 + half * 8) : 0);
                        __builtin_amdgcn_sched_barrier(0);  // one after the other, in few registers
                    }
                if (special_from < 0 && __ballot(special != 0)) special_from = pos;
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t] = E::mfma(vf[t][1], pf[1], E::mfma(vf[t][0], pf[0], o[t]));
            if (follows) load_v();
            pos = next;
            have[0] = next_have[0];
            have[1] = next_have[1];
        };
        if (pos + kUnit < pos_end && pos + 31 <= first_last && have[0] && have[1]) {
            // What is on its way is waited for here, where other loads and stores may be too; inside
            // the loop the waits then count on the order of the loop's own loads.
#pragma unroll
            for (int c = 0; c < NC; ++c) asm volatile("" : "+v"(kf[c]));
#pragma unroll
            for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(vf[t][0]), "+v"(vf[t][1]));
            do block(std::true_type{});
            while (pos + kUnit < pos_end && pos + 31 <= first_last && have[0] && have[1]);
        }
        while (pos < pos_end) block(std::false_type{});
        l = add_halves(l);
        if (special_from >= 0) {
            pages.fetch(special_from >> a.page_shift, lane);
            pages.settle();
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
        ms = m == -kInf ? -kInf : m * a.scale_log2 - E::kRaise;
        whole = cur.whole();
        begins = cur.unit0 == 0;
        f0 = cur.f0;
        nf = cur.nf;
        h = cur.h;
        final = whole && cur.q.kb == 0;
        more = cur.step();
    }
    if (bad_page && lane == 0) raise_status(a.status, kStatusBadPage);
}

// The many-rows form, for groups and prompts: a wave takes 32 columns, the workgroup eight
// (at head_dim 64 and 256: four) times as many, and all waves read the same 64 keys from LDS,
// which the next 64 are brought to meanwhile (global_load_lds: memory to LDS with no registers
// between).  The lanes of such a load pick their 16 bytes so that what 16 lanes read later,
// for an operand of a matrix instruction, lies in different banks.
//
// With eight waves two share a SIMD, and they are half a stage apart: while one multiplies, the
// other makes weights of its scores, which takes the vector unit about as long (1024 matrix
// cycles and 1000 of the other a stage), so both units work.  In step with each other, every
// wave's operands waited for one by one, the same loop took 350 us where this one takes 320.
// Reading the operands a group ahead, four at a time, is worth a further third of the product's
// time; nothing with a mask is in the products' path (see clean), for two paths cost copies of
// the accumulators and spills.
//
// 1145 rows behind 8192 shared tokens, 64 query and 8 key heads of 128, bf16: 320 us, 960
// TFLOP/s.  No unit is the bound: the matrix units are busy 44% of the time and LDS 24%.  Waves
// spend 39% of theirs on an issue slot or a result and 28% at the two barriers a stage and on loads,
// which are asked for in the half stage that ends by waiting for them.
// More columns a wave would need twice the accumulators, and leave one wave a SIMD and nothing
// to work while it waits.
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
    constexpr int NT = D / 32, NC = D / 16;
    constexpr int kStage = 8 * W::kBlock * 2, kJoin = W::kWaves * 32 * kPitch * 4;  // bytes
    __shared__ __attribute__((aligned(16))) char s_mem[2 * kStage > kJoin ? 2 * kStage : kJoin];
    __shared__ __attribute__((aligned(16))) int s_have[4][4];
    static_assert(__alignof__(s_have) == 16 && __alignof__(s_mem) == 16, "read as int4, float4 and eight 16-bit values");
    __shared__ int s_special;
    __shared__ uint32_t s_base[8];
    extern __shared__ uint32_t s_cum[];  // running units, n + 1, then the requests
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int n = kSet ? a.n_groups : a.R;
    const uint32_t total = plan<kSet, W::kThreads>(a, n, s_cum, s_base);
    const Split split(a, kSet, total);
    const int me = split.by_xcd();
    if (kSet == 0 && tid == 0) a.ends[me].units = 0;
    if (me >= split.workers) return;
    const int shift = a.page_shift - 4, in_page = (1 << shift) - 1;  // blocks of 16 in a page
    const int head_shift = __builtin_ctz(D) + a.page_shift;          // a head's elements in a page
    // where this lane's 16 bytes of each 1 KB of a block come from: K's keys with bits 2 and 3 of
    // their number swapped, V's halves of 16 tokens one after the other
    const int key = lane & 15, k_from = (lane >> 4) * 128 + ((key & 3) | ((key & 4) << 1) | ((key & 8) >> 1)) * 8;
    const int v_from = lane / 2 * 16 + ((lane ^ (lane >> 4)) & 1) * 8, v_at = (col * 2 + (half ^ ((col >> 3) & 1))) * 16;

    Cursor<kSet, W::kTile, W::kUnit> cur(split, me, tid == 0);
    do {
        cur.look(a, split, n, s_cum);
        const Work& q = cur.q;
        const int f0 = cur.f0, nf = cur.nf, h = cur.h;
        const int f = f0 + min(wave * 32 + col, nf - 1);
        s16x8 qf[NC];
        load_q<D>(a, qf, f, h, half);
        // The column's last key; the wave's earliest and latest of them, and the tile's latest.
        const int last = cur.last_of(a, f), first_last = cur.last_of(a, f0 + min(wave * 32, nf - 1));
        const int wave_end = wave * 32 >= nf ? 0 : cur.last_of(a, f0 + min(wave * 32 + 31, nf - 1)) + 1;
        const int tile_end = cur.last_of(a, f0 + nf - 1) + 1, tile_first = cur.last_of(a, f0);

        f32x16 o[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t] = f32x16{};
        float m = -kInf, mc = 0.f, l = 0.f;  // m of the raw scores, mc scaled; l this half's share of the sum
        bool large = false;
        int pos = q.kb + (int)(cur.unit0 * W::kUnit);
        const int pos_end = min(tile_end, q.kb + (int)(cur.unit1 * W::kUnit));
        const int stages = pos < pos_end ? (pos_end - pos + W::kUnit - 1) / W::kUnit : 0, pos0 = pos;

        // The first four waves each bring a block's K and the others its V, or each of four waves
        // the K and a stage later the V.  Where the blocks of 64 stages are stands in the lanes.
        uint32_t at_low = 0, at_high = 0;
        uint64_t there = 0, bad_pages = 0;
        const auto element = [&](int page, int p) {
            return (((size_t)(unsigned)page * (unsigned)a.Hkv + h) << head_shift) + (size_t)(p >> 4 & in_page) * W::kBlock;
        };
        const auto locate = [&](int t) {
            const int p = pos0 + (t + lane) * W::kUnit + (wave & 3) * 16;
            const bool wanted = t + lane < stages && p < q.ke;
            int page = wanted ? q.table[p >> a.page_shift] : 0;
            const bool bad = (unsigned)page >= (unsigned)a.n_pages;
            if (bad) page = 0;
            there = __ballot(wanted && !bad);
            bad_pages |= __ballot(bad);
            const size_t at = element(page, p);
            at_low = (uint32_t)at, at_high = (uint32_t)(at >> 32);
        };
        size_t at = 0;
        const auto find = [&](int t) {
            if (!(t & 63)) locate(t);
            at = (size_t)__builtin_amdgcn_readlane(at_high, t & 63) << 32 |
                 (uint32_t)__builtin_amdgcn_readlane(at_low, t & 63);
        };
        const auto bring = [&](int t, int kv) {
            const uint16_t* from = kv ? a.v + at + v_from : a.k + at + k_from;
            char* to = s_mem + (t & 1) * kStage + (kv * 4 + (wave & 3)) * (W::kBlock * 2);
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from + j * 512),
                                                 (__attribute__((address_space(3))) void*)(to + j * 1024), 16, 0, 0);
        };
        const auto bring_keys = [&](int t) {
            if (t >= stages) return;
            find(t);
            if (lane == 0) s_have[t & 3][wave & 3] = (int)(there >> (t & 63)) & 1;
            bring(t, 0);
        };
        const auto bring_values = [&](int t) {
            if (t >= stages) return;
            if (W::kWaves == 8) find(t);
            bring(t, 1);
        };
        const auto wait_loads = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };
        // Stage t's scores; its weights, from the scores; its second product, from the weights.
        f32x16 s[2];
        s16x8 pf[4];
        bool masked = false;
        const auto scores = [&](int t) {
            const char* mem = s_mem + (t & 1) * kStage + (half * 16 + (col & 15)) * 16 + (col >> 4) * (W::kBlock * 2);
            s[0] = s[1] = f32x16{};
            s16x8 kf[2][4];
            const auto read = [&](int g) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    kf[g & 1][j] = *(const s16x8*)(mem + (j & 1) * (W::kBlock * 4) + (g * 2 + j / 2) * 512);
            };
            const int4 have = *(const int4*)s_have[t & 3];
            read(0);
#pragma unroll
            for (int g = 0; g < NC / 2; ++g) {
                if (g + 1 < NC / 2) read(g + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j & 1] = E::mfma(kf[g & 1][j], qf[g * 2 + j / 2], s[j & 1]);
                __builtin_amdgcn_sched_barrier(0);
            }
            masked = pos0 + t * W::kUnit + 63 > first_last || !uniform(have.x & have.y & have.z & have.w);
        };
        const auto weights = [&](int t) {
            if (masked) {
                const int4 have = *(const int4*)s_have[t & 3];
                int left = last - (pos0 + t * W::kUnit) - half * 8;
                asm volatile("" : "+v"(left));  // so that no key's number takes a register in the loop
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int there = j < 8 ? have.x : j < 16 ? have.y : j < 24 ? have.z : have.w;
                    if ((j / 8) * 16 + j % 8 > left || !there) s[j / 16][j % 16] = -kInf;
                }
            }
            float mx = s[0][0];
#pragma unroll
            for (int j = 1; j < 32; ++j) mx = fmaxf(mx, s[j / 16][j % 16]);
            mx = max_halves(mx);
            if (__ballot((mx - m) * a.scale_log2 > kLag) || large) {
                const float m_new = fmaxf(m, mx);
                const float alpha = __builtin_amdgcn_exp2f((m - (m_new == -kInf ? 0.f : m_new)) * a.scale_log2);
                m = m_new;
                mc = m == -kInf ? 0.f : m * a.scale_log2 - E::kRaise;
                l *= alpha;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[i][j] *= alpha;
                large = any_large(m, a.scale_log2);
                if (large) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) s[j / 16][j % 16] -= m == -kInf ? 0.f : m;
                    mc = -E::kRaise;
                }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j / 16][j % 16], a.scale_log2, -mc));
                l += p;
                pf[j / 8][j % 8] = (short)E::bits(p);  // the weights, rounded for the matrix instruction
            }
        };
        const auto values = [&](int t) {
            const char* vl = s_mem + (t & 1) * kStage + 4 * (W::kBlock * 2) + v_at;
            s16x8 vf[2][4];
            const auto read = [&](int g) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    vf[g & 1][j] = *(const s16x8*)(vl + ((g & 1) * 2 + j / 2) * (W::kBlock * 2) + (g / 2 * 2 + (j & 1)) * 1024);
            };
            read(0);
#pragma unroll
            for (int g = 0; g < NT; ++g) {
                if (g + 1 < NT) read(g + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[g / 2 * 2 + (j & 1)] = E::mfma(vf[g & 1][j], pf[(g & 1) * 2 + j / 2], o[g / 2 * 2 + (j & 1)]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // Where a column of the tile does not see all of stage t, its weights there are zero, but
        // zero times what is not finite is not: the wave that brought a block's V removes such
        // values, and all behind the last key, before anyone reads them.  What is removed and
        // seen is added behind the loop, from the first such stage on.
        const auto clean = [&](int t) {
            if (t >= stages) return;
            const int p = pos0 + t * W::kUnit + (wave & 3) * 16;
            const bool is_there = uniform(s_have[t & 3][wave & 3]);
            if (is_there && pos0 + t * W::kUnit + 63 <= tile_first) return;
            char* block = s_mem + (t & 1) * kStage + (4 + (wave & 3)) * (W::kBlock * 2) + lane * 16;
            const int keys = is_there ? q.ke - p - ((lane ^ (lane >> 4)) & 1) * 8 : 0;
            uint32_t special = 0;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                s16x8 v = *(const s16x8*)(block + i * 1024);
                special |= clear_masked<E>(v, keys);
                *(s16x8*)(block + i * 1024) = v;
                __builtin_amdgcn_sched_barrier(0);  // one after the other, in few registers
            }
            if (__ballot(special != 0) && lane == 0) atomicMin(&s_special, t);
        };
        const int seen = wave_end > pos0 ? min(stages, (wave_end - pos0 + W::kUnit - 1) / W::kUnit) : 0;  // by the wave

        if (tid == 0) s_special = 1 << 30;
        __syncthreads();  // LDS is free
        const bool late = wave >= 4;  // half a stage behind: a barrier more before, one fewer after
#pragma unroll
        for (int c = 0; c < NC; ++c) asm volatile("" : "+v"(qf[c]));  // there, so that no later wait is for them
        if (!late) bring_keys(0);
        wait_loads();
        lds_barrier();
        if (late) {
            bring_values(0);
            lds_barrier();
        }
        // K of stage t + 1 and V of stage t come while the early waves make stage t's weights and the
        // late ones are still at its scores: into the halves of LDS whose readers the barrier
        // before has let go, to be read after the next.  (Four waves, one a SIMD: in one step.)
        for (int t = 0; t <= stages; ++t) {
            if (W::kWaves == 4) {
                bring_values(t);
                bring_keys(t + 1);
            }
            if (t > 0 && t <= seen) values(t - 1);
            if (t < seen) scores(t);
            if (W::kWaves == 8) {
                if (late) {
                    wait_loads();
                    clean(t);
                }
                __builtin_amdgcn_sched_barrier(0);
                lds_barrier();
                if (late)
                    bring_values(t + 1);
                else
                    bring_keys(t + 1);
            }
            if (t < seen) weights(t);
            if (!late) wait_loads();
            if (W::kWaves == 4) clean(t);
            __builtin_amdgcn_sched_barrier(0);
            lds_barrier();
        }
        if (W::kWaves == 8 && !late) lds_barrier();
        l = add_halves(l);
        if (bad_pages && lane == 0) raise_status(a.status, kStatusBadPage);
        const int special_from = uniform(s_special);
        if (special_from < stages) {
            for (pos = pos0 + special_from * W::kUnit; pos < min(pos_end, wave_end); pos += 32) {
                size_t at[2];
                bool have[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int p = pos + b * 16;
                    const int page = p < q.ke ? q.table[p >> a.page_shift] : -1;
                    have[b] = (unsigned)page < (unsigned)a.n_pages;
                    at[b] = element(have[b] ? page : 0, p);
                }
                s16x8 sees[2];
                int left = last - pos - half * 8;
                asm volatile("" : "+v"(left));
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    sees[j / 8][j % 8] = (j / 8) * 16 + j % 8 <= left && have[j / 8] ? (short)E::kOne : (short)0;
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    add_special<E>(o[t], *(const s16x8*)(a.v + at[0] + t * 512 + col * 16 + half * 8),
                                   *(const s16x8*)(a.v + at[1] + t * 512 + col * 16 + half * 8), sees[0], sees[1]);
            }
        }
        m = m == -kInf ? -kInf : m * a.scale_log2 - E::kRaise;

        const bool whole = cur.whole();
        __syncthreads();  // LDS is free
        finish_wave<E, kSet, NT>(a, (float*)s_mem + wave * (32 * kPitch), me, whole && q.kb == 0, whole, cur.unit0 == 0, f0, wave * 32, nf,
                                 h, m, l, o);
    } while (cur.step());
}

// Joins the parts of the segments that were split, where no prefix is shared.  Where worker w
// goes on with a segment that worker w - 1 began, workgroup (w, .) joins it, eight dims of a
// column to a thread.
template <class E>
__global__ __launch_bounds__(kT) void attend_join_kernel(AttendArgs a) {
    const AttendEnd e = a.ends[blockIdx.x];
    if (e.units == 0 || e.first != (int)blockIdx.x - 1) return;
    const int chunks = a.D / 8, c = blockIdx.y * (kT / chunks) + threadIdx.x / chunks, c8 = threadIdx.x % chunks;
    if (c >= e.nf) return;
    float m = -kInf, l = 0.f, acc[8] = {};
    join_parts(a, 0, e.first, e.last, c, c8, m, l, acc);
    store_row<E>(a, e.f0 + c, e.h, c8, m, l, acc);
}

// Joins everything where prefixes are shared: a workgroup the columns of a request with one
// key head (up to kAttendJoinItems of eight dims), from its own launch and its group's.
static_assert(kAttendJoinItems % kT == 0, "as many items to every thread");
template <class E>
__global__ __launch_bounds__(kT) void attend_join_shared_kernel(AttendArgs a) {
    const int r = blockIdx.x, h = blockIdx.y, chunks = a.D / 8;
    Request q;
    uint32_t bad = 0;
    if (request_of(a, r, q, bad) != 1) return;
    const uint32_t own_units = a.cum[0][a.R] * a.Hkv, common_units = a.cum[1][a.n_groups] * a.Hkv;
    if (own_units == 0) return;  // offsets out of all bounds (see plan)
    const Split own(a, 0, own_units), common(a, 1, common_units);
    const uint32_t u0 = a.cum[0][r] * a.Hkv, units = units_in(a, 0, q.ln + q.n - q.kb);
    const int tiles = tiles_in(a, 0, q.n), f0 = q.start * a.G;
    if (q.kb == 0 && own.worker_of(u0) == own.worker_of(u0 + a.Hkv * tiles * units - 1)) return;  // all done already
    Group g{};
    uint32_t g_u0 = 0;
    if (q.kb > 0) {
        g = shared_of(a, q.group, bad);
        g_u0 = a.cum[1][q.group] * a.Hkv;
    }
    const int end = min((blockIdx.z + 1) * kAttendJoinItems, (uint32_t)(q.n * a.G * chunks));
    for (int e = blockIdx.z * kAttendJoinItems + threadIdx.x; e < end; e += kT) {
        const int c = e / chunks, c8 = e % chunks;
        float m = -kInf, l = 0.f, acc[8] = {};
        if (q.kb == 0) {  // its whole tiles are done already
            const uint32_t u = u0 + (h * tiles + (c >> a.tile_shift[0])) * units;
            if (own.worker_of(u) == own.worker_of(u + units - 1)) continue;
        }
        join_item(a, 0, own, u0, tiles, units, f0 + c, c, h, c8, m, l, acc);
        if (g.ke > 0)
            join_item(a, 1, common, g_u0, tiles_in(a, 1, g.n), units_in(a, 1, g.ke), f0 + c, f0 + c - g.start * a.G, h, c8, m,
                      l, acc);
        store_row<E>(a, f0 + c, h, c8, m, l, acc);
    }
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
    if (a.n_groups)
        hipLaunchKernelGGL(attend_join_shared_kernel<E>,
                           dim3(a.R, a.Hkv, ((size_t)a.max_new * a.G * (D / 8) + kAttendJoinItems - 1) / kAttendJoinItems), dim3(kT), 0,
                           s, a);
    else
        hipLaunchKernelGGL(attend_join_kernel<E>, dim3(a.workers[0], a.tile[0] / (kT / (D / 8))), dim3(kT), 0, s, a);
    return hipGetLastError();
}

template <class E>
hipError_t run_dim(const AttendArgs& a, hipStream_t s) {
    return a.D == 64 ? run<E, 64>(a, s) : a.D == 128 ? run<E, 128>(a, s) : run<E, 256>(a, s);
}

// Two parts a worker, of as many columns a compute unit as the forms have.
size_t slots_bytes(int D) {
    const int columns = std::max(D <= 128 ? 128 : 64, D == 64 ? Wide<64>::kPerCu * Wide<64>::kTile
                                                       : D == 128 ? Wide<128>::kTile : Wide<256>::kTile);
    return round256((size_t)kAttendMaxCus * columns * 2 * (D + 2) * sizeof(float));
}
constexpr int kMaxWorkers = kAttendMaxCus * 3;  // of any form
size_t dense_bytes(int rows, int H, int D) { return round256((size_t)rows * H * (D + 2) * sizeof(float)); }

}  // namespace

size_t attend_ws_bytes(int R, int H, int D, int rows, int n_groups) {
    size_t n = slots_bytes(D) + round256(kMaxWorkers * sizeof(AttendEnd));
    if (n_groups)
        n += slots_bytes(D) + round256((size_t)(R + 1) * 4) + round256((size_t)(n_groups + 1) * 4) +
             2 * dense_bytes(rows, H, D);
    return n;
}

void attend_ws_layout(AttendArgs& a, void* ws) {
    char* p = (char*)ws;
    const auto take = [&](size_t bytes) {
        char* at = p;
        p += bytes;
        return at;
    };
    a.slots[0] = (float*)take(slots_bytes(a.D));
    a.ends = (AttendEnd*)take(round256(kMaxWorkers * sizeof(AttendEnd)));
    if (!a.n_groups) return;
    a.slots[1] = (float*)take(slots_bytes(a.D));
    a.cum[0] = (uint32_t*)take(round256((size_t)(a.R + 1) * 4));
    a.cum[1] = (uint32_t*)take(round256((size_t)(a.n_groups + 1) * 4));
    a.dense[0] = (float*)take(dense_bytes(a.rows, a.H, a.D));
    a.dense[1] = (float*)take(dense_bytes(a.rows, a.H, a.D));
}

void attend_forms(AttendArgs& a, int cus) {
    // The many-rows form where a request (a group) may have more columns than kWideFrom; else
    // workers of two waves where it may have more than the 32 of one.
    const int wide = a.D == 64 ? Wide<64>::kTile : a.D == 128 ? Wide<128>::kTile : Wide<256>::kTile;
    const int wide_per_cu = a.D == 64 ? Wide<64>::kPerCu : 1;
    cus = std::min(cus, kAttendMaxCus);
    for (int set = 0; set < 2; ++set) {
        const long long columns = (long long)(set ? a.rows : a.max_new) * a.G;
        // (at head_dim 256 the keys leave LDS for 4096 requests' running units beside them)
        const bool many = columns > kWideFrom && (set || a.D < 256 || a.R <= 4096);
        a.tile[set] = many ? wide : columns > 32 ? 64 : 32;
        a.unit[set] = columns > 32 ? 64 : 128;
        a.workers[set] = cus * (many ? wide_per_cu : a.D <= 128 ? 2 : 1);
        a.least[set] = many ? kWideLeast : 0;
        a.parts[set] = (uint32_t)kFewParts * a.Hkv * std::max(set ? a.n_groups : a.R, 1);
        a.tile_shift[set] = __builtin_ctz(a.tile[set]);
        a.unit_shift[set] = __builtin_ctz(a.unit[set]);
    }
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t s) {
    return a.dtype == DSPARK_F16 ? run_dim<F16>(a, s) : run_dim<Bf16>(a, s);
}

}  // namespace dspark
