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
#include "cache.h"
#include "common.h"

namespace dspark {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
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
    if ((q.ln + n + a.page - 1) / a.page > a.width) {
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

__device__ __forceinline__ int tiles_of(const AttendArgs& a, int n) { return (n * a.G + kAttendTile - 1) / kAttendTile; }
__device__ __forceinline__ int units_of(int keys) { return (keys + kAttendUnit - 1) / kAttendUnit; }

// Workers that have a unit at all, so that no part between two others is missing.
__device__ __forceinline__ int workers_of(const AttendArgs& a, uint32_t total) {
    return total < (uint32_t)a.workers ? (int)total : a.workers;
}
// Worker w's first unit, and the worker of unit u, when `workers` share `total` units.
__device__ __forceinline__ uint32_t first_unit(uint32_t total, int workers, int w) {
    return (uint32_t)((uint64_t)total * (uint32_t)w / (uint32_t)workers);
}
__device__ __forceinline__ int worker_of(uint32_t total, int workers, uint32_t u) {
    return (int)((((uint64_t)u + 1) * (uint32_t)workers - 1) / total);
}

__device__ __forceinline__ float* slot_of(const AttendArgs& a, int set, int worker, int which) {
    return a.slots[set] + (size_t)(worker * 2 + which) * (kAttendTile * (a.D + 2));
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
    const int workers = workers_of(a, total);
    const int wa = worker_of(total, workers, u0), wb = worker_of(total, workers, u0 + units - 1);
    for (int w = wa; w <= wb; ++w) {
        const float* s = slot_of(a, set, w, w == wa);
        join(m, l, acc, s[kAttendTile * a.D + col], s[kAttendTile * (a.D + 1) + col], s + col * a.D + c8 * 8);
    }
}

// Adds the shared keys' part of query row f (row G + head of the group) of key head h.
__device__ void join_shared(const AttendArgs& a, int group, int f, int h, int c8, float& m, float& l, float (&acc)[8]) {
    uint32_t bad = 0;
    const Group g = shared_of(a, group, bad);
    const int at = f - g.start * a.G;
    if (g.ke <= 0 || at < 0 || at >= g.n * a.G) return;
    const uint32_t* cum = a.cum[1];
    const uint32_t total = cum[a.n_groups] * a.Hkv, units = units_of(g.ke), tiles = tiles_of(a, g.n);
    const uint32_t u0 = cum[group] * a.Hkv + (h * tiles + at / kAttendTile) * units;
    const int workers = workers_of(a, total);
    if (worker_of(total, workers, u0) == worker_of(total, workers, u0 + units - 1)) {
        const size_t n = (size_t)a.Hkv * a.rows * a.G, i = (size_t)h * a.rows * a.G + f;
        join(m, l, acc, a.dense[n * a.D + i], a.dense[n * (a.D + 1) + i], a.dense + i * a.D + c8 * 8);
    } else {
        join_parts(a, 1, total, u0, units, at % kAttendTile, c8, m, l, acc);
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

// Values of V that are not finite, in a block whose columns do not all see the same keys.
// The product has run without them; counting, for each dim and column, the ones that the
// column sees gives what it comes to: a NaN, or infinities of both signs, give NaN, and
// infinities of one sign that infinity.  One product counts all three: a NaN counts 4096,
// +inf 64 and -inf 1, and a block's 32 keys stay below 64 of each.
template <class E>
__device__ __forceinline__ f32x16 add_special(f32x16 o, s16x8 v0, s16x8 v1, s16x8 sees0, s16x8 sees1) {
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
    return o;
}

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32, 64); }

// kSet 0: the requests' own keys; 1: the groups' shared ones.
template <class E, int D, int kSet>
__global__ __launch_bounds__(kT, D <= 128 ? 2 : 1) void attend_kernel(AttendArgs a) {
    constexpr int NT = D / 32, NC = D / 16;
    constexpr int kDims = D <= 128 ? D : 128;  // dims joined over the waves at a time
    constexpr int kPitch = kDims + 4;
    __shared__ float s_o[4][kAttendTile][kPitch];
    __shared__ float s_m[4][kAttendTile], s_l[4][kAttendTile];
    __shared__ uint32_t s_base[8];
    extern __shared__ uint32_t s_cum[];  // running units, n + 1
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int n = kSet ? a.n_groups : a.R;

    // Running units of the requests (groups).
    uint32_t base = 0, bad = 0;
    for (int i0 = 0; i0 < n; i0 += kT) {
        const int i = i0 + tid;
        uint32_t x = 0;
        if (i < n) {
            if (kSet) {
                const Group g = shared_of(a, i, bad);
                x = (uint32_t)tiles_of(a, g.n) * units_of(g.ke);
            } else {
                Request q;
                if (request_of(a, i, q, bad) == 1) x = (uint32_t)tiles_of(a, q.n) * units_of(q.ln + q.n - q.kb);
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
    const uint32_t total = base * a.Hkv;
    const int workers = workers_of(a, total);
    if ((int)blockIdx.x >= workers) return;
    uint32_t u = first_unit(total, workers, blockIdx.x);
    const uint32_t u_end = first_unit(total, workers, blockIdx.x + 1);

    while (u < u_end) {
        int i = 0;  // the request (group) of unit u
        for (int hi = n; hi - i > 1;) {
            const int mid = (i + hi) >> 1;
            if (s_cum[mid] * a.Hkv <= u) i = mid; else hi = mid;
        }
        i = __builtin_amdgcn_readfirstlane(i);
        int start, rows, kb, ke, ln = 0, group = -1;
        const int32_t* table;
        if (kSet) {
            uint32_t none = 0;
            const Group g = shared_of(a, i, none);
            start = g.start;
            rows = g.n;
            kb = 0;
            ke = g.ke;
            table = a.shared_table + (size_t)i * a.shared_width;
        } else {
            Request q;
            uint32_t none = 0;
            request_of(a, i, q, none);
            start = q.start;
            rows = q.n;
            kb = q.kb;
            ln = q.ln;
            ke = q.ln + q.n;
            group = q.group;
            table = a.table + (size_t)i * a.width;
        }
        const uint32_t units = units_of(ke - kb), tiles = tiles_of(a, rows);
        const uint32_t in = u - s_cum[i] * a.Hkv, seg = in / units, unit0 = in % units;
        const int h = seg / tiles, tile = seg % tiles;
        const uint32_t seg_u0 = u - unit0;
        const uint32_t unit1 = min(units, unit0 + (u_end - u));
        const int f0 = start * a.G + tile * kAttendTile;
        const int nf = min(kAttendTile, rows * a.G - tile * kAttendTile);

        if (kSet == 0 && kb > 0 && seg == 0 && unit0 == 0) {  // the request's table has to begin with the group's pages
            bool differs = false;
            for (int p = tid; p < kb / a.page; p += kT)
                differs |= table[p] != a.shared_table[(size_t)group * a.shared_width + p];
            if (differs) raise_status(a.status, kStatusBadPage);
        }

        // Q^T as the first product's second operand: this lane's column, dims 16 c + 8 half + 0..7.
        const int f = f0 + min(col, nf - 1);
        const uint16_t* qp = a.q + (size_t)(f / a.G) * a.q_stride + (size_t)(h * a.G + f % a.G) * D + half * 8;
        s16x8 qf[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) qf[c] = *(const s16x8*)(qp + c * 16);
        const int last = kSet ? ke - 1 : ln + f / a.G - start;  // the column's last key

        f32x16 o[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t] = f32x16{};
        float m = -kInf, l = 0.f;  // of the raw scores; l this half's share of the sum

        const int swapped = (col & 3) | ((col & 4) << 1) | ((col & 8) >> 1);  // key of this lane in its block of 16
        for (uint32_t unit = unit0; unit < unit1; ++unit) {
            const int pos = kb + (int)(unit * kAttendUnit) + wave * 32;
            if (pos >= ke) break;
            const uint16_t *kp[2], *vp[2];
            bool have[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int p = pos + b * kBlockTokens;
                have[b] = p < ke;
                int page = have[b] ? table[p / a.page] : 0;
                if (page < 0 || page >= a.n_pages) {
                    page = 0;
                    have[b] = false;
                    if (lane == 0) raise_status(a.status, kStatusBadPage);
                }
                const size_t block =
                    ((size_t)page * a.Hkv + h) * (a.page / kBlockTokens) + (have[b] ? p % a.page / kBlockTokens : 0);
                kp[b] = a.k + block * (kBlockTokens * D);
                vp[b] = a.v + block * (kBlockTokens * D);
            }
            s16x8 kf[NC], vf[NT][2];
            const uint16_t* kl = (col < 16 ? kp[0] : kp[1]) + half * 128 + swapped * 8;
#pragma unroll
            for (int c = 0; c < NC; ++c) kf[c] = *(const s16x8*)(kl + c * 256);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int b = 0; b < 2; ++b) vf[t][b] = *(const s16x8*)(vp[b] + (t * 32 + col) * 16 + half * 8);

            f32x16 s = {};
#pragma unroll
            for (int c = 0; c < NC; ++c) s = E::mfma(kf[c], qf[c], s);

            const int first_last = kSet ? ke - 1 : ln + f0 / a.G - start;  // the tile's earliest last key
            const bool masked = pos + 31 > first_last || !have[0] || !have[1];
            if (masked) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int key = pos + (j / 8) * 16 + half * 8 + j % 8;
                    if (key > last || !have[j / 8]) s[j] = -kInf;
                }
            }
            float mx = s[0];
#pragma unroll
            for (int j = 1; j < 16; ++j) mx = fmaxf(mx, s[j]);
            mx = fmaxf(mx, other_half(mx));
            const float m_new = fmaxf(m, mx);
            const float mc = m_new == -kInf ? 0.f : m_new * a.scale_log2;
            const float alpha = __builtin_amdgcn_exp2f(__builtin_fmaf(m, a.scale_log2, -mc));
            m = m_new;
            float sum = 0.f;
            s16x8 pf[2];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j], a.scale_log2, -mc));
                sum += p;
                pf[j / 8][j % 8] = (short)E::bits(p);  // weights of at most 1, rounded for the matrix instruction
            }
            l = l * alpha + sum;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j) o[t][j] *= alpha;

            if (masked) {
                bool special = false;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int k0 = pos + b * 16 + half * 8;
                    const int valid = have[b] ? ke - k0 : 0;  // keys of this lane's eight that the segment has
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (j >= valid) vf[t][b][j] = 0;
                            special |= ((uint16_t)vf[t][b][j] & E::kExp) == E::kExp;
                        }
                }
                if (__ballot(special)) {
                    s16x8 sees[2];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        sees[j / 8][j % 8] =
                            pos + (j / 8) * 16 + half * 8 + j % 8 <= last && have[j / 8] ? (short)E::kOne : (short)0;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        s16x8 fin[2];
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                fin[b][j] = ((uint16_t)vf[t][b][j] & E::kExp) == E::kExp ? (short)0 : vf[t][b][j];
                        o[t] = E::mfma(fin[1], pf[1], E::mfma(fin[0], pf[0], o[t]));
                        o[t] = add_special<E>(o[t], vf[t][0], vf[t][1], sees[0], sees[1]);
                    }
                    continue;
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t] = E::mfma(vf[t][1], pf[1], E::mfma(vf[t][0], pf[0], o[t]));
        }
        l += other_half(l);
        const float ms = m == -kInf ? -kInf : m * a.scale_log2;

        // The four waves' parts joined, column by column, eight dims to a thread.
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
                const int q = e / (kDims / 8), c8 = e % (kDims / 8);
                float jm = -kInf, jl = 0.f, acc[8] = {};
#pragma unroll
                for (int w = 0; w < 4; ++w) join(jm, jl, acc, s_m[w][q], s_l[w][q], &s_o[w][q][c8 * 8]);
                const int d8 = d0 / 8 + c8;
                if (whole && kSet == 0) {
                    if (group >= 0 && kb > 0) join_shared(a, group, f0 + q, h, d8, jm, jl, acc);
                    store_row<E>(a, f0 + q, h, d8, jm, jl, acc);
                    continue;
                }
                float *po, *pm, *pl;
                if (whole) {
                    const size_t all = (size_t)a.Hkv * a.rows * a.G, at = (size_t)h * a.rows * a.G + f0 + q;
                    po = a.dense + at * D;
                    pm = a.dense + all * D + at;
                    pl = a.dense + all * (D + 1) + at;
                } else {
                    float* slot = slot_of(a, kSet, blockIdx.x, unit0 == 0);
                    po = slot + q * D;
                    pm = slot + kAttendTile * D + q;
                    pl = slot + kAttendTile * (D + 1) + q;
                }
                *(float4*)(po + d8 * 8) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                *(float4*)(po + d8 * 8 + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
                if (d8 == 0) {
                    *pm = jm;
                    *pl = jl;
                }
            }
        }
        u = seg_u0 + unit1;
    }
}

// Joins the parts of the segments that were split, and gives zeros to rows that see nothing.
template <class E>
__global__ __launch_bounds__(kT) void attend_join_kernel(AttendArgs a) {
    const int r = blockIdx.x, h = blockIdx.y, tile = blockIdx.z;
    Request q;
    uint32_t bad = 0;
    const int state = request_of(a, r, q, bad);
    if (state < 0 || tile * kAttendTile >= q.n * a.G) return;
    const int f0 = q.start * a.G + tile * kAttendTile, nf = min(kAttendTile, q.n * a.G - tile * kAttendTile);
    const uint32_t *cum = a.cum[0], total = cum[a.R] * a.Hkv;
    const uint32_t units = state ? units_of(q.ln + q.n - q.kb) : 0;
    const uint32_t u0 = state ? cum[r] * a.Hkv + (h * tiles_of(a, q.n) + tile) * units : 0;
    const int workers = workers_of(a, total);
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

template <class E, int D>
hipError_t run(const AttendArgs& a, hipStream_t s) {
    if (a.n_groups) {
        hipLaunchKernelGGL((attend_kernel<E, D, 1>), dim3(a.workers), dim3(kT), (a.n_groups + 1) * sizeof(uint32_t), s,
                           a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((attend_kernel<E, D, 0>), dim3(a.workers), dim3(kT), (a.R + 1) * sizeof(uint32_t), s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(attend_join_kernel<E>, dim3(a.R, a.Hkv, (a.max_new * a.G + kAttendTile - 1) / kAttendTile),
                       dim3(kT), 0, s, a);
    return hipGetLastError();
}

template <class E>
hipError_t run_dim(const AttendArgs& a, hipStream_t s) {
    return a.D == 64 ? run<E, 64>(a, s) : a.D == 128 ? run<E, 128>(a, s) : run<E, 256>(a, s);
}

size_t slots_bytes(int D) { return round256((size_t)kAttendMaxWorkers * 2 * kAttendTile * (D + 2) * sizeof(float)); }
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
    const int w = cus * (a.D <= 128 ? 2 : 1);
    a.workers = w < kAttendMaxWorkers ? w : kAttendMaxWorkers;
    return a.dtype == DSPARK_F16 ? run_dim<F16>(a, s) : run_dim<Bf16>(a, s);
}

}  // namespace dspark
