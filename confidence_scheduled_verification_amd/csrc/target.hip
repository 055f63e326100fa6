// The target's choice at each row, from its logits: penalties for repeated tokens, biases and
// grammar masks, and the argmax, in one pass over the logits; and the record of what has been
// said, which the penalties read.
//
// Nearly all tokens lose by their logit alone.  While a workgroup streams a row (or a part of one), it
// knows a value that the row's best has at least, `floor`, and from it a logit below which no token
// can reach it: floor itself, or less where a penalty below nothing or a repetition below one could
// lift a token.  So the pass compares the largest of eight logits with that limit, a dozen
// instructions, and looks at tokens one by one only where it is reached: a few times a row.
// There the bits in LDS say whether a token is allowed, and whether anything changes it (it is seen,
// biased or drafted); if not, its logit is its value, and if so it is put on a list, whose values are
// computed at the end, side by side, in 64 bits and with the counts that only they need.
// Biases may lift a token as far as they like: those tokens are on the list from the start.  So is
// every changed one where the processed logits are wanted, or a frequency below nothing lifts tokens
// by how often they have been said.
//
// Bytes bound it where rows are many: 1152 bf16 rows of 129280 (298 MB, and 2000 said tokens, 100
// biases and a mask each) take 70 us, 4.4 TB/s; looking at every changed token took 126.  Without penalties,
// biases and masks the same rows take 57; of 151936 tokens, in two parts of which the second is small, 97 and
// 70, of 262144 132 and 107.  Groups of eight without an allowed token are not read, past a part's first 8192
// tokens (whose loads go out before the mask is there) and unless the processed logits are wanted.  Four rows of
// 129280, 32 workgroups each, take 12 us, of which the launch and loads that wait for each other (rows, bits,
// logits, counts) are all but one; a second launch to join the parts made it 16.  336 rows of 32771 in fp32,
// processed and written (89 MB): 34 us, 2.6 TB/s: rows of an odd length stand on no line, and a workgroup is
// through its part in four loads of a lane and a fifth for the last 32 groups.
#include <algorithm>

#include "common.h"
#include "tree.h"

namespace dspark {

namespace {

#define INLINE __attribute__((always_inline))
constexpr int kT = kTargetThreads, kWaves = kT / 64;
constexpr int kPerSimd = 7;           // waves that the registers leave room for
constexpr int kGroups = 2;            // of eight logits: a lane's loads under way, twice
constexpr int kMostChunk = 131072;    // tokens of a part: twice 16 KB of bits in LDS
constexpr int kLeastChunk = 4096;
constexpr int kWanted = 2 * kAttendMaxCus;  // workgroups, where there are few rows
constexpr int kList = 2048;           // changed tokens listed; where there are more, all of them are gone through
constexpr int kCounted = 4096;        // rows whose parts are counted in the workspace
constexpr int kHistoryT = 256, kWideT = 1024;
constexpr int kWideFrom = 256;        // tokens of a row that are gathered in LDS
constexpr int kMostInLds = 1 << 19;   // tokens of a vocabulary whose bits LDS takes, 64 KB (beside the answers' counts, half)
constexpr int kPromptSlice = 16384, kAnswerSlice = 2048;  // tokens to a workgroup
constexpr float kInf = __builtin_huge_valf();
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct F32 {
    typedef uint32_t T;
    static constexpr T kNegInf = 0xFF800000u;
    static __device__ __forceinline__ float value(T x) { return __uint_as_float(x); }
    static __device__ __forceinline__ T bits(float x) { return __float_as_uint(x); }
};
struct Bf16 {
    typedef uint16_t T;
    static constexpr T kNegInf = 0xFF80u;
    static __device__ __forceinline__ float value(T x) { return bf16_bits_to_f32(x); }
    static __device__ __forceinline__ T bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
};
struct F16 {
    typedef uint16_t T;
    static constexpr T kNegInf = 0xFC00u;
    static __device__ __forceinline__ float value(T x) { return (float)__builtin_bit_cast(_Float16, x); }
    static __device__ __forceinline__ T bits(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
};

// argmax_key's order in 64 bits, above the token's.  0 is below every value's key.
__device__ __forceinline__ uint64_t order_key(double x) {
    if (x != x) return ~0ull;
    const uint64_t b = x == 0.0 ? 0 : (uint64_t)__double_as_longlong(x);  // -0 as +0
    return b >> 63 ? ~b : b | 1ull << 63;
}

// The value of argmax_key's upper half.
__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float(key >> 31 ? (key == ~0u ? 0x7FC00000u : key & 0x7FFFFFFFu) : ~key);
}

struct Best {
    uint64_t key;
    uint32_t v;
    __device__ __forceinline__ void take(uint64_t k, uint32_t at) {
        if (k > key || (k == key && at < v)) {
            key = k;
            v = at;
        }
    }
};

__device__ __forceinline__ void wave_best(Best& b) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t k = shfl_xor_u64(b.key, d);
        const uint32_t v = __shfl_xor(b.v, d, 64);
        b.take(k, v);
    }
}

// The largest of a wave's numbers, by the data paths within and between rows of 16 lanes.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// Row j of request r, where it is one.
__device__ __forceinline__ bool row_of(const dspark_target_t& t, int r, int j, int& o, long long& start, int& n, uint32_t& bad) {
    o = t.offsets[r];
    const long long rows = (long long)t.offsets[r + 1] - o + t.lead;
    start = (long long)o + (long long)t.lead * r;
    if (o < 0 || rows < 0 || rows > t.max_new || start + rows > t.n_rows) {
        bad = kStatusBadRow;
        return false;
    }
    n = (int)rows;
    return j < n;
}

// Eight logits, wherever they stand (rows of an odd vocabulary are not aligned).  Of 16 bits they are read and
// written past the caches (1152 rows: 75 us, 78 through them); of 32 they are two pieces, between which a line's
// other half has to stay (340 rows processed: 35 us, 42 past the caches).
template <class E>
struct Eight {
    typedef typename E::T T;
    static constexpr int kParts = sizeof(T) / 2;
    typedef u32x4 __attribute__((aligned(2), may_alias)) any;
    u32x4 w[kParts];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) w[i] = kParts == 1 ? __builtin_nontemporal_load((const any*)p) : *((const any*)p + i);
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            if (kParts == 1) __builtin_nontemporal_store(w[i], (any*)p);
            else *((any*)p + i) = w[i];
    }
    __device__ __forceinline__ T bits(int k) const {
        return sizeof(T) == 4 ? (T)w[k / 4][k % 4] : (T)(w[0][k / 2 % 4] >> (k % 2 * 16));
    }
    __device__ __forceinline__ float value(int k) const { return E::value(bits(k)); }
    __device__ __forceinline__ void mask(uint32_t keep) {  // -inf where a bit is not set
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t on = (uint32_t)((int32_t)(keep << (31 - k)) >> 31);
            if (sizeof(T) == 4) {
                w[k / 4][k % 4] = (w[k / 4][k % 4] & on) | (0xFF800000u & ~on);
            } else {
                const uint32_t off = (0xFFFFu << (k % 2 * 16)) & ~on;
                w[0][k / 2 % 4] = (w[0][k / 2 % 4] & ~off) | ((uint32_t)E::kNegInf * 0x10001u & off);
            }
        }
    }
};

template <class E, bool kOut>
__global__ __launch_bounds__(kT, kPerSimd) void target_kernel(TargetArgs a) {
    typedef typename E::T T;
    const dspark_target_t& t = a.t;
    extern __shared__ uint32_t s_words[];  // bits of the part's tokens: changed ones, allowed ones
    __shared__ uint2 s_list[kList];        // changed tokens, and their logits
    __shared__ int s_draft[DSPARK_TARGET_MAX_ROWS], s_bias[kT];
    static_assert(DSPARK_TARGET_MAX_ROWS <= kT, "a draft to a lane");
    __shared__ uint32_t s_count, s_floor;
    __shared__ Best s_best[kWaves];
    // (a request's rows on different XCDs, every eighth workgroup being on the same: requests of many rows
    // would keep one busy longer than the others)
    const int part = blockIdx.x / t.R, j = blockIdx.y, r = (blockIdx.x % t.R + j) % t.R, tid = threadIdx.x;
    int o, n;
    long long start;
    uint32_t bad = 0;
    if (!row_of(t, r, j, o, start, n, bad)) {
        if (bad && part == 0 && j == 0 && tid == 0) raise_status(a.status, bad);
        return;
    }
    const size_t row = (size_t)(start + j);
    const T* logits = (const T*)t.logits + row * t.logits_stride;
    T* out = kOut ? (T*)t.adjusted + row * t.adjusted_stride : nullptr;
    const int lo = part * a.chunk, hi = min(t.V, lo + a.chunk), n_words = (hi - lo + 31) / 32;
    const int n_groups = (hi - lo) / 8;                                          // of eight tokens from lo on
    const int tail = tid < (hi - lo) % 8 ? lo + n_groups * 8 + tid : -1;  // and what is left, a token to a lane

    // What has a say in this row.
    const uint32_t* allowed = nullptr;
    bool nothing = false;  // is allowed
    if (t.allowed) {
        const long long pick = t.allowed_row ? t.allowed_row[row] : (long long)row;
        if (pick < -1 || pick >= t.n_allowed) {
            nothing = true;
            bad = kStatusBadRow;
        } else if (pick >= 0) {
            allowed = t.allowed + (size_t)pick * t.allowed_stride;
        }
    }
    const bool masked = allowed || nothing;
    const bool penalties = t.repetition || t.presence || t.frequency;
    const float repetition = t.repetition ? t.repetition[r] : 1.f, presence = t.presence ? t.presence[r] : 0.f,
                frequency = t.frequency ? t.frequency[r] : 0.f;
    const uint32_t *prompt = nullptr, *answered = nullptr;
    const int32_t* count = nullptr;
    if (penalties && a.seen) {
        prompt = a.seen + (size_t)r * 2 * a.words;
        answered = prompt + a.words;
        count = a.count + (size_t)r * t.V;
    }
    int b0 = 0, b1 = 0;
    if (t.bias_off) {
        b0 = t.bias_off[r];
        b1 = t.bias_off[r + 1];
        if (b0 < 0 || b1 < b0 || b1 > t.n_bias) {
            b0 = b1 = 0;
            bad = kStatusBadRow;
        }
    }
    const int n_draft = penalties && t.ver_tokens ? n : 0;
    const bool changes = prompt || n_draft || b1 > b0;  // anything
    // Every changed token is looked at, whatever its logit: where its value is wanted, or cannot be bounded.
    const bool every = changes && (kOut || !(frequency >= 0.f) || !(repetition > 0.f) || !(repetition < kInf) ||
                                   !(fabsf(presence) < kInf) || !(frequency < kInf));

    // The bits.  Their loads go out before the stream's first ones, so as not to wait behind those of all
    // workgroups.
    uint32_t *s_changed = s_words, *s_allowed = s_words + (a.seen || t.ver_tokens || t.bias_off ? a.chunk / 32 : 0);
    constexpr int kWords = kMostChunk / 32 / kT;  // a lane's
    uint32_t said[kWords], given[kWords], open[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const size_t at = lo / 32 + min(tid + i * kT, n_words - 1);
        said[i] = prompt ? answered[at] : 0;
        given[i] = prompt ? prompt[at] : 0;
        open[i] = allowed ? allowed[at] : 0;
    }
    const bool near = b1 - b0 <= kT;  // biases that are searched in LDS
    int draft = -1, bias = -1;        // this lane's token of each list
    if (tid < n_draft) {
        const bool on = tid >= t.lead && (t.anc ? (t.anc[row] >> (tid & 63) & 1) != 0 : tid <= j);
        const int at = o + tid - t.lead;
        if (on && at < t.n_nodes) draft = t.ver_tokens[at];
    }
    if (near && tid < b1 - b0) bias = t.bias_tok[b0 + tid];
    __builtin_amdgcn_sched_barrier(0);
    Eight<E> now[kGroups], ahead[kGroups];
    if (n_groups > 0) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) now[i].load(logits + lo + min(tid + i * kT, n_groups - 1) * 8);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (tid == 0) s_count = s_floor = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
        if (tid + i * kT < n_words) {
            if (changes) s_changed[tid + i * kT] = said[i] | given[i];
            if (masked) s_allowed[tid + i * kT] = open[i];
        }
    if (tid < n_draft) s_draft[tid] = draft;
    if (near && tid < b1 - b0) s_bias[tid] = bias;
    __syncthreads();
    const auto change = [&](int v) INLINE {
        if (v >= lo && v < hi) atomicOr(&s_changed[(v - lo) >> 5], 1u << (v & 31));
    };
    const auto bias_at = [&](int e) INLINE { return near ? s_bias[e] : t.bias_tok[b0 + e]; };
    if (draft >= 0) change(draft);
    for (int e = tid; e < b1 - b0; e += kT) {
        const int v = bias_at(e);
        if (v < 0 || v >= t.V || (e > 0 && bias_at(e - 1) >= v)) bad = kStatusBadRow;
        change(v);
    }
    if (bad && part == 0) raise_status(a.status, bad);
    __syncthreads();
    const uint8_t *changed_of = (const uint8_t*)s_changed, *allowed_of = (const uint8_t*)s_allowed;
    const auto is_allowed = [&](int v) { return !masked || (s_allowed[(v - lo) >> 5] >> (v & 31) & 1); };
    const auto is_changed = [&](int v) { return changes && (s_changed[(v - lo) >> 5] >> (v & 31) & 1); };

    // The place of v among the biases, -1 for none: at most one, in a list that does not rise too.
    const auto find = [&](int v) INLINE {
        for (int x0 = 0, x1 = b1 - b0; x0 < x1;) {
            const int mid = (x0 + x1) >> 1, at = bias_at(mid);
            if (at == v) return mid;
            if (at < v) x0 = mid + 1; else x1 = mid;
        }
        return -1;
    };
    // The value of token v, which is in the prompt (seen) or has been answered c times before the drafts.
    const auto value_of = [&](int v, float logit, bool seen, int c, bool biased, float by) INLINE {
        for (int i = 0; i < n_draft; ++i) c += s_draft[i] == v;
        double x = (double)logit;
        if (seen || c > 0) x = x > 0.0 ? x / (double)repetition : x * (double)repetition;
        if (c > 0) {
            x = x - (double)frequency * (double)c;
            x = x - (double)presence;
        }
        if (biased) x = x + (double)by;
        if (kOut) out[v] = E::bits((float)x);
        return x;
    };
    // The stream.  top: this lane's best unchanged token, as argmax_key has it; best: its best changed one;
    // floor: what the row's best has at least; limit: what a logit needs to reach it.
    uint64_t top = 0;
    Best best{0, ~0u};
    float limit = -kInf;
    uint32_t floor_key = 0;
    const float lift = fmaxf(-presence, 0.f), shrink = fminf(repetition, 1.f);
    const auto raise = [&](uint32_t key) INLINE {
        if (key <= floor_key) return;
        floor_key = key;
        if ((tid & 63) == 0) atomicMax(&s_floor, key);
        const float floor = key_value(key);
        limit = floor;
        if (penalties && !every && floor < kInf) {  // (a NaN stays one: nothing is below it)
            const float x = floor - lift - (fabsf(floor) + lift) * 0x1p-20f, y = x > 0.f ? x * shrink : x / shrink;
            limit = fminf(y - fabsf(y) * 0x1p-20f, floor);  // (2^-20 covers these roundings)
        }
    };
    const auto put = [&](int v, float logit) INLINE {
        const uint32_t at = atomicAdd(&s_count, 1u);
        if (at < kList) s_list[at] = make_uint2((uint32_t)v, __float_as_uint(logit));
    };
    // Of the eight tokens from v on those whose bits are set: to the list.
    const auto put_all = [&](int v, uint32_t bits, const Eight<E>& e) INLINE {
        uint32_t at = atomicAdd(&s_count, (uint32_t)__popc(bits));
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (bits >> k & 1) {
                if (at < kList) s_list[at] = make_uint2((uint32_t)(v + k), __float_as_uint(e.value(k)));
                ++at;
            }
    };
    const auto fetch = [&](int g0, Eight<E>(&e)[kGroups]) INLINE {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int g = min(g0 + i * kT, n_groups - 1);
            const bool skip = !kOut && masked && allowed_of[g] == 0;  // nothing allowed: not read
            e[i].load(logits + lo + (skip ? 0 : g * 8));
        }
    };
    const auto stream = [&](int g0, Eight<E>(&e)[kGroups]) INLINE {
        float m[kGroups], most = -kInf;
        if (kOut || every) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int g = g0 + i * kT, v = lo + g * 8;
                if (g >= n_groups) continue;
                if (kOut) {
                    Eight<E> x = e[i];
                    if (masked) x.mask(allowed_of[g]);
                    x.store(out + v);  // the changed ones once more, behind a barrier
                }
                const uint32_t changed = changed_of[g] & (masked ? allowed_of[g] : 0xFFu);
                if (every && changed) put_all(v, changed, e[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            m[i] = e[i].value(0);
#pragma unroll
            for (int k = 1; k < 8; ++k) m[i] = __builtin_elementwise_maximum(m[i], e[i].value(k));
            if (masked && allowed_of[min(g0 + i * kT, n_groups - 1)] == 0) m[i] = -kInf;  // (was not read)
            most = __builtin_elementwise_maximum(most, m[i]);
        }
        if (__ballot(!(most < limit))) {
            // Groups without a masked or a changed token have their largest logit for certain: of the wave's
            // lanes only those with the largest of these are left to be looked at, one as a rule.
            float sure = -kInf;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int g = g0 + i * kT;
                if (g < n_groups && (!masked || allowed_of[g] == 0xFFu) && (!changes || changed_of[g] == 0)) sure = fmaxf(sure, m[i]);
            }
            raise(max(wave_max((uint32_t)(argmax_key(sure, 0) >> 32)), *(volatile uint32_t*)&s_floor));
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int g = g0 + i * kT, v = lo + g * 8;
                const bool reaches = g < n_groups && !(m[i] < limit) && (!masked || allowed_of[g]);
                if (!__ballot(reaches)) continue;
                if (reaches) {
                    uint32_t bits = 0;  // of the tokens that reach the limit
#pragma unroll
                    for (int k = 0; k < 8; ++k) bits |= (!(e[i].value(k) < limit) ? 1u : 0u) << k;
                    if (masked) bits &= allowed_of[g];
                    const uint32_t changed = changes ? changed_of[g] & bits : 0;
                    for (bits &= ~changed; bits; bits &= bits - 1) {
                        const int at = __ffs(bits) - 1;
                        float x = e[i].value(0);
#pragma unroll
                        for (int k = 1; k < 8; ++k) x = at == k ? e[i].value(k) : x;
                        top = max(top, argmax_key(x, (uint32_t)(v + at)));
                    }
                    if (!every && changed) put_all(v, changed, e[i]);
                }
                raise(wave_max((uint32_t)(top >> 32)));
            }
        }
    };
    for (int g0 = tid; g0 - tid < n_groups; g0 += 2 * kT * kGroups) {
        fetch(g0 + kT * kGroups, ahead);
        stream(g0, now);
        if (g0 - tid + kT * kGroups >= n_groups) break;
        fetch(g0 + 2 * kT * kGroups, now);
        stream(g0 + kT * kGroups, ahead);
    }
    if (tail >= 0) {
        const bool on = is_allowed(tail), changed = is_changed(tail);
        if (kOut) out[tail] = on ? logits[tail] : E::kNegInf;
        if (on && changed) put(tail, E::value(logits[tail]));
        else if (on) top = max(top, argmax_key(E::value(logits[tail]), (uint32_t)tail));
    }
    if (!every)
        for (int e = tid; e < b1 - b0; e += kT) {
            const int v = bias_at(e);
            if (v >= lo && v < hi && is_allowed(v)) put(v, E::value(logits[v]));
        }
    if (kOut) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    // The list; or, where it was too short, every changed token of the part, 64 neighbours to a wave.
    const bool whole = s_count <= kList;
    const int many = whole ? (int)s_count : (n_words + 1) / 2 * 64;
    for (int i = tid; i < many; i += kT) {
        uint2 e;
        if (whole) {
            e = s_list[i];
        } else {
            const int v = lo + i;
            if (v >= hi || !is_changed(v) || !is_allowed(v)) continue;
            e = make_uint2((uint32_t)v, __float_as_uint(E::value(logits[v])));
        }
        const int v = (int)e.x, b = find(v);
        bool seen = false;
        int c = 0;
        if (prompt) {
            seen = prompt[v >> 5] >> (v & 31) & 1;
            if (!every || (answered[v >> 5] >> (v & 31) & 1)) c = count[v];  // (few: not worth waiting for their bits)
        }
        best.take(order_key(value_of(v, __uint_as_float(e.y), seen, c, b >= 0, b >= 0 ? t.bias_val[b0 + b] : 0.f)), e.x);
    }
    if (top) best.take(order_key((double)key_value((uint32_t)(top >> 32))), (uint32_t)key_index(top));

    wave_best(best);
    if ((tid & 63) == 0) s_best[tid >> 6] = best;
    __syncthreads();
    if (tid >= 64) return;
    best = s_best[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) best.take(s_best[w].key, s_best[w].v);
    if (a.parts > 1) {
        // The part that comes last joins all of the row's.  What the others have left is there when their
        // counts are: written through to where all of the device sees it, and waited for.  Where two requests
        // have the row (offsets that fall), every a.parts-th takes a.parts off, so that nothing is left
        // for the next call, and what is not there yet is no token of this one, or is passed over.
        TargetBest* parts = a.best + row * a.parts;
        int came = 0;
        if (tid == 0) {
            __hip_atomic_store(&parts[part].key, best.key, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(&parts[part].v, best.v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (a.came) came = (int)__hip_atomic_fetch_add(&a.came[row], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        if (!a.came || (uint32_t)(__builtin_amdgcn_readfirstlane(came) + 1) % (uint32_t)a.parts) return;
        asm volatile("" ::: "memory");
        for (int p = tid; p < a.parts; p += 64) {
            const uint64_t key = __hip_atomic_load(&parts[p].key, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const uint32_t v = __hip_atomic_load(&parts[p].v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (v < (uint32_t)t.V) best.take(key, v);
        }
        wave_best(best);
        if (tid == 0) __hip_atomic_fetch_sub(&a.came[row], (uint32_t)a.parts, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next call
    }
    if (tid == 0) {
        t.target[row] = best.key ? (int32_t)best.v : t.no_token;
        if (!best.key) raise_status(a.status, kStatusNoToken);
    }
}

// The same in a launch of its own, a wave to a row, for more rows than are counted.
__global__ __launch_bounds__(64) void target_join_kernel(TargetArgs a) {
    int o, n;
    long long start;
    uint32_t bad = 0;
    if (!row_of(a.t, blockIdx.x, blockIdx.y, o, start, n, bad)) return;
    const size_t row = (size_t)(start + blockIdx.y);
    Best best{0, ~0u};
    for (int p = threadIdx.x; p < a.parts; p += 64) {
        const TargetBest b = a.best[row * a.parts + p];
        best.take(b.key, b.v);
    }
    wave_best(best);
    if (threadIdx.x == 0) {
        a.t.target[row] = best.key ? (int32_t)best.v : a.t.no_token;
        if (!best.key) raise_status(a.status, kStatusNoToken);
    }
}

// A history row emptied: the counts only where there are any.  128 rows of 129280: 6.5 us.
__global__ __launch_bounds__(kHistoryT) void history_clear_kernel(dspark_history_t h, size_t words, const int32_t* rows,
                                                           uint32_t* status) {
    const int i = blockIdx.x, r = rows ? rows[i] : i;
    if (r < 0 || r >= h.rows) {
        if (blockIdx.y == 0 && threadIdx.x == 0) raise_status(status, kStatusBadRow);
        return;
    }
    uint32_t *prompt = h.seen + (size_t)r * 2 * words, *answered = prompt + words;
    int32_t* count = h.count + (size_t)r * h.V;
    for (size_t w = blockIdx.y * kHistoryT + threadIdx.x; w < words; w += (size_t)gridDim.y * kHistoryT) {
        for (uint32_t x = answered[w]; x; x &= x - 1) {
            const size_t v = w * 32 + __ffs(x) - 1;
            if (v < (size_t)h.V) count[v] = 0;
        }
        prompt[w] = 0;
        answered[w] = 0;
    }
}

// Entering tokens.  Few at a time (a step's answers) go to memory one by one; many are first gathered in
// LDS, a workgroup a slice of a row's tokens, for the frequent ones would have thousands of atomics wait
// for each other at the same words (128 prompts of 16000 tokens: 107 us one by one, 10 so; 128
// answers of 2000: 15 so).  Either way a bit that is set already needs no atomic.
__device__ __forceinline__ void set_bits(uint32_t* word, uint32_t bits) {
    if (bits & ~__hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicOr(word, bits);
}

// A workgroup's bits in LDS, `used` words, four to a lane at a time.
__device__ __forceinline__ void set_all(uint32_t* to, const uint32_t* s_bits, int used) {
    for (int w0 = threadIdx.x; w0 < used; w0 += 4 * kWideT) {
        uint32_t bits[4], have[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int w = w0 + i * kWideT;
            bits[i] = w < used ? s_bits[w] : 0;
            have[i] = __hip_atomic_load(to + min(w, used - 1), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (bits[i] & ~have[i]) atomicOr(to + w0 + i * kWideT, bits[i]);
    }
}

// The history row of tokens' row i; -1 where it is none (the first slice says so).
__device__ __forceinline__ int history_row(const dspark_history_t& h, const int32_t* rows, int i, bool first, uint32_t* status) {
    const int r = rows ? rows[i] : i;
    if (r >= 0 && r < h.rows) return r;
    if (first && threadIdx.x == 0) raise_status(status, kStatusBadRow);
    return -1;
}

__global__ __launch_bounds__(kHistoryT) void history_add_kernel(dspark_history_t h, size_t words, const int32_t* tokens,
                                                                int width, const int32_t* rows, int answered,
                                                                uint32_t* status) {
    const int i = blockIdx.x, r = history_row(h, rows, i, blockIdx.y == 0, status);
    if (r < 0) return;
    uint32_t* bits = h.seen + ((size_t)r * 2 + (answered ? 1 : 0)) * words;
    int32_t* count = h.count + (size_t)r * h.V;
    bool bad = false;
    for (size_t at = blockIdx.y * kHistoryT + threadIdx.x; at < (size_t)width; at += gridDim.y * kHistoryT) {
        const int v = tokens[(size_t)i * width + at];
        if (v < 0) continue;
        if (v >= h.V) {
            bad = true;
            continue;
        }
        set_bits(bits + (v >> 5), 1u << (v & 31));
        if (answered) atomicAdd(count + v, 1);
    }
    if (bad) raise_status(status, kStatusBadRow);
}

__global__ __launch_bounds__(kWideT) void history_prompt_kernel(dspark_history_t h, size_t words, const int32_t* tokens,
                                                                int width, const int32_t* rows, uint32_t* status) {
    extern __shared__ uint32_t s_bits[];  // of V tokens
    const int i = blockIdx.x, tid = threadIdx.x, r = history_row(h, rows, i, blockIdx.y == 0, status);
    if (r < 0) return;
    const int used = (h.V + 31) / 32, end = min(width, ((int)blockIdx.y + 1) * kPromptSlice);
    for (int w = tid; w < used; w += kWideT) s_bits[w] = 0;
    __syncthreads();
    bool bad = false;
    for (int at = blockIdx.y * kPromptSlice + tid; at < end; at += kWideT) {
        const int v = tokens[(size_t)i * width + at];
        if (v < 0) continue;
        if (v >= h.V) {
            bad = true;
            continue;
        }
        const uint32_t bit = 1u << (v & 31);
        if (!(s_bits[v >> 5] & bit)) atomicOr(&s_bits[v >> 5], bit);
    }
    if (bad) raise_status(status, kStatusBadRow);
    __syncthreads();
    uint32_t* prompt = h.seen + (size_t)r * 2 * words;
    set_all(prompt, s_bits, used);
}

// Answers: the bits first; a token's place among the bits that are set, from the bits before it, is then
// its place in a list of counts, and the lane that comes to a place first adds its count to memory's.
__global__ __launch_bounds__(kWideT) void history_answer_kernel(dspark_history_t h, size_t words, const int32_t* tokens,
                                                                int width, const int32_t* rows, uint32_t* status) {
    constexpr int kMine = kAnswerSlice / kWideT, kWords = kMostInLds / 2 / 32 / kWideT;  // a lane's tokens and words
    __shared__ uint32_t s_sum[kWideT / 64];
    __shared__ int s_times[kAnswerSlice];
    __shared__ uint16_t s_before[kWords * kWideT];  // bits set before each word
    extern __shared__ uint32_t s_bits[];            // of V tokens, whole pairs of words
    const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 63, r = history_row(h, rows, i, blockIdx.y == 0, status);
    if (r < 0) return;
    const int used = (h.V + 63) / 64 * 2;
    int mine[kMine];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        const int at = blockIdx.y * kAnswerSlice + k * kWideT + tid;
        mine[k] = at < width ? tokens[(size_t)i * width + at] : -1;
        if (mine[k] >= h.V) {
            mine[k] = -1;
            bad = true;
        }
        s_times[k * kWideT + tid] = 0;
    }
    if (bad) raise_status(status, kStatusBadRow);
    for (int w = tid; w < used; w += kWideT) s_bits[w] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMine; ++k)
        if (mine[k] >= 0) atomicOr(&s_bits[mine[k] >> 5], 1u << (mine[k] & 31));
    __syncthreads();
    uint32_t own = 0, before = 0;
#pragma unroll
    for (int k = 0; k < kWords; ++k)
        if (tid * kWords + k < used) own += __popc(s_bits[tid * kWords + k]);
    before = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t x = __shfl_up(before, d, 64);
        if (lane >= d) before += x;
    }
    if (lane == 63) s_sum[tid >> 6] = before;
    __syncthreads();
    before -= own;
    for (int w = 0; w < tid >> 6; ++w) before += s_sum[w];
#pragma unroll
    for (int k = 0; k < kWords; ++k)
        if (tid * kWords + k < used) {
            s_before[tid * kWords + k] = (uint16_t)before;
            before += __popc(s_bits[tid * kWords + k]);
        }
    __syncthreads();
    int place[kMine];
    bool first[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        first[k] = false;
        if (mine[k] < 0) continue;
        place[k] = s_before[mine[k] >> 5] + __popc(s_bits[mine[k] >> 5] & ((1u << (mine[k] & 31)) - 1));
        first[k] = atomicAdd(&s_times[place[k]], 1) == 0;
    }
    set_all(h.seen + ((size_t)r * 2 + 1) * words, s_bits, (h.V + 31) / 32);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMine; ++k)
        if (first[k]) atomicAdd(h.count + (size_t)r * h.V + mine[k], s_times[place[k]]);
}

template <class E>
hipError_t run(const TargetArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.t.R * (unsigned)a.parts, a.t.max_new);
    const size_t lds = ((a.seen || a.t.ver_tokens || a.t.bias_off ? 1 : 0) + (a.t.allowed ? 1 : 0)) * (size_t)a.chunk / 8;
    if (a.t.adjusted)
        hipLaunchKernelGGL((target_kernel<E, true>), grid, dim3(kT), lds, s, a);
    else
        hipLaunchKernelGGL((target_kernel<E, false>), grid, dim3(kT), lds, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1 || a.came) return e;
    hipLaunchKernelGGL(target_join_kernel, dim3(a.t.R, a.t.max_new), dim3(64), 0, s, a);
    return hipGetLastError();
}

}  // namespace

void target_split(int rows, int V, int& chunk, int& parts) {
    const long long want = ((long long)kWanted + rows - 1) / rows;
    const long long least = std::max<long long>((V + want - 1) / want, std::min(V, kLeastChunk));
    chunk = (int)std::min<long long>((least + 255) / 256 * 256, kMostChunk);
    parts = (int)(((long long)V + chunk - 1) / chunk);
}

// The counts have a place of their own in every call, whatever its rows, or what another call has left
// would be taken for them.
void target_ws_layout(TargetArgs& a, void* ws) {
    a.came = a.t.n_rows <= kCounted ? (uint32_t*)ws : nullptr;
    a.best = (TargetBest*)((uint32_t*)ws + kCounted);
}

size_t target_ws_bytes(long long n_rows, int parts) {
    return kCounted * sizeof(uint32_t) + (size_t)(n_rows * parts) * sizeof(TargetBest);
}

// Of every vocabulary up to V, however many rows: a larger one may have fewer (2097152 tokens of one row
// are 512 parts, 2097153 are 482).  Parts are as many as are wanted at most, and parts of kLeastChunk or
// more, unless kMostChunk makes them more.
int target_most_parts(int V) {
    const auto parts = [&](int chunk) { return (int)(((long long)V + chunk - 1) / chunk); };
    return std::max(std::min(kWanted, parts(kLeastChunk)), parts(kMostChunk));
}

hipError_t launch_target(const TargetArgs& a, hipStream_t s) {
    return a.t.dtype == DSPARK_F32 ? run<F32>(a, s) : a.t.dtype == DSPARK_F16 ? run<F16>(a, s) : run<Bf16>(a, s);
}

hipError_t launch_history_clear(const dspark_history_t& h, const int32_t* rows, int n, uint32_t* status, hipStream_t s) {
    const size_t words = dspark_history_words(h.V);
    const int slices = (int)std::min<size_t>((words + kHistoryT - 1) / kHistoryT, 64);
    hipLaunchKernelGGL(history_clear_kernel, dim3(n, slices), dim3(kHistoryT), 0, s, h, words, rows, status);
    return hipGetLastError();
}

hipError_t launch_history_add(const dspark_history_t& h, const int32_t* tokens, int n, int width, const int32_t* rows,
                              int answered, uint32_t* status, hipStream_t s) {
    const size_t words = dspark_history_words(h.V);
    if (width < kWideFrom || h.V > (answered ? kMostInLds / 2 : kMostInLds) || (long long)width > 65535ll * kAnswerSlice) {
        const int slices = std::min((width - 1) / kHistoryT + 1, 256);
        hipLaunchKernelGGL(history_add_kernel, dim3(n, slices), dim3(kHistoryT), 0, s, h, words, tokens, width, rows,
                           answered, status);
    } else if (answered) {
        hipLaunchKernelGGL(history_answer_kernel, dim3(n, (width + kAnswerSlice - 1) / kAnswerSlice), dim3(kWideT),
                           (h.V + 63) / 64 * 2 * sizeof(uint32_t), s, h, words, tokens, width, rows, status);
    } else {
        hipLaunchKernelGGL(history_prompt_kernel, dim3(n, (width + kPromptSlice - 1) / kPromptSlice), dim3(kWideT),
                           (h.V + 31) / 32 * sizeof(uint32_t), s, h, words, tokens, width, rows, status);
    }
    return hipGetLastError();
}

}  // namespace dspark
