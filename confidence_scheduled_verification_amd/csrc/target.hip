// The target's choice at each row, from its logits: penalties for repeated tokens, biases and
// grammar masks, and the argmax, in one pass over the logits; and the record of what has been
// said, which the penalties read.
//
// Few tokens of a row are changed at all: those seen, biased, or drafted on the row's path.  Each
// of these has one owner, who takes it out of the bits of what is left and computes its value in
// 64 bits by itself; the others compare as they are, in fp32, eight at a time under eight bits.
// So the pass over the logits costs what an argmax costs, and the counts are read only at the
// few tokens that have any.
//
// A workgroup takes a part of a row (all of it where there are rows enough):
//   1. the bits of the tokens that the row's mask allows go to LDS;
//   2. biased tokens and the path's are owned by their entry in the list;
//   3. seen ones by their bit: they are gathered in a list in LDS, so that the lanes share them
//      evenly however they cluster, and several of their loads are under way at a time;
//   4. the rest is streamed.
// Every value has an order key, and the largest key with the lowest token wins.
#include <algorithm>

#include "common.h"
#include "tree.h"

namespace dspark {

namespace {

constexpr int kT = 256;
constexpr int kGroups = 4;             // of eight logits, that a lane has under way
constexpr int kMostChunk = 131072;     // tokens of a part: 16 KB of bits in LDS
constexpr int kList = 2048;            // seen tokens gathered at a time
constexpr float kInf = __builtin_huge_valf();

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

// Row j of request r, where it is one (the first workgroup of a request says what does not fit).
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

// Where `tok` is in the request's biases [b0, b1), -1 if it is not there.  In a list that does not
// rise it may not be found; each token has at most one place either way.
__device__ __forceinline__ int find_bias(const int32_t* bias_tok, int b0, int b1, int tok) {
    while (b0 < b1) {
        const int mid = b0 + ((b1 - b0) >> 1), t = bias_tok[mid];
        if (t == tok) return mid;
        if (t < tok) b0 = mid + 1; else b1 = mid;
    }
    return -1;
}

template <class E, bool kOut>
__global__ __launch_bounds__(kT) void target_kernel(TargetArgs a) {
    typedef typename E::T T;
    const dspark_target_t& t = a.t;
    // bits of the part's tokens, with a word before them and one behind: [0] allowed and without an
    // owner so far; [1] (kOut) owned
    extern __shared__ uint32_t s_words[];
    __shared__ uint32_t s_list[kList];
    __shared__ int s_path[DSPARK_TARGET_MAX_ROWS];
    __shared__ uint32_t s_count, s_limit;
    __shared__ Best s_best[kT / 64];
    const int r = blockIdx.x, j = blockIdx.y, part = blockIdx.z, tid = threadIdx.x;
    int o, n;
    long long start;
    uint32_t bad = 0;
    if (!row_of(t, r, j, o, start, n, bad)) {
        if (bad && j == 0 && part == 0 && tid == 0) raise_status(a.status, bad);
        return;
    }
    const size_t row = (size_t)(start + j);
    const int lo = part * a.chunk, hi = min(t.V, lo + a.chunk), n_words = (hi - lo + 31) / 32;
    uint32_t *s_left = s_words + 1, *s_owned = s_words + (a.chunk / 32 + 2) + 1;
    const T* logits = (const T*)t.logits + row * t.logits_stride;
    T* out = kOut ? (T*)t.adjusted + row * t.adjusted_stride : nullptr;

    // 1. what is allowed
    const uint32_t* allowed = nullptr;
    bool nothing = false;
    if (t.allowed) {
        long long pick = t.allowed_row ? t.allowed_row[row] : (long long)row;
        if (pick < -1 || pick >= t.n_allowed) {
            nothing = true;
            bad = kStatusBadRow;
        } else if (pick >= 0) {
            allowed = t.allowed + (size_t)pick * t.allowed_stride + lo / 32;
        }
    }
    for (int w = tid; w <= n_words; w += kT) {
        uint32_t x = 0;
        if (w < n_words && !nothing) {
            x = allowed ? allowed[w] : ~0u;
            const int rest = hi - lo - w * 32;
            if (rest < 32) x &= (1u << rest) - 1;
        }
        s_left[w] = x;
        if (kOut) s_owned[w] = 0;
    }
    if (tid == 0) {
        s_words[0] = 0;
        if (kOut) s_owned[-1] = 0;
    }

    const bool penalties = t.repetition || t.presence || t.frequency;
    const uint32_t *prompt = nullptr, *answered = nullptr;
    const int32_t* count = nullptr;
    if (penalties && a.seen) {
        prompt = a.seen + (size_t)r * 2 * a.words + lo / 32;
        answered = prompt + a.words;
        count = a.count + (size_t)r * t.V;
    }
    const double repetition = t.repetition ? t.repetition[r] : 1.f, presence = t.presence ? t.presence[r] : 0.f,
                 frequency = t.frequency ? t.frequency[r] : 0.f;
    const int n_path = penalties && t.ver_tokens ? n : 0;
    if (n_path) {
        const uint64_t word = t.anc ? t.anc[row] : 0;
        for (int i = tid; i < n; i += kT) {
            const bool on = i >= t.lead && (t.anc ? (word >> (i & 63) & 1) != 0 : i <= j);
            const int at = o + i - t.lead;
            s_path[i] = on && at < t.n_nodes ? t.ver_tokens[at] : -1;
        }
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
    __syncthreads();

    // 2. biased tokens and the path's
    Best best{0, ~0u};
    const auto put = [&](int v, double x) {
        best.take(order_key(x), (uint32_t)v);
        if (kOut) out[v] = E::bits((float)x);
    };
    const auto penalised = [&](int v, bool seen, int c) {
        double x = (double)E::value(logits[v]);
        if (seen || c > 0) x = x > 0.0 ? x / repetition : x * repetition;
        x = x - frequency * (double)c;
        if (c > 0) x = x - presence;
        return x;
    };
    // The owner of v takes it; false where it is not allowed.
    const auto own = [&](int v) {
        const int w = (v - lo) >> 5;
        const uint32_t bit = 1u << ((v - lo) & 31);
        if (kOut) atomicOr(&s_owned[w], bit);
        if (atomicAnd(&s_left[w], ~bit) & bit) return true;
        if (kOut) out[v] = E::kNegInf;
        return false;
    };
    const auto on_path = [&](int v) {
        int c = 0;
        for (int i = 0; i < n_path; ++i) c += s_path[i] == v;
        return c;
    };
    const auto listed = [&](int v, int c) {  // the value of a token of one of the lists, c times on the path
        bool seen = false;
        if (prompt) {
            const int w = (v - lo) >> 5, bit = (v - lo) & 31;
            seen = prompt[w] >> bit & 1;
            if (answered[w] >> bit & 1) c += count[v];
        }
        return penalised(v, seen, c);
    };
    for (int e = b0 + tid; e < b1; e += kT) {
        const int v = t.bias_tok[e];
        if (v < 0 || v >= t.V || (e > b0 && t.bias_tok[e - 1] >= v)) bad = kStatusBadRow;
        if (v < lo || v >= hi || find_bias(t.bias_tok, b0, b1, v) != e || !own(v)) continue;
        put(v, listed(v, on_path(v)) + (double)t.bias_val[e]);
    }
    for (int i = tid; i < n_path; i += kT) {
        const int v = s_path[i];
        if (v < lo || v >= hi) continue;
        int first = 0;
        while (s_path[first] != v) ++first;
        if (first != i || find_bias(t.bias_tok, b0, b1, v) >= 0 || !own(v)) continue;
        put(v, listed(v, on_path(v)));
    }
    if (bad && part == 0) raise_status(a.status, bad);

    // 3. seen tokens, as many at a time as the list takes: words that did not fit come again
    if (prompt) {
        for (bool more = true; more;) {
            __syncthreads();
            if (tid == 0) {
                s_count = 0;
                s_limit = ~0u;
            }
            __syncthreads();
            for (int w = tid; w < n_words; w += kT) {
                const uint32_t left = s_left[w], said = answered[w] & left, seen = (prompt[w] & left) | said;
                if (!seen) continue;
                const uint32_t at = atomicAdd(&s_count, (uint32_t)__popc(seen));
                if (at + __popc(seen) > kList) {
                    atomicMin(&s_limit, at);
                    continue;
                }
                s_left[w] = left & ~seen;
                if (kOut) s_owned[w] |= seen;
                uint32_t to = at;
                for (uint32_t x = seen; x; x &= x - 1) {
                    const int b = __ffs(x) - 1;
                    s_list[to++] = (uint32_t)(lo + w * 32 + b) | (said >> b & 1) << 31;
                }
            }
            __syncthreads();
            const uint32_t n_list = min(s_count, s_limit);
            more = s_limit != ~0u;
            for (uint32_t i = tid; i < n_list; i += kT) {
                const int v = (int)(s_list[i] & 0x7FFFFFFFu);
                put(v, penalised(v, true, s_list[i] >> 31 ? count[v] : 0));
            }
        }
    }
    __syncthreads();

    // 4. the others, in groups of eight from the last boundary of eight values in memory on
    const int before = (int)(((uintptr_t)(logits + lo) / sizeof(T)) & 7), first = lo - before;
    const int n_groups = (hi - first + 7) / 8;
    const uint8_t *left = (const uint8_t*)s_left, *owned = (const uint8_t*)s_owned;
    const auto eight = [&](const uint8_t* bits, int g) {  // of group g's tokens
        const int at = g * 8 - before;
        const uint32_t x = bits[at >> 3];
        return before ? ((x | (uint32_t)bits[(at >> 3) + 1] << 8) >> (at & 7)) & 0xFFu : x;
    };
    struct Eight {
        T x[8];
    };
    const auto load = [&](int g) {
        const int v = first + g * 8;
        Eight e;
        if (v >= 0 && v + 8 <= t.V) {
            typedef uint4 alias __attribute__((may_alias));
            const alias* p = (const alias*)(logits + v);
            uint4 w[sizeof(e) / 16];
#pragma unroll
            for (int i = 0; i < (int)(sizeof(e) / 16); ++i) w[i] = p[i];
            __builtin_memcpy(&e, w, sizeof(e));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) e.x[i] = v + i >= 0 && v + i < t.V ? logits[v + i] : E::kNegInf;
        }
        return e;
    };
    float top = -kInf;  // of this lane's groups; NaN where there is one
    int top_group = -1;
    for (int g0 = tid; g0 < n_groups; g0 += kT * kGroups) {
        Eight e[kGroups];
        uint32_t bits[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int g = g0 + i * kT;
            bits[i] = g < n_groups ? eight(left, g) : 0;
            e[i] = load(bits[i] ? g : 0);  // (a group without bits is not read)
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int g = g0 + i * kT;
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t on = (uint32_t)((int32_t)(bits[i] << (31 - k)) >> 31);
                x[k] = __uint_as_float((__float_as_uint(E::value(e[i].x[k])) & on) | (0xFF800000u & ~on));
            }
            float m = x[0];
#pragma unroll
            for (int k = 1; k < 8; ++k) m = __builtin_elementwise_maximum(m, x[k]);
            if (m > top) top_group = g;
            top = __builtin_elementwise_maximum(top, m);
            if (kOut && g < n_groups) {
                const int v = first + g * 8;
                const uint32_t skip = eight(owned, g);
                if (!skip && v >= lo && v + 8 <= hi && ((uintptr_t)(out + v) & 15) == 0) {
                    Eight y;
#pragma unroll
                    for (int k = 0; k < 8; ++k) y.x[k] = bits[i] >> k & 1 ? e[i].x[k] : E::kNegInf;
                    typedef uint4 alias __attribute__((may_alias));
                    uint4 w[sizeof(y) / 16];
                    __builtin_memcpy(w, &y, sizeof(y));
#pragma unroll
                    for (int q = 0; q < (int)(sizeof(y) / 16); ++q) ((alias*)(out + v))[q] = w[q];
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (v + k >= lo && v + k < hi && !(skip >> k & 1)) out[v + k] = bits[i] >> k & 1 ? e[i].x[k] : E::kNegInf;
                }
            }
        }
    }
    if (top > -kInf) {
        const Eight e = load(top_group);
        const uint32_t bits = eight(left, top_group);
#pragma unroll
        for (int k = 7; k >= 0; --k)
            if ((bits >> k & 1) && E::value(e.x[k]) == top) best.take(order_key((double)top), (uint32_t)(first + top_group * 8 + k));
    } else {  // a NaN, or nothing above -inf: this lane's groups once more, value by value
        for (int g = tid; g < n_groups; g += kT) {
            const uint32_t bits = eight(left, g);
            for (int k = 0; k < 8; ++k)
                if (bits >> k & 1) {
                    const int v = first + g * 8 + k;
                    best.take(order_key((double)E::value(logits[v])), (uint32_t)v);
                }
        }
    }

    wave_best(best);
    if ((tid & 63) == 0) s_best[tid >> 6] = best;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kT / 64; ++w) best.take(s_best[w].key, s_best[w].v);
        if (a.parts > 1) {
            a.best[row * a.parts + part] = TargetBest{best.key, best.v, 0};
        } else {
            t.target[row] = best.key ? (int32_t)best.v : -1;
            if (!best.key) raise_status(a.status, kStatusNoToken);
        }
    }
}

// The best of a row's parts: a wave to a row.
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
        a.t.target[row] = best.key ? (int32_t)best.v : -1;
        if (!best.key) raise_status(a.status, kStatusNoToken);
    }
}

// A history row emptied: the counts only where there are any.
__global__ __launch_bounds__(kT) void history_clear_kernel(dspark_history_t h, size_t words, const int32_t* rows,
                                                           uint32_t* status) {
    const int i = blockIdx.x, r = rows ? rows[i] : i;
    if (r < 0 || r >= h.rows) {
        if (blockIdx.y == 0 && threadIdx.x == 0) raise_status(status, kStatusBadRow);
        return;
    }
    uint32_t *prompt = h.seen + (size_t)r * 2 * words, *answered = prompt + words;
    int32_t* count = h.count + (size_t)r * h.V;
    for (size_t w = blockIdx.y * kT + threadIdx.x; w < words; w += (size_t)gridDim.y * kT) {
        for (uint32_t x = answered[w]; x; x &= x - 1) {
            const size_t v = w * 32 + __ffs(x) - 1;
            if (v < (size_t)h.V) count[v] = 0;
        }
        prompt[w] = 0;
        answered[w] = 0;
    }
}

// A bit that is set already needs no atomic: of a prompt's tokens most have been there before.
__global__ __launch_bounds__(kT) void history_add_kernel(dspark_history_t h, size_t words, const int32_t* tokens,
                                                         int width, const int32_t* rows, int answered, uint32_t* status) {
    const int i = blockIdx.x, r = rows ? rows[i] : i;
    if (r < 0 || r >= h.rows) {
        if (blockIdx.y == 0 && threadIdx.x == 0) raise_status(status, kStatusBadRow);
        return;
    }
    uint32_t* bits = h.seen + ((size_t)r * 2 + (answered ? 1 : 0)) * words;
    int32_t* count = h.count + (size_t)r * h.V;
    bool bad = false;
    for (int at = blockIdx.y * kT + threadIdx.x; at < width; at += gridDim.y * kT) {
        const int v = tokens[(size_t)i * width + at];
        if (v < 0) continue;
        if (v >= h.V) {
            bad = true;
            continue;
        }
        const uint32_t bit = 1u << (v & 31);
        if (!(__hip_atomic_load(bits + (v >> 5), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) & bit)) atomicOr(bits + (v >> 5), bit);
        if (answered) atomicAdd(count + v, 1);
    }
    if (bad) raise_status(status, kStatusBadRow);
}

template <class E>
hipError_t run(const TargetArgs& a, hipStream_t s) {
    const size_t lds = (size_t)(a.chunk / 32 + 2) * 4;
    const dim3 grid(a.t.R, a.t.max_new, a.parts);
    if (a.t.adjusted)
        hipLaunchKernelGGL((target_kernel<E, true>), grid, dim3(kT), 2 * lds, s, a);
    else
        hipLaunchKernelGGL((target_kernel<E, false>), grid, dim3(kT), lds, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    hipLaunchKernelGGL(target_join_kernel, dim3(a.t.R, a.t.max_new), dim3(64), 0, s, a);
    return hipGetLastError();
}

}  // namespace

// About four workgroups a compute unit, none of fewer than 4096 tokens.
constexpr int kPerCu = 4, kLeastChunk = 4096;

void target_split(int n_rows, int V, int num_cu, int& chunk, int& parts) {
    const long long want = ((long long)kPerCu * std::min(num_cu, kAttendMaxCus) + n_rows - 1) / n_rows;
    const long long least = std::max<long long>((V + want - 1) / want, std::min(V, kLeastChunk));
    chunk = (int)std::min<long long>((least + 255) / 256 * 256, kMostChunk);
    parts = (int)(((long long)V + chunk - 1) / chunk);
}

size_t target_ws_parts(int n_rows, int V) {
    return std::max<size_t>((size_t)kPerCu * kAttendMaxCus + n_rows, (size_t)n_rows * (((size_t)V + kMostChunk - 1) / kMostChunk));
}

hipError_t launch_target(const TargetArgs& a, hipStream_t s) {
    return a.t.dtype == DSPARK_F32 ? run<F32>(a, s) : a.t.dtype == DSPARK_F16 ? run<F16>(a, s) : run<Bf16>(a, s);
}

hipError_t launch_history_clear(const dspark_history_t& h, const int32_t* rows, int n, uint32_t* status, hipStream_t s) {
    const size_t words = dspark_history_words(h.V);
    const int slices = (int)std::min<size_t>((words + kT - 1) / kT, 64);
    hipLaunchKernelGGL(history_clear_kernel, dim3(n, slices), dim3(kT), 0, s, h, words, rows, status);
    return hipGetLastError();
}

hipError_t launch_history_add(const dspark_history_t& h, const int32_t* tokens, int n, int width, const int32_t* rows,
                              int answered, uint32_t* status, hipStream_t s) {
    const int slices = std::min((width + kT - 1) / kT, 256);
    hipLaunchKernelGGL(history_add_kernel, dim3(n, slices), dim3(kT), 0, s, h, dspark_history_words(h.V), tokens, width,
                       rows, answered, status);
    return hipGetLastError();
}

}  // namespace dspark
