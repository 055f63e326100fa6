// Trees of drafts: chains merged into one tree a request, depths and ancestors of the nodes,
// the accepted path, and that path's keys and values moved together.
//
// A request has at most 64 nodes, so one wave holds a tree, a node (or a chain's token) to a
// lane, and sets of nodes are 64-bit words: comparing is a ballot, counting a population
// count, and a number among the set's members the count of those before.
//
// Merging, planning and accepting are launches and their loads, which wait for each other: 2.8, 2.7 and 3.0 us
// for 16 requests (kernels, under the profiler), 3.2 and 3.7 for planning and accepting 256, whatever the
// trees. More than 64 requests are merged in two launches, counts and then writes: 4.2 and 3.5 us for 256.
#include <algorithm>

#include "common.h"
#include "tree.h"

namespace dspark {

namespace {

constexpr int kWaves = 4, kT = kWaves * 64;  // requests a workgroup

__device__ __forceinline__ uint64_t below(int n) { return n >= 64 ? ~0ull : (1ull << n) - 1; }
__device__ __forceinline__ uint64_t shfl64(uint64_t x, int lane) {
    const uint32_t lo = __shfl((uint32_t)x, lane, 64), hi = __shfl((uint32_t)(x >> 32), lane, 64);
    return (uint64_t)hi << 32 | lo;
}

// One request's chains: lane s K + i holds token i of chain s.  The token's node is that of the
// lowest chain that begins with the same i + 1 tokens; `made` are the lanes that are that one
// themselves.  Chain s agrees with chain t up to token i where a ballot of equal tokens has
// the bits s K .. s K + i.
struct Chains {  // a lane's token, and how many of its chain's count
    int token, len;
};
__device__ __forceinline__ Chains chains_of(const int32_t* tokens, const int32_t* prefix_len, int r, int S, int K) {
    const int lane = threadIdx.x & 63, s = lane / K;
    const bool in = s < S;
    return Chains{in ? tokens[(size_t)r * S * K + lane] : 0, in ? prefix_len ? prefix_len[r * S + s] : K : 0};
}
struct Merged {
    int token, node, parent;
    uint64_t made;
};
__device__ __forceinline__ Merged merged(Chains c, int S, int K, uint32_t& bad) {
    const int lane = threadIdx.x & 63, s = lane / K, i = lane % K;
    if (c.len < 0 || c.len > K) {
        c.len = 0;
        bad = kStatusBadRow;
    }
    Merged m;
    m.token = c.token;
    const bool valid = i < c.len;
    const uint64_t want = below(i + 1) << (s * K & 63);
    int first = s;
    bool open = valid;
    for (int t = 0; t < S; ++t) {
        const int other = __shfl(m.token, t * K + i, 64), there = __shfl((int)valid, t * K + i, 64);
        const uint64_t same = __ballot(valid && there && other == m.token);
        if (open && (same & want) == want) {
            first = t;
            open = false;
        }
    }
    m.made = __ballot(valid && first == s);
    m.node = __popcll(m.made & below(first * K + i)) + 1;
    const int before = __shfl(m.node, lane > 0 ? lane - 1 : 0, 64);
    m.parent = i == 0 ? 0 : before;
    return m;
}

// What a merge writes of request r, whose nodes begin at o.
struct MergeOut {
    int32_t *counts, *offsets, *ver_tokens, *parent;
};
__device__ __forceinline__ void write_merged(const MergeOut& out, const Merged& m, int r, int R, int o) {
    const int lane = threadIdx.x & 63;
    if (m.made >> lane & 1) {
        out.ver_tokens[o + m.node - 1] = m.token;
        out.parent[o + r + m.node] = m.parent;
    }
    if (lane == 0) {
        out.parent[o + r] = -1;
        out.offsets[r] = o;
        if (r == R - 1) out.offsets[R] = o + __popcll(m.made);
    }
}

// Few requests: one workgroup, kEach requests to a wave, whose chains are all asked for at once.
constexpr int kMergeWaves = 16;
template <int kEach>
__global__ __launch_bounds__(kMergeWaves * 64) void merge_kernel(const int32_t* tokens, const int32_t* prefix_len, int R, int S,
                                                                 int K, MergeOut out, uint32_t* status) {
    __shared__ int s_n[kEach * kMergeWaves];
    const int lane = threadIdx.x & 63, r0 = (threadIdx.x >> 6) * kEach;
    Chains c[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) c[k] = r0 + k < R ? chains_of(tokens, prefix_len, r0 + k, S, K) : Chains{0, 0};
    Merged m[kEach];
    uint32_t bad = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        m[k] = merged(c[k], S, K, bad);
        if (lane == 0) s_n[r0 + k] = __popcll(m[k].made);
    }
    if (__ballot(bad != 0) && lane == 0) raise_status(status, kStatusBadRow);
    __syncthreads();
    int o = lane < r0 ? s_n[lane] : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) o += __shfl_xor(o, d, 64);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        if (r0 + k >= R) return;
        if (lane == 0) out.counts[r0 + k] = __popcll(m[k].made);
        write_merged(out, m[k], r0 + k, R, o);
        o += __popcll(m[k].made);
    }
}

__global__ __launch_bounds__(kT) void merge_count_kernel(const int32_t* tokens, const int32_t* prefix_len, int R, int S,
                                                         int K, int32_t* counts, uint32_t* status) {
    const int r = blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (r >= R) return;
    uint32_t bad = 0;
    const Merged m = merged(chains_of(tokens, prefix_len, r, S, K), S, K, bad);
    if (__ballot(bad != 0) && (threadIdx.x & 63) == 0) raise_status(status, kStatusBadRow);
    if ((threadIdx.x & 63) == 0) counts[r] = __popcll(m.made);
}

// Every workgroup adds up the counts before its requests itself (R of them at most 8192), so
// that no launch is spent on a running sum.
__global__ __launch_bounds__(kT) void merge_write_kernel(const int32_t* tokens, const int32_t* prefix_len, int R, int S,
                                                         int K, MergeOut out) {
    __shared__ int s_sum[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r0 = blockIdx.x * kWaves, r = r0 + wave;
    int sum = 0;
    for (int i = threadIdx.x; i < r0; i += kT) sum += out.counts[i];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    int o = 0;
    for (int w = 0; w < kWaves; ++w) o += s_sum[w];
    for (int i = r0; i < r && i < R; ++i) o += out.counts[i];
    if (r >= R) return;
    uint32_t bad = 0;
    const Merged m = merged(chains_of(tokens, prefix_len, r, S, K), S, K, bad);
    write_merged(out, m, r, R, o);
}

__global__ __launch_bounds__(kT) void tree_plan_kernel(const int32_t* parent, int n_rows, const int32_t* offsets,
                                                       int lead, int R, int max_new, int32_t* depth, uint64_t* anc,
                                                       uint32_t* status) {
    const int lane = threadIdx.x & 63, r = blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (r >= R) return;
    const int o = offsets[r];
    const long long n = (long long)offsets[r + 1] - o + lead, start = (long long)o + (long long)lead * r;
    if (o < 0 || n < 0 || n > max_new || start + n > n_rows) {
        if (lane == 0) raise_status(status, kStatusBadRow);
        return;
    }
    const bool in = lane < n;
    int up = in ? parent[start + lane] : -1;
    bool dead = in && (up < -1 || up >= lane);
    if (dead || up < 0) up = lane;
    uint64_t word = 1ull << lane;
#pragma unroll
    for (int step = 0; step < 6; ++step) {  // each covers twice as many generations
        word |= shfl64(word, up);
        const int gone = __shfl((int)dead, up, 64);
        up = __shfl(up, up, 64);
        dead |= gone != 0;
    }
    if (__ballot(dead) && lane == 0) raise_status(status, kStatusBadRow);
    if (in) {
        depth[start + lane] = dead ? 0 : __popcll(word) - 1;
        anc[start + lane] = dead ? 0 : word;
    }
}

// Lane j holds node j, so a step down the path is a ballot of the nodes that hang on the current
// one and say its target, without memory: only later nodes count, so it ends.
__global__ __launch_bounds__(kT) void accept_tree_kernel(const int32_t* ver_tokens, int n_nodes, const int32_t* offsets,
                                                         const int32_t* parent, const int32_t* target, int R, int K,
                                                         int32_t* accept_len, int32_t* path, int32_t* next_prev0,
                                                         int32_t* out_tokens, uint32_t* status) {
    const int lane = threadIdx.x & 63, r = blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (r >= R) return;
    const int o = offsets[r];
    const long long L = (long long)offsets[r + 1] - o;
    const bool ok = o >= 0 && L >= 0 && L < kTreeNodes && o + L <= n_nodes;
    int accepted = 0, bonus = -1, mine = -1, said = -1;  // mine, said: lane i's entry of path and of out_tokens
    if (ok) {
        const bool node = lane >= 1 && lane <= L;
        const int up = node ? parent[(size_t)o + r + lane] : -1, token = node ? ver_tokens[o + lane - 1] : -1;
        const int choice = lane <= L ? target[(size_t)o + r + lane] : -1;
        int at = 0;
        for (;;) {
            bonus = __shfl(choice, at, 64);
            if (accepted == K) break;
            const uint64_t next = __ballot(node && lane > at && up == at && token == bonus);
            if (!next) break;
            at = (int)__ffsll((unsigned long long)next) - 1;
            if (lane == accepted) {
                mine = at;
                said = bonus;
            }
            ++accepted;
        }
        if (lane == accepted) said = bonus;
    } else if (lane == 0) {
        raise_status(status, kStatusBadAllocation);
    }
    if (lane == 0) {
        accept_len[r] = accepted;
        next_prev0[r] = bonus;
    }
    if (lane < K) path[(size_t)r * K + lane] = mine;
    if (out_tokens && lane <= K) out_tokens[(size_t)r * (K + 1) + lane] = said;
}

// A row of V in a block of 16 tokens: the tokens' values of one dim, two to a word.
typedef uint32_t u32x8 __attribute__((ext_vector_type(8), aligned(16)));
__device__ __forceinline__ uint32_t value_at(const u32x8& row, int i) { return row[i >> 1] >> (16 * (i & 1)) & 0xFFFFu; }
__device__ __forceinline__ void put_at(u32x8& row, int i, uint32_t x) {
    const uint32_t w = row[i >> 1];
    row[i >> 1] = i & 1 ? (w & 0xFFFFu) | x << 16 : (w & 0xFFFF0000u) | x;
}

// A workgroup takes a request's K or its V in a layer.  Nodes move towards the front and in rising order, so
// what one takes the place of has been read, or is none of the path's: a thread keeps to its dims and
// waits for nobody.  Of K it moves 16 bytes, eight dims of a token; of V it reads the whole row of a dim in
// the block that tokens come to, 32 bytes, sets their values in it (from the same row, or from other
// blocks, where they are read alone) and writes it back: the block is this request's own.
//
// Waiting bounds it: the page ids come after the path and the lengths, the data after them.  256 requests
// of up to 28 nodes, 16 layers of 8 key heads of 128: 23 us, of which 67 MB read and written would take 14;
// with two bytes of V at a time 34, with K and V one after the other 41, with some layers one after the
// other 76.  The workgroups of a request stand together in the grid: with the layers together it takes 31.
// (The compiler keeps the rows of V that a thread has under way in LDS, 16 KB of a workgroup's 17.5.)
__global__ __launch_bounds__(kT) void keep_path_kernel(dspark_cache_t c, const int32_t* path, int K,
                                                       const int32_t* accept_len, const int32_t* granted, int lead,
                                                       uint32_t* status) {
    constexpr int kAtOnce = 4;  // tokens of K, and rows of V, under way
    __shared__ int s_from[kTreeNodes], s_to[kTreeNodes], s_n;
    __shared__ size_t s_from_at[kTreeNodes], s_to_at[kTreeNodes];
    const int r = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
    const int ln = c.len[r], n = accept_len[r];
    if (ln < 0 || (granted && granted[r] == 0)) return;
    const int shift = __builtin_ctz(c.page_size), D = c.head_dim;
    if (tid < 64) {
        bool bad = n < 0 || n > K, gone = false;
        int from = 0, to = 0;
        size_t from_at = 0, to_at = 0;
        const bool in = !bad && lane < n;
        if (in) {
            from = path[(size_t)r * K + lane];
            const int prev = lane ? path[(size_t)r * K + lane - 1] : lead - 1;
            to = lead + lane;
            bad = from <= prev || from >= kTreeNodes || ((long long)ln + from) >> shift >= c.width;
        }
        const bool moves = in && from != to;
        bad = __ballot(bad) != 0;
        if (!bad && moves) {
            const long long p = (long long)ln + from, q = (long long)ln + to;
            const int fp = c.table[(size_t)r * c.width + (p >> shift)], tp = c.table[(size_t)r * c.width + (q >> shift)];
            gone = (unsigned)fp >= (unsigned)c.n_pages || (unsigned)tp >= (unsigned)c.n_pages || c.ref[tp] > 1;
            // the token's block in its page's first head, in values of a head
            from_at = (((size_t)(unsigned)fp * c.n_kv_heads << shift) + (p & (c.page_size - 16))) * D;
            to_at = (((size_t)(unsigned)tp * c.n_kv_heads << shift) + (q & (c.page_size - 16))) * D;
            from = (int)(p & 15);
            to = (int)(q & 15);
        }
        gone = __ballot(gone) != 0;
        if (lane == 0 && blockIdx.x == 0 && (bad || gone)) raise_status(status, bad ? kStatusBadRow : kStatusBadPage);
        const uint64_t all = bad || gone ? 0 : __ballot(moves);
        if (all >> lane & 1) {
            const int at = __popcll(all & below(lane));
            s_from[at] = from;
            s_to[at] = to;
            s_from_at[at] = from_at;
            s_to_at[at] = to_at;
        }
        if (lane == 0) s_n = __popcll(all);
    }
    __syncthreads();
    const int moved = __builtin_amdgcn_readfirstlane(s_n);
    if (moved == 0) return;
    const size_t layer = (size_t)(blockIdx.x >> 1) * c.n_pages * c.n_kv_heads * c.page_size * D;
    if (blockIdx.x & 1) {
        for (int e = tid; e < c.n_kv_heads * (D / 8); e += kT) {
            uint16_t* p = (uint16_t*)c.k + layer + ((size_t)(e / (D / 8)) << shift) * D + (size_t)(e % (D / 8)) * 128;
            for (int i0 = 0; i0 < moved; i0 += kAtOnce) {
                uint4 x[kAtOnce];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    const int at = min(i0 + i, moved - 1);
                    x[i] = *(const uint4*)(p + s_from_at[at] + s_from[at] * 8);
                }
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (i0 + i < moved) *(uint4*)(p + s_to_at[i0 + i] + s_to[i0 + i] * 8) = x[i];
            }
        }
        return;
    }
    const int rows = c.n_kv_heads * D;
    for (int e0 = tid; e0 < rows; e0 += kT * kAtOnce) {
        uint16_t* p[kAtOnce];
#pragma unroll
        for (int d = 0; d < kAtOnce; ++d) {
            const int e = min(e0 + d * kT, rows - 1);
            p[d] = (uint16_t*)c.v + layer + ((size_t)(e / D) << shift) * D + (size_t)(e % D) * 16;
        }
        for (int i = 0; i < moved;) {
            const size_t block = s_to_at[i];
            u32x8 x[kAtOnce];
#pragma unroll
            for (int d = 0; d < kAtOnce; ++d) x[d] = *(const u32x8*)(p[d] + block);
            for (; i < moved && s_to_at[i] == block; ++i) {
                const int from = __builtin_amdgcn_readfirstlane(s_from[i]), to = __builtin_amdgcn_readfirstlane(s_to[i]);
                const size_t source = s_from_at[i];
                uint32_t y[kAtOnce];
#pragma unroll
                for (int d = 0; d < kAtOnce; ++d) y[d] = source == block ? value_at(x[d], from) : p[d][source + from];
#pragma unroll
                for (int d = 0; d < kAtOnce; ++d) put_at(x[d], to, y[d]);
            }
#pragma unroll
            for (int d = 0; d < kAtOnce; ++d)
                if (e0 + d * kT < rows) *(u32x8*)(p[d] + block) = x[d];
        }
    }
}

// The requests up to which one workgroup merges them. Whole calls, one after the other in a graph: 3.4 us for 16
// requests, 4.2 for 32 and 6.2 for 64, where counting and writing, two launches, take 5.4, 5.6 and 5.7, and
// outside a graph the host 3 more for the second.
constexpr int kMergeAtOnce = 4 * kMergeWaves;
static_assert(kMergeAtOnce <= 64, "a request's count to a lane");

int groups(int R) { return (R + kWaves - 1) / kWaves; }

}  // namespace

hipError_t launch_tree_merge(const int32_t* tokens, const int32_t* prefix_len, int R, int S, int K, int32_t* counts,
                             int32_t* offsets, int32_t* ver_tokens, int32_t* parent, uint32_t* status, hipStream_t s) {
    const MergeOut out{counts, offsets, ver_tokens, parent};
    if (R <= kMergeAtOnce) {
        const auto kernel = R <= kMergeWaves ? merge_kernel<1> : R <= 2 * kMergeWaves ? merge_kernel<2> : merge_kernel<4>;
        hipLaunchKernelGGL(kernel, dim3(1), dim3(kMergeWaves * 64), 0, s, tokens, prefix_len, R, S, K, out, status);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(merge_count_kernel, dim3(groups(R)), dim3(kT), 0, s, tokens, prefix_len, R, S, K, counts, status);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(merge_write_kernel, dim3(groups(R)), dim3(kT), 0, s, tokens, prefix_len, R, S, K, out);
    return hipGetLastError();
}

hipError_t launch_tree_plan(const int32_t* parent, int n_rows, const int32_t* offsets, int lead, int R, int max_new,
                            int32_t* depth, uint64_t* anc, uint32_t* status, hipStream_t s) {
    hipLaunchKernelGGL(tree_plan_kernel, dim3(groups(R)), dim3(kT), 0, s, parent, n_rows, offsets, lead, R, max_new,
                       depth, anc, status);
    return hipGetLastError();
}

hipError_t launch_accept_tree(const int32_t* ver_tokens, int n_nodes, const int32_t* offsets, const int32_t* parent,
                              const int32_t* target, int R, int K, int32_t* accept_len, int32_t* path,
                              int32_t* next_prev0, int32_t* out_tokens, uint32_t* status, hipStream_t s) {
    hipLaunchKernelGGL(accept_tree_kernel, dim3(groups(R)), dim3(kT), 0, s, ver_tokens, n_nodes, offsets, parent,
                       target, R, K, accept_len, path, next_prev0, out_tokens, status);
    return hipGetLastError();
}

hipError_t launch_keep_path(const dspark_cache_t& c, const int32_t* path, int K, const int32_t* accept_len,
                            const int32_t* granted, int lead, int R, uint32_t* status, hipStream_t s) {
    hipLaunchKernelGGL(keep_path_kernel, dim3(2 * c.layers, R), dim3(kT), 0, s, c, path, K, accept_len, granted, lead, status);
    return hipGetLastError();
}

}  // namespace dspark
