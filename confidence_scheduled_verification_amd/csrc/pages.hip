// Pages of the cache: handing them out, taking them back, sharing and copying them, and
// moving the live ones together.  A page is free where its reference count is 0, and the
// lowest free pages go first, in the order of the requests, so that every result is a
// function of the tables and counts alone.
//
// Ranking the free pages: the counts are cut into slices of 4096, sixteen pages to a thread.
// A first launch counts each slice; in the second each workgroup adds up the slices before
// its own, ranks its free pages by one scan, and gives the page of rank k to the request that
// holds place k of the running needs, found by bisection in LDS.  Two launches, whatever the
// sizes; nothing is kept between calls.
//
// What bounds them: the launches and a few loads that wait for each other, where only numbers
// are moved (trim and reserve together: 15 us for 64 requests and 16 for 1024 over a nearly
// full cache; with the free pages of a slice found one by one by bisection over the counts, 37),
// and the copy of the pages elsewhere, read and written once.  64 forks, a last page of 64
// tokens, 8 heads of 128 and 8 layers each (268 MB): the copy is 50 of 66 us, 5.4 TB/s; 24 whole
// copies (710 MB) 133 of 157 us, 5.3; 6000 of 12000 pages made compact (3.1 GB) 605 of 634 us, 5.2.
// A large library copy reaches 5.5.
#include <algorithm>

#include "cache.h"
#include "common.h"

namespace dspark {

namespace {

constexpr int kT = 256;

__device__ __forceinline__ int pages_of(long long tokens, int page) { return (int)((tokens + page - 1) / page); }

// Inclusive scan over the 256 threads of a workgroup.
__device__ int block_scan(int x, int* tmp) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 63) tmp[w] = x;
    __syncthreads();
    for (int i = 0; i < w; ++i) x += tmp[i];
    return x;
}

__device__ int block_sum(int x, int* tmp) {
#pragma unroll
    for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = x;
    __syncthreads();
    return tmp[0] + tmp[1] + tmp[2] + tmp[3];
}

// A thread's sixteen pages of slice b, one after the other: bit i says whether page first + i
// has a count above zero (live) or not (free).
constexpr int kOwn = kPageSlice / kT;
static_assert(kOwn == 16, "four 16-byte loads to a thread");

__device__ uint32_t own_pages(const dspark_cache_t& c, int b, bool live, int& first) {
    first = b * kPageSlice + (int)threadIdx.x * kOwn;
    uint32_t bits = 0;
    if (first + kOwn <= c.n_pages && ((uintptr_t)c.ref & 15u) == 0) {
        int4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = ((const int4*)(c.ref + first))[i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            bits |= (uint32_t)(x[i].x > 0) << (4 * i) | (uint32_t)(x[i].y > 0) << (4 * i + 1) |
                    (uint32_t)(x[i].z > 0) << (4 * i + 2) | (uint32_t)(x[i].w > 0) << (4 * i + 3);
        return live ? bits : ~bits & 0xFFFFu;
    }
    for (int i = 0; i < kOwn && first + i < c.n_pages; ++i) bits |= (uint32_t)((c.ref[first + i] > 0) == live) << i;
    return bits;
}

__device__ void count_slice(const dspark_cache_t& c, int b, bool live, int32_t* out, int* tmp) {
    int first;
    const int n = block_sum(__popc(own_pages(c, b, live, first)), tmp);
    if (threadIdx.x == 0) out[b] = n;
}

// The free pages of slice b in order, in LDS; returns how many.
__device__ int list_free(const dspark_cache_t& c, int b, int* list, int* tmp) {
    int first;
    uint32_t mine = own_pages(c, b, false, first);
    const int upto = block_scan(__popc(mine), tmp);
    for (int k = upto - __popc(mine); mine; mine &= mine - 1) list[k++] = first + __ffs(mine) - 1;
    __syncthreads();
    if (threadIdx.x == kT - 1) tmp[4] = upto;
    __syncthreads();
    return tmp[4];
}

// Counts of the slices before b, and of all.
__device__ void slices_before(const int32_t* cnt, int n, int b, int& before, int& all, int* tmp) {
    int x = 0, y = 0;
    for (int i = threadIdx.x; i < n; i += kT) {
        const int c = cnt[i];
        y += c;
        if (i < b) x += c;
    }
    before = block_sum(x, tmp);
    all = block_sum(y, tmp);
}

// Running sums of need[0..n) in LDS: cum[i] = need[0] + ... + need[i-1], cum[n] the total.
__device__ void running_needs(const int32_t* need, int n, int* cum, int* tmp) {
    for (int i = threadIdx.x; i < n; i += kT) cum[i] = need[i];
    __syncthreads();
    const int per = (n + kT - 1) / kT, i0 = min(n, (int)threadIdx.x * per), i1 = min(n, i0 + per);
    int x = 0;
    for (int i = i0; i < i1; ++i) x += cum[i];
    int base = block_scan(x, tmp) - x;
    for (int i = i0; i < i1; ++i) {
        const int y = cum[i];
        cum[i] = base;
        base += y;
    }
    if (threadIdx.x == kT - 1) cum[n] = base;
    __syncthreads();
}

// The largest i in [0, n) with cum[i] <= k, for cum[0] = 0 <= k < cum[n]: the request that
// place k belongs to (requests without a need share their start with the next one).
__device__ __forceinline__ int owner_of(const int* cum, int n, int k) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= k) lo = mid; else hi = mid;
    }
    return lo;
}

// Pages that are handed out when `free_n` are free: the places of the requests that are
// served, the running needs up to the first one that does not fit.
__device__ __forceinline__ int served(const int* cum, int n, int free_n) {
    int lo = 0, hi = n + 1;  // largest i in [0, n] with cum[i] <= free_n
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= free_n) lo = mid; else hi = mid;
    }
    return cum[lo];
}

// Pages that row r holds if it covers `ln` tokens: they lie in the row's first entries, so
// the count is found from entry ceil(ln / page) - 1 on.  -1 where that entry holds none.
__device__ int held_pages(const dspark_cache_t& c, const int32_t* row, int ln) {
    const int lane = threadIdx.x & 63;
    const int first = pages_of(ln, c.page_size);
    if (first > c.width) return -1;
    if (first > 0 && row[first - 1] < 0) return -1;
    for (int i0 = first; i0 < c.width; i0 += 64) {
        const int i = i0 + lane;
        const uint64_t none = __ballot(i >= c.width || row[i] < 0);
        if (none) return i0 + (int)__ffsll((unsigned long long)none) - 1;
    }
    return c.width;
}

// First launch of reserve: blocks [0, ns) count the free pages of their slices, the others
// find the needs of four requests each, a wave a request.
__global__ __launch_bounds__(kT) void reserve_needs_kernel(dspark_cache_t c, const int32_t* offsets, int lead, int R,
                                                           int ns, int32_t* cnt, int32_t* need, int32_t* have,
                                                           uint32_t* status) {
    __shared__ int tmp[8];
    if ((int)blockIdx.x < ns) {
        count_slice(c, blockIdx.x, false, cnt, tmp);
        return;
    }
    const int r = (blockIdx.x - ns) * 4 + (threadIdx.x >> 6);
    if (r >= R) return;
    const int ln = c.len[r];
    int nd = 0, hv = 0;
    if (ln >= 0) {
        const long long n = (long long)offsets[r + 1] - offsets[r] + lead;
        hv = held_pages(c, c.table + (size_t)r * c.width, ln);
        const long long want = (ln + n + c.page_size - 1) / c.page_size;
        uint32_t bad = 0;
        if (n < 0 || hv < 0) bad = kStatusBadRow;
        else if (want > c.width) bad = kStatusNoPages;
        if (bad) {
            nd = 0;
            hv = -1;
            if ((threadIdx.x & 63) == 0) raise_status(status, bad);
        } else {
            nd = want > hv ? (int)(want - hv) : 0;
        }
    } else {
        hv = -1;
    }
    if ((threadIdx.x & 63) == 0) {
        need[r] = nd;
        have[r] = hv;
    }
}

__global__ __launch_bounds__(kT) void reserve_assign_kernel(dspark_cache_t c, int R, int ns, const int32_t* cnt,
                                                            const int32_t* need, const int32_t* have,
                                                            int32_t* granted, uint32_t* status) {
    extern __shared__ int cum[];  // R + 1
    __shared__ int list[kPageSlice], tmp[8];
    const int b = blockIdx.x;
    int before, all;
    slices_before(cnt, ns, b, before, all, tmp);
    running_needs(need, R, cum, tmp);
    const int give = served(cum, R, all);
    if (b == 0) {
        bool short_of = false;
        for (int r = threadIdx.x; r < R; r += kT) {
            const bool ok = have[r] >= 0 && (need[r] == 0 || cum[r + 1] <= all);
            granted[r] = ok;
            short_of |= have[r] >= 0 && !ok;
        }
        if (short_of) raise_status(status, kStatusNoPages);
    }
    if (before >= give) return;
    const int count = list_free(c, b, list, tmp);
    for (int i = threadIdx.x; i < count && before + i < give; i += kT) {
        const int p = list[i], k = before + i, r = owner_of(cum, R, k);
        c.table[(size_t)r * c.width + have[r] + (k - cum[r])] = p;
        c.ref[p] = 1;
    }
}

// Takes the pages from entry `first` of the row on out of it: an exchange takes each entry
// once, however many rows of the list name the row.
__device__ void drop_pages(const dspark_cache_t& c, int row, int first, uint32_t* status) {
    int32_t* t = c.table + (size_t)row * c.width;
    bool bad = false;
    for (int i = first + (int)(threadIdx.x & 63); i < c.width; i += 64) {
        if (t[i] < 0) continue;
        const int p = atomicExch(&t[i], -1);
        if (p < 0) continue;
        if (p >= c.n_pages) {
            bad = true;
        } else if (atomicSub(&c.ref[p], 1) <= 0) {
            atomicAdd(&c.ref[p], 1);
            bad = true;
        }
    }
    if (bad) raise_status(status, kStatusBadPage);
}

// A wave a row; more rows than kTrimBlocks hold are taken in rounds, since a grid has at most
// 2^32 threads and a table may have 2^31 rows.
constexpr int kTrimBlocks = 1 << 20;

__global__ __launch_bounds__(kT) void trim_kernel(dspark_cache_t c, const int32_t* rows, int n, const int32_t* keep,
                                                  uint32_t* status) {
    for (long long i = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); i < n; i += (long long)gridDim.x * 4) {
        const int row = rows ? rows[i] : (int)i;
        const int kp = keep ? keep[i] : 0;
        if (row < 0 || row >= c.rows) {
            if ((threadIdx.x & 63) == 0) raise_status(status, kStatusBadRow);
            continue;
        }
        drop_pages(c, row, pages_of(kp > 0 ? kp : 0, c.page_size), status);
        if ((threadIdx.x & 63) == 0) atomicMin(&c.len[row], kp < 0 ? -1 : kp);
    }
}

__global__ __launch_bounds__(kT) void commit_kernel(dspark_cache_t c, const int32_t* accept_len,
                                                    const int32_t* granted, int lead, int R, uint32_t* status) {
    const int r = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r >= R) return;
    const int ln = c.len[r];
    if (ln < 0 || (granted && granted[r] == 0)) return;
    const int acc = accept_len[r];
    const long long kp = (long long)ln + lead + acc;
    const long long first = (kp + c.page_size - 1) / c.page_size;
    if (acc < 0 || first > c.width || kp > INT32_MAX ||
        (first > 0 && c.table[(size_t)r * c.width + first - 1] < 0)) {
        if ((threadIdx.x & 63) == 0) raise_status(status, kStatusBadRow);
        return;
    }
    drop_pages(c, r, (int)first, status);
    if ((threadIdx.x & 63) == 0) c.len[r] = (int)kp;
}

// First launch of fork: slices counted as above; the other blocks check 256 forks each.
// lens keeps the parent's tokens as they were before the call (-1: the fork is refused),
// since a parent may be another fork's destination.  A destination is taken by the first
// fork that names it.
__global__ __launch_bounds__(kT) void fork_needs_kernel(dspark_cache_t c, const int32_t* src, const int32_t* dst,
                                                        int n, int deep, int ns, int32_t* cnt, int32_t* need,
                                                        int32_t* lens, uint32_t* status) {
    __shared__ int tmp[8];
    __shared__ int tile[kT];
    if ((int)blockIdx.x < ns) {
        count_slice(c, blockIdx.x, false, cnt, tmp);
        return;
    }
    const int i0 = (blockIdx.x - ns) * kT;
    const int i = i0 + threadIdx.x;
    const int a = i < n ? src[i] : -1, d = i < n ? dst[i] : -1;
    bool good = i < n && a >= 0 && a < c.rows && d >= 0 && d < c.rows && a != d;
    for (int j0 = 0; j0 <= i0; j0 += kT) {
        __syncthreads();
        tile[threadIdx.x] = j0 + (int)threadIdx.x < n ? dst[j0 + threadIdx.x] : -1;
        __syncthreads();
        const int m = min(kT, i - j0);
        for (int j = 0; j < m; ++j) good &= tile[j] != d;
    }
    int nd = 0, ln = -1;
    if (good) {
        ln = c.len[a];
        const int first = ln > 0 ? pages_of(ln, c.page_size) : 0;
        good = ln >= 0 && first <= c.width && (first == 0 || c.table[(size_t)a * c.width + first - 1] >= 0) &&
               c.len[d] <= 0 && c.table[(size_t)d * c.width] < 0;
        if (good) nd = deep ? first : (ln % c.page_size ? 1 : 0);
    }
    if (i < n) {
        need[i] = nd;
        lens[i] = good ? ln : -1;
        if (!good) raise_status(status, kStatusBadRow);
    }
}

// Blocks [0, ns) hand the free pages of their slices out and list the copies; the others
// share the whole pages, a wave a fork.  A page that is shared has a count above 0 before
// and after, so the two do not meet.
__global__ __launch_bounds__(kT) void fork_assign_kernel(dspark_cache_t c, const int32_t* src, const int32_t* dst,
                                                         int n, int deep, int ns, const int32_t* cnt,
                                                         const int32_t* need, const int32_t* lens, int32_t* forked,
                                                         int32_t* from, int32_t* to, int32_t* n_copies,
                                                         uint32_t* status) {
    extern __shared__ int cum[];  // n + 1
    __shared__ int list[kPageSlice], tmp[8];
    const int b = blockIdx.x;
    int before, all;
    slices_before(cnt, ns, b < ns ? b : 0, before, all, tmp);
    running_needs(need, n, cum, tmp);
    if (b >= ns) {
        const int f = (b - ns) * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
        if (f >= n) return;
        const bool fits = cum[f + 1] <= all;
        const int ln = lens[f];
        const bool go = ln >= 0 && fits;
        if (lane == 0) {
            forked[f] = go;
            if (ln >= 0 && !fits) raise_status(status, kStatusNoPages);
        }
        if (!go) return;
        const int whole = deep ? 0 : ln / c.page_size;
        const int32_t* s = c.table + (size_t)src[f] * c.width;
        int32_t* t = c.table + (size_t)dst[f] * c.width;
        for (int i = lane; i < whole; i += 64) {
            const int p = s[i];
            t[i] = p;
            if (p >= 0 && p < c.n_pages) atomicAdd(&c.ref[p], 1);
            else raise_status(status, kStatusBadPage);
        }
        if (lane == 0) c.len[dst[f]] = ln;
        return;
    }
    const int give = served(cum, n, all);
    if (b == 0 && threadIdx.x == 0) *n_copies = give;
    if (before >= give) return;
    const int count = list_free(c, b, list, tmp);
    for (int i = threadIdx.x; i < count && before + i < give; i += kT) {
        const int p = list[i], k = before + i, f = owner_of(cum, n, k);
        const int at = (deep ? 0 : lens[f] / c.page_size) + (k - cum[f]);
        from[k] = c.table[(size_t)src[f] * c.width + at];
        to[k] = p;
        c.table[(size_t)dst[f] * c.width + at] = p;
        c.ref[p] = 1;
    }
}

__global__ __launch_bounds__(kT) void compact_count_kernel(dspark_cache_t c, int32_t* cnt) {
    __shared__ int tmp[8];
    count_slice(c, blockIdx.x, true, cnt, tmp);
}

// Ranks: with n_live live pages, `low` of them below n_live, the live page p at or above
// n_live is move number (live pages before p) - low, and the free page p below n_live is
// the destination of move number p - (live pages before p).  page_map holds the new place,
// -1 for a free page, and -2 - k for a page that move k takes away.
__global__ __launch_bounds__(kT) void compact_rank_kernel(dspark_cache_t c, int ns, const int32_t* cnt, int32_t* from,
                                                          int32_t* to, int32_t* page_map, int32_t* n_live,
                                                          int32_t* n_moves) {
    __shared__ int tmp[8];
    const int b = blockIdx.x;
    int before, all;
    slices_before(cnt, ns, b, before, all, tmp);
    const int edge = all / kPageSlice;  // the slice that n_live lies in
    int low, unused;
    slices_before(cnt, ns, edge, low, unused, tmp);
    int first;
    uint32_t at_edge = edge < ns ? own_pages(c, edge, true, first) : 0;
    if (edge < ns) at_edge &= all <= first ? 0u : all - first >= kOwn ? 0xFFFFu : (1u << (all - first)) - 1u;
    low += block_sum(__popc(at_edge), tmp);
    if (b == 0 && threadIdx.x == 0) {
        *n_live = all;
        *n_moves = all - low;
    }
    const uint32_t mine = own_pages(c, b, true, first);
    int rank = before + block_scan(__popc(mine), tmp) - __popc(mine);  // live pages before p
    for (int i = 0; i < kOwn && first + i < c.n_pages; ++i) {
        const int p = first + i;
        const bool live = mine >> i & 1;
        int m = -1;
        if (live && p < all) {
            m = p;
        } else if (live) {
            from[rank - low] = p;
            m = -2 - (rank - low);
        } else if (p < all) {
            to[p - rank] = p;
        }
        page_map[p] = m;
        rank += live;
    }
}

__device__ __forceinline__ uint4* page_part(const dspark_cache_t& c, int kv, int layer, int p, size_t bytes) {
    return (uint4*)((char*)(kv ? c.v : c.k) + ((size_t)layer * c.n_pages + p) * bytes);
}

// Copies of whole pages, every layer's K and V: 16 KB of one page's part at a time.
__device__ void copy_pages(const dspark_cache_t& c, const int32_t* from, const int32_t* to, int n, int block,
                           int blocks, uint32_t* status) {
    const size_t bytes = (size_t)c.n_kv_heads * c.page_size * c.head_dim * 2;
    const int vecs = (int)(bytes / 16);
    const int pieces = (vecs + 4 * kT - 1) / (4 * kT);
    const long long total = (long long)n * c.layers * 2 * pieces;
    for (long long w = block; w < total; w += blocks) {
        const int piece = (int)(w % pieces);
        const long long x = w / pieces;
        const int kv = (int)(x & 1), layer = (int)((x >> 1) % c.layers), k = (int)((x >> 1) / c.layers);
        const int a = from[k], d = to[k];
        if (a < 0 || a >= c.n_pages || d < 0 || d >= c.n_pages) {
            if (threadIdx.x == 0) raise_status(status, kStatusBadPage);
            continue;
        }
        const uint4* s = page_part(c, kv, layer, a, bytes);
        uint4* t = page_part(c, kv, layer, d, bytes);
        uint4 r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = (piece * 4 + i) * kT + threadIdx.x;
            if (at < vecs) r[i] = s[at];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = (piece * 4 + i) * kT + threadIdx.x;
            if (at < vecs) t[at] = r[i];
        }
    }
}

__global__ __launch_bounds__(kT) void copy_pages_kernel(dspark_cache_t c, const int32_t* from, const int32_t* to,
                                                        const int32_t* n, uint32_t* status) {
    copy_pages(c, from, to, *n, blockIdx.x, gridDim.x, status);
}

// The moves: counts and data by blocks [tb, grid), the tables' entries by blocks [0, tb).
// page_map is read in either of its two states, -2 - k and the new place, which say the same.
__global__ __launch_bounds__(kT) void compact_move_kernel(dspark_cache_t c, int tb, const int32_t* from,
                                                          const int32_t* to, const int32_t* n_moves,
                                                          int32_t* page_map, uint32_t* status) {
    if ((int)blockIdx.x < tb) {
        const size_t n = (size_t)c.rows * c.width;
        for (size_t i = (size_t)blockIdx.x * kT + threadIdx.x; i < n; i += (size_t)tb * kT) {
            const int p = c.table[i];
            if (p < 0) continue;
            int m = -1;
            if (p < c.n_pages) {
                m = __hip_atomic_load(&page_map[p], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                if (m <= -2) m = to[-2 - m];
            }
            if (m < 0) raise_status(status, kStatusBadPage);
            if (m != p) c.table[i] = m;
        }
        return;
    }
    const int block = blockIdx.x - tb, blocks = gridDim.x - tb, n = *n_moves;
    for (int k = block * kT + threadIdx.x; k < n; k += blocks * kT) {
        const int a = from[k], d = to[k];
        c.ref[d] = c.ref[a];
        c.ref[a] = 0;
        __hip_atomic_store(&page_map[a], d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    copy_pages(c, from, to, n, block, blocks, status);
}

int copy_blocks(const dspark_cache_t& c, long long most, int cus) {
    const size_t bytes = (size_t)c.n_kv_heads * c.page_size * c.head_dim * 2;
    const long long pieces = (long long)((bytes / 16 + 4 * kT - 1) / (4 * kT)) * c.layers * 2 * most;
    const long long cap = (long long)cus * 8;
    return (int)(pieces < 1 ? 1 : pieces < cap ? pieces : cap);
}

}  // namespace

hipError_t launch_reserve(const dspark_cache_t& c, const int32_t* offsets, int lead, int R, int32_t* granted,
                          uint32_t* status, int32_t* ws, hipStream_t s) {
    const int ns = page_slices(c.n_pages);
    int32_t *cnt = ws, *need = cnt + ns, *have = need + R;
    hipLaunchKernelGGL(reserve_needs_kernel, dim3(ns + (R + 3) / 4), dim3(kT), 0, s, c, offsets, lead, R, ns, cnt,
                       need, have, status);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(reserve_assign_kernel, dim3(ns), dim3(kT), (R + 1) * sizeof(int), s, c, R, ns, cnt, need, have,
                       granted, status);
    return hipGetLastError();
}

hipError_t launch_trim(const dspark_cache_t& c, const int32_t* rows, int n, const int32_t* keep, uint32_t* status,
                       hipStream_t s) {
    const int blocks = (int)std::min(((long long)n + 3) / 4, (long long)kTrimBlocks);
    hipLaunchKernelGGL(trim_kernel, dim3(blocks), dim3(kT), 0, s, c, rows, n, keep, status);
    return hipGetLastError();
}

hipError_t launch_commit(const dspark_cache_t& c, const int32_t* accept_len, const int32_t* granted, int lead, int R,
                         uint32_t* status, hipStream_t s) {
    hipLaunchKernelGGL(commit_kernel, dim3((R + 3) / 4), dim3(kT), 0, s, c, accept_len, granted, lead, R, status);
    return hipGetLastError();
}

hipError_t launch_fork(const dspark_cache_t& c, const int32_t* src, const int32_t* dst, int n, int deep,
                       int32_t* forked, uint32_t* status, int32_t* ws, int cus, hipStream_t s) {
    const int ns = page_slices(c.n_pages);
    int32_t *cnt = ws, *need = cnt + ns, *lens = need + n, *from = lens + n, *to = from + c.n_pages,
            *n_copies = to + c.n_pages;
    hipLaunchKernelGGL(fork_needs_kernel, dim3(ns + (n + kT - 1) / kT), dim3(kT), 0, s, c, src, dst, n, deep, ns, cnt,
                       need, lens, status);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(fork_assign_kernel, dim3(ns + (n + 3) / 4), dim3(kT), (n + 1) * sizeof(int), s, c, src, dst, n,
                       deep, ns, cnt, need, lens, forked, from, to, n_copies, status);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    long long most = deep ? (long long)n * c.width : n;
    if (most > c.n_pages) most = c.n_pages;
    hipLaunchKernelGGL(copy_pages_kernel, dim3(copy_blocks(c, most, cus)), dim3(kT), 0, s, c, from, to, n_copies,
                       status);
    return hipGetLastError();
}

hipError_t launch_compact(const dspark_cache_t& c, int32_t* page_map, int32_t* n_live, uint32_t* status, int32_t* ws,
                          int cus, hipStream_t s) {
    const int ns = page_slices(c.n_pages);
    int32_t *cnt = ws, *from = cnt + ns, *to = from + c.n_pages, *n_moves = to + c.n_pages;
    hipLaunchKernelGGL(compact_count_kernel, dim3(ns), dim3(kT), 0, s, c, cnt);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(compact_rank_kernel, dim3(ns), dim3(kT), 0, s, c, ns, cnt, from, to, page_map, n_live, n_moves);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const long long entries = (long long)c.rows * c.width;
    const int tb = (int)(entries < (long long)kT * cus ? (entries + kT - 1) / kT : cus);
    hipLaunchKernelGGL(compact_move_kernel, dim3(tb + copy_blocks(c, c.n_pages / 2, cus)), dim3(kT), 0, s, c, tb, from,
                       to, n_moves, page_map, status);
    return hipGetLastError();
}

}  // namespace dspark
