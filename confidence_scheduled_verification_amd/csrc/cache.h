// Internal launchers of the paged cache (pages.hip, append.hip, attend.hip) and the
// host helpers that the C entry points share.  Argument checks happen in cache_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dspark.h"

namespace dspark {

// Error text of this thread and the current device's compute units (api.hip).
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char* where);
int num_cu();

constexpr uint32_t kStatusBadPage = 32u;
constexpr uint32_t kStatusBadRow = 64u;
constexpr uint32_t kStatusNoPages = 128u;

constexpr int kBlockTokens = 16;    // tokens of one block of a page
constexpr int kPageSlice = 4096;    // reference counts that one workgroup counts

inline int page_slices(int n_pages) { return (n_pages + kPageSlice - 1) / kPageSlice; }

// Workspace of reserve, fork and compact, in 32-bit words: each slice's count, then two
// words per request or fork, then two per page (the copies' sources and destinations).
inline size_t pages_ws_words(int n_pages, int n) {
    return (size_t)page_slices(n_pages) + 2 * (size_t)n + 2 * (size_t)n_pages + 8;
}

hipError_t launch_reserve(const dspark_cache_t& c, const int32_t* offsets, int lead, int R, int32_t* granted,
                          uint32_t* status, int32_t* ws, hipStream_t s);
hipError_t launch_trim(const dspark_cache_t& c, const int32_t* rows, int n, const int32_t* keep, uint32_t* status,
                       hipStream_t s);
// granted: NULL where every request of the step was served
hipError_t launch_commit(const dspark_cache_t& c, const int32_t* accept_len, const int32_t* granted, int lead, int R,
                         uint32_t* status, hipStream_t s);
hipError_t launch_fork(const dspark_cache_t& c, const int32_t* src, const int32_t* dst, int n, int deep,
                       int32_t* forked, uint32_t* status, int32_t* ws, int num_cu, hipStream_t s);
hipError_t launch_compact(const dspark_cache_t& c, int32_t* page_map, int32_t* n_live, uint32_t* status, int32_t* ws,
                          int num_cu, hipStream_t s);

struct AppendArgs {
    const uint16_t* k_new;
    const uint16_t* v_new;
    int64_t k_stride, v_stride;  // elements between rows
    uint16_t* k;                 // the layer's pages
    uint16_t* v;
    const int32_t* table;
    const int32_t* len;
    const int32_t* ref;
    const int32_t* offsets;
    int lead, R, rows, max_new, Hkv, D, page, page_shift, n_pages, width;
    uint32_t* status;
};
hipError_t launch_append(const AppendArgs& a, hipStream_t s);

// Attention: a launch's workers share its units of keys evenly, so a segment (the rows of
// one request or group, a tile of them, with one key head) is split over consecutive
// workers where it has to be.  A worker leaves a split segment's part in one of its two
// slots: slot 0 for the segment that an earlier worker began, slot 1 for the one that it
// begins and does not end.
constexpr int kAttendMaxCus = 256;  // compute units that a launch uses
constexpr int kAttendJoinItems = 1024;  // eight dims of a column each: what a joining workgroup takes
// Tokens of one table row, at most: positions are 32-bit numbers, and the kernels look up to 64
// stages of 64 keys and a unit past the last one before they compare.
constexpr long long kAttendMaxTokens = (1ll << 31) - 8192;

// A worker's first segment, where an earlier worker began it (units = 0: it did not): the
// workers that have parts of it, and its columns.
struct AttendEnd {
    uint32_t units;
    int first, last, f0, nf, h;
};

struct AttendArgs {
    const uint16_t* q;
    int64_t q_stride, out_stride;  // elements between rows
    const uint16_t* k;             // the layer's pages
    const uint16_t* v;
    const int32_t* table;
    const int32_t* len;
    const int32_t* offsets;
    int lead, R, rows, max_new, H, Hkv, G, D, dtype, page, page_shift, n_pages, width;
    float scale_log2;  // the scores' scale times log2(e)
    int n_groups, shared_width;
    const int32_t* group_off;
    const int32_t* shared_table;
    const int32_t* shared_pages;
    uint16_t* out;
    float* lse;
    uint32_t* status;
    // the launches' forms (attend_forms): [0] the requests' own keys, [1] the shared ones;
    // tile: columns (row, head of the group) taken together, unit: keys dealt to workers at a time
    int tile[2], unit[2], tile_shift[2], unit_shift[2], workers[2];
    int least[2];       // units that are worth a worker; 0: all units over `parts`
    uint32_t parts[2];  // of the key heads of all requests (groups), a few each
    float* slots[2];   // parts of split segments: of the requests' own keys, of the shared ones
    float* dense[2];   // with shared prefixes: the parts of whole segments, [Hkv][rows G][D], then maxima and sums
    AttendEnd* ends;   // [workers[0]]
    uint32_t* cum[2];  // with shared prefixes: running units (of one key head) of the requests, of the groups
};
void attend_forms(AttendArgs& a, int num_cu);  // from the sizes and the device
size_t attend_ws_bytes(int R, int H, int D, int rows, int n_groups);
void attend_ws_layout(AttendArgs& a, void* ws);
hipError_t launch_attend(const AttendArgs& a, hipStream_t s);

}  // namespace dspark
