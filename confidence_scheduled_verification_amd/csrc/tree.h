// Internal launchers of drafted trees and of the target's choice (tree.hip, rotary.hip,
// target.hip).  Argument checks happen in cache_api.hip and target_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "cache.h"
#include "dspark.h"

namespace dspark {

constexpr uint32_t kStatusNoToken = 256u;
constexpr int kTreeNodes = DSPARK_TREE_MAX_NODES;

hipError_t launch_tree_merge(const int32_t* tokens, const int32_t* prefix_len, int R, int S, int K, int32_t* counts,
                             int32_t* offsets, int32_t* ver_tokens, int32_t* parent, uint32_t* status, hipStream_t s);
hipError_t launch_tree_plan(const int32_t* parent, int n_rows, const int32_t* offsets, int lead, int R, int max_new,
                            int32_t* depth, uint64_t* anc, uint32_t* status, hipStream_t s);
hipError_t launch_accept_tree(const int32_t* ver_tokens, int n_nodes, const int32_t* offsets, const int32_t* parent,
                              const int32_t* target, int R, int K, int32_t* accept_len, int32_t* path,
                              int32_t* next_prev0, int32_t* out_tokens, uint32_t* status, hipStream_t s);
hipError_t launch_keep_path(const dspark_cache_t& c, const int32_t* path, int K, const int32_t* accept_len,
                            const int32_t* granted, int lead, int R, uint32_t* status, hipStream_t s);

// The append of rotated rows: AppendArgs for K and V, and the queries beside them.
struct RotaryArgs {
    AppendArgs a;
    const uint16_t* q;
    uint16_t* q_out;
    int64_t q_stride, q_out_stride;
    const uint64_t* turns;
    const int32_t* depth;
    int H, dim, first, interleaved, dtype;
    float attention;
};
hipError_t launch_append_rotary(const RotaryArgs& a, hipStream_t s);

hipError_t launch_history_clear(const dspark_history_t& h, const int32_t* rows, int n, uint32_t* status, hipStream_t s);
hipError_t launch_history_add(const dspark_history_t& h, const int32_t* tokens, int n, int width, const int32_t* rows,
                              int answered, uint32_t* status, hipStream_t s);

// The order key of a part's best value and that token (key 0: none).
struct TargetBest {
    uint64_t key;
    uint32_t v, pad;
};
struct TargetArgs {
    dspark_target_t t;
    const uint32_t* seen;  // NULL: no history
    const int32_t* count;
    size_t words;      // of a history row's bits
    int chunk, parts;  // tokens of a part of a row (a multiple of 256), and parts of a row
    // where a row has several parts: the parts of each row that have come, 0 between the calls (NULL: a launch
    // of its own joins them), and what each of them has, [n_rows, parts]
    uint32_t* came;
    TargetBest* best;
    uint32_t* status;
};
constexpr int kTargetThreads = 512;  // of a workgroup
// How as many rows of V tokens are taken apart.
void target_split(int rows, int V, int& chunk, int& parts);
void target_ws_layout(TargetArgs& a, void* ws);
size_t target_ws_bytes(long long n_rows, int parts);
int target_most_parts(int V);  // of up to V tokens, however many rows there are
hipError_t launch_target(const TargetArgs& a, hipStream_t s);

}  // namespace dspark
