// C entry points of the paged cache: argument checks and launches.  Semantics of every
// entry point are documented in include/dspark.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "cache.h"
#include "dspark.h"
#include "tree.h"

using dspark::fail;
using dspark::hip_fail;

namespace {

// The pages' bookkeeping, which every call needs.
int check_pages(const dspark_cache_t* c, const char* who) {
    if (!c) return fail(DSPARK_EINVAL, "%s: NULL cache", who);
    if (c->n_pages < 1 || c->n_pages > DSPARK_CACHE_MAX_PAGES)
        return fail(DSPARK_EUNSUPPORTED, "%s: %d pages, 1 to %d are supported", who, c->n_pages, DSPARK_CACHE_MAX_PAGES);
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
        return fail(DSPARK_EUNSUPPORTED, "%s: page_size %d, a power of two from 16 to 256 is supported", who,
                    c->page_size);
    if (c->rows < 0 || c->width < 1 || (long long)c->rows * c->width > INT32_MAX)
        return fail(DSPARK_EUNSUPPORTED, "%s: a table of %d rows and %d entries", who, c->rows, c->width);
    if ((c->rows > 0 && (!c->table || !c->len)) || !c->ref) return fail(DSPARK_EINVAL, "%s: table, len or ref is NULL", who);
    return DSPARK_OK;
}

// The pages' contents, for the calls that read or write them.
int check_data(const dspark_cache_t* c, const char* who) {
    const int rc = check_pages(c, who);
    if (rc != DSPARK_OK) return rc;
    if (!c->k || !c->v) return fail(DSPARK_EINVAL, "%s: the cache has no k or no v", who);
    if (((uintptr_t)c->k | (uintptr_t)c->v) & 15u) return fail(DSPARK_EINVAL, "%s: k and v must be 16-byte aligned", who);
    if (c->layers < 1) return fail(DSPARK_EINVAL, "%s: %d layers", who, c->layers);
    if (c->dtype != DSPARK_BF16 && c->dtype != DSPARK_F16)
        return fail(DSPARK_EUNSUPPORTED, "%s: dtype %d, bf16 and fp16 are supported", who, c->dtype);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(DSPARK_EUNSUPPORTED, "%s: head_dim %d, 64, 128 and 256 are supported", who, c->head_dim);
    if (c->n_kv_heads < 1 || c->n_kv_heads > 1024)
        return fail(DSPARK_EUNSUPPORTED, "%s: %d key heads, 1 to 1024 are supported", who, c->n_kv_heads);
    return DSPARK_OK;
}

int check_requests(const dspark_cache_t* c, int R, int lead, const char* who) {
    if (R < 0 || R > c->rows) return fail(DSPARK_ERANGE, "%s: R %d outside [0, %d], the table's rows", who, R, c->rows);
    if (R > DSPARK_CACHE_MAX_REQUESTS)
        return fail(DSPARK_EUNSUPPORTED, "%s: %d requests exceed %d", who, R, DSPARK_CACHE_MAX_REQUESTS);
    if (lead != 0 && lead != 1) return fail(DSPARK_ERANGE, "%s: lead %d, 0 or 1 is meant", who, lead);
    return DSPARK_OK;
}

int check_ws(const void* ws, size_t have, size_t need, const char* who) {
    if (!ws || have < need)
        return fail(DSPARK_EWORKSPACE, "%s: workspace of %zu bytes needed, %zu given%s", who, need, have,
                    ws ? "" : " (NULL)");
    if ((uintptr_t)ws & 15u) return fail(DSPARK_EINVAL, "%s: workspace must be 16-byte aligned", who);
    return DSPARK_OK;
}

// Rows of a packed tensor: 16-byte loads from each row's heads.
int check_rows(const void* p, int64_t stride, int heads, int D, const char* who, const char* what) {
    if (!p) return fail(DSPARK_EINVAL, "%s: %s is NULL", who, what);
    if ((uintptr_t)p & 15u) return fail(DSPARK_EINVAL, "%s: %s must be 16-byte aligned", who, what);
    if (stride < (int64_t)heads * D || stride % 8 || stride > INT32_MAX)
        return fail(DSPARK_EINVAL, "%s: rows of %s lie %lld elements apart, a multiple of 8 from %d on is needed", who,
                    what, (long long)stride, heads * D);
    return DSPARK_OK;
}

int done(hipError_t e, const char* who) { return e == hipSuccess ? DSPARK_OK : hip_fail(e, who); }

size_t layer_elems(const dspark_cache_t* c) {
    return (size_t)c->n_pages * c->n_kv_heads * c->page_size * c->head_dim;
}

// The rows of an append, checked; any: there are some.
int append_args(const dspark_cache_t* c, int layer, const void* k_new, int64_t k_stride, const void* v_new,
                int64_t v_stride, int n_rows, const int32_t* offsets, int lead, int R, int max_new, uint32_t* status,
                const char* who, dspark::AppendArgs& a, bool& any) {
    int rc = check_data(c, who);
    if (rc != DSPARK_OK || (rc = check_requests(c, R, lead, who)) != DSPARK_OK) return rc;
    if (layer < 0 || layer >= c->layers) return fail(DSPARK_ERANGE, "%s: layer %d outside [0, %d)", who, layer, c->layers);
    if (n_rows < 0 || max_new < 0) return fail(DSPARK_ERANGE, "%s: n_rows %d, max_new %d", who, n_rows, max_new);
    if (R == 0 || n_rows == 0 || max_new == 0) return DSPARK_OK;
    if ((rc = check_rows(k_new, k_stride, c->n_kv_heads, c->head_dim, who, "k_new")) != DSPARK_OK ||
        (rc = check_rows(v_new, v_stride, c->n_kv_heads, c->head_dim, who, "v_new")) != DSPARK_OK)
        return rc;
    if (!offsets) return fail(DSPARK_EINVAL, "%s: offsets is NULL", who);
    const size_t at = layer * layer_elems(c);
    a = dspark::AppendArgs{(const uint16_t*)k_new, (const uint16_t*)v_new, k_stride, v_stride, (uint16_t*)c->k + at,
                           (uint16_t*)c->v + at, c->table, c->len, c->ref, offsets, lead, R, n_rows, max_new,
                           c->n_kv_heads, c->head_dim, c->page_size, __builtin_ctz(c->page_size), c->n_pages, c->width,
                           status};
    any = true;
    return DSPARK_OK;
}

// Whether n rows of `used` elements at x and of `out_used` at out touch.  Rows as far apart from one another may
// lie between each other, as parts of the same wider rows do.
bool touch(int n, const void* x, int64_t stride, int64_t used, const void* out, int64_t out_stride, int64_t out_used) {
    const uintptr_t x0 = (uintptr_t)x, y0 = (uintptr_t)out, x1 = x0 + ((uintptr_t)(n - 1) * stride + used) * 2,
                    y1 = y0 + ((uintptr_t)(n - 1) * out_stride + out_used) * 2;
    if (x0 >= y1 || y0 >= x1) return false;
    if (stride != out_stride) return true;
    const int64_t row = stride * 2, apart = (((int64_t)(y0 - x0)) % row + row) % row;
    return apart < used * 2 || row - apart < out_used * 2;
}

int attend(const dspark_cache_t* c, int layer, const void* q, int64_t q_stride, int n_rows, int H,
           const int32_t* offsets, int lead, int R, int max_new, const uint64_t* anc, float scale, int n_groups,
           const int32_t* group_off, const int32_t* shared_table, int shared_width, const int32_t* shared_pages,
           void* out, int64_t out_stride, float* lse, uint32_t* status, void* ws, size_t ws_bytes, void* stream,
           const char* who) {
    int rc = check_data(c, who);
    if (rc != DSPARK_OK || (rc = check_requests(c, R, lead, who)) != DSPARK_OK) return rc;
    if (layer < 0 || layer >= c->layers) return fail(DSPARK_ERANGE, "%s: layer %d outside [0, %d)", who, layer, c->layers);
    if (n_rows < 0 || max_new < 0) return fail(DSPARK_ERANGE, "%s: n_rows %d, max_new %d", who, n_rows, max_new);
    if (H < 1 || H % c->n_kv_heads || H > 65535)
        return fail(DSPARK_EINVAL, "%s: %d query heads over %d key heads", who, H, c->n_kv_heads);
    if (!(scale > 0.f) || !isfinite(scale * 1.44269504f))
        return fail(DSPARK_ERANGE, "%s: scale %g must be positive and finite", who, (double)scale);
    if (n_groups < 0 || n_groups > DSPARK_CACHE_MAX_GROUPS)
        return fail(DSPARK_EUNSUPPORTED, "%s: %d groups, at most %d are supported", who, n_groups, DSPARK_CACHE_MAX_GROUPS);
    if (n_groups > 0 && (!group_off || !shared_table || !shared_pages || shared_width < 1))
        return fail(DSPARK_EINVAL, "%s: groups need group_off, shared_table and shared_pages", who);
    if (R == 0 || n_rows == 0 || max_new == 0) return DSPARK_OK;
    if ((rc = check_rows(q, q_stride, H, c->head_dim, who, "q")) != DSPARK_OK ||
        (rc = check_rows(out, out_stride, H, c->head_dim, who, "out")) != DSPARK_OK)
        return rc;
    if (!offsets) return fail(DSPARK_EINVAL, "%s: offsets is NULL", who);
    const long long tokens = (long long)c->width * c->page_size, shared_tokens = (long long)shared_width * c->page_size;
    dspark::AttendArgs a{};
    a.lead = lead;
    a.R = R;
    a.rows = (int)std::min<long long>(n_rows, (long long)R * max_new);  // rows past those belong to no request
    a.max_new = std::min(max_new, n_rows);                              // (more would not lie in the tensors)
    a.H = H;
    a.Hkv = c->n_kv_heads;
    a.G = H / c->n_kv_heads;
    a.D = c->head_dim;
    a.n_groups = n_groups;
    dspark::attend_forms(a, dspark::num_cu());
    // The work is numbered with 32 bits: columns, the units of the requests' own keys and those of
    // the groups', as many as these sizes allow, and the joining launch's grid.
    const auto tiles = [&](int set, long long columns) { return (columns + a.tile[set] - 1) / a.tile[set]; };
    const auto units = [&](int set, long long keys) { return (long long)a.Hkv * (keys / a.unit[set] + 1); };
    const bool fits = (long long)a.rows * H <= INT32_MAX - 1023 && tokens <= dspark::kAttendMaxTokens &&
                      std::min(R * tiles(0, (long long)a.max_new * a.G), R + tiles(0, (long long)a.rows * a.G)) *
                              units(0, tokens) <= INT32_MAX;
    const bool groups_fit =
        !n_groups || (shared_tokens <= dspark::kAttendMaxTokens &&
                      (n_groups + tiles(1, (long long)a.rows * a.G)) * units(1, shared_tokens) <= INT32_MAX &&
                      (long long)a.max_new * a.G * (a.D / 8) <= 65535ll * dspark::kAttendJoinItems);
    if (!fits || !groups_fit)
        return fail(DSPARK_EUNSUPPORTED, "%s: %d rows of %d heads over up to %lld tokens are too many for one call", who,
                    n_rows, H, tokens);
    if ((rc = check_ws(ws, ws_bytes, dspark::attend_ws_bytes(R, H, a.D, a.rows, n_groups), who)) != DSPARK_OK) return rc;
    const size_t at = layer * layer_elems(c);
    a.q = (const uint16_t*)q;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.k = (const uint16_t*)c->k + at;
    a.v = (const uint16_t*)c->v + at;
    a.table = c->table;
    a.len = c->len;
    a.offsets = offsets;
    a.anc = anc;
    a.dtype = c->dtype;
    a.page = c->page_size;
    a.page_shift = __builtin_ctz(c->page_size);
    a.n_pages = c->n_pages;
    a.width = c->width;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    a.shared_width = shared_width;
    a.group_off = group_off;
    a.shared_table = shared_table;
    a.shared_pages = shared_pages;
    a.out = (uint16_t*)out;
    a.lse = lse;
    a.status = status;
    dspark::attend_ws_layout(a, ws);
    return done(dspark::launch_attend(a, (hipStream_t)stream), who);
}

}  // namespace

extern "C" {

size_t dspark_pages_workspace_bytes(int n_pages, int n) {
    if (n_pages < 1 || n < 0) return 0;
    return dspark::pages_ws_words(n_pages, n) * sizeof(int32_t);
}

int dspark_pages_reserve(const dspark_cache_t* c, const int32_t* offsets, int lead, int R, int32_t* granted,
                         uint32_t* status, void* ws, size_t ws_bytes, void* stream) {
    const char* who = "pages_reserve";
    int rc = check_pages(c, who);
    if (rc != DSPARK_OK || (rc = check_requests(c, R, lead, who)) != DSPARK_OK) return rc;
    if (R == 0) return DSPARK_OK;
    if (!offsets || !granted) return fail(DSPARK_EINVAL, "%s: a required pointer is NULL", who);
    if ((rc = check_ws(ws, ws_bytes, dspark_pages_workspace_bytes(c->n_pages, R), who)) != DSPARK_OK) return rc;
    return done(dspark::launch_reserve(*c, offsets, lead, R, granted, status, (int32_t*)ws, (hipStream_t)stream), who);
}

int dspark_pages_trim(const dspark_cache_t* c, const int32_t* rows, int n, const int32_t* keep, uint32_t* status,
                      void* stream) {
    const char* who = "pages_trim";
    const int rc = check_pages(c, who);
    if (rc != DSPARK_OK) return rc;
    if (n < 0 || (!rows && n > c->rows))
        return fail(DSPARK_ERANGE, "%s: %d rows, the table has %d", who, n, c->rows);
    if (n == 0) return DSPARK_OK;
    return done(dspark::launch_trim(*c, rows, n, keep, status, (hipStream_t)stream), who);
}

int dspark_pages_commit_granted(const dspark_cache_t* c, const int32_t* accept_len, const int32_t* granted, int lead,
                                int R, uint32_t* status, void* stream) {
    const char* who = "pages_commit";
    int rc = check_pages(c, who);
    if (rc != DSPARK_OK || (rc = check_requests(c, R, lead, who)) != DSPARK_OK) return rc;
    if (R == 0) return DSPARK_OK;
    if (!accept_len) return fail(DSPARK_EINVAL, "%s: accept_len is NULL", who);
    return done(dspark::launch_commit(*c, accept_len, granted, lead, R, status, (hipStream_t)stream), who);
}

int dspark_pages_commit(const dspark_cache_t* c, const int32_t* accept_len, int lead, int R, uint32_t* status,
                        void* stream) {
    return dspark_pages_commit_granted(c, accept_len, nullptr, lead, R, status, stream);
}

int dspark_pages_fork(const dspark_cache_t* c, const int32_t* src, const int32_t* dst, int n, int deep,
                      int32_t* forked, uint32_t* status, void* ws, size_t ws_bytes, void* stream) {
    const char* who = "pages_fork";
    int rc = check_data(c, who);
    if (rc != DSPARK_OK) return rc;
    if (n < 0) return fail(DSPARK_ERANGE, "%s: %d forks", who, n);
    if (n > DSPARK_CACHE_MAX_REQUESTS)
        return fail(DSPARK_EUNSUPPORTED, "%s: %d forks exceed %d", who, n, DSPARK_CACHE_MAX_REQUESTS);
    if ((long long)n * c->width > INT32_MAX) return fail(DSPARK_EUNSUPPORTED, "%s: %d forks of %d pages", who, n, c->width);
    if (n == 0) return DSPARK_OK;
    if (!src || !dst || !forked) return fail(DSPARK_EINVAL, "%s: a required pointer is NULL", who);
    if ((rc = check_ws(ws, ws_bytes, dspark_pages_workspace_bytes(c->n_pages, n), who)) != DSPARK_OK) return rc;
    return done(dspark::launch_fork(*c, src, dst, n, deep != 0, forked, status, (int32_t*)ws, dspark::num_cu(),
                                    (hipStream_t)stream), who);
}

int dspark_pages_compact(const dspark_cache_t* c, int32_t* page_map, int32_t* n_live, uint32_t* status, void* ws,
                         size_t ws_bytes, void* stream) {
    const char* who = "pages_compact";
    int rc = check_data(c, who);
    if (rc != DSPARK_OK) return rc;
    if (!page_map || !n_live) return fail(DSPARK_EINVAL, "%s: a required pointer is NULL", who);
    if ((rc = check_ws(ws, ws_bytes, dspark_pages_workspace_bytes(c->n_pages, 0), who)) != DSPARK_OK) return rc;
    return done(dspark::launch_compact(*c, page_map, n_live, status, (int32_t*)ws, dspark::num_cu(),
                                       (hipStream_t)stream), who);
}

int dspark_cache_append(const dspark_cache_t* c, int layer, const void* k_new, int64_t k_stride, const void* v_new,
                        int64_t v_stride, int n_rows, const int32_t* offsets, int lead, int R, int max_new,
                        uint32_t* status, void* stream) {
    const char* who = "cache_append";
    dspark::AppendArgs a;
    bool any = false;
    const int rc = append_args(c, layer, k_new, k_stride, v_new, v_stride, n_rows, offsets, lead, R, max_new, status, who, a, any);
    if (rc != DSPARK_OK || !any) return rc;
    return done(dspark::launch_append(a, (hipStream_t)stream), who);
}

size_t dspark_cache_attend_workspace_bytes(int R, int H, int head_dim, int max_new, int n_groups) {
    if (R < 1 || H < 1 || max_new < 1 || n_groups < 0) return 0;
    return dspark::attend_ws_bytes(R, H, head_dim, (int)std::min<long long>((long long)R * max_new, INT32_MAX), n_groups);
}

int dspark_cache_attend(const dspark_cache_t* c, int layer, const void* q, int64_t q_stride, int n_rows, int H,
                        const int32_t* offsets, int lead, int R, int max_new, float scale, int n_groups,
                        const int32_t* group_off, const int32_t* shared_table, int shared_width,
                        const int32_t* shared_pages, void* out, int64_t out_stride, float* lse, uint32_t* status,
                        void* ws, size_t ws_bytes, void* stream) {
    return attend(c, layer, q, q_stride, n_rows, H, offsets, lead, R, max_new, nullptr, scale, n_groups, group_off,
                  shared_table, shared_width, shared_pages, out, out_stride, lse, status, ws, ws_bytes, stream,
                  "cache_attend");
}

int dspark_cache_attend_tree(const dspark_cache_t* c, int layer, const void* q, int64_t q_stride, int n_rows, int H,
                             const int32_t* offsets, int lead, int R, int max_new, const uint64_t* anc, float scale,
                             int n_groups, const int32_t* group_off, const int32_t* shared_table, int shared_width,
                             const int32_t* shared_pages, void* out, int64_t out_stride, float* lse, uint32_t* status,
                             void* ws, size_t ws_bytes, void* stream) {
    const char* who = "cache_attend_tree";
    if (max_new > dspark::kTreeNodes)
        return fail(DSPARK_EUNSUPPORTED, "%s: trees of %d nodes exceed %d", who, max_new, dspark::kTreeNodes);
    if (!anc && R > 0 && n_rows > 0 && max_new > 0) return fail(DSPARK_EINVAL, "%s: anc is NULL", who);
    return attend(c, layer, q, q_stride, n_rows, H, offsets, lead, R, max_new, anc, scale, n_groups, group_off,
                  shared_table, shared_width, shared_pages, out, out_stride, lse, status, ws, ws_bytes, stream, who);
}

// One layer's K, V and Q of a step's rows turned to their positions.
int dspark_cache_append_rotary(const dspark_cache_t* c, int layer, const dspark_rotary_t* rotary, const void* q,
                               int64_t q_stride, int H, void* q_out, int64_t q_out_stride, const void* k_new,
                               int64_t k_stride, const void* v_new, int64_t v_stride, int n_rows,
                               const int32_t* offsets, int lead, int R, int max_new, const int32_t* depth,
                               uint32_t* status, void* stream) {
    const char* who = "cache_append_rotary";
    dspark::RotaryArgs g{};
    bool any = false;
    int rc = append_args(c, layer, k_new, k_stride, v_new, v_stride, n_rows, offsets, lead, R, max_new, status, who, g.a, any);
    if (rc != DSPARK_OK) return rc;
    if (!rotary) return fail(DSPARK_EINVAL, "%s: rotary is NULL", who);
    if (rotary->dim < 16 || rotary->dim % 16 || rotary->first < 0 || rotary->first % 8 ||
        rotary->first > c->head_dim - rotary->dim)
        return fail(DSPARK_EINVAL, "%s: %d dims from %d on, of %d, cannot be turned", who, rotary->dim, rotary->first, c->head_dim);
    if (!isfinite(rotary->attention))
        return fail(DSPARK_ERANGE, "%s: attention %g must be finite", who, (double)rotary->attention);
    if (H < 1 || H > 65535) return fail(DSPARK_EINVAL, "%s: %d query heads", who, H);
    if (!any) return DSPARK_OK;
    if (!rotary->turns) return fail(DSPARK_EINVAL, "%s: turns is NULL", who);
    if ((rc = check_rows(q, q_stride, H, c->head_dim, who, "q")) != DSPARK_OK ||
        (rc = check_rows(q_out, q_out_stride, H, c->head_dim, who, "q_out")) != DSPARK_OK)
        return rc;
    const int64_t wide = (int64_t)H * c->head_dim, narrow = (int64_t)c->n_kv_heads * c->head_dim;
    if (q == q_out ? q_stride != q_out_stride && n_rows > 1 : touch(n_rows, q, q_stride, wide, q_out, q_out_stride, wide))
        return fail(DSPARK_EINVAL, "%s: q and q_out overlap", who);
    if (touch(n_rows, k_new, k_stride, narrow, q_out, q_out_stride, wide) ||
        touch(n_rows, v_new, v_stride, narrow, q_out, q_out_stride, wide))
        return fail(DSPARK_EINVAL, "%s: q_out and k_new or v_new overlap", who);
    g.q = (const uint16_t*)q;
    g.q_out = (uint16_t*)q_out;
    g.q_stride = q_stride;
    g.q_out_stride = q_out_stride;
    g.turns = rotary->turns;
    g.depth = depth;
    g.H = H;
    g.dim = rotary->dim;
    g.first = rotary->first;
    g.interleaved = rotary->interleaved != 0;
    g.dtype = c->dtype;
    g.attention = rotary->attention;
    return done(dspark::launch_append_rotary(g, (hipStream_t)stream), who);
}

int dspark_cache_keep_path(const dspark_cache_t* c, const int32_t* path, int K, const int32_t* accept_len,
                           const int32_t* granted, int lead, int R, uint32_t* status, void* stream) {
    const char* who = "cache_keep_path";
    int rc = check_data(c, who);
    if (rc != DSPARK_OK || (rc = check_requests(c, R, lead, who)) != DSPARK_OK) return rc;
    if (K < 0 || K >= dspark::kTreeNodes) return fail(DSPARK_ERANGE, "%s: K %d outside [0, %d)", who, K, dspark::kTreeNodes);
    if (c->layers > 65535) return fail(DSPARK_EUNSUPPORTED, "%s: %d layers", who, c->layers);
    if (R == 0) return DSPARK_OK;
    if (!accept_len || (K > 0 && !path)) return fail(DSPARK_EINVAL, "%s: a required pointer is NULL", who);
    return done(dspark::launch_keep_path(*c, path, K, accept_len, granted, lead, R, status, (hipStream_t)stream), who);
}

}  // extern "C"
