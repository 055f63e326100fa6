// C entry points of drafted trees, rotary frequencies and target tokens: argument checks and
// launches.  Semantics of every entry point are documented in include/dspark.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "cache.h"
#include "dspark.h"
#include "tree.h"

using dspark::fail;
using dspark::hip_fail;
using dspark::kTreeNodes;

namespace {

constexpr int kMostTokens = 1 << 30;  // of a vocabulary
constexpr long long kMostThreads = (1ll << 32) - 1;  // of a launch along its requests
constexpr int kMostHistoryRows = (int)(kMostThreads / 1024);

int done(hipError_t e, const char* who) { return e == hipSuccess ? DSPARK_OK : hip_fail(e, who); }

int check_step(int R, int lead, int n_rows, int max_new, int most, const char* who) {
    if (R < 0 || n_rows < 0 || max_new < 0)
        return fail(DSPARK_ERANGE, "%s: R %d, n_rows %d, max_new %d", who, R, n_rows, max_new);
    if (lead != 0 && lead != 1) return fail(DSPARK_ERANGE, "%s: lead %d, 0 or 1 is meant", who, lead);
    if (R > DSPARK_CACHE_MAX_REQUESTS)
        return fail(DSPARK_EUNSUPPORTED, "%s: %d requests exceed %d", who, R, DSPARK_CACHE_MAX_REQUESTS);
    if (max_new > most) return fail(DSPARK_EUNSUPPORTED, "%s: %d rows of a request exceed %d", who, max_new, most);
    return DSPARK_OK;
}

int check_history(const dspark_history_t* h, const char* who) {
    if (!h) return fail(DSPARK_EINVAL, "%s: NULL history", who);
    if (h->rows < 0 || h->V < 1) return fail(DSPARK_ERANGE, "%s: a history of %d rows of %d tokens", who, h->rows, h->V);
    if (h->V > kMostTokens) return fail(DSPARK_EUNSUPPORTED, "%s: %d tokens exceed %d", who, h->V, kMostTokens);
    if (h->rows > 0 && (!h->seen || !h->count)) return fail(DSPARK_EINVAL, "%s: seen or count is NULL", who);
    if (((uintptr_t)h->seen | (uintptr_t)h->count) & 15u)
        return fail(DSPARK_EINVAL, "%s: seen and count must be 16-byte aligned", who);
    return DSPARK_OK;
}

}  // namespace

extern "C" {

int dspark_tree_merge(const int32_t* tokens, const int32_t* prefix_len, int R, int S, int K, int32_t* counts,
                      int32_t* offsets, int32_t* ver_tokens, int32_t* parent, uint32_t* status, void* stream) {
    const char* who = "tree_merge";
    if (R < 0 || S < 1 || K < 1) return fail(DSPARK_ERANGE, "%s: R %d, S %d, K %d", who, R, S, K);
    if ((long long)S * K >= kTreeNodes)
        return fail(DSPARK_EUNSUPPORTED, "%s: %d chains of %d tokens, together fewer than %d are supported", who, S, K,
                    kTreeNodes);
    if (R > DSPARK_CACHE_MAX_REQUESTS)
        return fail(DSPARK_EUNSUPPORTED, "%s: %d requests exceed %d", who, R, DSPARK_CACHE_MAX_REQUESTS);
    if (R == 0) return DSPARK_OK;
    if (!tokens || !counts || !offsets || !ver_tokens || !parent)
        return fail(DSPARK_EINVAL, "%s: a required pointer is NULL", who);
    return done(dspark::launch_tree_merge(tokens, prefix_len, R, S, K, counts, offsets, ver_tokens, parent, status,
                                          (hipStream_t)stream), who);
}

int dspark_tree_plan(const int32_t* parent, int n_rows, const int32_t* offsets, int lead, int R, int max_new,
                     int32_t* depth, uint64_t* anc, uint32_t* status, void* stream) {
    const char* who = "tree_plan";
    const int rc = check_step(R, lead, n_rows, max_new, kTreeNodes, who);
    if (rc != DSPARK_OK) return rc;
    if (R == 0 || n_rows == 0 || max_new == 0) return DSPARK_OK;
    if (!parent || !offsets || !depth || !anc) return fail(DSPARK_EINVAL, "%s: a required pointer is NULL", who);
    return done(dspark::launch_tree_plan(parent, n_rows, offsets, lead, R, max_new, depth, anc, status,
                                         (hipStream_t)stream), who);
}

int dspark_accept_tree(const int32_t* ver_tokens, int n_nodes, const int32_t* offsets, const int32_t* parent,
                       const int32_t* target, int R, int K, int32_t* accept_len, int32_t* path, int32_t* next_prev0,
                       int32_t* out_tokens, uint32_t* status, void* stream) {
    const char* who = "accept_tree";
    if (R < 0 || n_nodes < 0 || K < 0 || K >= kTreeNodes)
        return fail(DSPARK_ERANGE, "%s: R %d, n_nodes %d, K %d (below %d)", who, R, n_nodes, K, kTreeNodes);
    if ((long long)n_nodes + R > INT32_MAX) return fail(DSPARK_EUNSUPPORTED, "%s: %d nodes of %d requests", who, n_nodes, R);
    if (R == 0) return DSPARK_OK;
    if ((n_nodes > 0 && !ver_tokens) || !offsets || !parent || !target || !accept_len || (K > 0 && !path) || !next_prev0)
        return fail(DSPARK_EINVAL, "%s: a required pointer is NULL", who);
    return done(dspark::launch_accept_tree(ver_tokens, n_nodes, offsets, parent, target, R, K, accept_len, path,
                                           next_prev0, out_tokens, status, (hipStream_t)stream), who);
}

int dspark_rotary_frequencies(int scaling, int dim, double base, double factor, double original, double low,
                              double high, double* freq) {
    const char* who = "rotary_frequencies";
    if (!freq) return fail(DSPARK_EINVAL, "%s: freq is NULL", who);
    if (dim < 2 || dim % 2) return fail(DSPARK_EINVAL, "%s: %d dims", who, dim);
    if (scaling < DSPARK_ROTARY_NONE || scaling > DSPARK_ROTARY_RAMP)
        return fail(DSPARK_EINVAL, "%s: unknown scaling %d", who, scaling);
    const bool stretched = scaling == DSPARK_ROTARY_BANDS || scaling == DSPARK_ROTARY_RAMP;
    if (!(base > 1) || !isfinite(base) || (scaling != DSPARK_ROTARY_NONE && (!(factor >= 1) || !isfinite(factor))) ||
        (stretched && (!(original > 0) || !isfinite(original) || !(low > 0) || !(low < high) || !isfinite(high))))
        return fail(DSPARK_ERANGE, "%s: base %g, factor %g, original %g, low %g, high %g", who, base, factor, original, low,
                    high);
    const double turn = 6.283185307179586476925286766559;
    const auto pair_of = [&](double turns) { return dim * log(original / (turn * turns)) / (2 * log(base)); };
    double a = 0, b = 1;
    if (scaling == DSPARK_ROTARY_RAMP) {
        a = std::max(floor(pair_of(high)), 0.0);
        b = std::min(ceil(pair_of(low)), dim - 1.0);
    }
    for (int i = 0; i < dim / 2; ++i) {
        const double f = pow(base, -2.0 * i / dim);
        double kept = 1;  // of the frequency as it is; the rest is divided by the factor
        if (scaling == DSPARK_ROTARY_LINEAR) kept = 0;
        if (scaling == DSPARK_ROTARY_BANDS)
            kept = std::min(std::max((original * f / turn - low) / (high - low), 0.0), 1.0);
        if (scaling == DSPARK_ROTARY_RAMP) kept = 1 - std::min(std::max((i - a) / std::max(b - a, 0.001), 0.0), 1.0);
        freq[i] = scaling == DSPARK_ROTARY_NONE ? f : f * (kept + (1 - kept) / factor);
    }
    return DSPARK_OK;
}

int dspark_rotary_turns(const double* freq, int n, uint64_t* turns) {
    const char* who = "rotary_turns";
    if (n < 0) return fail(DSPARK_ERANGE, "%s: %d frequencies", who, n);
    if (n == 0) return DSPARK_OK;
    if (!freq || !turns) return fail(DSPARK_EINVAL, "%s: a required pointer is NULL", who);
    for (int i = 0; i < n; ++i)
        if (!isfinite(freq[i])) return fail(DSPARK_ERANGE, "%s: frequency %d is not finite", who, i);
    for (int i = 0; i < n; ++i) {
        // In 80-bit arithmetic (64 bits of mantissa), as the fraction in [0, 1) of a turn; whole turns say nothing.
        const long double f = (long double)freq[i] / 6.283185307179586476925286766559005768L, part = f - floorl(f);
        const long double scaled = floorl(part * 18446744073709551616.0L + 0.5L);
        turns[i] = scaled >= 18446744073709551616.0L ? 0 : (uint64_t)scaled;
    }
    return DSPARK_OK;
}

size_t dspark_history_words(int V) { return V < 1 ? 0 : ((size_t)V + 127) / 128 * 4; }

int dspark_history_clear(const dspark_history_t* h, const int32_t* rows, int n, uint32_t* status, void* stream) {
    const char* who = "history_clear";
    const int rc = check_history(h, who);
    if (rc != DSPARK_OK) return rc;
    if (n < 0 || (!rows && n > h->rows)) return fail(DSPARK_ERANGE, "%s: %d rows, the history has %d", who, n, h->rows);
    if (n > kMostHistoryRows) return fail(DSPARK_EUNSUPPORTED, "%s: %d rows exceed %d", who, n, kMostHistoryRows);
    if (n == 0) return DSPARK_OK;
    return done(dspark::launch_history_clear(*h, rows, n, status, (hipStream_t)stream), who);
}

int dspark_history_add(const dspark_history_t* h, const int32_t* tokens, int n, int width, const int32_t* rows,
                       int answered, uint32_t* status, void* stream) {
    const char* who = "history_add";
    const int rc = check_history(h, who);
    if (rc != DSPARK_OK) return rc;
    if (n < 0 || (!rows && n > h->rows)) return fail(DSPARK_ERANGE, "%s: %d rows, the history has %d", who, n, h->rows);
    if (width < 0) return fail(DSPARK_ERANGE, "%s: width %d", who, width);
    if (n > kMostHistoryRows) return fail(DSPARK_EUNSUPPORTED, "%s: %d rows exceed %d", who, n, kMostHistoryRows);
    if (n == 0 || width == 0) return DSPARK_OK;
    if (!tokens) return fail(DSPARK_EINVAL, "%s: tokens is NULL", who);
    return done(dspark::launch_history_add(*h, tokens, n, width, rows, answered, status, (hipStream_t)stream), who);
}

size_t dspark_target_workspace_bytes(int n_rows, int V) {
    if (n_rows < 1 || V < 1 || V > kMostTokens) return 0;
    return dspark::target_ws_bytes(n_rows, dspark::target_most_parts(V));
}

int dspark_target_tokens(const dspark_target_t* t, uint32_t* status, void* ws, size_t ws_bytes, void* stream) {
    const char* who = "target_tokens";
    if (!t) return fail(DSPARK_EINVAL, "%s: NULL call", who);
    const int rc = check_step(t->R, t->lead, t->n_rows, t->max_new, t->anc ? kTreeNodes : DSPARK_TARGET_MAX_ROWS, who);
    if (rc != DSPARK_OK) return rc;
    if (t->V < 1) return fail(DSPARK_ERANGE, "%s: V %d", who, t->V);
    if (t->V > kMostTokens) return fail(DSPARK_EUNSUPPORTED, "%s: %d tokens exceed %d", who, t->V, kMostTokens);
    if (t->dtype != DSPARK_F32 && t->dtype != DSPARK_BF16 && t->dtype != DSPARK_F16)
        return fail(DSPARK_EINVAL, "%s: unknown dtype %d", who, t->dtype);
    if (t->n_nodes < 0 || t->n_bias < 0 || t->n_allowed < 0)
        return fail(DSPARK_ERANGE, "%s: n_nodes %d, n_bias %d, n_allowed %d", who, t->n_nodes, t->n_bias, t->n_allowed);
    if (t->no_token < -1 || t->no_token >= t->V)
        return fail(DSPARK_ERANGE, "%s: no_token %d outside -1 .. %d", who, t->no_token, t->V - 1);
    if (t->history) {
        const int bad = check_history(t->history, who);
        if (bad != DSPARK_OK) return bad;
        if (t->history->rows < t->R || t->history->V != t->V)
            return fail(DSPARK_EINVAL, "%s: a history of %d rows of %d tokens for %d requests of %d", who,
                        t->history->rows, t->history->V, t->R, t->V);
    }
    if (t->R == 0 || t->n_rows == 0 || t->max_new == 0) return DSPARK_OK;
    if (!t->logits || !t->offsets || !t->target) return fail(DSPARK_EINVAL, "%s: a required pointer is NULL", who);
    const size_t size = t->dtype == DSPARK_F32 ? 4 : 2;
    if ((uintptr_t)t->logits % size || (uintptr_t)t->adjusted % size)
        return fail(DSPARK_EINVAL, "%s: logits and adjusted must be aligned to their type", who);
    if (t->logits_stride < t->V || t->logits_stride > INT64_MAX / 8 / t->n_rows ||
        (t->adjusted && (t->adjusted_stride < t->V || t->adjusted_stride > INT64_MAX / 8 / t->n_rows)))
        return fail(DSPARK_EINVAL, "%s: rows lie %lld and %lld elements apart, %d or more are needed", who,
                    (long long)t->logits_stride, (long long)t->adjusted_stride, t->V);
    if (t->adjusted) {
        const uintptr_t x0 = (uintptr_t)t->logits, y0 = (uintptr_t)t->adjusted,
                        x1 = x0 + ((size_t)(t->n_rows - 1) * t->logits_stride + t->V) * size,
                        y1 = y0 + ((size_t)(t->n_rows - 1) * t->adjusted_stride + t->V) * size;
        if (x0 < y1 && y0 < x1) return fail(DSPARK_EINVAL, "%s: logits and adjusted overlap", who);
    }
    if (t->bias_off && t->n_bias > 0 && (!t->bias_tok || !t->bias_val))
        return fail(DSPARK_EINVAL, "%s: biases need bias_tok and bias_val", who);
    if (t->allowed && (t->allowed_stride < ((int64_t)t->V + 31) / 32 || (uintptr_t)t->allowed % 4))
        return fail(DSPARK_EINVAL, "%s: masks need rows of %lld words, 4-byte aligned", who, ((long long)t->V + 31) / 32);
    if (t->allowed && !t->allowed_row && t->n_allowed < t->n_rows)
        return fail(DSPARK_EINVAL, "%s: %d masks for %d rows", who, t->n_allowed, t->n_rows);
    if (!t->allowed && t->allowed_row) return fail(DSPARK_EINVAL, "%s: allowed_row without allowed", who);
    dspark::TargetArgs a{};
    a.t = *t;
    a.status = status;
    if (t->history) {
        a.seen = t->history->seen;
        a.count = t->history->count;
        a.words = dspark_history_words(t->V);
    }
    dspark::target_split((int)std::min<long long>(t->n_rows, (long long)t->R * t->max_new), t->V, a.chunk, a.parts);
    const size_t need = a.parts > 1 ? dspark::target_ws_bytes(t->n_rows, a.parts) : 0;
    if (need > ws_bytes || (need && !ws))
        return fail(DSPARK_EWORKSPACE, "%s: workspace of %zu bytes needed, %zu given%s", who, need, ws_bytes,
                    ws ? "" : " (NULL)");
    if ((uintptr_t)ws & 15u) return fail(DSPARK_EINVAL, "%s: workspace must be 16-byte aligned", who);
    if ((long long)t->R * a.parts > kMostThreads / dspark::kTargetThreads)
        return fail(DSPARK_EUNSUPPORTED, "%s: %d requests of %d parts each are too many for one call", who, t->R, a.parts);
    if (need) dspark::target_ws_layout(a, ws);
    return done(dspark::launch_target(a, (hipStream_t)stream), who);
}

}  // extern "C"
