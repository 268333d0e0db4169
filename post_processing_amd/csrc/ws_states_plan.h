// ws_states_plan.h -- host-side checks and launch geometry of the operators
// over rows of hidden states (ws_states.h).
//
// Plain C++17 with no HIP dependency, so the same code the library runs can
// be compiled and tested on a host without a GPU.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "ws_logits_plan.h"
#include "ws_states.h"

namespace ws {

inline bool stride_ok(int64_t stride, int32_t width) {
    return stride >= width && stride <= WS_MAX_ROW_STRIDE;
}

inline int validate_states(const ws_states* t) {
    if (!t) return WS_E_INVALID_ARG;
    if (t->device < 0) return WS_E_INVALID_ARG;
    if (t->dtype != WS_DTYPE_F32 && t->dtype != WS_DTYPE_F16 && t->dtype != WS_DTYPE_BF16)
        return WS_E_INVALID_ARG;
    if (t->rows < 0 || t->rows > WS_MAX_ROWS) return WS_E_INVALID_ARG;
    if (t->width < 1 || t->width > WS_MAX_WIDTH) return WS_E_INVALID_ARG;
    return stride_ok(t->row_stride, t->width) ? WS_OK : WS_E_INVALID_ARG;
}

// The same rows of the same elements.
inline bool same_rows(const Extent& a, const Extent& b) {
    return a.at == b.at && a.dtype == b.dtype && (a.stride == b.stride || a.rows <= 1);
}

inline Extent extent_of(const ws_states& t, const void* at, int64_t stride) {
    return {at, t.rows, t.width, stride, t.dtype};
}

// ---- embedding -----------------------------------------------------------------

inline int validate_embed(const ws_states* t, const ws_embed_args* a) {
    const int v = validate_states(t);
    if (v != WS_OK) return v;
    if (!a || a->vocab < 1 || a->vocab > WS_MAX_TOKENS) return WS_E_INVALID_ARG;
    if (!stride_ok(a->table_stride, t->width) || !std::isfinite(a->scale)) return WS_E_INVALID_ARG;
    if (t->rows == 0) return WS_OK;
    const Extent out = extent_of(*t, a->out, t->row_stride);
    const Extent table = {a->table, a->vocab, t->width, a->table_stride, t->dtype};
    const Extent ids = {a->ids, 1, t->rows, t->rows, WS_DTYPE_F32};
    if (!a->table || !a->out || !a->ids) return WS_E_INVALID_ARG;
    if (!out.aligned() || !table.aligned() || !ids.aligned()) return WS_E_INVALID_ARG;
    return disjoint(out, table) && disjoint(out, ids) ? WS_OK : WS_E_INVALID_ARG;
}

inline int validate_weight_dtype(const ws_states& t, int32_t dtype) {
    return dtype == t.dtype || dtype == WS_DTYPE_F32 ? WS_OK : WS_E_INVALID_ARG;
}

inline int validate_embed_grad(const ws_states* t, const ws_embed_grad_args* a) {
    const int v = validate_states(t);
    if (v != WS_OK) return v;
    if (!a || a->vocab < 1 || a->vocab > WS_MAX_TOKENS) return WS_E_INVALID_ARG;
    if (!stride_ok(a->grad_stride, t->width) || !std::isfinite(a->scale)) return WS_E_INVALID_ARG;
    if (validate_weight_dtype(*t, a->grad_dtype) != WS_OK) return WS_E_INVALID_ARG;
    if (a->accumulate != 0 && a->accumulate != 1) return WS_E_INVALID_ARG;
    const Extent grad = {a->grad_table, a->vocab, t->width, a->grad_stride, a->grad_dtype};
    if (!a->grad_table || !grad.aligned()) return WS_E_INVALID_ARG;
    if (t->rows == 0) return WS_OK;
    const Extent rows = extent_of(*t, a->grad_out, t->row_stride);
    const Extent ids = {a->ids, 1, t->rows, t->rows, WS_DTYPE_F32};
    if (!a->grad_out || !a->ids || !rows.aligned() || !ids.aligned()) return WS_E_INVALID_ARG;
    return disjoint(grad, rows) && disjoint(grad, ids) ? WS_OK : WS_E_INVALID_ARG;
}

// (with arguments that validate_embed_grad has passed)
inline int validate_embed_grad_workspace(const ws_states& t, const ws_embed_grad_args& a,
                                         size_t needed) {
    const Extent buffers[] = {extent_of(t, a.grad_out, t.row_stride),
                              {a.ids, 1, t.rows, t.rows, WS_DTYPE_F32},
                              {a.grad_table, a.vocab, t.width, a.grad_stride, a.grad_dtype}};
    return validate_apart(a.workspace, a.workspace_bytes, needed, buffers, 3);
}

inline int64_t slots_in(int32_t width, int32_t dtype) {
    const int64_t vec = 16 / logit_bytes(dtype);
    return (width + vec - 1) / vec;
}

// Lookup: a workgroup of 256 threads takes 256 / lanes rows, `lanes` (a power
// of two) threads to a row's 16-byte slots.
constexpr int kLookupThreads = 256;

struct EmbedPlan {
    int32_t lanes = 8;
    int64_t groups = 0;
};

inline EmbedPlan plan_embed(const ws_states& t) {
    EmbedPlan p;
    const int64_t slots = slots_in(t.width, t.dtype);
    while (p.lanes < slots && p.lanes < kLookupThreads) p.lanes *= 2;
    const int64_t each = kLookupThreads / p.lanes;
    p.groups = (t.rows + each - 1) / each;
    return p;
}

// Gradient: tokens sorted in tiles of kSortTile, one digit of kDigitBits a pass;
// the sorted rows are added in blocks of `block` rows.  Blocks are small while
// workgroups are few (the rows of a block come one after the other).
constexpr int kSortThreads = 1024, kSortTile = 2048, kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kOwnTiles = 2;       // up to here every tile counts all tokens for itself:
                                   // 2,100 rows 22.6 us, 26.2 with a launch that counts;
                                   // 8,192 rows of one token 35 (one address), 27
constexpr int kScanTiles = 64;     // up to here every tile sums the counts for itself
constexpr int kScanDigits = 16;    // a cache line of them
constexpr int kMostGroups = 8192, kLeastRows = 8, kBlockRows = 32, kSumGroups = 512;
constexpr int kSumThreads = 256, kLeastLanes = 8;
constexpr int kMostRows = kBlockRows * kSumThreads / kLeastLanes;   // of a workgroup
static_assert(kMostRows >= WS_MAX_ROWS / kMostGroups, "a workgroup's rows");
constexpr int kClearRows = 16;     // of the table, by one workgroup
// Few rows go without a sort, a workgroup a row and kSumThreads slots at most: 777 x
// 1,000 FP32 into 5,003 rows 9.5 us, sorted 17.8; 1,000 x 64 BF16 into 50,000 7.9 and
// 17.4; 512 x 4,096 BF16 into 1,000 10.7 and 18.5, into 32,768, whose zeros are most of
// it, 41 and 42.  Not where that makes more than kFewGroups workgroups, each of which
// reads all tokens (512 x 16,384 BF16 27 us, sorted 23), nor where one token's rows
// could be more than kFewBytes for one workgroup to add (1,024 x 4,096 BF16 of one token
// 98 us, sorted 32).  Below that one token of all rows costs up to half as much again:
// 777 x 1,000 FP32 into 5,003 36 us, sorted 26; 512 x 4,096 BF16 into 1,000 23 and 23,
// into 32,768 66 and 50.
constexpr int kFewRows = 1024, kFewGroups = 2048;
constexpr int64_t kFewBytes = 2 << 20;

struct EmbedGradPlan {
    bool few = false;              // one launch without a sort
    int32_t tiles = 0;
    int32_t passes = 0;
    int32_t block = kBlockRows;    // sorted rows added one after the other
    int32_t blocks = 0;
    int32_t lanes = kLeastLanes;   // threads to a block; the blocks of a workgroup lie
                                   // side by side
    int32_t columns = 0;           // workgroups over a row's slots
    size_t keys_at[2] = {0, 0}, rows_at[2] = {0, 0}, counts_at = 0, partial_at = 0;
    size_t workspace = 0;
};

inline size_t round16(size_t n) { return (n + 15) / 16 * 16; }

inline EmbedGradPlan plan_embed_grad(const ws_states& t, int32_t vocab) {
    EmbedGradPlan p;
    if (t.rows == 0) return p;
    const int64_t n = t.rows;
    p.tiles = (int32_t)((n + kSortTile - 1) / kSortTile);
    // Keys are 0..vocab, vocab standing for no token.
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;
    p.passes = (bits + kDigitBits - 1) / kDigitBits;
    const int64_t slots = slots_in(t.width, t.dtype);
    while (p.lanes < slots && p.lanes < kSumThreads) p.lanes *= 2;
    p.columns = (int32_t)((slots + kSumThreads - 1) / kSumThreads);
    if (n <= kFewRows) {
        int32_t lanes = p.lanes;   // few, for a token of many rows is one workgroup's work
        while (lanes > 64 && n * ((slots + lanes / 2 - 1) / (lanes / 2)) <= kFewGroups) lanes /= 2;
        const int64_t columns = (slots + lanes - 1) / lanes;
        p.few = n * columns <= kFewGroups && n * lanes * 16 <= kFewBytes;
        if (p.few) {
            p.lanes = lanes;
            p.columns = (int32_t)columns;
        }
    }
    const int64_t beside = kSumThreads / p.lanes, most = kMostGroups * beside;
    int64_t block = n * p.columns / (kSumGroups * beside);
    block = block < kLeastRows ? kLeastRows : block > kBlockRows ? kBlockRows : block;
    if (n > block * most) block = (n + most - 1) / most;
    p.block = (int32_t)block;
    p.blocks = (int32_t)((n + block - 1) / block);
    const size_t each = round16((size_t)n * 4);
    size_t at = 0;
    for (int i = 0; i < 2; ++i) {
        p.keys_at[i] = at;
        p.rows_at[i] = at + each;
        at += 2 * each;
    }
    p.counts_at = at;
    if (p.tiles > 1) at += (size_t)(p.tiles + 1) * kDigits * 4;   // and the tiles' sums
    // Two rows of FP32 sums a block: of the token that began before it, and of
    // the one that goes on behind it.
    p.partial_at = at;
    at += (size_t)p.blocks * 2 * round16((size_t)t.width * 4);
    p.workspace = at;
    return p;
}

// ---- layer norm ------------------------------------------------------------------

inline bool in_place_or_apart(const Extent& out, const Extent& in) {
    return same_rows(out, in) || disjoint(out, in);
}

inline int validate_layernorm(const ws_states* t, const ws_layernorm_args* a) {
    const int v = validate_states(t);
    if (v != WS_OK) return v;
    if (!a || validate_weight_dtype(*t, a->weight_dtype) != WS_OK) return WS_E_INVALID_ARG;
    if (!stride_ok(a->y_stride, t->width)) return WS_E_INVALID_ARG;
    if (!(a->eps >= 0.0f) || !std::isfinite(a->eps)) return WS_E_INVALID_ARG;
    if (t->rows == 0) return WS_OK;
    const Extent x = extent_of(*t, a->x, t->row_stride), y = extent_of(*t, a->y, a->y_stride);
    const Extent weight = {a->weight, a->weight ? 1 : 0, t->width, t->width, a->weight_dtype};
    const Extent bias = {a->bias, a->bias ? 1 : 0, t->width, t->width, a->weight_dtype};
    const Extent stats = {a->stats, a->stats ? 1 : 0, 2ll * t->rows, 2ll * t->rows, WS_DTYPE_F32};
    if (!a->x || !a->y || !x.aligned() || !y.aligned() || !aligned_to(a->stats, 8))
        return WS_E_INVALID_ARG;
    if (!weight.aligned() || !bias.aligned()) return WS_E_INVALID_ARG;
    if (!in_place_or_apart(y, x) || !disjoint(y, weight) || !disjoint(y, bias) ||
        !disjoint(y, stats) || !disjoint(stats, x) || !disjoint(stats, weight) ||
        !disjoint(stats, bias))
        return WS_E_INVALID_ARG;
    return WS_OK;
}

inline int validate_layernorm_grad(const ws_states* t, const ws_layernorm_grad_args* a) {
    const int v = validate_states(t);
    if (v != WS_OK) return v;
    if (!a || a->reserved != 0) return WS_E_INVALID_ARG;
    if (validate_weight_dtype(*t, a->weight_dtype) != WS_OK) return WS_E_INVALID_ARG;
    if (!stride_ok(a->grad_y_stride, t->width)) return WS_E_INVALID_ARG;
    if (a->grad_x && !stride_ok(a->grad_x_stride, t->width)) return WS_E_INVALID_ARG;
    if (!a->grad_x && !a->grad_weight && !a->grad_bias) return WS_E_INVALID_ARG;
    const Extent gw = {a->grad_weight, a->grad_weight ? 1 : 0, t->width, t->width, a->weight_dtype};
    const Extent gb = {a->grad_bias, a->grad_bias ? 1 : 0, t->width, t->width, a->weight_dtype};
    if (!gw.aligned() || !gb.aligned() || !disjoint(gw, gb)) return WS_E_INVALID_ARG;
    if (t->rows == 0) return WS_OK;
    const Extent x = extent_of(*t, a->x, t->row_stride);
    const Extent gy = extent_of(*t, a->grad_y, a->grad_y_stride);
    Extent gx = extent_of(*t, a->grad_x, a->grad_x_stride);
    if (!a->grad_x) gx.rows = 0;
    const Extent weight = {a->weight, a->weight ? 1 : 0, t->width, t->width, a->weight_dtype};
    const Extent stats = {a->stats, 1, 2ll * t->rows, 2ll * t->rows, WS_DTYPE_F32};
    if (!a->x || !a->grad_y || !a->stats || !x.aligned() || !gy.aligned() || !gx.aligned() ||
        !weight.aligned() || !aligned_to(a->stats, 8))
        return WS_E_INVALID_ARG;
    if (!in_place_or_apart(gx, x) || !in_place_or_apart(gx, gy) || !disjoint(gx, weight) ||
        !disjoint(gx, stats))
        return WS_E_INVALID_ARG;
    for (const Extent* out : {&gw, &gb})
        if (!disjoint(*out, x) || !disjoint(*out, gy) || !disjoint(*out, gx) ||
            !disjoint(*out, weight) || !disjoint(*out, stats))
            return WS_E_INVALID_ARG;
    return WS_OK;
}

// (with arguments that validate_layernorm_grad has passed)
inline int validate_layernorm_grad_workspace(const ws_states& t, const ws_layernorm_grad_args& a,
                                             size_t needed) {
    const auto vector = [&](const void* p) -> Extent {
        return {p, p ? 1 : 0, t.width, t.width, a.weight_dtype};
    };
    Extent gx = extent_of(t, a.grad_x, a.grad_x_stride);
    if (!a.grad_x) gx.rows = 0;
    const Extent buffers[] = {extent_of(t, a.x, t.row_stride),
                              extent_of(t, a.grad_y, a.grad_y_stride),
                              gx,
                              {a.stats, 1, 2ll * t.rows, 2ll * t.rows, WS_DTYPE_F32},
                              vector(a.weight),
                              vector(a.grad_weight),
                              vector(a.grad_bias)};
    return validate_apart(a.workspace, a.workspace_bytes, needed, buffers, 7);
}

constexpr int kNormThreads = 256, kLongThreads = 1024, kLongGroups = 1 << 20;

// Rows held in registers: `held` slots by each of `threads` threads (less than a
// wave: rows side by side in one), `groups` workgroups that take rows in turn.  0:
// rows that do not fit, or have no slot.
struct NormPlan {
    int32_t threads = kNormThreads;
    int32_t held = 0;
    int32_t groups = 0;
};

// Waves at work at a time, four to a SIMD.
constexpr int32_t kNormCus = 256;
constexpr int64_t kNormWaves = kNormCus * 16;

inline NormPlan plan_held(const ws_states& t, int64_t most) {
    NormPlan p;
    const int64_t slots = slots_in(t.width, t.dtype);
    if (slots > most || t.width < 16 / logit_bytes(t.dtype)) return p;
    // (Thread counts between powers of two leave waves' room unused past 192: 384 and
    // 768 threads with two slots each took 67 and 78 us for 5,120 and 12,288 BF16
    // elements, 56 and 56 with three of 256 and 512.)
    struct Shape { int16_t threads, held; };
    constexpr Shape kShapes[] = {{8, 1},   {16, 1},  {32, 1},  {64, 1},  {64, 2},   {192, 1}, {256, 1},
                                 {256, 2}, {256, 3}, {512, 2}, {512, 3}, {1024, 2}, {512, 6}, {1024, 4}};
    for (const Shape& shape : kShapes) {
        p.threads = shape.threads;
        p.held = shape.held;
        if (p.threads * p.held >= slots) break;
    }
    const int64_t beside = p.threads < 64 ? 64 / p.threads : 1;
    const int64_t most_groups = kNormWaves / (p.threads < 64 ? 1 : p.threads / 64);
    const int64_t groups = (t.rows + beside - 1) / beside;
    p.groups = (int32_t)(groups < most_groups ? groups : most_groups);
    return p;
}

inline NormPlan plan_layernorm(const ws_states& t) { return plan_held(t, 4096); }

// Sums over the rows: `groups` workgroups' sums of every column, then their sum.
// Workgroups of one wave are four times as many: 65,536 x 1,024 BF16 takes 116 us
// with 512 of them, 88 with 2,048.  Each has kLeastEach rows (or the joining takes
// longer than the rows: 300 x 4,096 BF16 13.5 us with one a group, 11.4 with four, 4,000
// x 256 13.5 and 11.0), but where there are few at all.
constexpr int64_t kColumnGroups = 512, kLeastEach = 4, kFewSums = 256;

struct NormGradPlan {
    int32_t threads = kNormThreads;
    int32_t held = 0;
    int32_t columns = 1;   // of rows that are not held: workgroups over the columns
    int32_t groups = 1;    // over the rows
    int32_t row_groups = 0;   // of rows that are held, without sums
    size_t workspace = 0;
};

inline NormGradPlan plan_layernorm_grad(const ws_states& t) {
    NormGradPlan p;
    NormPlan held = plan_held(t, t.dtype == WS_DTYPE_F32 ? 4096 : 2048);
    // The sums fill the registers of 1,024 threads with two slots each: 12,288 BF16
    // elements 122 us for 5,461 rows, 89 with three of 512 threads.
    if (held.threads == 192) held.threads = 256;
    if (held.threads > 256) {
        held.threads = 512;
        held.held = (int32_t)((slots_in(t.width, t.dtype) + 511) / 512);
        if (held.held == 7) held.held = 8;
        if (held.held > 2 && held.groups > kNormCus) held.groups = kNormCus;
    }
    p.threads = held.threads;
    p.held = held.held;
    if (t.rows == 0) {
        p.groups = 0;
    } else if (p.held > 0) {
        const int64_t most = p.threads <= 64 ? 4 * kColumnGroups : kColumnGroups;
        int64_t each = (t.rows + most - 1) / most;
        if (each < kLeastEach && t.rows >= kFewSums) each = kLeastEach;
        const int64_t groups = (t.rows + each - 1) / each;
        p.groups = (int32_t)(groups < held.groups ? groups : held.groups);
        p.row_groups = held.groups;
    } else {
        p.columns = (int32_t)((slots_in(t.width, t.dtype) + kNormThreads - 1) / kNormThreads);
        int64_t groups = kColumnGroups / p.columns;
        const int64_t most = (t.rows + 7) / 8;
        if (groups > most) groups = most;
        p.groups = (int32_t)(groups < 1 ? 1 : groups);
    }
    p.workspace = (size_t)p.groups * 2 * round16((size_t)t.width * 4);
    return p;
}

}  // namespace ws
