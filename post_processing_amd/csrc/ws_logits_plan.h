// ws_logits_plan.h -- host-side checks and launch geometry of the operators
// over rows of logits (ws_logits.h).
//
// Plain C++17 with no HIP dependency, so the same code the library runs can
// be compiled and tested on a host without a GPU.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "ws_logits.h"

namespace ws {

inline int64_t logit_bytes(int32_t dtype) { return dtype == WS_DTYPE_F32 ? 4 : 2; }

inline bool aligned_to(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// A matrix of `rows` rows in memory.
struct Extent {
    const void* at;
    int64_t rows, width, stride;   // elements
    int32_t dtype;

    uintptr_t begin() const { return (uintptr_t)at; }
    uintptr_t bytes() const {
        return rows == 0 ? 0 : (uintptr_t)(((rows - 1) * stride + width) * logit_bytes(dtype));
    }
    bool aligned() const { return aligned_to(at, (uintptr_t)logit_bytes(dtype)); }
};

// Whether no byte belongs to both: apart, or between each other's rows.  An array (one
// row) may lie in a matrix's padding.  Two matrices whose rows interleave need equal
// steps, where two rows lie a fixed distance modulo the step apart, wherever the two
// extents meet; of other steps they have to lie apart.
inline bool disjoint(const Extent& a, const Extent& b) {
    if (a.rows == 0 || b.rows == 0) return true;
    const Extent& low = a.begin() < b.begin() ? a : b;
    const Extent& high = a.begin() < b.begin() ? b : a;
    const uintptr_t apart = high.begin() - low.begin();
    if (apart >= low.bytes()) return true;
    if (low.rows == 1) return false;   // reaches the other's first row
    const uintptr_t step = (uintptr_t)(low.stride * logit_bytes(low.dtype));
    if (high.rows > 1 && step != (uintptr_t)(high.stride * logit_bytes(high.dtype))) return false;
    // From the lower one's row to the next row of the upper one, and back.
    const uintptr_t into = apart % step;
    return into >= (uintptr_t)(low.width * logit_bytes(low.dtype)) &&
           step - into >= (uintptr_t)(high.width * logit_bytes(high.dtype));
}

inline int validate_rows(const ws_rows* r) {
    if (!r) return WS_E_INVALID_ARG;
    if (r->device < 0) return WS_E_INVALID_ARG;
    if (r->dtype != WS_DTYPE_F32 && r->dtype != WS_DTYPE_F16 && r->dtype != WS_DTYPE_BF16)
        return WS_E_INVALID_ARG;
    if (r->rows < 0 || r->rows > WS_MAX_ROWS) return WS_E_INVALID_ARG;
    if (r->vocab < 1 || r->vocab > WS_MAX_SCORES) return WS_E_INVALID_ARG;
    if (r->row_stride < r->vocab || r->row_stride > WS_MAX_ROW_STRIDE) return WS_E_INVALID_ARG;
    if (!(r->temperature >= WS_MIN_TEMPERATURE && r->temperature <= WS_MAX_TEMPERATURE))
        return WS_E_INVALID_ARG;
    if (r->reserved != 0) return WS_E_INVALID_ARG;
    return WS_OK;
}

// Bytes from the first to one past the last element of a matrix of rows.
inline int64_t rows_extent(const ws_rows& r, int64_t stride) {
    if (r.rows == 0) return 0;
    return ((int64_t)(r.rows - 1) * stride + r.vocab) * logit_bytes(r.dtype);
}

// The gradient's matrix: the logits themselves, or apart from them, or between
// their rows (equal strides: two rows then lie a fixed distance modulo the
// stride apart, wherever the two extents meet).
inline int validate_gradient(const ws_rows& r, const void* logits, const void* grad,
                             int64_t stride) {
    if (stride < r.vocab || stride > WS_MAX_ROW_STRIDE) return WS_E_INVALID_ARG;
    if (r.rows == 0) return WS_OK;
    if (!grad || !aligned_to(grad, (uintptr_t)logit_bytes(r.dtype))) return WS_E_INVALID_ARG;
    if (grad == logits)
        return stride == r.row_stride || r.rows == 1 ? WS_OK : WS_E_INVALID_ARG;
    const uintptr_t a = (uintptr_t)logits, b = (uintptr_t)grad;
    const uintptr_t an = (uintptr_t)rows_extent(r, r.row_stride);
    const uintptr_t bn = (uintptr_t)rows_extent(r, stride);
    const uintptr_t apart = a < b ? b - a : a - b;
    if (apart >= (a < b ? an : bn)) return WS_OK;
    if (stride != r.row_stride) return WS_E_INVALID_ARG;
    const uintptr_t step = (uintptr_t)(stride * logit_bytes(r.dtype));
    const uintptr_t row = (uintptr_t)(r.vocab * logit_bytes(r.dtype));
    const uintptr_t into = apart % step;
    return into >= row && step - into >= row ? WS_OK : WS_E_INVALID_ARG;
}

inline bool logits_ok(const ws_rows& r, const void* logits) {
    return logits && aligned_to(logits, (uintptr_t)logit_bytes(r.dtype));
}

// Two arrays that come together or not at all; where they come, both aligned.
inline bool paired(const void* a, const void* b, uintptr_t align_a, uintptr_t align_b) {
    return (a != nullptr) == (b != nullptr) && aligned_to(a, align_a) && aligned_to(b, align_b);
}

inline int validate_top_k(const ws_rows& r, int32_t top_k) {
    const int32_t most = r.vocab < WS_MAX_K ? r.vocab : WS_MAX_K;
    return top_k >= 0 && top_k <= most ? WS_OK : WS_E_INVALID_ARG;
}

inline int validate_logprobs(const ws_rows* r, const ws_logprobs_args* a) {
    const int v = validate_rows(r);
    if (v != WS_OK) return v;
    if (!a || a->reserved != 0) return WS_E_INVALID_ARG;
    if (validate_top_k(*r, a->top_k) != WS_OK) return WS_E_INVALID_ARG;
    if (r->rows == 0) return WS_OK;
    if (!logits_ok(*r, a->logits)) return WS_E_INVALID_ARG;
    if (!paired(a->targets, a->logprob, 4, 4)) return WS_E_INVALID_ARG;
    if ((a->top != nullptr) != (a->top_k > 0)) return WS_E_INVALID_ARG;
    if (!aligned_to(a->entropy, 4) || !aligned_to(a->top, 8) || !aligned_to(a->stats, 8))
        return WS_E_INVALID_ARG;
    return WS_OK;
}

inline int validate_logprobs_grad(const ws_rows* r, const ws_logprobs_grad_args* a) {
    const int v = validate_rows(r);
    if (v != WS_OK) return v;
    if (!a || a->reserved != 0) return WS_E_INVALID_ARG;
    if (a->top_k < 0 || a->top_k > WS_MAX_K) return WS_E_INVALID_ARG;
    if (r->rows > 0) {
        if (!logits_ok(*r, a->logits)) return WS_E_INVALID_ARG;
        if (!a->stats || !aligned_to(a->stats, 8)) return WS_E_INVALID_ARG;
        if (!paired(a->targets, a->grad_logprob, 4, 4)) return WS_E_INVALID_ARG;
        if (!paired(a->entropy, a->grad_entropy, 4, 4)) return WS_E_INVALID_ARG;
        if (!paired(a->top, a->grad_top, 8, 4)) return WS_E_INVALID_ARG;
        if ((a->top != nullptr) != (a->top_k > 0)) return WS_E_INVALID_ARG;
    }
    return validate_gradient(*r, a->logits, a->grad_logits, a->grad_stride);
}

inline int validate_teacher(int32_t teacher_k, int32_t mode) {
    if (teacher_k < 1 || teacher_k > WS_DISTILL_MAX_K) return WS_E_INVALID_ARG;
    return mode == WS_DISTILL_RENORM || mode == WS_DISTILL_TAIL ? WS_OK : WS_E_INVALID_ARG;
}

inline int validate_distill(const ws_rows* r, const ws_distill_args* a) {
    const int v = validate_rows(r);
    if (v != WS_OK) return v;
    if (!a || a->reserved[0] != 0 || a->reserved[1] != 0) return WS_E_INVALID_ARG;
    if (validate_teacher(a->teacher_k, a->mode) != WS_OK) return WS_E_INVALID_ARG;
    if (a->tail && a->mode != WS_DISTILL_TAIL) return WS_E_INVALID_ARG;
    if (r->rows == 0) return WS_OK;
    if (!logits_ok(*r, a->logits)) return WS_E_INVALID_ARG;
    if (!a->teacher || !aligned_to(a->teacher, 8)) return WS_E_INVALID_ARG;
    if (!a->loss || !aligned_to(a->loss, 4)) return WS_E_INVALID_ARG;
    if (!aligned_to(a->stats, 8) || !aligned_to(a->tail, 4)) return WS_E_INVALID_ARG;
    if (!paired(a->grad_logits, a->grad_loss, 1, 4)) return WS_E_INVALID_ARG;
    if (!a->grad_logits) return WS_OK;
    return validate_gradient(*r, a->logits, a->grad_logits, a->grad_stride);
}

inline int validate_distill_grad(const ws_rows* r, const ws_distill_grad_args* a) {
    const int v = validate_rows(r);
    if (v != WS_OK) return v;
    if (!a || validate_teacher(a->teacher_k, a->mode) != WS_OK) return WS_E_INVALID_ARG;
    if (r->rows > 0) {
        if (!logits_ok(*r, a->logits)) return WS_E_INVALID_ARG;
        if (!a->teacher || !aligned_to(a->teacher, 8)) return WS_E_INVALID_ARG;
        if (!a->stats || !aligned_to(a->stats, 8)) return WS_E_INVALID_ARG;
        if ((a->tail != nullptr) != (a->mode == WS_DISTILL_TAIL)) return WS_E_INVALID_ARG;
        if (!aligned_to(a->tail, 4)) return WS_E_INVALID_ARG;
        if (!a->grad_loss || !aligned_to(a->grad_loss, 4)) return WS_E_INVALID_ARG;
    }
    return validate_gradient(*r, a->logits, a->grad_logits, a->grad_stride);
}

inline int validate_workspace(const void* workspace, size_t given, size_t needed) {
    if (needed == 0) return WS_OK;
    if (!workspace || !aligned_to(workspace, 16) || given < needed) return WS_E_INVALID_ARG;
    return WS_OK;
}

// The `needed` bytes of workspace that a call writes: they must be there, and belong to
// none of its other buffers.
inline int validate_apart(const void* workspace, size_t given, size_t needed,
                          const Extent* buffers, int count) {
    const int v = validate_workspace(workspace, given, needed);
    if (v != WS_OK || needed == 0) return v;
    const int64_t words = (int64_t)((needed + 3) / 4);
    const Extent space = {workspace, 1, words, words, WS_DTYPE_F32};
    for (int i = 0; i < count; ++i)
        if (!disjoint(space, buffers[i])) return WS_E_INVALID_ARG;
    return WS_OK;
}

// The buffers of a sampling call, what is left out being nowhere; the first
// kSampleOutputs are written.
constexpr int kSampleOutputs = 2, kSampleBuffers = 8;

struct SampleBuffers {
    Extent at[kSampleBuffers];

    SampleBuffers(const ws_rows& r, const ws_sample_args& a) {
        const void* arrays[] = {a.token, a.logprob, a.uniform, a.temperature, a.top_k, a.top_p, a.min_p};
        for (int i = 0; i < kSampleBuffers - 1; ++i)
            at[i] = {arrays[i], arrays[i] ? 1 : 0, r.rows, r.rows, WS_DTYPE_F32};
        at[kSampleBuffers - 1] = {a.logits, r.rows, r.vocab, r.row_stride, r.dtype};
    }
};

inline int validate_sample(const ws_rows* r, const ws_sample_args* a) {
    const int v = validate_rows(r);
    if (v != WS_OK) return v;
    if (!a) return WS_E_INVALID_ARG;
    if (r->rows == 0) return WS_OK;
    if (!logits_ok(*r, a->logits)) return WS_E_INVALID_ARG;
    if (!a->uniform || !a->token) return WS_E_INVALID_ARG;
    const SampleBuffers buffers(*r, *a);
    for (const Extent& b : buffers.at)
        if (!b.aligned()) return WS_E_INVALID_ARG;
    for (int i = 0; i < kSampleOutputs; ++i)
        for (int j = i + 1; j < kSampleBuffers; ++j)
            if (!disjoint(buffers.at[i], buffers.at[j])) return WS_E_INVALID_ARG;
    return WS_OK;
}

// (with arguments that validate_sample has passed)
inline int validate_sample_workspace(const ws_rows& r, const ws_sample_args& a, size_t needed) {
    const SampleBuffers buffers(r, a);
    return validate_apart(a.workspace, a.workspace_bytes, needed, buffers.at, kSampleBuffers);
}

// ---------------------------------------------------------------------------
// Launch geometry and workspaces.

inline int64_t slots_of(const ws_rows& r) {
    const int64_t vec = 16 / logit_bytes(r.dtype);
    return (r.vocab + vec - 1) / vec;
}

// Whether every row starts on 16 bytes.
inline bool rows_aligned(const ws_rows& r, const void* logits) {
    return aligned_to(logits, 16) &&
           (r.rows == 1 || (r.row_stride * logit_bytes(r.dtype)) % 16 == 0);
}

// Whether slots go past the caches: matrices of more than half the 256 MB
// last-level cache, of which the next reader would find little (MI355X, other
// inputs from pass to pass: 4,096 x 131,072 BF16 with entropy 174 us through
// them, 165 past; gradient of 4,096 x 65,536 189 and 176; 2,048 x 50,001 with the
// best 20, 205 MB, 49 and 45; smaller ones, which the cache holds, lose: 64 x
// 32,768 FP16 7.6 and 10.1, gradient of 255 x 50,001 12.9 and 15.4).
constexpr int64_t kStreamBytes = 128ll << 20;

inline bool streams(const ws_rows& r) {
    return (int64_t)r.rows * r.vocab * logit_bytes(r.dtype) > kStreamBytes;
}

// A row is split into `parts` of `chunk` 16-byte slots, the last of which takes
// what is left (fewer than `parts` slots more, and one more still when the
// row's start is not aligned); a second kernel joins them.
constexpr int kMaxRowParts = 64;
constexpr int kBatchSlots = 4;      // slots a thread has in flight in a pass
constexpr int kHeldLeast = 16;      // from here a row has a slot that lies in it whole

// Workgroups a row is split over.  The join costs about 4 us (MI355X, best 20;
// 2 us without), so rows are split that would take a workgroup longer than
// that and only while they leave CUs idle: 131,072 BF16 logits with the best 20
// in 1 / 8 / 16 parts 17.0 / 11.3 / 10.6 us for 16 rows, 1 / 4 / 8 parts 17.3 /
// 15.0 / 14.6 us for 64 rows, 1 / 2 parts 28.6 / 23.3 us for 256; 32,768 logits
// 7.7 us whole, 10.5 in 4 parts.
constexpr int64_t kSplitSlots = 6144, kPartSlots = 1024, kSplitGroups = 512;

inline int64_t row_parts(const ws_rows& r) {
    const int64_t slots = slots_of(r);
    if (slots <= kSplitSlots) return 1;
    int64_t parts = kSplitGroups / r.rows;
    if (parts > slots / kPartSlots) parts = slots / kPartSlots;
    if (parts > kMaxRowParts) parts = kMaxRowParts;
    return parts < 1 ? 1 : parts;
}

// Threads of a workgroup that takes `slots` slots: one wave for short rows
// (MI355X, 4,096 rows of 4,096 BF16 logits with the best 20: 15.4 us with one
// wave, 20.1 with four; of 8,192 logits 23.4 and 22.2), sixteen for long ones,
// where fewer rows are in flight at once (4,096 rows with entropy: of 131,072
// logits 185 us with four waves, 172 with sixteen; of 100,001 152 and 141; of
// 81,920, which end amid a batch, 120 and 129), four otherwise.
constexpr int64_t kWaveSlots = 512, kWideSlots = 12288;

inline int32_t row_threads(int64_t slots) {
    return slots <= kWaveSlots ? 64 : slots < kWideSlots ? 256 : 1024;
}

struct LogprobsPlan {
    int32_t threads = 256;
    int32_t parts = 1;
    int32_t chunk = 0;
    size_t workspace = 0;
};

inline LogprobsPlan plan_logprobs(const ws_rows& r, int32_t top_k) {
    LogprobsPlan p;
    if (r.rows == 0) return p;
    p.parts = (int32_t)row_parts(r);
    p.chunk = (int32_t)(slots_of(r) / p.parts);
    p.threads = row_threads(p.chunk);
    // Keys of the best K and the sums (three FP32) of every part.
    if (p.parts > 1)
        p.workspace = (size_t)r.rows * (size_t)p.parts * (8u * (size_t)top_k + 12u);
    return p;
}

// Gradients: parts of a row as above, each workgroup reading the row's named
// tokens for itself.  2,048 slots a workgroup (MI355X, 4,096 rows of 65,536 BF16
// with entropy, in us: 1,024 slots 195, 2,048 189, 4,096 205, 8,192 221), and
// enough of them for few rows (255 rows of 50,001 FP16: 512 workgroups 14.8,
// 1,024 12.8, 2,048 14.9, 4,096 17.2).
constexpr int64_t kGradSlots = 2048, kGradLeast = 256, kGradGroups = 1024;

struct GradPlan {
    int32_t parts = 1;
    int32_t chunk = 0;
};

inline GradPlan plan_grad(const ws_rows& r) {
    GradPlan p;
    const int64_t slots = slots_of(r);
    int64_t parts = (slots + kGradSlots - 1) / kGradSlots;
    int64_t want = (kGradGroups + r.rows - 1) / r.rows;
    if (want > slots / kGradLeast) want = slots / kGradLeast;
    if (parts < want) parts = want;
    p.parts = (int32_t)parts;
    p.chunk = (int32_t)(slots / parts);
    return p;
}

// ws_distill: the loss as ws_logprobs splits its rows, with a limit to a part
// from the marks of the listed tokens in LDS (a byte a slot).  With a gradient,
// rows that fit the registers of one workgroup (`held` slots a thread) are done
// in one kernel; longer ones, and few 16-bit rows that take sixteen waves, by
// the loss and then the gradient.  A 16-bit slot is twice the elements to work
// through on the CU that holds it, so splitting its row pays until there are
// rows for a third of the CUs (MI355X, 32 entries with a tail, whole calls in us,
// held and in three kernels; 131,072 BF16 logits: 4 rows 20.5 and 13.7, 64 rows
// 23.4 and 21.3, 80 rows 23.7 and 23.8, 128 rows 25.5 and 28.5; 98,301: 64 rows
// 20.8 and 20.0, 80 rows 21.1 and 21.7; 51,197, eight waves: 4 rows 13.4 and
// 15.2, 64 rows 14.4 and 18.7; 65,536 FP32: 4 rows 12.3 and 13.0, 64 rows 15.1
// and 20.2).
constexpr int kHeldSlots = 16;
constexpr int kHeldRows = 80;
constexpr int kMaxMarkedSlots = 32768;

struct DistillPlan {
    int32_t threads = 256;
    int32_t held = 0;
    int32_t parts = 1;
    int32_t chunk = 0;
    int32_t mark_bytes = 0;
    size_t tail_at = 0, sums_at = 0;   // offsets in the workspace
    size_t workspace = 0;
};

// aligned: as rows_aligned says; without it a row may take one slot more, and
// the workspace (which is asked for before the rows' address is known) is at
// least that of aligned rows.
inline DistillPlan plan_distill(const ws_rows& r, int32_t mode, bool gradient, bool aligned) {
    DistillPlan p;
    if (r.rows == 0) return p;
    const int64_t slots = slots_of(r);
    const int64_t most = slots + (aligned ? 0 : 1);
    if (gradient && most <= kHeldSlots * 1024 && r.vocab >= kHeldLeast &&
        (most <= kHeldSlots * 512 || r.dtype == WS_DTYPE_F32 || r.rows >= kHeldRows)) {
        p.held = kHeldSlots;
        p.threads = most <= kHeldSlots * 256 ? 256 : most <= kHeldSlots * 512 ? 512 : 1024;
        p.chunk = (int32_t)slots;
    } else {
        int64_t parts = row_parts(r);
        const int64_t marked = kMaxMarkedSlots - kMaxRowParts;
        if (mode == WS_DISTILL_TAIL && parts < slots / marked + 1) parts = slots / marked + 1;
        p.parts = (int32_t)parts;
        p.chunk = (int32_t)(slots / parts);
        p.threads = row_threads(p.chunk);
        if (gradient) {
            p.tail_at = (size_t)r.rows * sizeof(ws_row_stats);
            p.sums_at = p.tail_at + (size_t)r.rows * sizeof(float);
        }
        p.workspace = p.sums_at;
        if (p.parts > 1) p.workspace += (size_t)r.rows * (size_t)p.parts * 12u;
    }
    // A byte a slot: the part's, and past them what a batch of kBatchSlots
    // slots a thread reaches.
    if (mode == WS_DISTILL_TAIL)
        p.mark_bytes = p.held > 0 ? p.held * p.threads
                                  : (p.chunk + p.parts + kBatchSlots * p.threads + 15) / 16 * 16;
    return p;
}

// ws_sample: a workgroup a row; few long rows are read by `parts` workgroups
// each, whose waves leave 24 bytes and their lanes' largest logits in the
// workspace, and drawn from by a second kernel (as row_parts splits rows: more
// parts for more rows brought nothing, 300 x 50,001 FP32 33 us whole and 36 in
// three).
//
// A CU has 1,024 threads of the kernel at work.  One row of them while rows are
// few, or long (the longest row's nucleus is then waited for: 1,024 x 131,072 BF16
// with mixed settings 131 us, 166 with two rows of 512 threads); two of 512 where
// rows come in more than one round and are shorter (2,000 x 32,768 FP16 mixed 77 us
// and 115 with one of 1,024; 600 x 50,001 BF16 with the best 50 30 and 38); 256
// threads for rows that give more no whole slot.
//
// Up to 512 rows, one turn of 512 threads for two of 1,024: what reads the row once
// gains, an undecided row's nucleus, whose list is as long as the workgroup, loses, the
// more the longer the row.  Microseconds with 512 and 1,024, for all kept, mixed
// settings and the best 50: 300 x 70,001 BF16 43 and 50, 80 and 64, 18 and 28; 300 x
// 50,001 FP32 32 and 39, 69 and 51, 20 and 29; 300 x 131,072 BF16 56 and 57, 112 and
// 89, 27 and 36; but 300 x 131,072 FP32 60 and 67, 132 and 98, 48 and 54, and 300 x
// 200,003 BF16 85 and 94, 263 and 135, 34 and 42: 512 up to kSampleWide slots.
constexpr int kMaxSampleParts = 32;
constexpr int64_t kSampleSlots = 1024;   // of a part, at least
constexpr int64_t kSampleShort = 1024, kSampleLong = 8192, kSampleWide = 16384;   // slots of a row
constexpr int kSampleGroups = 256;       // workgroups of 1,024 threads at work at a time
constexpr int kStretchBytes = 24 + 64 * 4;

inline int32_t sample_threads(int64_t rows, int64_t slots) {
    if (slots <= kSampleShort) return 256;
    if (rows <= kSampleGroups) return 1024;
    return slots <= (rows <= 2 * kSampleGroups ? kSampleWide : kSampleLong) ? 512 : 1024;
}

struct SamplePlan {
    int32_t threads = 1024;
    int32_t parts = 1;
    int32_t chunk = 0;
    int32_t unit = 0;
    size_t workspace = 0;
};

inline SamplePlan plan_sample(const ws_rows& r) {
    SamplePlan p;
    if (r.rows == 0) return p;
    const int64_t slots = slots_of(r);
    p.threads = sample_threads(r.rows, slots);
    if (slots > kSplitSlots) {
        int64_t parts = kSplitGroups / r.rows;
        if (parts > slots / kSampleSlots) parts = slots / kSampleSlots;
        if (parts > kMaxSampleParts) parts = kMaxSampleParts;
        if (parts > 1) p.parts = (int32_t)parts;
    }
    p.chunk = (int32_t)(slots / p.parts);
    if (p.parts > 1)
        p.workspace = (size_t)r.rows * (size_t)p.parts * 4u * (size_t)kStretchBytes;
    // Sums of `vocab` weights of at most 1 stay at 2^62 or below.
    int bits = 0;
    while ((1ll << bits) < r.vocab) ++bits;
    p.unit = 62 - bits;
    return p;
}

}  // namespace ws
