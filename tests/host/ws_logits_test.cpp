// Host-only driver for the checks and launch geometry of the operators over
// rows of logits (ws_logits_plan.h): compiled with g++ and no HIP by
// tests/test_logits_host.py.
//   ws_logits_test selftest  -> argument checks
//   ws_logits_test layout    -> "struct field offset" for the ABI structs
#include <cmath>
#include <cstddef>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <limits>

#include "ws_fp64.h"
#include "ws_logits_plan.h"

static int failures = 0;
#define CHECK(cond)                                                    \
    do {                                                               \
        if (!(cond)) {                                                 \
            std::printf("FAIL %s:%d %s\n", __FILE__, __LINE__, #cond); \
            ++failures;                                                \
        }                                                              \
    } while (0)

template <typename T>
static T* at(uintptr_t a) {
    return reinterpret_cast<T*>(a);
}

static ws_rows rows() {
    ws_rows r;
    std::memset(&r, 0, sizeof r);
    r.dtype = WS_DTYPE_BF16;
    r.rows = 8;
    r.vocab = 1000;
    r.row_stride = 1024;
    r.temperature = 1.0f;
    return r;
}

static ws_logprobs_args logprobs() {
    ws_logprobs_args a;
    std::memset(&a, 0, sizeof a);
    a.logits = at<void>(0x10000);
    a.targets = at<int32_t>(0x80000);
    a.logprob = at<float>(0x81000);
    a.entropy = at<float>(0x82000);
    a.top = at<ws_topk_entry>(0x83000);
    a.stats = at<ws_row_stats>(0x84000);
    a.top_k = 20;
    return a;
}

static ws_logprobs_grad_args logprobs_grad() {
    ws_logprobs_grad_args a;
    std::memset(&a, 0, sizeof a);
    a.logits = at<void>(0x10000);
    a.stats = at<ws_row_stats>(0x84000);
    a.targets = at<int32_t>(0x80000);
    a.grad_logprob = at<float>(0x81000);
    a.grad_logits = at<void>(0x100000);
    a.grad_stride = 1000;
    return a;
}

static ws_distill_args distill() {
    ws_distill_args a;
    std::memset(&a, 0, sizeof a);
    a.logits = at<void>(0x10000);
    a.teacher = at<ws_topk_entry>(0x80000);
    a.loss = at<float>(0x90000);
    a.teacher_k = 32;
    a.mode = WS_DISTILL_TAIL;
    return a;
}

static ws_distill_grad_args distill_grad() {
    ws_distill_grad_args a;
    std::memset(&a, 0, sizeof a);
    a.logits = at<void>(0x10000);
    a.teacher = at<ws_topk_entry>(0x80000);
    a.stats = at<ws_row_stats>(0x90000);
    a.tail = at<float>(0x91000);
    a.grad_loss = at<float>(0x92000);
    a.grad_logits = at<void>(0x100000);
    a.grad_stride = 1000;
    a.teacher_k = 32;
    a.mode = WS_DISTILL_TAIL;
    return a;
}

// Launch geometry over the whole range of shapes: what the kernels assume of
// their parts, marks and workspaces.
static void plans() {
    using namespace ws;
    const int64_t vocabs[] = {1,     2,     7,      8,      9,      15,      16,       17,
                              511,   512,   2047,   2048,   4096,   4104,    32768,    49151,
                              49152, 49160, 65536,  65537,  98303,  98304,   131071,   131072,
                              131073, 261632, 262144, 262145, 1000003, 20000003, WS_MAX_SCORES};
    const int32_t counts[] = {1, 2, 3, 8, 63, 64, 65, 127, 255, 256, 257, 511, 512, 513, 1024,
                              4096, 100000, WS_MAX_ROWS};
    for (int32_t dtype : {WS_DTYPE_F32, WS_DTYPE_F16, WS_DTYPE_BF16})
        for (int64_t vocab : vocabs)
            for (int32_t count : counts) {
                ws_rows r = rows();
                r.dtype = dtype;
                r.rows = count;
                r.vocab = (int32_t)vocab;
                r.row_stride = vocab;
                const int64_t slots = slots_of(r);
                const LogprobsPlan lp = plan_logprobs(r, 32 < vocab ? 32 : (int32_t)vocab);
                CHECK(lp.parts >= 1 && lp.parts <= kMaxRowParts && lp.chunk >= 1);
                CHECK((int64_t)(lp.parts - 1) * lp.chunk + lp.chunk <= slots);
                CHECK(slots - (int64_t)(lp.parts - 1) * lp.chunk < lp.chunk + lp.parts);
                CHECK(lp.parts == 1 || lp.chunk >= WS_MAX_K);
                CHECK(lp.parts == 1 ? lp.workspace == 0
                                    : lp.workspace >= (size_t)count * lp.parts * (8u * 32 + 12));
                const GradPlan g = plan_grad(r);
                CHECK(g.parts >= 1 && g.chunk >= 1 && (int64_t)g.parts * g.chunk <= slots);
                CHECK(g.parts == 1 || g.chunk >= kGradLeast);
                for (int mode : {WS_DISTILL_RENORM, WS_DISTILL_TAIL})
                    for (bool gradient : {false, true}) {
                        const DistillPlan any = plan_distill(r, mode, gradient, false);
                        const DistillPlan even = plan_distill(r, mode, gradient, true);
                        CHECK(any.workspace >= even.workspace);
                        for (const DistillPlan& p : {any, even}) {
                            if (p.held > 0) {
                                CHECK(gradient && p.parts == 1 && r.vocab >= kHeldLeast);
                                CHECK(slots <= (int64_t)p.held * p.threads);
                                CHECK(mode != WS_DISTILL_TAIL || p.mark_bytes == p.held * p.threads);
                                CHECK(p.workspace == 0);
                                continue;
                            }
                            const int64_t last = slots - (int64_t)(p.parts - 1) * p.chunk + 1;   // unaligned
                            CHECK(p.parts >= 1 && p.chunk >= 1 && last >= p.chunk);
                            CHECK(mode == WS_DISTILL_TAIL
                                      ? p.mark_bytes >= last + (kBatchSlots - 1) * p.threads &&
                                            p.mark_bytes <= 60 * 1024 && p.mark_bytes % 16 == 0
                                      : p.mark_bytes == 0);
                            size_t need = gradient ? (size_t)count * 12 : 0;
                            if (p.parts > 1) need += (size_t)count * (size_t)p.parts * 12;
                            CHECK(p.workspace >= need);
                        }
                        if (any.held > 0) CHECK(slots + 1 <= (int64_t)any.held * any.threads);
                    }
            }
}

// Which rows a workgroup holds for loss and gradient: the sides that measured
// faster (see kHeldRows).
static void held_rows() {
    const struct {
        int32_t dtype, rows, vocab;
        bool held;
    } cases[] = {{WS_DTYPE_BF16, 4, 131072, false}, {WS_DTYPE_BF16, 64, 131072, false},
                 {WS_DTYPE_F16, 79, 98301, false},  {WS_DTYPE_BF16, 80, 131072, true},
                 {WS_DTYPE_BF16, 4, 51197, true},   {WS_DTYPE_F16, 64, 51197, true},
                 {WS_DTYPE_F32, 4, 65536, true},    {WS_DTYPE_F32, 32, 50001, true},
                 {WS_DTYPE_F32, 64, 65541, false},  {WS_DTYPE_BF16, 4096, 131073, false}};
    for (const auto& c : cases) {
        ws_rows r = rows();
        r.dtype = c.dtype;
        r.rows = c.rows;
        r.vocab = c.vocab;
        r.row_stride = c.vocab;
        for (int mode : {WS_DISTILL_RENORM, WS_DISTILL_TAIL})
            CHECK((ws::plan_distill(r, mode, true, true).held > 0) == c.held);
    }
}

// The kernels' own exponential against the 80-bit one: its series leaves 5e-18,
// its argument 6e-17, and its last two steps round to 1.6e-16; near 0, and with
// it 1 minus a teacher's probabilities, half a step of the result.
static void exponential() {
    double worst = 0.0;
    for (int i = 0; i <= 288000; ++i) {
        const double x = -200.0 + i * 1e-3;
        const long double want = expl((long double)x);
        const double off = (double)fabsl(((long double)ws::small_exp(x) - want) / want);
        if (off > worst) worst = off;
    }
    CHECK(worst < 3e-16);
    for (double x : {-1e-16, -1e-12, -1e-10, -1e-8, -1e-4, 1e-12, 1e-8})
        CHECK(fabsl((1.0L - ws::small_exp(x)) + expm1l((long double)x)) <= 1.2e-16L);
    CHECK(ws::small_exp(0.0) == 1.0);
    CHECK(ws::small_exp(-200.5) == 0.0);
    CHECK(ws::small_exp(-std::numeric_limits<double>::infinity()) == 0.0);
    CHECK(ws::small_exp(std::numeric_limits<double>::infinity()) ==
          std::numeric_limits<double>::infinity());
    CHECK(std::isnan(ws::small_exp(std::numeric_limits<double>::quiet_NaN())));
}

#define REFUSED(make, check, field, value)             \
    do {                                               \
        ws_rows r = rows();                            \
        auto a = make();                               \
        a.field = value;                               \
        CHECK(check(&r, &a) == WS_E_INVALID_ARG);      \
    } while (0)

static int selftest() {
    using namespace ws;
    const float inf = std::numeric_limits<float>::infinity();
    {
        ws_rows r = rows();
        CHECK(validate_rows(&r) == WS_OK);
        CHECK(validate_rows(nullptr) == WS_E_INVALID_ARG);
#define BAD(field, value)                                \
    do {                                                 \
        ws_rows b = rows();                              \
        b.field = value;                                 \
        CHECK(validate_rows(&b) == WS_E_INVALID_ARG);    \
    } while (0)
        BAD(device, -1);
        BAD(dtype, 3);
        BAD(dtype, -1);
        BAD(rows, -1);
        BAD(rows, WS_MAX_ROWS + 1);
        BAD(vocab, 0);
        BAD(vocab, WS_MAX_SCORES + 1);
        BAD(row_stride, 999);
        BAD(row_stride, 0);
        BAD(row_stride, WS_MAX_ROW_STRIDE + 1);
        BAD(temperature, 0.0f);
        BAD(temperature, -1.0f);
        BAD(temperature, inf);
        BAD(temperature, inf - inf);
        BAD(reserved, 1);
#undef BAD
        r.rows = 0;
        CHECK(validate_rows(&r) == WS_OK);
        r.rows = WS_MAX_ROWS;
        r.vocab = WS_MAX_SCORES;
        r.row_stride = WS_MAX_ROW_STRIDE;
        CHECK(validate_rows(&r) == WS_OK);
        CHECK(rows_extent(r, r.row_stride) > 0);       // no overflow at the limits
    }
    {
        ws_rows r = rows();
        ws_logprobs_args a = logprobs();
        CHECK(validate_logprobs(&r, &a) == WS_OK);
        CHECK(validate_logprobs(&r, nullptr) == WS_E_INVALID_ARG);
        a.targets = nullptr;
        a.logprob = nullptr;
        a.entropy = nullptr;
        a.top = nullptr;
        a.top_k = 0;
        CHECK(validate_logprobs(&r, &a) == WS_OK);     // statistics alone
        a.logits = nullptr;
        CHECK(validate_logprobs(&r, &a) == WS_E_INVALID_ARG);
        r.rows = 0;
        CHECK(validate_logprobs(&r, &a) == WS_OK);     // nothing to read
        REFUSED(logprobs, validate_logprobs, logits, at<void>(0x10001));
        REFUSED(logprobs, validate_logprobs, targets, nullptr);
        REFUSED(logprobs, validate_logprobs, logprob, nullptr);
        REFUSED(logprobs, validate_logprobs, logprob, at<float>(0x81002));
        REFUSED(logprobs, validate_logprobs, entropy, at<float>(0x81001));
        REFUSED(logprobs, validate_logprobs, top, nullptr);
        REFUSED(logprobs, validate_logprobs, top, at<ws_topk_entry>(0x83004));
        REFUSED(logprobs, validate_logprobs, stats, at<ws_row_stats>(0x84004));
        REFUSED(logprobs, validate_logprobs, top_k, 0);
        REFUSED(logprobs, validate_logprobs, top_k, -1);
        REFUSED(logprobs, validate_logprobs, top_k, WS_MAX_K + 1);
        REFUSED(logprobs, validate_logprobs, reserved, 1);
        r = rows();
        r.vocab = 19;                                   // fewer tokens than top_k
        a = logprobs();
        CHECK(validate_logprobs(&r, &a) == WS_E_INVALID_ARG);
        r.vocab = 20;
        CHECK(validate_logprobs(&r, &a) == WS_OK);
        r.dtype = WS_DTYPE_F32;
        a.logits = at<void>(0x10002);
        CHECK(validate_logprobs(&r, &a) == WS_E_INVALID_ARG);
    }
    {
        ws_rows r = rows();
        ws_logprobs_grad_args a = logprobs_grad();
        CHECK(validate_logprobs_grad(&r, &a) == WS_OK);
        CHECK(validate_logprobs_grad(&r, nullptr) == WS_E_INVALID_ARG);
        a.grad_logits = at<void>(0x10000);              // in place: the same stride
        CHECK(validate_logprobs_grad(&r, &a) == WS_E_INVALID_ARG);
        a.grad_stride = r.row_stride;
        CHECK(validate_logprobs_grad(&r, &a) == WS_OK);
        a.grad_logits = at<void>(0x10000 + 2 * 1000);   // beside the logits, in their padding
        CHECK(validate_logprobs_grad(&r, &a) == WS_E_INVALID_ARG);
        a.grad_logits = at<void>(0x10000 - 2);
        CHECK(validate_logprobs_grad(&r, &a) == WS_E_INVALID_ARG);
        a.grad_logits = at<void>(0x10000 + 2 * (7 * 1024 + 1000));   // right behind them
        CHECK(validate_logprobs_grad(&r, &a) == WS_OK);
        r.rows = 1;                                     // one row has no stride
        a = logprobs_grad();
        a.grad_logits = at<void>(0x10000);
        CHECK(validate_logprobs_grad(&r, &a) == WS_OK);
        REFUSED(logprobs_grad, validate_logprobs_grad, logits, nullptr);
        REFUSED(logprobs_grad, validate_logprobs_grad, stats, nullptr);
        REFUSED(logprobs_grad, validate_logprobs_grad, stats, at<ws_row_stats>(0x84004));
        REFUSED(logprobs_grad, validate_logprobs_grad, targets, nullptr);
        REFUSED(logprobs_grad, validate_logprobs_grad, grad_logprob, nullptr);
        REFUSED(logprobs_grad, validate_logprobs_grad, entropy, at<float>(0x1000));
        REFUSED(logprobs_grad, validate_logprobs_grad, grad_entropy, at<float>(0x1000));
        REFUSED(logprobs_grad, validate_logprobs_grad, top, at<ws_topk_entry>(0x1000));
        REFUSED(logprobs_grad, validate_logprobs_grad, grad_top, at<float>(0x1000));
        REFUSED(logprobs_grad, validate_logprobs_grad, top_k, 3);
        REFUSED(logprobs_grad, validate_logprobs_grad, top_k, WS_MAX_K + 1);
        REFUSED(logprobs_grad, validate_logprobs_grad, grad_logits, nullptr);
        REFUSED(logprobs_grad, validate_logprobs_grad, grad_logits, at<void>(0x100001));
        REFUSED(logprobs_grad, validate_logprobs_grad, grad_stride, 999);
        REFUSED(logprobs_grad, validate_logprobs_grad, grad_stride, WS_MAX_ROW_STRIDE + 1);
        REFUSED(logprobs_grad, validate_logprobs_grad, reserved, 1);
    }
    {
        // Rows of logits and of gradients in turn in one buffer: every distance
        // against a count of the elements both hold.
        for (int64_t vocab : {1, 3, 5})
            for (int64_t stride : {5, 8, 10, 11})
                for (int32_t count : {1, 2, 4})
                    for (int64_t gstride : {stride, stride + 1})
                        for (int64_t d = -60; d <= 60; ++d) {
                            ws_rows r = rows();
                            r.rows = count;
                            r.vocab = (int32_t)vocab;
                            r.row_stride = stride;
                            ws_logprobs_grad_args a = logprobs_grad();
                            a.grad_logits = at<void>((uintptr_t)(0x10000 + 2 * d));
                            a.grad_stride = gstride;
                            bool both = false;
                            for (int32_t i = 0; i < count; ++i)
                                for (int32_t j = 0; j < count; ++j) {
                                    const int64_t apart = d + j * gstride - i * stride;
                                    both |= apart < vocab && apart > -vocab;
                                }
                            const int64_t extent = (count - 1) * stride + vocab;
                            const int64_t gextent = (count - 1) * gstride + vocab;
                            const bool meet = d < extent && -d < gextent;
                            const bool ok = d == 0 ? gstride == stride || count == 1
                                            : gstride == stride || count == 1 ? !both : !meet;
                            CHECK((validate_logprobs_grad(&r, &a) == WS_OK) == ok);
                        }
    }
    {
        ws_rows r = rows();
        ws_distill_args a = distill();
        CHECK(validate_distill(&r, &a) == WS_OK);
        CHECK(validate_distill(&r, nullptr) == WS_E_INVALID_ARG);
        a.grad_logits = at<void>(0x100000);
        a.grad_loss = at<float>(0x91000);
        a.grad_stride = 1000;
        CHECK(validate_distill(&r, &a) == WS_OK);
        a.grad_stride = 0;
        CHECK(validate_distill(&r, &a) == WS_E_INVALID_ARG);
        REFUSED(distill, validate_distill, logits, nullptr);
        REFUSED(distill, validate_distill, teacher, nullptr);
        REFUSED(distill, validate_distill, teacher, at<ws_topk_entry>(0x80004));
        REFUSED(distill, validate_distill, loss, nullptr);
        REFUSED(distill, validate_distill, stats, at<ws_row_stats>(0x84004));
        REFUSED(distill, validate_distill, grad_loss, at<float>(0x91000));
        REFUSED(distill, validate_distill, grad_logits, at<void>(0x100000));
        REFUSED(distill, validate_distill, teacher_k, 0);
        REFUSED(distill, validate_distill, teacher_k, WS_DISTILL_MAX_K + 1);
        REFUSED(distill, validate_distill, mode, 2);
        REFUSED(distill, validate_distill, mode, -1);
        REFUSED(distill, validate_distill, reserved[0], 1);
        REFUSED(distill, validate_distill, reserved[1], 1);
        a = distill();
        a.mode = WS_DISTILL_RENORM;
        a.tail = at<float>(0x92000);                    // no tail without WS_DISTILL_TAIL
        CHECK(validate_distill(&r, &a) == WS_E_INVALID_ARG);
    }
    {
        ws_rows r = rows();
        ws_distill_grad_args a = distill_grad();
        CHECK(validate_distill_grad(&r, &a) == WS_OK);
        CHECK(validate_distill_grad(&r, nullptr) == WS_E_INVALID_ARG);
        REFUSED(distill_grad, validate_distill_grad, logits, nullptr);
        REFUSED(distill_grad, validate_distill_grad, teacher, nullptr);
        REFUSED(distill_grad, validate_distill_grad, stats, nullptr);
        REFUSED(distill_grad, validate_distill_grad, tail, nullptr);
        REFUSED(distill_grad, validate_distill_grad, mode, WS_DISTILL_RENORM);   // tail set
        REFUSED(distill_grad, validate_distill_grad, grad_loss, nullptr);
        REFUSED(distill_grad, validate_distill_grad, grad_logits, nullptr);
        REFUSED(distill_grad, validate_distill_grad, grad_logits, at<void>(0x10010));
        REFUSED(distill_grad, validate_distill_grad, teacher_k, 0);
        REFUSED(distill_grad, validate_distill_grad, teacher_k, WS_DISTILL_MAX_K + 1);
    }
    CHECK(validate_workspace(nullptr, 0, 0) == WS_OK);
    CHECK(validate_workspace(nullptr, 64, 64) == WS_E_INVALID_ARG);
    CHECK(validate_workspace(at<void>(0x1000), 63, 64) == WS_E_INVALID_ARG);
    CHECK(validate_workspace(at<void>(0x1008), 64, 64) == WS_E_INVALID_ARG);
    CHECK(validate_workspace(at<void>(0x1000), 64, 64) == WS_OK);
    plans();
    held_rows();
    exponential();
    std::printf("%d failures\n", failures);
    return failures ? 1 : 0;
}

#define F(s, f) std::printf(#s " " #f " %zu\n", offsetof(s, f))
static int layout() {
    std::printf("ws_rows sizeof %zu\n", sizeof(ws_rows));
    F(ws_rows, device); F(ws_rows, dtype); F(ws_rows, rows); F(ws_rows, vocab);
    F(ws_rows, row_stride); F(ws_rows, temperature); F(ws_rows, reserved);
    std::printf("ws_row_stats sizeof %zu\n", sizeof(ws_row_stats));
    F(ws_row_stats, max); F(ws_row_stats, logsum);
    std::printf("ws_logprobs_args sizeof %zu\n", sizeof(ws_logprobs_args));
    F(ws_logprobs_args, logits); F(ws_logprobs_args, targets); F(ws_logprobs_args, logprob);
    F(ws_logprobs_args, entropy); F(ws_logprobs_args, top); F(ws_logprobs_args, stats);
    F(ws_logprobs_args, workspace); F(ws_logprobs_args, workspace_bytes);
    F(ws_logprobs_args, top_k); F(ws_logprobs_args, reserved);
    std::printf("ws_logprobs_grad_args sizeof %zu\n", sizeof(ws_logprobs_grad_args));
    F(ws_logprobs_grad_args, logits); F(ws_logprobs_grad_args, stats);
    F(ws_logprobs_grad_args, targets); F(ws_logprobs_grad_args, grad_logprob);
    F(ws_logprobs_grad_args, entropy); F(ws_logprobs_grad_args, grad_entropy);
    F(ws_logprobs_grad_args, top); F(ws_logprobs_grad_args, grad_top);
    F(ws_logprobs_grad_args, grad_logits); F(ws_logprobs_grad_args, grad_stride);
    F(ws_logprobs_grad_args, top_k); F(ws_logprobs_grad_args, reserved);
    std::printf("ws_distill_args sizeof %zu\n", sizeof(ws_distill_args));
    F(ws_distill_args, logits); F(ws_distill_args, teacher); F(ws_distill_args, loss);
    F(ws_distill_args, stats); F(ws_distill_args, tail); F(ws_distill_args, grad_loss);
    F(ws_distill_args, grad_logits); F(ws_distill_args, grad_stride);
    F(ws_distill_args, workspace); F(ws_distill_args, workspace_bytes);
    F(ws_distill_args, teacher_k); F(ws_distill_args, mode); F(ws_distill_args, reserved);
    std::printf("ws_distill_grad_args sizeof %zu\n", sizeof(ws_distill_grad_args));
    F(ws_distill_grad_args, logits); F(ws_distill_grad_args, teacher);
    F(ws_distill_grad_args, stats); F(ws_distill_grad_args, tail);
    F(ws_distill_grad_args, grad_loss); F(ws_distill_grad_args, grad_logits);
    F(ws_distill_grad_args, grad_stride); F(ws_distill_grad_args, teacher_k);
    F(ws_distill_grad_args, mode);
    return 0;
}

int main(int argc, char** argv) {
    if (argc == 2 && std::strcmp(argv[1], "selftest") == 0) return selftest();
    if (argc == 2 && std::strcmp(argv[1], "layout") == 0) return layout();
    std::fprintf(stderr, "usage: ws_logits_test selftest|layout\n");
    return 2;
}
