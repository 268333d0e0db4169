// Host-only driver for the checks and launch geometry of sampling
// (ws_logits_plan.h): compiled with g++ and no HIP by tests/test_sample_host.py.
//   ws_sample_test selftest  -> argument checks and plans
//   ws_sample_test layout    -> "struct field offset" for the ABI structs
#include <cstddef>
#include <cstdio>
#include <cstring>
#include <initializer_list>

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

static ws_sample_args sample() {
    ws_sample_args a;
    std::memset(&a, 0, sizeof a);
    a.logits = at<void>(0x10000);
    a.uniform = at<float>(0x80000);
    a.temperature = at<float>(0x81000);
    a.top_k = at<int32_t>(0x82000);
    a.top_p = at<float>(0x83000);
    a.min_p = at<float>(0x84000);
    a.token = at<int32_t>(0x85000);
    a.logprob = at<float>(0x86000);
    return a;
}

template <typename F>
static int with(F change) {
    ws_rows r = rows();
    ws_sample_args a = sample();
    change(r, a);
    return ws::validate_sample(&r, &a);
}

#define NO(...) \
    CHECK(with([](ws_rows& r, ws_sample_args& a) { (void)r; (void)a; __VA_ARGS__; }) == WS_E_INVALID_ARG)
#define YES(...) \
    CHECK(with([](ws_rows& r, ws_sample_args& a) { (void)r; (void)a; __VA_ARGS__; }) == WS_OK)

static void test_arguments() {
    const ws_rows r = rows();
    const ws_sample_args a = sample();
    CHECK(ws::validate_sample(nullptr, &a) == WS_E_INVALID_ARG);
    CHECK(ws::validate_sample(&r, nullptr) == WS_E_INVALID_ARG);
    YES();
    YES(a.temperature = nullptr; a.top_k = nullptr; a.top_p = nullptr; a.min_p = nullptr;
        a.logprob = nullptr);
    NO(a.logits = nullptr);
    NO(a.uniform = nullptr);
    NO(a.token = nullptr);
    NO(a.logits = at<void>(0x10001));
    YES(a.logits = at<void>(0x10002));
    NO(a.uniform = at<float>(0x80002));
    NO(a.temperature = at<float>(0x81002));
    NO(a.top_k = at<int32_t>(0x82001));
    NO(a.top_p = at<float>(0x83003));
    NO(a.min_p = at<float>(0x84002));
    NO(a.token = at<int32_t>(0x85002));
    NO(a.logprob = at<float>(0x86001));
    NO(r.temperature = 0.0f);          // the rows' own must hold, array or not
    NO(r.rows = -1);
    NO(r.vocab = 0);
    NO(r.row_stride = 999);
    YES(r.rows = 0; std::memset(&a, 0, sizeof a));
}

// Outputs and the workspace over each other buffer of the call, and beside it.
static void test_buffers_lie_apart() {
    const uintptr_t inputs[][2] = {{0x10000, 7 * 2048 + 2000}, {0x80000, 32}, {0x81000, 32},
                                   {0x82000, 32}, {0x83000, 32}, {0x84000, 32}};
    for (const auto& in : inputs) {
        const uintptr_t first = in[0], end = in[0] + in[1];
        for (const uintptr_t b : {first - 28, first, end - 4}) {
            CHECK(with([&](ws_rows&, ws_sample_args& a) { a.token = at<int32_t>(b); }) == WS_E_INVALID_ARG);
            CHECK(with([&](ws_rows&, ws_sample_args& a) { a.logprob = at<float>(b); }) == WS_E_INVALID_ARG);
        }
        for (const uintptr_t b : {first - 32, end}) {
            CHECK(with([&](ws_rows&, ws_sample_args& a) { a.token = at<int32_t>(b); }) == WS_OK);
            CHECK(with([&](ws_rows&, ws_sample_args& a) { a.logprob = at<float>(b); }) == WS_OK);
        }
    }
    NO(a.logprob = at<float>(0x85000));                    // the tokens
    NO(a.logprob = at<float>(0x85000 + 28));
    YES(a.logprob = at<float>(0x85000 + 32));
    YES(a.temperature = a.top_p = a.min_p = a.uniform);    // inputs may be one array
    YES(a.logits = at<void>(0x80000));                     // and lie in each other
    YES(a.token = at<int32_t>(0x10000 + 2000));            // the last row ends before the
    NO(a.token = at<int32_t>(0x10000 + 2020));             // padding's 48 bytes do
    NO(r.rows = 100; r.row_stride = 1000; a.token = at<int32_t>(0x10000 + 2000));

    const ws_rows r = rows();
    const size_t needed = 0x400;
    const auto workspace = [&](uintptr_t b) {
        ws_sample_args a = sample();
        a.workspace = at<void>(b);
        a.workspace_bytes = needed;
        return ws::validate_sample_workspace(r, a, needed);
    };
    for (const uintptr_t first : {0x10000, 0x80000, 0x81000, 0x82000, 0x83000, 0x84000, 0x85000, 0x86000}) {
        CHECK(workspace(first) == WS_E_INVALID_ARG);
        CHECK(workspace(first - needed + 16) == WS_E_INVALID_ARG);
        CHECK(workspace(first - needed) == WS_OK);
    }
    CHECK(workspace(0x85000 + 32) == WS_OK);
    CHECK(workspace(0x10000 + 7 * 2048 + 2000) == WS_OK);
    ws_sample_args few = sample();
    few.logprob = nullptr;
    few.temperature = nullptr;
    few.workspace = at<void>(0x86000 - needed + 16);
    few.workspace_bytes = needed;
    CHECK(ws::validate_sample_workspace(r, few, needed) == WS_OK);
    few.workspace = nullptr;
    CHECK(ws::validate_sample_workspace(r, few, needed) == WS_E_INVALID_ARG);
    CHECK(ws::validate_sample_workspace(r, few, 0) == WS_OK);
}

static void test_plans() {
    for (int32_t dtype : {WS_DTYPE_F32, WS_DTYPE_F16, WS_DTYPE_BF16})
        for (int64_t count : {1ll, 2ll, 15ll, 16ll, 17ll, 64ll, 256ll, 257ll, 512ll, 513ll, 1ll << 22})
            for (int32_t vocab : {1, 7, 8, 9, 8192, 8193, 24576, 49152, 49160, 131072, 200003, 1 << 30}) {
                ws_rows r = rows();
                r.dtype = dtype;
                r.rows = (int32_t)count;
                r.vocab = vocab;
                r.row_stride = vocab;
                const ws::SamplePlan p = ws::plan_sample(r);
                CHECK(p.threads == 256 || p.threads == 512 || p.threads == 1024);
                CHECK(p.parts >= 1 && p.parts <= ws::kMaxSampleParts);
                CHECK(count * p.parts < (1ll << 31));
                CHECK((int64_t)p.chunk * p.parts <= ws::slots_of(r));
                CHECK(ws::slots_of(r) - (int64_t)p.chunk * p.parts < p.parts);
                CHECK(p.parts == 1 || p.chunk >= ws::kSampleSlots);
                CHECK(p.workspace == (p.parts > 1 ? (size_t)count * p.parts * 4 * ws::kStretchBytes : 0));
                // The sum of a row's weights in fixed point fits 63 bits.
                CHECK(p.unit >= 32 && p.unit <= 62 && ((int64_t)vocab << p.unit) > 0);
                CHECK(((int64_t)vocab << p.unit) <= (1ll << 62));
            }
}

// The threads of a row's workgroup, on both sides of each border of the rule.
static void test_threads() {
    struct Rule { int32_t rows, vocab, dtype, threads; };
    const Rule rules[] = {
        {1, 8192, WS_DTYPE_BF16, 256},      {5000, 4096, WS_DTYPE_F32, 256},
        {256, 8193, WS_DTYPE_BF16, 1024},   {256, 200003, WS_DTYPE_F16, 1024},
        {257, 8193, WS_DTYPE_BF16, 512},    {300, 50001, WS_DTYPE_F32, 512},
        {512, 131072, WS_DTYPE_BF16, 512},  {512, 65536, WS_DTYPE_F32, 512},
        {512, 131073, WS_DTYPE_BF16, 1024}, {300, 65537, WS_DTYPE_F32, 1024},
        {257, 200003, WS_DTYPE_F16, 1024},  {513, 65536, WS_DTYPE_BF16, 512},
        {513, 65537, WS_DTYPE_BF16, 1024},  {1024, 131072, WS_DTYPE_BF16, 1024},
    };
    for (const Rule& rule : rules) {
        ws_rows r = rows();
        r.rows = rule.rows;
        r.vocab = rule.vocab;
        r.row_stride = rule.vocab;
        r.dtype = rule.dtype;
        CHECK(ws::plan_sample(r).threads == rule.threads);
    }
}

static void layout() {
#define FIELD(f) std::printf("ws_sample_args " #f " %zu\n", offsetof(ws_sample_args, f))
    std::printf("ws_sample_args sizeof %zu\n", sizeof(ws_sample_args));
    FIELD(logits); FIELD(uniform); FIELD(temperature); FIELD(top_k); FIELD(top_p); FIELD(min_p);
    FIELD(token); FIELD(logprob); FIELD(workspace); FIELD(workspace_bytes);
}

int main(int argc, char** argv) {
    if (argc == 2 && !std::strcmp(argv[1], "layout")) {
        layout();
        return 0;
    }
    test_arguments();
    test_buffers_lie_apart();
    test_plans();
    test_threads();
    std::printf("%d failures\n", failures);
    return failures != 0;
}
