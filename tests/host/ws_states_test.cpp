// Host-only driver for the checks and launch geometry of the operators over
// rows of hidden states (ws_states_plan.h): compiled with g++ and no HIP by
// tests/test_states_host.py.
//   ws_states_test selftest  -> argument checks and plans
//   ws_states_test layout    -> "struct field offset" for the ABI structs
#include <cstddef>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <limits>
#include <vector>

#include "ws_states_plan.h"

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

static const float kInf = std::numeric_limits<float>::infinity();
static const float kNan = std::numeric_limits<float>::quiet_NaN();

static ws_states states() {
    ws_states t;
    std::memset(&t, 0, sizeof t);
    t.dtype = WS_DTYPE_BF16;
    t.rows = 8;
    t.width = 100;
    t.row_stride = 128;
    return t;
}

static ws_embed_args embed() {
    ws_embed_args a;
    std::memset(&a, 0, sizeof a);
    a.table = at<void>(0x100000);
    a.table_stride = 100;
    a.ids = at<int32_t>(0x80000);
    a.out = at<void>(0x10000);
    a.vocab = 50;
    a.scale = 1.0f;
    return a;
}

static ws_embed_grad_args embed_grad() {
    ws_embed_grad_args a;
    std::memset(&a, 0, sizeof a);
    a.grad_out = at<void>(0x10000);
    a.ids = at<int32_t>(0x80000);
    a.grad_table = at<void>(0x100000);
    a.grad_stride = 100;
    a.vocab = 50;
    a.grad_dtype = WS_DTYPE_F32;
    a.scale = 1.0f;
    return a;
}

static ws_layernorm_args norm() {
    ws_layernorm_args a;
    std::memset(&a, 0, sizeof a);
    a.x = at<void>(0x10000);
    a.weight = at<void>(0x80000);
    a.bias = at<void>(0x81000);
    a.y = at<void>(0x20000);
    a.y_stride = 100;
    a.stats = at<ws_norm_stats>(0x82000);
    a.weight_dtype = WS_DTYPE_F32;
    a.eps = 1e-5f;
    return a;
}

static ws_layernorm_grad_args norm_grad() {
    ws_layernorm_grad_args a;
    std::memset(&a, 0, sizeof a);
    a.x = at<void>(0x10000);
    a.stats = at<ws_norm_stats>(0x82000);
    a.weight = at<void>(0x80000);
    a.grad_y = at<void>(0x20000);
    a.grad_y_stride = 100;
    a.grad_x = at<void>(0x30000);
    a.grad_x_stride = 100;
    a.grad_weight = at<void>(0x83000);
    a.grad_bias = at<void>(0x84000);
    a.weight_dtype = WS_DTYPE_F32;
    return a;
}

template <typename A, typename F>
static bool refused(int (*validate)(const ws_states*, const A*), A a, F change) {
    ws_states t = states();
    change(t, a);
    return validate(&t, &a) == WS_E_INVALID_ARG;
}

template <typename A, typename F>
static bool taken(int (*validate)(const ws_states*, const A*), A a, F change) {
    ws_states t = states();
    change(t, a);
    return validate(&t, &a) == WS_OK;
}

#define NO(V, A, ...) \
    CHECK(refused(ws::V, A(), [](ws_states& t, auto& a) { (void)t; (void)a; __VA_ARGS__; }))
#define YES(V, A, ...) \
    CHECK(taken(ws::V, A(), [](ws_states& t, auto& a) { (void)t; (void)a; __VA_ARGS__; }))

template <typename A>
static void shapes(int (*validate)(const ws_states*, const A*), A a) {
    CHECK(validate(nullptr, &a) == WS_E_INVALID_ARG);
    const ws_states good = states();
    CHECK(validate(&good, nullptr) == WS_E_INVALID_ARG);
    CHECK(validate(&good, &a) == WS_OK);
    const auto bad = [&](auto change) {
        ws_states t = states();
        change(t);
        CHECK(validate(&t, &a) == WS_E_INVALID_ARG);
    };
    bad([](ws_states& t) { t.device = -1; });
    bad([](ws_states& t) { t.dtype = 3; });
    bad([](ws_states& t) { t.dtype = -1; });
    bad([](ws_states& t) { t.rows = -1; });
    bad([](ws_states& t) { t.rows = WS_MAX_ROWS + 1; });
    bad([](ws_states& t) { t.width = 0; });
    bad([](ws_states& t) { t.width = WS_MAX_WIDTH + 1; });
    bad([](ws_states& t) { t.row_stride = 99; });
    bad([](ws_states& t) { t.row_stride = WS_MAX_ROW_STRIDE + 1; });
}

static void test_embed() {
    shapes(ws::validate_embed, embed());
    NO(validate_embed, embed, a.vocab = 0);
    NO(validate_embed, embed, a.vocab = WS_MAX_TOKENS + 1);
    NO(validate_embed, embed, a.table_stride = 99);
    NO(validate_embed, embed, a.scale = kInf);
    NO(validate_embed, embed, a.scale = kNan);
    NO(validate_embed, embed, a.table = nullptr);
    NO(validate_embed, embed, a.ids = nullptr);
    NO(validate_embed, embed, a.out = nullptr);
    NO(validate_embed, embed, a.table = at<void>(0x100001));
    NO(validate_embed, embed, a.out = at<void>(0x10001));
    NO(validate_embed, embed, a.ids = at<int32_t>(0x80002));
    YES(validate_embed, embed, a.out = at<void>(0x10002));
    NO(validate_embed, embed, a.out = at<void>(0x100000 - 200));     // the last rows reach in
    NO(validate_embed, embed, a.out = at<void>(0x80000 - 16));       // over the indices
    YES(validate_embed, embed, t.rows = 0; a.table = nullptr; a.out = nullptr; a.ids = nullptr);
    NO(validate_embed, embed, t.rows = 0; a.vocab = 0);
    YES(validate_embed, embed, t.row_stride = WS_MAX_ROW_STRIDE; t.rows = 1);
}

static void test_embed_grad() {
    shapes(ws::validate_embed_grad, embed_grad());
    NO(validate_embed_grad, embed_grad, a.vocab = 0);
    NO(validate_embed_grad, embed_grad, a.vocab = WS_MAX_TOKENS + 1);
    NO(validate_embed_grad, embed_grad, a.grad_stride = 99);
    NO(validate_embed_grad, embed_grad, a.scale = -kInf);
    NO(validate_embed_grad, embed_grad, a.grad_dtype = WS_DTYPE_F16);
    YES(validate_embed_grad, embed_grad, a.grad_dtype = WS_DTYPE_BF16);
    NO(validate_embed_grad, embed_grad, a.accumulate = 2);
    NO(validate_embed_grad, embed_grad, a.grad_table = nullptr);
    NO(validate_embed_grad, embed_grad, a.grad_table = at<void>(0x100002));
    NO(validate_embed_grad, embed_grad, a.grad_out = nullptr);
    NO(validate_embed_grad, embed_grad, a.grad_out = at<void>(0x10001));
    NO(validate_embed_grad, embed_grad, a.ids = nullptr);
    NO(validate_embed_grad, embed_grad, a.grad_table = at<void>(0x10000));
    YES(validate_embed_grad, embed_grad, t.rows = 0; a.grad_out = nullptr; a.ids = nullptr);
    NO(validate_embed_grad, embed_grad, t.rows = 0; a.grad_table = nullptr);
}

static void test_norm() {
    shapes(ws::validate_layernorm, norm());
    NO(validate_layernorm, norm, a.weight_dtype = WS_DTYPE_F16);
    YES(validate_layernorm, norm, a.weight_dtype = WS_DTYPE_BF16);
    NO(validate_layernorm, norm, a.y_stride = 99);
    NO(validate_layernorm, norm, a.eps = -1e-9f);
    NO(validate_layernorm, norm, a.eps = kInf);
    NO(validate_layernorm, norm, a.eps = kNan);
    YES(validate_layernorm, norm, a.eps = 0.0f);
    NO(validate_layernorm, norm, a.x = nullptr);
    NO(validate_layernorm, norm, a.y = nullptr);
    YES(validate_layernorm, norm, a.weight = nullptr; a.bias = nullptr; a.stats = nullptr);
    NO(validate_layernorm, norm, a.weight = at<void>(0x80002));
    NO(validate_layernorm, norm, a.bias = at<void>(0x81001));
    NO(validate_layernorm, norm, a.stats = at<ws_norm_stats>(0x82004));
    YES(validate_layernorm, norm, a.y = at<void>(0x10000); a.y_stride = 128);
    NO(validate_layernorm, norm, a.y = at<void>(0x10000));            // another stride
    YES(validate_layernorm, norm, a.y = at<void>(0x10000); t.rows = 1);
    NO(validate_layernorm, norm, a.y = at<void>(0x10002); a.y_stride = 128);
    YES(validate_layernorm, norm, t.row_stride = 200; a.y_stride = 200; a.y = at<void>(0x10000 + 200));
    NO(validate_layernorm, norm, t.row_stride = 200; a.y_stride = 200; a.y = at<void>(0x10000 + 198));
    NO(validate_layernorm, norm, t.row_stride = 200; a.y_stride = 200; a.y = at<void>(0x10000 + 202));
    NO(validate_layernorm, norm, a.stats = at<ws_norm_stats>(0x20000));
    NO(validate_layernorm, norm, a.stats = at<ws_norm_stats>(0x10000));
    NO(validate_layernorm, norm, a.weight = at<void>(0x20000));
    YES(validate_layernorm, norm, t.rows = 0; a.x = nullptr; a.y = nullptr);
    NO(validate_layernorm, norm, t.rows = 0; a.eps = -1.0f);
}

static void test_norm_grad() {
    shapes(ws::validate_layernorm_grad, norm_grad());
    NO(validate_layernorm_grad, norm_grad, a.reserved = 1);
    NO(validate_layernorm_grad, norm_grad, a.weight_dtype = WS_DTYPE_F16);
    NO(validate_layernorm_grad, norm_grad, a.grad_y_stride = 99);
    NO(validate_layernorm_grad, norm_grad, a.grad_x_stride = 99);
    YES(validate_layernorm_grad, norm_grad, a.grad_x = nullptr; a.grad_x_stride = 0);
    NO(validate_layernorm_grad, norm_grad, a.grad_x = nullptr; a.grad_weight = nullptr;
       a.grad_bias = nullptr);
    YES(validate_layernorm_grad, norm_grad, a.grad_weight = nullptr; a.grad_bias = nullptr);
    NO(validate_layernorm_grad, norm_grad, a.x = nullptr);
    NO(validate_layernorm_grad, norm_grad, a.stats = nullptr);
    NO(validate_layernorm_grad, norm_grad, a.stats = at<ws_norm_stats>(0x82004));
    NO(validate_layernorm_grad, norm_grad, a.grad_y = nullptr);
    YES(validate_layernorm_grad, norm_grad, a.weight = nullptr);
    YES(validate_layernorm_grad, norm_grad, a.grad_x = at<void>(0x20000));
    YES(validate_layernorm_grad, norm_grad, a.grad_x = at<void>(0x10000); a.grad_x_stride = 128);
    NO(validate_layernorm_grad, norm_grad, a.grad_x = at<void>(0x10000));
    NO(validate_layernorm_grad, norm_grad, a.grad_bias = at<void>(0x83000));
    NO(validate_layernorm_grad, norm_grad, a.grad_bias = at<void>(0x80000));
    NO(validate_layernorm_grad, norm_grad, a.grad_weight = at<void>(0x30000));
    NO(validate_layernorm_grad, norm_grad, a.grad_weight = at<void>(0x83002));
    YES(validate_layernorm_grad, norm_grad, t.rows = 0; a.x = nullptr; a.stats = nullptr;
        a.grad_y = nullptr; a.grad_x = nullptr);
    NO(validate_layernorm_grad, norm_grad, t.rows = 0; a.grad_x = nullptr; a.grad_weight = nullptr;
       a.grad_bias = nullptr);
}

// The extents' rule against every byte of small matrices.
static void test_disjoint() {
    const auto bytes = [](const ws::Extent& e, std::vector<int>& mark, int as) {
        bool met = false;
        for (int64_t r = 0; r < e.rows; ++r)
            for (int64_t i = 0; i < e.width * 2; ++i) {
                int& m = mark[e.begin() + r * e.stride * 2 + i];
                met |= m != 0 && m != as;
                m = as;
            }
        return met;
    };
    for (int64_t sa : {3, 4, 7})
        for (int64_t sb : {3, 4, 7})
            for (int64_t wa : {1, 2, 3})
                for (int64_t wb : {1, 3})
                    for (int64_t ra : {0, 1, 3})
                        for (int64_t rb : {1, 4})
                            for (uintptr_t b = 2; b < 120; b += 2) {
                                const ws::Extent x = {at<void>(60), ra, wa, sa, WS_DTYPE_BF16};
                                const ws::Extent y = {at<void>(b), rb, wb, sb, WS_DTYPE_BF16};
                                std::vector<int> mark(400, 0);
                                bytes(x, mark, 1);
                                const bool met = bytes(y, mark, 2);
                                CHECK(ws::disjoint(x, y) == ws::disjoint(y, x));
                                if (ws::disjoint(x, y)) CHECK(!met);
                                // Equal strides and enough rows: exactly.
                                if (!met && (sa == sb || ra == 0)) CHECK(ws::disjoint(x, y) || ra == 1 || rb == 1);
                            }
}

// An array against a matrix's rows, exactly: between them, over them, and behind the
// last one.
static void test_array_and_matrix() {
    for (int64_t rows : {1, 2, 3})
        for (int64_t width : {1, 3, 5})
            for (int64_t stride : {5, 8})
                for (int64_t n : {1, 2, 3, 4, 9, 40})
                    for (uintptr_t b = 4; b < 240; b += 2)
                        for (int32_t dtype : {WS_DTYPE_BF16, WS_DTYPE_F32}) {
                            const ws::Extent m = {at<void>(100), rows, width, stride, WS_DTYPE_BF16};
                            const ws::Extent array = {at<void>(b), 1, n, n, dtype};
                            const uintptr_t end = b + (uintptr_t)(n * ws::logit_bytes(dtype));
                            bool met = false;
                            for (int64_t r = 0; r < rows; ++r) {
                                const uintptr_t from = 100 + (uintptr_t)(r * stride * 2);
                                met |= b < from + (uintptr_t)(width * 2) && from < end;
                            }
                            CHECK(ws::disjoint(m, array) == !met);
                            CHECK(ws::disjoint(array, m) == !met);
                        }
    // Through the calls: indices, statistics and weights in the rows' padding.
    YES(validate_embed, embed, a.ids = at<int32_t>(0x10000 + 200));
    NO(validate_embed, embed, a.ids = at<int32_t>(0x10000 + 196));
    NO(validate_embed, embed, a.ids = at<int32_t>(0x10000 + 228));
    YES(validate_layernorm, norm, t.row_stride = 400; t.rows = 3; a.y_stride = 400;
        a.stats = at<ws_norm_stats>(0x20000 + 200); a.weight = at<void>(0x20000 + 224));
    NO(validate_layernorm, norm, t.row_stride = 400; t.rows = 3; a.y_stride = 400;
       a.weight = at<void>(0x20000 + 404));
    YES(validate_layernorm_grad, norm_grad, t.row_stride = 400; a.grad_weight = at<void>(0x10000 + 200));
    NO(validate_layernorm_grad, norm_grad, t.row_stride = 400; a.grad_weight = at<void>(0x10000 + 404));
}

// A workspace over a call's buffers, byte by byte around each of them.
static void test_workspaces_lie_apart() {
    const ws_states t = states();
    const auto around = [](uintptr_t from, uintptr_t bytes, size_t needed, auto validate) {
        for (const uintptr_t b : {from - needed, from + (bytes + 15) / 16 * 16})
            CHECK(validate(b) == WS_OK);
        for (const uintptr_t b : {from - needed + 16, from, from + (bytes - 1) / 16 * 16})
            CHECK(validate(b) == WS_E_INVALID_ARG);
    };
    const size_t needed = 0x1000;
    const uintptr_t rows = (7 * 128 + 100) * 2;
    const auto embed = [&](uintptr_t b) {
        ws_embed_grad_args a = embed_grad();
        a.workspace = at<void>(b);
        a.workspace_bytes = needed;
        return ws::validate_embed_grad_workspace(t, a, needed);
    };
    around(0x10000, rows, needed, embed);                  // grad_out
    around(0x80000, 8 * 4, needed, embed);                 // ids
    around(0x100000, 50 * 100 * 4, needed, embed);         // grad_table
    ws_embed_grad_args none = embed_grad();
    CHECK(ws::validate_embed_grad_workspace(t, none, needed) == WS_E_INVALID_ARG);
    CHECK(ws::validate_embed_grad_workspace(t, none, 0) == WS_OK);
    // In the rows' padding, and a workspace larger than needed, whose rest is not used.
    ws_states wide = states();
    wide.row_stride = 0x2000;
    none.workspace = at<void>(0x10000 + 0x100);
    none.workspace_bytes = 0x100000;
    CHECK(ws::validate_embed_grad_workspace(wide, none, needed) == WS_OK);
    CHECK(ws::validate_embed_grad_workspace(wide, none, 0x4000) == WS_E_INVALID_ARG);

    const auto norm = [&](uintptr_t b) {
        ws_layernorm_grad_args a = norm_grad();
        a.grad_weight = at<void>(0x50000);                 // apart from each other by more
        a.grad_bias = at<void>(0x60000);                   // than the workspace
        a.stats = at<ws_norm_stats>(0x70000);
        a.workspace = at<void>(b);
        a.workspace_bytes = needed;
        return ws::validate_layernorm_grad_workspace(t, a, needed);
    };
    around(0x10000, rows, needed, norm);                   // x
    around(0x20000, (7 * 100 + 100) * 2, needed, norm);    // grad_y
    around(0x30000, (7 * 100 + 100) * 2, needed, norm);    // grad_x
    around(0x50000, 400, needed, norm);
    around(0x60000, 400, needed, norm);
    around(0x70000, 64, needed, norm);                     // stats
    around(0x80000, 400, needed, norm);                    // weight
    ws_layernorm_grad_args parts = norm_grad();            // what is left out is nowhere
    parts.grad_x = parts.grad_bias = nullptr;
    parts.weight = nullptr;
    parts.workspace = at<void>(0x80000 - needed + 0x100);
    parts.workspace_bytes = needed;
    CHECK(ws::validate_layernorm_grad_workspace(t, parts, needed) == WS_OK);
}

static void test_plans() {
    for (int32_t dtype : {WS_DTYPE_F32, WS_DTYPE_F16, WS_DTYPE_BF16})
        for (int64_t rows : {1ll, 2ll, 31ll, 2048ll, 2049ll, 100000ll, 1ll << 22})
            for (int32_t width : {1, 7, 8, 9, 64, 1000, 4096, 65537, WS_MAX_WIDTH}) {
                ws_states t = states();
                t.dtype = dtype;
                t.rows = (int32_t)rows;
                t.width = width;
                t.row_stride = width;
                const ws::EmbedPlan e = ws::plan_embed(t);
                CHECK(e.lanes <= ws::kLookupThreads && (e.lanes & (e.lanes - 1)) == 0);
                CHECK(e.groups * (ws::kLookupThreads / e.lanes) >= rows && e.groups < (1ll << 31));
                for (int32_t vocab : {1, 2, 511, 512, 262143, 262144, WS_MAX_TOKENS}) {
                    const ws::EmbedGradPlan g = ws::plan_embed_grad(t, vocab);
                    CHECK(vocab >> (g.passes * ws::kDigitBits) == 0);
                    CHECK((int64_t)g.tiles * ws::kSortTile >= rows);
                    CHECK((int64_t)g.blocks * g.block >= rows && (int64_t)(g.blocks - 1) * g.block < rows);
                    CHECK((int64_t)g.blocks * g.columns < (1ll << 31));
                    CHECK(g.lanes >= ws::kLeastLanes && ws::kSumThreads % g.lanes == 0);
                    CHECK(g.block * (ws::kSumThreads / g.lanes) <= ws::kMostRows);
                    CHECK((int64_t)g.lanes * g.columns >= ws::slots_in(t.width, t.dtype));
                    CHECK(!g.few || (rows <= ws::kFewRows && rows * g.columns <= ws::kFewGroups));
                    CHECK(g.keys_at[1] % 16 == 0 && g.rows_at[1] % 16 == 0 && g.counts_at % 16 == 0 &&
                          g.partial_at % 16 == 0);
                }
                const ws::NormPlan f = ws::plan_layernorm(t);
                CHECK(f.held == 0 || (f.groups >= 1 && f.groups <= rows));
                const ws::NormGradPlan n = ws::plan_layernorm_grad(t);
                CHECK(n.groups >= 1 && n.groups <= rows);
                CHECK(n.held == 0 || (n.row_groups >= n.groups && n.row_groups <= rows));
                CHECK(n.workspace >= (size_t)n.groups * 2 * 4 * (size_t)width);
                CHECK(n.held == 0 || (int64_t)n.threads * n.held >= ws::slots_in(t.width, t.dtype));
            }
}

// Which launches the GPU tests' sizes take, so that each path stays tested: how many
// tiles sort, the rows of a block, and the workgroups over a row.
static void test_paths() {
    struct Path { int32_t rows, width, dtype; bool few; int32_t tiles, block, columns; };
    const Path paths[] = {
        {150, 5000, WS_DTYPE_BF16, true, 1, 0, 0},     {203, 67, WS_DTYPE_BF16, true, 1, 0, 0},
        {700, 520, WS_DTYPE_BF16, true, 1, 0, 0},      {777, 1000, WS_DTYPE_F32, true, 1, 0, 0},
        {1025, 5000, WS_DTYPE_BF16, false, 1, 8, 3},   {1025, 5000, WS_DTYPE_F32, false, 1, 10, 5},
        {1025, 1, WS_DTYPE_BF16, false, 1, 8, 1},      {1100, 67, WS_DTYPE_F16, false, 1, 8, 1},
        {2100, 67, WS_DTYPE_F32, false, 2, 8, 1},      {4500, 67, WS_DTYPE_BF16, false, 3, 8, 1},
        {1100, 20, WS_DTYPE_F32, false, 1, 8, 1},      {3000, 20, WS_DTYPE_F32, false, 2, 8, 1},
        {5000, 20, WS_DTYPE_F32, false, 3, 8, 1},      {1100, 300, WS_DTYPE_F32, false, 1, 8, 1},
        {5000, 300, WS_DTYPE_F16, false, 3, 8, 1},     {2100, 2051, WS_DTYPE_F32, false, 2, 12, 3},
        {5000, 2051, WS_DTYPE_F32, false, 3, 29, 3},   {16384, 2100, WS_DTYPE_BF16, false, 8, 32, 2},
        {262200, 1032, WS_DTYPE_BF16, false, 129, 33, 1}, {1500, 520, WS_DTYPE_BF16, false, 1, 8, 1},
        {2100, 520, WS_DTYPE_BF16, false, 2, 8, 1},    {5000, 520, WS_DTYPE_BF16, false, 3, 8, 1},
        {140000, 40, WS_DTYPE_BF16, false, 69, 8, 1},
    };
    for (const Path& path : paths) {
        ws_states t = states();
        t.rows = path.rows;
        t.width = t.row_stride = path.width;
        t.dtype = path.dtype;
        const ws::EmbedGradPlan p = ws::plan_embed_grad(t, 900);
        CHECK(p.few == path.few && p.tiles == path.tiles);
        if (!p.few) CHECK(p.block == path.block && p.columns == path.columns);
    }
}

static void layout() {
#define SIZE(T) std::printf(#T " sizeof %zu\n", sizeof(T))
#define FIELD(T, f) std::printf(#T " " #f " %zu\n", offsetof(T, f))
    SIZE(ws_states);
    FIELD(ws_states, device); FIELD(ws_states, dtype); FIELD(ws_states, rows);
    FIELD(ws_states, width); FIELD(ws_states, row_stride);
    SIZE(ws_norm_stats);
    FIELD(ws_norm_stats, mean); FIELD(ws_norm_stats, inverse);
    SIZE(ws_embed_args);
    FIELD(ws_embed_args, table); FIELD(ws_embed_args, table_stride); FIELD(ws_embed_args, ids);
    FIELD(ws_embed_args, out); FIELD(ws_embed_args, vocab); FIELD(ws_embed_args, scale);
    SIZE(ws_embed_grad_args);
    FIELD(ws_embed_grad_args, grad_out); FIELD(ws_embed_grad_args, ids);
    FIELD(ws_embed_grad_args, grad_table); FIELD(ws_embed_grad_args, grad_stride);
    FIELD(ws_embed_grad_args, workspace); FIELD(ws_embed_grad_args, workspace_bytes);
    FIELD(ws_embed_grad_args, vocab); FIELD(ws_embed_grad_args, grad_dtype);
    FIELD(ws_embed_grad_args, accumulate); FIELD(ws_embed_grad_args, scale);
    SIZE(ws_layernorm_args);
    FIELD(ws_layernorm_args, x); FIELD(ws_layernorm_args, weight); FIELD(ws_layernorm_args, bias);
    FIELD(ws_layernorm_args, y); FIELD(ws_layernorm_args, y_stride);
    FIELD(ws_layernorm_args, stats); FIELD(ws_layernorm_args, weight_dtype);
    FIELD(ws_layernorm_args, eps);
    SIZE(ws_layernorm_grad_args);
    FIELD(ws_layernorm_grad_args, x); FIELD(ws_layernorm_grad_args, stats);
    FIELD(ws_layernorm_grad_args, weight); FIELD(ws_layernorm_grad_args, grad_y);
    FIELD(ws_layernorm_grad_args, grad_y_stride); FIELD(ws_layernorm_grad_args, grad_x);
    FIELD(ws_layernorm_grad_args, grad_x_stride); FIELD(ws_layernorm_grad_args, grad_weight);
    FIELD(ws_layernorm_grad_args, grad_bias); FIELD(ws_layernorm_grad_args, workspace);
    FIELD(ws_layernorm_grad_args, workspace_bytes); FIELD(ws_layernorm_grad_args, weight_dtype);
    FIELD(ws_layernorm_grad_args, reserved);
}

int main(int argc, char** argv) {
    if (argc == 2 && !std::strcmp(argv[1], "layout")) {
        layout();
        return 0;
    }
    test_embed();
    test_embed_grad();
    test_norm();
    test_norm_grad();
    test_disjoint();
    test_array_and_matrix();
    test_workspaces_lie_apart();
    test_plans();
    test_paths();
    std::printf("%d failures\n", failures);
    return failures != 0;
}
