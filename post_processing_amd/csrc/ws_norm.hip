// ws_norm.hip -- layer norm forward and backward (ws_states.h), written for
// gfx950 (CDNA4, wave64).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ws_enqueue.h"
#include "ws_lanes.h"
#include "ws_state_slots.h"
#include "ws_states.h"
#include "ws_states_plan.h"

namespace ws {
namespace {

struct NormParams {
    const void* x;
    const void* weight;
    const void* bias;
    void* y;
    ws_norm_stats* stats;
    int64_t x_stride, y_stride;
    int32_t width;
    int32_t weight_f32;
    float inv_width;
    float eps;
};

// One row a workgroup, read again for each of its three passes: the mean, the
// deviations from it, the result.
template <typename L, int NT>
__global__ void __launch_bounds__(NT) norm_long_kernel(NormParams p) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC;
    __shared__ float waves[3][NT / 64];
    const int64_t row = blockIdx.x;
    const Elem* x = static_cast<const Elem*>(p.x) + row * p.x_stride;
    Elem* y = static_cast<Elem*>(p.y) + row * p.y_stride;
    const int first = threadIdx.x * VEC;

    float sum = 0.0f;
    for (int c = first; c < p.width; c += NT * VEC) {
        float v[VEC];
        L::unpack(load_columns<L>(x, c, p.width), v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum += v[j];
    }
    float mean = group_sum<NT>(sum, waves[0]) * p.inv_width;
    // The deviations' own sum takes back the mean's rounding, which a row far
    // from 0 would otherwise carry into its variance and its result.
    float left = 0.0f, square = 0.0f;
    for (int c = first; c < p.width; c += NT * VEC) {
        float v[VEC];
        L::unpack(load_columns<L>(x, c, p.width), v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float d = c + j < p.width ? v[j] - mean : 0.0f;
            left += d;
            square = fmaf(d, d, square);
        }
    }
    const float shift = group_sum<NT>(left, waves[1]) * p.inv_width;
    const float var = fmaxf(group_sum<NT>(square, waves[2]) * p.inv_width - shift * shift, 0.0f);
    const float inverse = 1.0f / sqrtf(var + p.eps);
    if (p.stats && threadIdx.x == 0) p.stats[row] = {mean + shift, inverse};
    for (int c = first; c < p.width; c += NT * VEC) {
        float v[VEC], g[VEC], b[VEC];
        L::unpack(load_columns<L>(x, c, p.width), v);
        if (p.weight) load_either<L>(p.weight, p.weight_f32, c, p.width, g);
        if (p.bias) load_either<L>(p.bias, p.weight_f32, c, p.width, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            v[j] = (v[j] - mean - shift) * inverse;
            if (p.weight) v[j] *= g[j];
            if (p.bias) v[j] += b[j];
        }
        store_columns<L>(y, c, p.width, v);
    }
}

struct NormGradParams {
    const void* x;
    const ws_norm_stats* stats;
    const void* weight;
    const void* grad_y;
    void* grad_x;
    float* partial;      // [groups][2][padded width]
    void* grad_weight;
    void* grad_bias;
    int64_t x_stride, y_stride, grad_stride;
    int64_t partial_stride;
    int32_t rows;
    int32_t width;
    int32_t weight_f32;
    int32_t columns;
    int32_t groups;
    float inv_width;
};

// The gradient of one row a workgroup, in two passes over it.
template <typename L, int NT>
__global__ void __launch_bounds__(NT) norm_grad_long_kernel(NormGradParams p) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC;
    __shared__ float waves[2][NT / 64];
    const int64_t row = blockIdx.x;
    const Elem* x = static_cast<const Elem*>(p.x) + row * p.x_stride;
    const Elem* gy = static_cast<const Elem*>(p.grad_y) + row * p.y_stride;
    Elem* gx = static_cast<Elem*>(p.grad_x) + row * p.grad_stride;
    const ws_norm_stats s = p.stats[row];
    const int first = threadIdx.x * VEC;

    float level = 0.0f, along = 0.0f;
    for (int c = first; c < p.width; c += NT * VEC) {
        float v[VEC], d[VEC], g[VEC];
        L::unpack(load_columns<L>(x, c, p.width), v);
        L::unpack(load_columns<L>(gy, c, p.width), d);
        if (p.weight) load_either<L>(p.weight, p.weight_f32, c, p.width, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if (p.weight) d[j] *= g[j];
            level += d[j];
            along = fmaf(d[j], (v[j] - s.mean) * s.inverse, along);
        }
    }
    level = group_sum<NT>(level, waves[0]) * p.inv_width;
    along = group_sum<NT>(along, waves[1]) * p.inv_width;
    for (int c = first; c < p.width; c += NT * VEC) {
        float v[VEC], d[VEC], g[VEC];
        L::unpack(load_columns<L>(x, c, p.width), v);
        L::unpack(load_columns<L>(gy, c, p.width), d);
        if (p.weight) load_either<L>(p.weight, p.weight_f32, c, p.width, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if (p.weight) d[j] *= g[j];
            const float u = (v[j] - s.mean) * s.inverse;
            d[j] = s.inverse * (d[j] - level - u * along);
        }
        store_columns<L>(gx, c, p.width, d);
    }
}

// Sums over rows: a workgroup's share of the rows for a tile of the columns,
// a slot of columns a thread.
template <typename L, int NT>
__global__ void __launch_bounds__(NT) norm_columns_kernel(NormGradParams p) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC;
    const int tile = blockIdx.x % (uint32_t)p.columns;
    const int64_t group = blockIdx.x / (uint32_t)p.columns;
    const int c = (tile * NT + (int)threadIdx.x) * VEC;
    if (c >= p.width) return;
    const Elem* x = static_cast<const Elem*>(p.x);
    const Elem* gy = static_cast<const Elem*>(p.grad_y);
    float gw[VEC], gb[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) gw[j] = gb[j] = 0.0f;
    for (int64_t row = group; row < p.rows; row += p.groups) {
        const ws_norm_stats s = p.stats[row];
        float v[VEC], d[VEC];
        L::unpack(load_columns<L>(x + row * p.x_stride, c, p.width), v);
        L::unpack(load_columns<L>(gy + row * p.y_stride, c, p.width), d);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            gw[j] = fmaf(d[j], (v[j] - s.mean) * s.inverse, gw[j]);
            gb[j] += d[j];
        }
    }
    float* out = p.partial + group * 2 * p.partial_stride;
    store_either<L>(out, true, c, p.width, gw);
    store_either<L>(out + p.partial_stride, true, c, p.width, gb);
}

// The groups' sums of a column, one column a thread.
template <typename L>
__global__ void __launch_bounds__(kNormThreads) norm_join_kernel(NormGradParams p) {
    const int c = blockIdx.x * kNormThreads + (int)threadIdx.x;
    if (c >= p.width) return;
    float gw = 0.0f, gb = 0.0f;
    for (int g = 0; g < p.groups; ++g) {
        const float* in = p.partial + (int64_t)g * 2 * p.partial_stride + c;
        gw += in[0];
        gb += in[p.partial_stride];
    }
    if (p.grad_weight) {
        if (p.weight_f32) static_cast<float*>(p.grad_weight)[c] = gw;
        else static_cast<typename L::Elem*>(p.grad_weight)[c] = L::down(gw);
    }
    if (p.grad_bias) {
        if (p.weight_f32) static_cast<float*>(p.grad_bias)[c] = gb;
        else static_cast<typename L::Elem*>(p.grad_bias)[c] = L::down(gb);
    }
}

// ---------------------------------------------------------------------------

#define WS_BY_DTYPE(dtype, CALL)                             \
    do {                                                     \
        if ((dtype) == WS_DTYPE_F32) { CALL(F32); }          \
        else if ((dtype) == WS_DTYPE_F16) { CALL(F16); }     \
        else { CALL(BF16); }                                 \
    } while (0)

template <typename L>
int run_norm(const ws_states& t, const NormParams& p, hipStream_t s) {
    return launch(norm_long_kernel<L, kNormThreads>, t.rows, kNormThreads, p, s);
}

template <typename L>
int run_norm_grad(const ws_states& t, const NormGradPlan& plan, const NormGradParams& p,
                  hipStream_t s) {
    // The sums over rows first: grad_x may take the place of x or grad_y.
    if (p.grad_weight || p.grad_bias) {
        int v = launch(norm_columns_kernel<L, kNormThreads>, (int64_t)plan.columns * plan.groups,
                       kNormThreads, p, s);
        if (v != WS_OK) return v;
        v = launch(norm_join_kernel<L>, (p.width + kNormThreads - 1) / kNormThreads, kNormThreads,
                   p, s);
        if (v != WS_OK) return v;
    }
    if (!p.grad_x || t.rows == 0) return WS_OK;
    return launch(norm_grad_long_kernel<L, kNormThreads>, t.rows, kNormThreads, p, s);
}

}  // namespace
}  // namespace ws

extern "C" int ws_layernorm(const ws_states* states, const ws_layernorm_args* args, void* stream) {
    using namespace ws;
    int v = ws::validate_layernorm(states, args);
    if (v != WS_OK) return v;
    if (states->rows == 0) return WS_OK;
    v = ws::device_ready(states->device);
    if (v != WS_OK) return v;
    ws::NormParams p{};
    p.x = args->x;
    p.weight = args->weight;
    p.bias = args->bias;
    p.y = args->y;
    p.stats = args->stats;
    p.x_stride = states->row_stride;
    p.y_stride = args->y_stride;
    p.width = states->width;
    p.weight_f32 = args->weight_dtype == WS_DTYPE_F32;
    p.inv_width = (float)(1.0 / states->width);
    p.eps = args->eps;
    const hipStream_t s = static_cast<hipStream_t>(stream);
#define CALL(L) return run_norm<L>(*states, p, s)
    WS_BY_DTYPE(states->dtype, CALL);
#undef CALL
}

extern "C" int ws_layernorm_grad_workspace(const ws_states* states, size_t* bytes) {
    const int v = ws::validate_states(states);
    if (v != WS_OK) return v;
    if (!bytes) return WS_E_INVALID_ARG;
    *bytes = ws::plan_layernorm_grad(*states).workspace;
    return WS_OK;
}

extern "C" int ws_layernorm_grad(const ws_states* states, const ws_layernorm_grad_args* args,
                                 void* stream) {
    using namespace ws;
    int v = ws::validate_layernorm_grad(states, args);
    if (v != WS_OK) return v;
    const ws::NormGradPlan plan = ws::plan_layernorm_grad(*states);
    const bool sums = args->grad_weight || args->grad_bias;
    v = ws::validate_workspace(args->workspace, args->workspace_bytes, sums ? plan.workspace : 0);
    if (v != WS_OK) return v;
    v = ws::device_ready(states->device);
    if (v != WS_OK) return v;
    ws::NormGradParams p{};
    p.x = args->x;
    p.stats = args->stats;
    p.weight = args->weight;
    p.grad_y = args->grad_y;
    p.grad_x = args->grad_x;
    p.partial = static_cast<float*>(args->workspace);
    p.grad_weight = args->grad_weight;
    p.grad_bias = args->grad_bias;
    p.x_stride = states->row_stride;
    p.y_stride = args->grad_y_stride;
    p.grad_stride = args->grad_x_stride;
    p.partial_stride = (int64_t)(ws::round16((size_t)states->width * 4) / 4);
    p.rows = states->rows;
    p.width = states->width;
    p.weight_f32 = args->weight_dtype == WS_DTYPE_F32;
    p.columns = plan.columns;
    p.groups = plan.groups;
    p.inv_width = (float)(1.0 / states->width);
    const hipStream_t s = static_cast<hipStream_t>(stream);
#define CALL(L) return run_norm_grad<L>(*states, plan, p, s)
    WS_BY_DTYPE(states->dtype, CALL);
#undef CALL
}
