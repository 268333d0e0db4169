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
    int32_t rows;
    int32_t width;
    int32_t weight_f32;
    float inv_width;
    float eps;
};

// A row's mean and deviation from its slots in registers.  The mean is summed
// first and the deviations from it after, never squares of far-off values; and the
// deviations' own sum takes back the mean's rounding, which a row far from 0 would
// otherwise carry into its variance and its result.
//
// Rows up to 65,536 bytes: the next row is on its way while one is worked on,
// weights stay in registers but for 1,024 threads' four 16-bit slots (8,200 BF16
// elements: 80 us for 8,183 rows with them read again, 57 with 512 threads' three
// slots and theirs; 32,768 elements: 105 us for 2,048 with 512 threads, 74), and each
// element is read and written once (counted: 134.6 MB read, 134.8 written for 16,384
// x 4,096 BF16).  HBM bounds it: 52.6 us for that, 5.1 TB/s, where a large copy runs at
// 4.9; three passes over the row in a workgroup a row took 75.7.  (Slots read and
// written past the caches, which carry the gradient of rows of logits to 6 TB/s, have
// not been tried here.)  64 rows take 3.9 us: a launch, one row's latency and two sums
// over four waves.
// NT threads to a row; rows of less than a wave's slots lie side by side in one,
// whose lanes would else be idle (200,000 x 256 BF16 68 us with a wave a row, 40 with
// two rows a wave).
constexpr int group_threads(int nt) { return nt < 64 ? 64 : nt; }

// A product that its uses all see rounded: fused into a subtraction here and not
// there, the mean would be two numbers, and the deviations' sum that of one of them.
__device__ __forceinline__ float rounded(float v) {
    asm volatile("" : "+v"(v));
    return v;
}

// A row's statistics from its first mean and the sums of the deviations from it and of
// their squares: `shift` takes back the first mean's rounding.  Comparisons keep what the
// formulas carry: the variance of a row that holds a NaN or an infinity is NaN (where a
// maximum with 0 would make it 0), and the mean of one whose infinities have one sign is
// that infinity, not its sum with deviations' that are NaN.
__device__ __forceinline__ ws_norm_stats row_stats(float mean, float left, float square,
                                                   const NormParams& p, float& shift) {
    shift = left * p.inv_width;
    const float var = square * p.inv_width - shift * shift;
    const float inverse = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + p.eps);
    return {__builtin_isnan(shift) ? mean : mean + shift, inverse};
}

// Has the compiler unpack the slots again instead of keeping twice the registers
// (4,096 x 32,768 BF16 142 us, 154 unpacked).
template <int R>
__device__ __forceinline__ void stay_packed(uint4 (&w)[R]) {
#pragma unroll
    for (int i = 0; i < R; ++i)
        asm volatile("" : "+v"(w[i].x), "+v"(w[i].y), "+v"(w[i].z), "+v"(w[i].w));
}

template <typename L, int NT, int R>
__global__ void __launch_bounds__(group_threads(NT)) norm_kernel(NormParams p) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC;
    constexpr bool kHold = NT <= 512 || R * VEC <= 16;   // the weights too
    constexpr int kRows = group_threads(NT) / NT;   // side by side
    __shared__ float first[kRows > 1 ? 1 : NT / 64];
    __shared__ float2 second[kRows > 1 ? 1 : NT / 64];
    const HeldSlots<L, NT, R> slots(p.width);
    const Elem* x = static_cast<const Elem*>(p.x);
    Elem* y = static_cast<Elem*>(p.y);
    float g[kHold ? R : 1][VEC], b[kHold ? R : 1][VEC];
    if constexpr (kHold) {
        slots.weights(p.weight, p.weight_f32, 1.0f, g);
        slots.weights(p.bias, p.weight_f32, 0.0f, b);
    }
    uint4 w[R];
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / NT;
    slots.load(x + (row < p.rows ? row : p.rows - 1) * p.x_stride, w);
    // (a row side by side with the last one may lie behind it)
    for (int64_t base = (int64_t)blockIdx.x * kRows; base < p.rows; base += step, row += step) {
        uint4 own[R];
#pragma unroll
        for (int i = 0; i < R; ++i) own[i] = w[i];
        const int64_t next = row + step;
        slots.load(x + (next < p.rows ? next : p.rows - 1) * p.x_stride, w);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float v[VEC];
            L::unpack(own[i], v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += slots.mine(i, j) ? v[j] : 0.0f;
        }
        const float mean = rounded(group_sum<NT>(sum, first) * p.inv_width);
        if constexpr (!kHold) stay_packed(own);
        float2 far = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float v[VEC];
            L::unpack(own[i], v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = slots.mine(i, j) ? v[j] - mean : 0.0f;
                far.x += d;
                far.y = fmaf(d, d, far.y);
            }
        }
        far = group_sums<NT>(far, second);
        if constexpr (!kHold) stay_packed(own);
        float shift;
        const ws_norm_stats stats = row_stats(mean, far.x, far.y, p, shift);
        const float inverse = stats.inverse;
        if (kRows > 1 && row >= p.rows) continue;
        if (p.stats && threadIdx.x % NT == 0) p.stats[row] = stats;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (!slots.any(i)) continue;
            float v[VEC], g_own[VEC], b_own[VEC];
            L::unpack(own[i], v);
            if constexpr (!kHold) {
                if (p.weight) load_either<L>(p.weight, p.weight_f32, slots.at[i], p.width, g_own);
                if (p.bias) load_either<L>(p.bias, p.weight_f32, slots.at[i], p.width, b_own);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                v[j] = (v[j] - mean - shift) * inverse;
                if constexpr (kHold) {
                    v[j] = fmaf(v[j], g[i][j], b[i][j]);
                } else {
                    if (p.weight) v[j] *= g_own[j];
                    if (p.bias) v[j] += b_own[j];
                }
            }
            store_loose<L>(y + row * p.y_stride + slots.at[i], L::pack(v));
        }
    }
}

// Longer rows, and those of less than a slot: one a workgroup (of one wave for those
// of less than a slot), read again for each of its three passes, which for the most
// part come from the caches (2,048 x 65,536 BF16 163 us, 3.3 TB/s).
template <typename L, int NT>
__global__ void __launch_bounds__(NT) norm_long_kernel(NormParams p) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC;
    __shared__ float waves[3][NT / 64];
    const int64_t row = (int64_t)blockIdx.y * kLongGroups + blockIdx.x;
    if (row >= p.rows) return;
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
    const float mean = rounded(group_sum<NT>(sum, waves[0]) * p.inv_width);
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
    left = group_sum<NT>(left, waves[1]);
    square = group_sum<NT>(square, waves[2]);
    float shift;
    const ws_norm_stats stats = row_stats(mean, left, square, p, shift);
    const float inverse = stats.inverse;
    if (p.stats && threadIdx.x == 0) p.stats[row] = stats;
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

// The sum over a wave's lanes NT apart, in each of them.
template <int NT>
__device__ __forceinline__ float apart_sum(float v) {
    const int lane = threadIdx.x & 63;
    if constexpr (NT <= 8) v += xor_lane_f<8>(v, lane);
    if constexpr (NT <= 16) v += xor_lane_f<16>(v, lane);
    return v + xor_lane_f<32>(v, lane);
}

// Rows held as norm_kernel's: grad_x, and in registers the workgroup's rows'
// sums for the weight's and the bias's gradient, which it leaves in the workspace.
// SUMS: with those.  One pass over x and grad_y serves both: 16,384 x 4,096 BF16
// 75 us (5.4 TB/s; 269.7 MB read, 151.0 written, 16.8 of them the workgroups' sums)
// and 5 for joining the sums; with a kernel for each, 219 in all.
template <typename L, int NT, int R, bool SUMS>
__global__ void __launch_bounds__(group_threads(NT)) norm_grad_kernel(NormGradParams p) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC;
    constexpr int kRows = group_threads(NT) / NT;
    __shared__ float2 waves[2][kRows > 1 ? 1 : NT / 64];
    const HeldSlots<L, NT, R> slots(p.width);
    const Elem* x = static_cast<const Elem*>(p.x);
    const Elem* gy = static_cast<const Elem*>(p.grad_y);
    float g[R][VEC], gw[SUMS ? R : 1][VEC], gb[SUMS ? R : 1][VEC];
    slots.weights(p.weight, p.weight_f32, 1.0f, g);
    if constexpr (SUMS) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) gw[i][j] = gb[i][j] = 0.0f;
    }
    uint4 wx[R], wy[R];
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / NT;
    int64_t next = row < p.rows ? row : p.rows - 1;
    slots.load(x + next * p.x_stride, wx);
    slots.load(gy + next * p.y_stride, wy);
    ws_norm_stats ahead = p.stats[next];
    int turn = 0;
    for (int64_t base = (int64_t)blockIdx.x * kRows; base < p.rows; base += step, row += step) {
        float u[R][VEC], d[R][VEC];
        const ws_norm_stats s = ahead;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            L::unpack(wx[i], u[i]);
            L::unpack(wy[i], d[i]);
        }
        next = row + step < p.rows ? row + step : p.rows - 1;
        slots.load(x + next * p.x_stride, wx);
        slots.load(gy + next * p.y_stride, wy);
        ahead = p.stats[next];
        float2 sums = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                u[i][j] = (u[i][j] - s.mean) * s.inverse;
                if constexpr (SUMS) {
                    if (kRows > 1 && row >= p.rows) continue;
                    gw[i][j] = fmaf(d[i][j], u[i][j], gw[i][j]);
                    gb[i][j] += d[i][j];
                }
                d[i][j] *= g[i][j];
                const float m = slots.mine(i, j) ? d[i][j] : 0.0f;
                sums.x += m;
                sums.y += slots.mine(i, j) ? m * u[i][j] : 0.0f;
            }
        if (!p.grad_x) continue;
        sums = group_sums<NT>(sums, waves[turn]);
        turn ^= 1;
        if (kRows > 1 && row >= p.rows) continue;
        const float level = sums.x * p.inv_width, along = sums.y * p.inv_width;
        Elem* gx = static_cast<Elem*>(p.grad_x) + row * p.grad_stride;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (!slots.any(i)) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                d[i][j] = s.inverse * (d[i][j] - level - u[i][j] * along);
            store_loose<L>(gx + slots.at[i], L::pack(d[i]));
        }
    }
    if constexpr (SUMS) {
        float* out = p.partial + (int64_t)blockIdx.x * 2 * p.partial_stride;
        if constexpr (kRows > 1) {   // the rows side by side
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    gw[i][j] = apart_sum<NT>(gw[i][j]);
                    gb[i][j] = apart_sum<NT>(gb[i][j]);
                }
            if (threadIdx.x >= NT) return;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (!slots.any(i)) continue;
            store_either<L>(out, true, slots.at[i], p.width, gw[i]);
            store_either<L>(out + p.partial_stride, true, slots.at[i], p.width, gb[i]);
        }
    }
}

// The gradient of one longer row a workgroup, in two passes over it.
template <typename L, int NT>
__global__ void __launch_bounds__(NT) norm_grad_long_kernel(NormGradParams p) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC;
    __shared__ float waves[2][NT / 64];
    const int64_t row = (int64_t)blockIdx.y * kLongGroups + blockIdx.x;
    if (row >= p.rows) return;
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
    constexpr int U = 4;   // rows on their way
    for (int64_t row = group; row < p.rows; row += U * p.groups) {
        uint4 wx[U], wy[U];
        ws_norm_stats s[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t at = row + i * p.groups < p.rows ? row + i * p.groups : row;
            wx[i] = load_columns<L>(x + at * p.x_stride, c, p.width);
            wy[i] = load_columns<L>(gy + at * p.y_stride, c, p.width);
            s[i] = p.stats[at];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (row + i * p.groups >= p.rows) break;
            float v[VEC], d[VEC];
            L::unpack(wx[i], v);
            L::unpack(wy[i], d);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                gw[j] = fmaf(d[j], (v[j] - s[i].mean) * s[i].inverse, gw[j]);
                gb[j] += d[j];
            }
        }
    }
    float* out = p.partial + group * 2 * p.partial_stride;
    store_either<L>(out, true, c, p.width, gw);
    store_either<L>(out + p.partial_stride, true, c, p.width, gb);
}

// The groups' sums of a column: 64 columns a workgroup, whose 64 shares of
// sixteen lanes take the groups in turn, four columns a lane.
constexpr int kJoinThreads = 1024, kJoinColumns = 64, kJoinShares = kJoinThreads / 16;

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

template <int J>
__device__ __forceinline__ float4 xor_lane4(float4 v, int lane) {
    return make_float4(xor_lane_f<J>(v.x, lane), xor_lane_f<J>(v.y, lane),
                       xor_lane_f<J>(v.z, lane), xor_lane_f<J>(v.w, lane));
}

template <typename L>
__global__ void __launch_bounds__(kJoinThreads) norm_join_kernel(NormGradParams p) {
    constexpr int U = 8;   // loads in flight
    __shared__ float4 part[kJoinThreads / 64][16];
    const int lane = threadIdx.x % 16u, share = threadIdx.x / 16u;
    const int tiles = (p.width + kJoinColumns - 1) / kJoinColumns;
    const bool bias = (int)blockIdx.x >= tiles;
    const int c = ((int)blockIdx.x - (bias ? tiles : 0)) * kJoinColumns + lane * 4;
    const float* in = p.partial + (bias ? p.partial_stride : 0) + c;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < p.width) {   // a row of the workspace is whole in fours
        for (int from = share; from < p.groups; from += U * kJoinShares) {
            float4 v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int g = from + i * kJoinShares < p.groups ? from + i * kJoinShares : from;
                v[i] = *reinterpret_cast<const float4*>(in + (int64_t)g * 2 * p.partial_stride);
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (from + i * kJoinShares < p.groups) sum = add4(sum, v[i]);
        }
    }
    sum = add4(sum, xor_lane4<16>(sum, threadIdx.x & 63));
    sum = add4(sum, xor_lane4<32>(sum, threadIdx.x & 63));
    if ((threadIdx.x & 63) < 16) part[threadIdx.x >> 6][lane] = sum;
    __syncthreads();
    if (share != 0) return;
    sum = part[0][lane];
#pragma unroll
    for (int i = 1; i < kJoinThreads / 64; ++i) sum = add4(sum, part[i][lane]);
    void* out = bias ? p.grad_bias : p.grad_weight;
    if (!out) return;
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (c + j < p.width) {
            if (p.weight_f32) static_cast<float*>(out)[c + j] = v[j];
            else static_cast<typename L::Elem*>(out)[c + j] = L::down(v[j]);
        }
}

// ---------------------------------------------------------------------------

// A workgroup a row.  A side of a grid has less than 2^32 threads, which 2^22 rows
// of 1,024 would not be.
dim3 long_grid(int64_t rows) {
    return rows <= kLongGroups ? dim3((uint32_t)rows)
                               : dim3(kLongGroups, (uint32_t)((rows + kLongGroups - 1) / kLongGroups));
}

template <typename L>
int run_norm(const ws_states& t, const NormParams& p, hipStream_t s) {
    const NormPlan plan = plan_layernorm(t);
#define PICK(NT, R)                           \
    if (plan.threads == NT && plan.held == R) \
    return launch(norm_kernel<L, NT, R>, plan.groups, group_threads(NT), p, s)
    PICK(8, 1);
    PICK(16, 1);
    PICK(32, 1);
    PICK(64, 1);
    PICK(64, 2);
    PICK(192, 1);
    PICK(256, 1);
    PICK(256, 2);
    PICK(256, 3);
    PICK(512, 2);
    PICK(512, 3);
    PICK(512, 6);
    PICK(1024, 2);
    PICK(1024, 4);
#undef PICK
    const dim3 grid = long_grid(t.rows);
    if (t.width < L::VEC) return launch_grid(norm_long_kernel<L, 64>, grid, 64, p, s);
    return launch_grid(norm_long_kernel<L, kLongThreads>, grid, kLongThreads, p, s);
}

template <typename L, bool SUMS>
int run_norm_grad_held(const NormGradPlan& plan, const NormGradParams& p, hipStream_t s) {
    const int64_t groups = SUMS ? plan.groups : plan.row_groups;
#define PICK(NT, R)                                  \
    if (plan.threads == NT && plan.held == R)        \
    return launch(norm_grad_kernel<L, NT, R, SUMS>, groups, group_threads(NT), p, s)
    PICK(8, 1);
    PICK(16, 1);
    PICK(32, 1);
    PICK(64, 1);
    PICK(64, 2);
    PICK(256, 1);
    PICK(256, 2);
    PICK(256, 3);
    PICK(512, 2);
    PICK(512, 3);
    if constexpr (L::VEC == 4) {   // of 16 bits they would not fit the registers
        PICK(512, 5);
        PICK(512, 6);
        PICK(512, 8);
    }
#undef PICK
    return launch(norm_grad_kernel<L, 512, 4, SUMS>, groups, 512, p, s);
}

template <typename L>
int run_norm_grad(const ws_states& t, const NormGradPlan& plan, const NormGradParams& p,
                  hipStream_t s) {
    const bool sums = p.grad_weight || p.grad_bias;
    int v = WS_OK;
    if (t.rows > 0 && plan.held > 0) {
        v = sums ? run_norm_grad_held<L, true>(plan, p, s) : run_norm_grad_held<L, false>(plan, p, s);
    } else if (t.rows > 0) {
        // The sums over rows first: grad_x may take the place of x or grad_y.
        if (sums)
            v = launch(norm_columns_kernel<L, kNormThreads>, (int64_t)plan.columns * plan.groups,
                       kNormThreads, p, s);
        const dim3 grid = long_grid(t.rows);
        if (v == WS_OK && p.grad_x)
            v = t.width < L::VEC
                    ? launch_grid(norm_grad_long_kernel<L, 64>, grid, 64, p, s)
                    : launch_grid(norm_grad_long_kernel<L, kLongThreads>, grid, kLongThreads, p, s);
    }
    if (v != WS_OK || !sums) return v;
    return launch(norm_join_kernel<L>, 2 * ((p.width + kJoinColumns - 1) / kJoinColumns),
                  kJoinThreads, p, s);
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
    p.rows = states->rows;
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
    v = ws::validate_layernorm_grad_workspace(*states, *args, sums ? plan.workspace : 0);
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
