// ws_logits.hip -- the operators over rows of logits (ws_logits.h), written
// for gfx950 (CDNA4, wave64): one workgroup a row.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "ws_lanes.h"
#include "ws_logits.h"
#include "ws_logits_plan.h"

namespace ws {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f;
// A finite stand-in below every difference z - max that matters: at the
// highest temperature exp((z - max) / tau) is 0 from -1.04e5 on, and 0 times a
// finite number is 0 where 0 times -inf would be NaN.
constexpr float kFar = -1.0e6f;

struct F32 {
    using type = float;
    static __device__ __forceinline__ float load(const void* p, int64_t i) {
        return static_cast<const float*>(p)[i];
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, float v) {
        static_cast<float*>(p)[i] = v;
    }
};

struct F16 {
    using type = uint16_t;
    static __device__ __forceinline__ float load(const void* p, int64_t i) {
        return (float)static_cast<const _Float16*>(p)[i];
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, float v) {
        static_cast<_Float16*>(p)[i] = (_Float16)v;
    }
};

// Round to nearest even; a NaN stays one.
__device__ __forceinline__ uint16_t bf16_bits(float v) {
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7fffffffu) > 0x7f800000u) return (uint16_t)((u >> 16) | 0x40u);
    return (uint16_t)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

struct BF16 {
    using type = uint16_t;
    static __device__ __forceinline__ float load(const void* p, int64_t i) {
        return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, float v) {
        static_cast<uint16_t*>(p)[i] = bf16_bits(v);
    }
};

// Order-preserving unsigned image of an FP32 value: NaN -> -inf and -0 -> +0
// first, then larger values have larger images.
__device__ __forceinline__ uint32_t order_image(float v) {
    uint32_t b = __float_as_uint(v);
    b = (b & 0x7fffffffu) > 0x7f800000u ? 0xff800000u : b;
    b = b == 0x80000000u ? 0u : b;
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// (value descending, index ascending) as one integer, larger = better; 0 is
// below every key.
__device__ __forceinline__ uint64_t order_key(float v, uint32_t index) {
    return ((uint64_t)order_image(v) << 32) | (uint32_t)~index;
}

template <typename T, typename Op>
__device__ __forceinline__ T wave_reduce(T v, int lane, Op op) {
    if constexpr (sizeof(T) == 8) {
        v = op(v, xor_lane64<32>(v, lane));
        v = op(v, xor_lane64<16>(v, lane));
        v = op(v, xor_lane64<8>(v, lane));
        v = op(v, xor_lane64<4>(v, lane));
        v = op(v, xor_lane64<2>(v, lane));
        v = op(v, xor_lane64<1>(v, lane));
    } else {
        v = op(v, __uint_as_float(xor_lane32<32>(__float_as_uint(v), lane)));
        v = op(v, __uint_as_float(xor_lane32<16>(__float_as_uint(v), lane)));
        v = op(v, __uint_as_float(xor_lane32<8>(__float_as_uint(v), lane)));
        v = op(v, __uint_as_float(xor_lane32<4>(__float_as_uint(v), lane)));
        v = op(v, __uint_as_float(xor_lane32<2>(__float_as_uint(v), lane)));
        v = op(v, __uint_as_float(xor_lane32<1>(__float_as_uint(v), lane)));
    }
    return v;
}

// The same result in every thread of the workgroup; scratch holds one T per
// wave and may be reused after the call.
template <typename T, typename Op>
__device__ __forceinline__ T group_reduce(T v, T* scratch, Op op) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = wave_reduce(v, lane, op);
    if (lane == 0) scratch[wave] = v;
    __syncthreads();
    T r = scratch[0];
    for (int w = 1; w < kThreads / 64; ++w) r = op(r, scratch[w]);
    __syncthreads();
    return r;
}

struct AddF {
    __device__ float operator()(float a, float b) const { return a + b; }
};
struct MaxF {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct MaxKey {
    __device__ uint64_t operator()(uint64_t a, uint64_t b) const { return umax64(a, b); }
};

__device__ __forceinline__ bool listed(const uint32_t* ids, int k, uint32_t j) {
    for (int i = 0; i < k; ++i)
        if (ids[i] == j) return true;
    return false;
}

// Row sums with respect to the row's maximum m (-FLT_MAX or more, so that a
// difference from it is never inf - inf in a row without +inf):
//   s = sum e_j, u = sum e_j (z_j - m), e_j = 2^((z_j - m) c), c = log2(e) / tau.
struct Sums {
    float m, s, u;
};

template <typename L>
__device__ Sums row_sums(const void* logits, int64_t at, int V, float c, const uint32_t* ids,
                         int k, float* scratch) {
    float m = -FLT_MAX;
    for (int j = threadIdx.x; j < V; j += kThreads)
        if (!listed(ids, k, j)) m = fmaxf(m, L::load(logits, at + j));
    m = group_reduce(m, scratch, MaxF());
    float s = 0.0f, u = 0.0f;
    for (int j = threadIdx.x; j < V; j += kThreads) {
        if (listed(ids, k, j)) continue;
        const float d = L::load(logits, at + j) - m;
        const float e = __builtin_amdgcn_exp2f(d * c);
        s += e;
        u += e * fmaxf(d, kFar);
    }
    Sums r;
    r.m = m;
    r.s = group_reduce(s, scratch, AddF());
    r.u = group_reduce(u, scratch, AddF());
    return r;
}

struct LogprobsParams {
    const void* logits;
    int64_t stride;
    const int32_t* targets;
    float* logprob;
    float* entropy;
    ws_topk_entry* top;
    ws_row_stats* stats;
    int32_t vocab;
    int32_t k;
    float c;         // log2(e) / tau
    float inv_tau;
};

template <typename L>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(LogprobsParams p) {
    __shared__ float scratch[kThreads / 64];
    __shared__ uint64_t keys[kThreads / 64];
    const int64_t row = blockIdx.x;
    const int64_t at = row * p.stride;
    const Sums r = row_sums<L>(p.logits, at, p.vocab, p.c, nullptr, 0, scratch);
    const bool empty = r.s == 0.0f;
    const float logsum = empty ? -INFINITY : logf(r.s);
    if (threadIdx.x == 0) {
        if (p.stats) p.stats[row] = {empty ? -INFINITY : r.m, logsum};
        if (p.entropy) p.entropy[row] = empty ? 0.0f : logsum - r.u * p.inv_tau / r.s;
        if (p.logprob) {
            const int32_t t = p.targets[row];
            float v = 0.0f;
            if (t >= 0 && t < p.vocab)
                v = empty ? -INFINITY : (L::load(p.logits, at + t) - r.m) * p.inv_tau - logsum;
            else if (t != -1)
                v = NAN;
            p.logprob[row] = v;
        }
    }
    uint64_t bound = ~0ull;
    for (int i = 0; i < p.k; ++i) {
        uint64_t best = 0;
        for (int j = threadIdx.x; j < p.vocab; j += kThreads) {
            const uint64_t key = order_key(L::load(p.logits, at + j), (uint32_t)j);
            if (key < bound) best = umax64(best, key);
        }
        bound = group_reduce(best, keys, MaxKey());
        if (threadIdx.x == 0) {
            const int32_t j = (int32_t)~(uint32_t)bound;
            const float v =
                empty ? -INFINITY : (L::load(p.logits, at + j) - r.m) * p.inv_tau - logsum;
            p.top[row * p.k + i] = {v, j};
        }
    }
}

struct GradParams {
    const void* logits;
    void* grad;
    int64_t stride, grad_stride;
    const ws_row_stats* stats;
    const ws_topk_entry* entries;   // alternatives, or the teacher's entries
    const float* grad_entries;      // [rows][k] upstream of the alternatives
    const int32_t* targets;
    const float* grad_target;       // [rows]
    const float* entropy;
    const float* grad_entropy;
    const float* tail;              // distillation
    const float* grad_loss;
    int32_t vocab;
    int32_t k;
    int32_t mode;
    float c, inv_tau;
};

// A distillation row's teacher entries in LDS.
struct Teacher {
    uint32_t ids[WS_DISTILL_MAX_K];   // 0xffffffff: absent
    double q[WS_DISTILL_MAX_K];
    double logq[WS_DISTILL_MAX_K];
    double rest;                      // q_t
    double mass;                      // M
    int distinct;
    bool bad;                         // an index outside the row
};

__device__ void read_teacher(const ws_topk_entry* e, int k, int mode, int V, Teacher* t) {
    for (int i = threadIdx.x; i < k; i += kThreads) {
        t->ids[i] = (uint32_t)e[i].index;
        t->logq[i] = (double)e[i].score;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        t->bad = false;
        t->distinct = 0;
        double high = -INFINITY;
        for (int i = 0; i < k; ++i) {
            if (t->ids[i] == 0xffffffffu) continue;
            if (t->ids[i] >= (uint32_t)V) t->bad = true;
            if (!listed(t->ids, i, t->ids[i])) ++t->distinct;
            if (!(t->logq[i] <= high)) high = t->logq[i];
        }
        double sum = 0.0;
        const double shift = mode == WS_DISTILL_RENORM && high != -INFINITY ? high : 0.0;
        for (int i = 0; i < k; ++i) {
            t->q[i] = t->ids[i] == 0xffffffffu ? 0.0 : exp(t->logq[i] - shift);
            sum += t->q[i];
        }
        t->rest = 0.0;
        t->mass = sum;
        if (mode == WS_DISTILL_RENORM) {
            if (sum != 0.0) {
                for (int i = 0; i < k; ++i) {
                    t->q[i] /= sum;
                    t->logq[i] -= shift + log(sum);
                }
                t->mass = sum / sum;
            }
        } else if (t->distinct < V) {
            t->rest = sum < 1.0 ? 1.0 - sum : 0.0;
            t->mass = sum + t->rest;
        }
    }
    __syncthreads();
}

struct DistillParams {
    const void* logits;
    int64_t stride;
    const ws_topk_entry* teacher;
    float* loss;
    ws_row_stats* stats;
    float* tail;
    int32_t vocab, k, mode;
    float c, inv_tau;
};

template <typename L>
__global__ void __launch_bounds__(kThreads) distill_kernel(DistillParams p) {
    __shared__ float scratch[kThreads / 64];
    __shared__ Teacher t;
    const int64_t row = blockIdx.x;
    const int64_t at = row * p.stride;
    read_teacher(p.teacher + row * p.k, p.k, p.mode, p.vocab, &t);
    const bool tail_mode = p.mode == WS_DISTILL_TAIL;
    // The unlisted tokens' sums apart from the listed ones', so that a small
    // tail is summed, never the difference of two sums near 1.
    const Sums r = row_sums<L>(p.logits, at, p.vocab, p.c, t.ids, tail_mode ? p.k : 0, scratch);
    if (threadIdx.x != 0) return;
    float m = r.m, s = r.s;
    if (tail_mode && !t.bad) {
        for (int i = 0; i < p.k; ++i)
            if (t.ids[i] != 0xffffffffu) m = fmaxf(m, L::load(p.logits, at + t.ids[i]));
        s = s == 0.0f ? 0.0f : s * __builtin_amdgcn_exp2f((r.m - m) * p.c);
        for (int i = 0; i < p.k; ++i)
            if (t.ids[i] != 0xffffffffu && !listed(t.ids, i, t.ids[i]))
                s += __builtin_amdgcn_exp2f((L::load(p.logits, at + t.ids[i]) - m) * p.c);
    }
    const bool empty = s == 0.0f;
    const double logsum = empty ? -INFINITY : log((double)s);
    const double tail = r.s == 0.0f ? -(double)INFINITY
                                    : ((double)r.m - (double)m) * p.inv_tau + log((double)r.s) - logsum;
    double loss = 0.0;
    for (int i = 0; i < p.k && !t.bad; ++i) {
        if (t.q[i] == 0.0) continue;
        const double logp =
            empty ? -(double)INFINITY
                  : ((double)L::load(p.logits, at + t.ids[i]) - (double)m) * p.inv_tau - logsum;
        loss += t.q[i] * (t.logq[i] - logp);
    }
    if (t.rest > 0.0) loss += t.rest * (log(t.rest) - tail);
    p.loss[row] = t.bad ? NAN : (float)loss;
    if (p.stats) p.stats[row] = {empty ? -INFINITY : m, t.bad ? NAN : (float)logsum};
    if (p.tail) p.tail[row] = (float)tail;
}

// dz_j = p_j (a + b log p_j) for most tokens of a row; the few that a target,
// an alternative or a teacher entry names get their own term on top.
template <typename L, bool DISTILL>
__global__ void __launch_bounds__(kThreads) grad_kernel(GradParams p) {
    __shared__ Teacher t;
    const int64_t row = blockIdx.x;
    const int64_t at = row * p.stride, to = row * p.grad_stride;
    const ws_row_stats st = p.stats[row];
    if (st.logsum == -INFINITY) {
        for (int j = threadIdx.x; j < p.vocab; j += kThreads) L::store(p.grad, to + j, 0.0f);
        return;
    }
    float a = 0.0f, b = 0.0f, scale = p.inv_tau;
    int target = -1;
    float gt = 0.0f;
    // log2 of the sum that p's exponent is measured against.  An unlisted token
    // of a row with a tail uses the unlisted tokens' own, so that a tail too
    // small for FP32 still divides: p_j (M - q_t / p_t) = p_j / p_t (M p_t - q_t).
    float base = st.logsum * kLog2e;
    const float listed_base = base;
    float a_listed = 0.0f;
    if constexpr (DISTILL) {
        read_teacher(p.entries + row * p.k, p.k, p.mode, p.vocab, &t);
        a = a_listed = (float)t.mass;
        if (p.mode == WS_DISTILL_TAIL && t.rest > 0.0) {
            const double tail = (double)p.tail[row];
            a = tail == -INFINITY ? 0.0f : (float)(t.mass * exp(tail) - t.rest);
            if (tail != -INFINITY) base = (float)(((double)st.logsum + tail) * 1.4426950408889634074);
        }
        scale *= p.grad_loss[row];
        if (t.bad) a = NAN;
    } else {
        for (int i = threadIdx.x; i < p.k; i += kThreads)
            t.ids[i] = (uint32_t)p.entries[row * p.k + i].index;
        __syncthreads();
        for (int i = 0; i < p.k; ++i) {
            if (t.ids[i] == 0xffffffffu) continue;
            a -= p.grad_entries[row * p.k + i];
            if (t.ids[i] >= (uint32_t)p.vocab) a = NAN;
        }
        if (p.targets) {
            target = p.targets[row];
            if (target != -1) {
                gt = p.grad_target[row];
                a -= gt;
                if (target < 0 || target >= p.vocab) a = NAN;
            }
        }
        if (p.entropy) {
            const float gh = p.grad_entropy[row];
            b = -gh;
            a -= gh * p.entropy[row];
        }
    }
    for (int j = threadIdx.x; j < p.vocab; j += kThreads) {
        const float d = L::load(p.logits, at + j) - st.max;
        float v = a;
        if (b != 0.0f) v += b * fmaxf(d * p.inv_tau - st.logsum, kFar);
        float extra = 0.0f;
        bool named = false;
        for (int i = 0; i < p.k; ++i)
            if (t.ids[i] == (uint32_t)j) {
                named = true;
                extra += DISTILL ? -(float)t.q[i] : p.grad_entries[row * p.k + i];
            }
        if (DISTILL && named) v = a_listed;
        const float prob =
            __builtin_amdgcn_exp2f(d * p.c - (DISTILL && named ? listed_base : base));
        if (!DISTILL && j == target) extra += gt;
        v = prob * v + extra;
        L::store(p.grad, to + j, v * scale);
    }
}

// ---------------------------------------------------------------------------

int device_ready(int32_t device) {
    int ndev = 0;
    if (hipGetDeviceCount(&ndev) != hipSuccess || device >= ndev) return WS_E_NO_DEVICE;
    int cur = -1;
    if (hipGetDevice(&cur) != hipSuccess) return WS_E_HIP;
    return cur == device ? WS_OK : WS_E_INVALID_ARG;
}

#define WS_BY_DTYPE(dtype, CALL)                        \
    do {                                                \
        if ((dtype) == WS_DTYPE_F32) { CALL(F32); }     \
        else if ((dtype) == WS_DTYPE_F16) { CALL(F16); } \
        else { CALL(BF16); }                            \
    } while (0)

int launched() { return hipGetLastError() == hipSuccess ? WS_OK : WS_E_HIP; }

float scale_c(const ws_rows& r) { return (float)(1.4426950408889634074 / (double)r.temperature); }
float scale_inv(const ws_rows& r) { return (float)(1.0 / (double)r.temperature); }

int run_distill_grad(const ws_rows& r, const GradParams& g, hipStream_t s) {
#define CALL(L) grad_kernel<L, true><<<r.rows, kThreads, 0, s>>>(g)
    WS_BY_DTYPE(r.dtype, CALL);
#undef CALL
    return launched();
}

}  // namespace
}  // namespace ws

extern "C" int ws_logprobs_workspace(const ws_rows* rows, int32_t top_k, size_t* bytes) {
    const int v = ws::validate_rows(rows);
    if (v != WS_OK) return v;
    if (!bytes || ws::validate_top_k(*rows, top_k) != WS_OK) return WS_E_INVALID_ARG;
    *bytes = 0;
    return WS_OK;
}

extern "C" int ws_logprobs(const ws_rows* rows, const ws_logprobs_args* args, void* stream) {
    int v = ws::validate_logprobs(rows, args);
    if (v != WS_OK) return v;
    if (rows->rows == 0) return WS_OK;
    v = ws::device_ready(rows->device);
    if (v != WS_OK) return v;
    const ws_rows& r = *rows;
    ws::LogprobsParams p{args->logits, r.row_stride, args->targets, args->logprob, args->entropy,
                         args->top, args->stats, r.vocab, args->top_k, ws::scale_c(r),
                         ws::scale_inv(r)};
    const hipStream_t s = static_cast<hipStream_t>(stream);
#define CALL(L) ws::logprobs_kernel<ws::L><<<r.rows, ws::kThreads, 0, s>>>(p)
    WS_BY_DTYPE(r.dtype, CALL);
#undef CALL
    return ws::launched();
}

extern "C" int ws_logprobs_grad(const ws_rows* rows, const ws_logprobs_grad_args* args,
                                void* stream) {
    int v = ws::validate_logprobs_grad(rows, args);
    if (v != WS_OK) return v;
    if (rows->rows == 0) return WS_OK;
    v = ws::device_ready(rows->device);
    if (v != WS_OK) return v;
    const ws_rows& r = *rows;
    ws::GradParams g{};
    g.logits = args->logits;
    g.grad = args->grad_logits;
    g.stride = r.row_stride;
    g.grad_stride = args->grad_stride;
    g.stats = args->stats;
    g.entries = args->top;
    g.grad_entries = args->grad_top;
    g.targets = args->targets;
    g.grad_target = args->grad_logprob;
    g.entropy = args->entropy;
    g.grad_entropy = args->grad_entropy;
    g.vocab = r.vocab;
    g.k = args->top_k;
    g.c = ws::scale_c(r);
    g.inv_tau = ws::scale_inv(r);
    const hipStream_t s = static_cast<hipStream_t>(stream);
#define CALL(L) ws::grad_kernel<ws::L, false><<<r.rows, ws::kThreads, 0, s>>>(g)
    WS_BY_DTYPE(r.dtype, CALL);
#undef CALL
    return ws::launched();
}

extern "C" int ws_distill_workspace(const ws_rows* rows, int32_t mode, int32_t gradient,
                                    size_t* bytes) {
    const int v = ws::validate_rows(rows);
    if (v != WS_OK) return v;
    if (!bytes || ws::validate_teacher(1, mode) != WS_OK || (gradient != 0 && gradient != 1))
        return WS_E_INVALID_ARG;
    *bytes = ws::distill_workspace_bytes(*rows, mode, gradient == 1);
    return WS_OK;
}

extern "C" int ws_distill(const ws_rows* rows, const ws_distill_args* args, void* stream) {
    int v = ws::validate_distill(rows, args);
    if (v != WS_OK) return v;
    const ws_rows& r = *rows;
    if (r.rows == 0) return WS_OK;
    const bool gradient = args->grad_logits != nullptr;
    v = ws::validate_workspace(args->workspace, args->workspace_bytes,
                               ws::distill_workspace_bytes(r, args->mode, gradient));
    if (v != WS_OK) return v;
    v = ws::device_ready(r.device);
    if (v != WS_OK) return v;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    ws::DistillParams p{args->logits, r.row_stride, args->teacher, args->loss, args->stats,
                        args->tail, r.vocab, args->teacher_k, args->mode, ws::scale_c(r),
                        ws::scale_inv(r)};
    if (gradient) {
        if (!p.stats) p.stats = static_cast<ws_row_stats*>(args->workspace);
        if (!p.tail)
            p.tail = reinterpret_cast<float*>(static_cast<ws_row_stats*>(args->workspace) + r.rows);
    }
#define CALL(L) ws::distill_kernel<ws::L><<<r.rows, ws::kThreads, 0, s>>>(p)
    WS_BY_DTYPE(r.dtype, CALL);
#undef CALL
    v = ws::launched();
    if (v != WS_OK || !gradient) return v;
    ws::GradParams g{};
    g.logits = args->logits;
    g.grad = args->grad_logits;
    g.stride = r.row_stride;
    g.grad_stride = args->grad_stride;
    g.stats = p.stats;
    g.entries = args->teacher;
    g.tail = p.tail;
    g.grad_loss = args->grad_loss;
    g.vocab = r.vocab;
    g.k = args->teacher_k;
    g.mode = args->mode;
    g.c = p.c;
    g.inv_tau = p.inv_tau;
    return ws::run_distill_grad(r, g, s);
}

extern "C" int ws_distill_grad(const ws_rows* rows, const ws_distill_grad_args* args,
                               void* stream) {
    int v = ws::validate_distill_grad(rows, args);
    if (v != WS_OK) return v;
    if (rows->rows == 0) return WS_OK;
    v = ws::device_ready(rows->device);
    if (v != WS_OK) return v;
    const ws_rows& r = *rows;
    ws::GradParams g{};
    g.logits = args->logits;
    g.grad = args->grad_logits;
    g.stride = r.row_stride;
    g.grad_stride = args->grad_stride;
    g.stats = args->stats;
    g.entries = args->teacher;
    g.tail = args->tail;
    g.grad_loss = args->grad_loss;
    g.vocab = r.vocab;
    g.k = args->teacher_k;
    g.mode = args->mode;
    g.c = ws::scale_c(r);
    g.inv_tau = ws::scale_inv(r);
    return ws::run_distill_grad(r, g, static_cast<hipStream_t>(stream));
}
