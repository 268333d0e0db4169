// ws_logits.hip -- the operators over rows of logits (ws_logits.h), written
// for gfx950 (CDNA4, wave64).
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "ws_lanes.h"
#include "ws_logits.h"
#include "ws_logits_plan.h"
#include "ws_logits_rows.h"

namespace ws {
namespace {

constexpr int kThreads = 256;

template <typename L>
__device__ __forceinline__ float lload(const void* p, int64_t i) {
    return L::up(static_cast<const typename L::Elem*>(p)[i]);
}
template <typename L>
__device__ __forceinline__ void lstore(void* p, int64_t i, float v) {
    static_cast<typename L::Elem*>(p)[i] = L::down(v);
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

__device__ __forceinline__ bool listed(const uint32_t* ids, int k, uint32_t j) {
    for (int i = 0; i < k; ++i)
        if (ids[i] == j) return true;
    return false;
}

template <typename L>
__device__ Sums row_sums(const void* logits, int64_t at, int V, float c, const uint32_t* ids,
                         int k, float* scratch) {
    float m = -FLT_MAX;
    for (int j = threadIdx.x; j < V; j += kThreads)
        if (!listed(ids, k, j)) m = fmaxf(m, lload<L>(logits, at + j));
    m = group_reduce(m, scratch, MaxF());
    float s = 0.0f, u = 0.0f;
    for (int j = threadIdx.x; j < V; j += kThreads) {
        if (listed(ids, k, j)) continue;
        const float d = lload<L>(logits, at + j) - m;
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

// ---------------------------------------------------------------------------
// Forward: one pass over the row.
//
// Each thread keeps running sums of its own slots against its own running
// maximum (raised once per batch of slots), joined across lanes, waves and, for
// a row split over several workgroups, parts.
//
// Best K: a thread also keeps its best slot (largest slot maximum, the first
// one) and the second largest slot maximum.  The K-th largest of the threads'
// best values is a lower bound t on the row's K-th best: K threads reach it, so
// every element of the best K lies at or above t in one of those threads' slots
// - in its best slot, or, only if its second largest slot maximum reaches t as
// well, in any of its slots.  So after the pass about K slots are read again
// instead of a selection running inside the pass.

// A row's best keys as they are collected, in LDS.
template <typename L, int NT>
struct Best {
    static constexpr int kScan = NT < 128 ? NT : 128;   // threads that read slots again
    static constexpr int kRoom = kScan * L::VEC + WS_MAX_K;
    static constexpr int kListed = 64;
    uint64_t keys[kRoom];
    uint64_t sorted[WS_MAX_K];
    uint32_t tops[NT / 64 * 32];   // each wave's 32 largest thread bests, descending
    int single[kListed];           // slots to read again
    int thread[kListed];           // threads all of whose slots are read again
    int above, picked, singles, threads, count;
};

// K-th largest over the workgroup of one value a thread (K <= 32); every
// thread gets it.  The caller has synchronised since `tops` was last read.
template <int NT>
__device__ __forceinline__ uint32_t group_kth_largest(uint32_t v, int k, uint32_t* tops) {
    const int lane = threadIdx.x & 63;
    v = wave_sort<true>(v, lane);
    if constexpr (NT > 64) {
        static_assert(NT == 256, "one or four waves");
        const int wave = threadIdx.x >> 6;
        if (lane < 32) tops[wave * 32 + lane] = v;
        __syncthreads();
        // Lists 0 and 2 in the lower half of the lanes, 1 and 3 in the upper:
        // the larger of one list and the other reversed are the 32 largest of
        // both, a bitonic sequence; sorted, the halves meet the same way.
        const int half = lane & 32, i = lane & 31;
        const uint32_t a = tops[half + i], b = tops[64 + half + 31 - i];
        v = bitonic_stages<64, 16, true>(a > b ? a : b, lane);
        const uint32_t w = (uint32_t)__builtin_amdgcn_ds_bpermute((lane ^ 63) * 4, (int)v);
        v = bitonic_stages<64, 16, true>(v > w ? v : w, lane);
    }
    return (uint32_t)__builtin_amdgcn_readlane((int)v, k - 1);
}

// Keeps the K best of the collected keys, in order, at the list's start.
template <typename L, int NT>
__device__ __forceinline__ int keep_best(Best<L, NT>& b, int k) {
    const int n = b.count;
    for (int i = threadIdx.x; i < n; i += NT) {
        const uint64_t x = b.keys[i];
        const int r = keys_above(b.keys, n, x);
        if (r < k) b.sorted[r] = x;
    }
    __syncthreads();
    const int kept = n < k ? n : k;
    if ((int)threadIdx.x < kept) b.keys[threadIdx.x] = b.sorted[threadIdx.x];
    if (threadIdx.x == 0) b.count = kept;
    __syncthreads();
    return kept;
}

// What a thread remembers of its slots for the best K.
struct SlotTrack {
    float best, second;   // largest and second largest slot maximum
    int slot;             // first slot of the largest
};

// The K best keys of a part of a row into b.sorted; returns how many there are
// (K, or the part's elements if fewer).  all: read every slot again (a row
// with a NaN, which the running maxima skip).
template <typename L, int NT>
__device__ __forceinline__ int select_best(const Part<L>& part, SlotTrack t, bool all, int k,
                                           Best<L, NT>& b) {
    const int tid = threadIdx.x;
    const bool has = tid < part.n;
    const uint32_t best = has ? value_image(t.best) : 0;
    const uint32_t second = value_image(t.second);
    if (tid == 0) b.above = b.picked = b.singles = b.threads = b.count = 0;
    uint32_t bound = group_kth_largest<NT>(best, k, b.tops);
    __syncthreads();
    // Threads at the bound may be more than K when their bests are equal.
    if (has && best >= bound) {
        atomicAdd(&b.picked, 1);
        if (best > bound) atomicAdd(&b.above, 1);
    }
    __syncthreads();
    int last = 0x7fffffff;   // of the threads at the bound, those whose slot is not beyond
    if (b.picked > Best<L, NT>::kListed) {
        const int above = b.above;
        const uint32_t early =
            group_kth_largest<NT>(has && best == bound ? ~(uint32_t)t.slot : 0u, k - above, b.tops);
        last = (int)~early;
        __syncthreads();
    }
    const int rounds_per_thread = (part.n + NT - 1) / NT;
    if (has && !all && (best > bound || (best == bound && t.slot <= last))) {
        // A second slot at the bound counts only if it is not beyond `last`; it
        // comes at least NT slots after the first when both are at the bound.
        const bool more = second > bound ||
                          (second == bound && (best > bound || (int64_t)t.slot + NT <= last));
        if (more) b.thread[atomicAdd(&b.threads, 1)] = tid;
        else b.single[atomicAdd(&b.singles, 1)] = t.slot;
    }
    __syncthreads();
    const uint32_t edge = last == 0x7fffffff ? 0xffffffffu
                                             : (uint32_t)(part.e0 + last * L::VEC + L::VEC - 1);
    uint64_t least = all ? 0 : ((uint64_t)bound << 32) | (uint32_t)~edge;
    const int singles = b.singles;
    const int items = all ? part.n : singles + b.threads * rounds_per_thread;
    for (int from = 0;; from += Best<L, NT>::kScan) {
        const int item = from + tid;
        if (tid < Best<L, NT>::kScan && item < items) {
            int slot = item;
            if (!all) {
                if (item < singles) {
                    slot = b.single[item];
                } else {
                    const int j = item - singles;
                    slot = b.thread[j / rounds_per_thread] + (j % rounds_per_thread) * NT;
                }
            }
            if (slot < part.n) {
                float v[L::VEC];
                part.load_any(slot, v);
#pragma unroll
                for (int j = 0; j < L::VEC; ++j) {
                    const int e = part.e0 + slot * L::VEC + j;
                    const uint64_t key = value_key(v[j], (uint32_t)e);
                    if (key >= least && e >= 0 && e < part.vocab)
                        b.keys[atomicAdd(&b.count, 1)] = key;
                }
            }
        }
        __syncthreads();
        const bool more = from + Best<L, NT>::kScan < items;
        if (!more || b.count > WS_MAX_K) {
            const int kept = keep_best(b, k);
            if (!more) return kept;
            if (kept == k) least = umax64(least, b.sorted[k - 1]);
        }
    }
}

struct LogprobsParams {
    const void* logits;
    int64_t stride;
    const int32_t* targets;
    float* logprob;
    float* entropy;
    ws_topk_entry* top;
    ws_row_stats* stats;
    Sums* sums;         // [rows][parts], when a row has several parts
    uint64_t* keys;     // [rows][parts][k]
    int32_t vocab;
    int32_t k;
    int32_t chunk;      // slots of a part
    int32_t parts;
    float c;            // log2(e) / tau
    float inv_tau;
};

// Row outputs from its sums; `sorted` holds its best keys.  Called by every
// thread of a workgroup.
template <typename L>
__device__ __forceinline__ void write_logprobs(const LogprobsParams& p, int64_t row, Sums t,
                                               const uint64_t* sorted) {
    const bool empty = t.s == 0.0f;
    const float logsum = empty ? -INFINITY : logf(t.s);
    if (threadIdx.x == 0) {
        if (p.stats) p.stats[row] = {empty ? -INFINITY : t.m, logsum};
        if (p.entropy) p.entropy[row] = empty ? 0.0f : logsum - t.u * p.inv_tau / t.s;
        if (p.logprob) {
            const int32_t j = p.targets[row];
            float v = 0.0f;
            if (j >= 0 && j < p.vocab) {
                const float z =
                    L::up(static_cast<const typename L::Elem*>(p.logits)[row * p.stride + j]);
                v = empty ? -INFINITY : (z - t.m) * p.inv_tau - logsum;
            } else if (j != -1) {
                v = NAN;
            }
            p.logprob[row] = v;
        }
    }
    if ((int)threadIdx.x < p.k) {
        const uint64_t key = sorted[threadIdx.x];
        const float z = image_value((uint32_t)(key >> 32));
        ws_topk_entry e;
        e.score = empty ? -INFINITY : (z - t.m) * p.inv_tau - logsum;
        e.index = (int32_t)~(uint32_t)key;
        p.top[row * p.k + threadIdx.x] = e;
    }
}

constexpr int kBatch = 4;   // slots a thread has in flight

struct Nothing {
    static constexpr uint64_t* sorted = nullptr;
};
template <bool ON, typename T>
struct Select {
    using Type = T;
};
template <typename T>
struct Select<false, T> {
    using Type = Nothing;
};

template <typename L, int NT, bool ENT, bool TOPK>
__global__ void __launch_bounds__(NT) logprobs_kernel(LogprobsParams p) {
    constexpr int VEC = L::VEC;
    __shared__ Sums wave_sums[NT / 64];
    __shared__ typename Select<TOPK, Best<L, NT>>::Type best;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x / (uint32_t)p.parts;
    const int index = (int)(blockIdx.x % (uint32_t)p.parts);
    Part<L> part;
    part.init(p.logits, row * p.stride, p.vocab, p.chunk, p.parts, index);

    Sums a;
    a.init();
    SlotTrack t{-INFINITY, -INFINITY, tid};
    // The running sums over U slots of values, the first at `slot`, NT apart.
    const auto take = [&](auto& v, int slot) {
        constexpr int U = sizeof(v) / sizeof(v[0]);
        float top = a.m;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float m = fmaxf(v[i][0], v[i][1]);
#pragma unroll
            for (int j = 2; j < VEC; ++j) m = fmaxf(m, v[i][j]);
            top = fmaxf(top, m);
            if constexpr (TOPK) {
                t.second = __builtin_amdgcn_fmed3f(m, t.best, t.second);
                t.slot = m > t.best ? slot + i * NT : t.slot;
                t.best = fmaxf(t.best, m);
            }
        }
        a.raise<ENT>(top, p.c);
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = v[i][j] - a.m;
                const float e = __builtin_amdgcn_exp2f(d * p.c);
                a.s += e;
                if constexpr (ENT) a.u = fmaf(e, fmaxf(d, kFar), a.u);
            }
    };
    int s = tid;
    if (s < part.full_from) {   // the slot that sticks out in front
        float v[1][VEC];
        part.load_edge(s, v[0]);
        take(v, s);
        s += NT;
    }
    for (; s < part.full_to; s += kBatch * NT) {
        float v[kBatch][VEC];
        uint4 w[kBatch];
        if (s + (kBatch - 1) * NT < part.full_to) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) w[i] = part.load(s + i * NT);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) L::unpack(w[i], v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (s + i * NT < part.full_to) w[i] = part.load(s + i * NT);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (s + i * NT < part.full_to) {
                    L::unpack(w[i], v[i]);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) v[i][j] = -INFINITY;
                }
            }
        }
        take(v, s);
    }
    // The slot that sticks out behind belongs to the thread next in turn.
    const int tail = part.full_to > part.full_from ? part.full_to : part.full_from;
    if (tail < part.n && tail % NT == tid) {
        float v[1][VEC];
        part.load_edge(tail, v[0]);
        take(v, tail);
    }

    a = wave_join<ENT>(a, p.c, lane);
    if constexpr (NT > 64) {
        if (lane == 0) wave_sums[tid >> 6] = a;
        __syncthreads();
        a = join_in_order<ENT>(wave_sums, NT / 64, p.c);
    }
    int kept = 0;
    if constexpr (TOPK) {
        kept = select_best<L, NT>(part, t, a.s != a.s, p.k, best);
    }
    if (p.parts == 1) {
        write_logprobs<L>(p, row, a, best.sorted);
    } else {
        if (tid == 0) p.sums[blockIdx.x] = a;
        if constexpr (TOPK) {
            if (tid < p.k)
                p.keys[(int64_t)blockIdx.x * p.k + tid] = tid < kept ? best.sorted[tid] : 0;
        }
    }
}

// Joins the parts of a row (at most 64): one wave a row.


template <typename L, bool ENT>
__global__ void __launch_bounds__(64) logprobs_join_kernel(LogprobsParams p) {
    __shared__ uint64_t keys[WS_MAX_K * WS_MAX_K + WS_MAX_K];
    __shared__ uint64_t sorted[WS_MAX_K];
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    Sums a;
    a.init();
    if (lane < p.parts) a = p.sums[row * p.parts + lane];
    if (p.k > 0) {
        const uint64_t* in = p.keys + row * p.parts * p.k;
        // The K-th largest of the lists' leading keys, as many from each as
        // fill a wave, bounds the K-th best from below.
        const int lead = 64 / p.parts < p.k ? 64 / p.parts : p.k;
        uint64_t x = 0;
        if (lane < p.parts * lead) x = in[lane / lead * p.k + lane % lead];
        x = wave_sort<true>(x, lane);
        const uint64_t least = umax64(readlane64(x, p.k - 1), 1);
        int n = 0;
        const int all = p.parts * p.k;
        for (int i = 0; i < all; i += 64) {
            const uint64_t key = i + lane < all ? in[i + lane] : 0;
            const uint64_t hit = __ballot(key >= least);
            if (key >= least) keys[n + lanes_below(hit)] = key;
            n += __popcll(hit);
        }
        wave_lds_sync();
        for (int i = lane; i < n; i += 64) {
            const uint64_t key = keys[i];
            const int r = keys_above(keys, n, key);
            if (r < p.k) sorted[r] = key;
        }
        wave_lds_sync();
    }
    a = wave_join<ENT>(a, p.c, lane);
    write_logprobs<L>(p, row, a, sorted);
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
            if (t.ids[i] != 0xffffffffu) m = fmaxf(m, lload<L>(p.logits, at + t.ids[i]));
        s = s == 0.0f ? 0.0f : s * __builtin_amdgcn_exp2f((r.m - m) * p.c);
        for (int i = 0; i < p.k; ++i)
            if (t.ids[i] != 0xffffffffu && !listed(t.ids, i, t.ids[i]))
                s += __builtin_amdgcn_exp2f((lload<L>(p.logits, at + t.ids[i]) - m) * p.c);
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
                  : ((double)lload<L>(p.logits, at + t.ids[i]) - (double)m) * p.inv_tau - logsum;
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
        for (int j = threadIdx.x; j < p.vocab; j += kThreads) lstore<L>(p.grad, to + j, 0.0f);
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
        const float d = lload<L>(p.logits, at + j) - st.max;
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
        lstore<L>(p.grad, to + j, v * scale);
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

// Enqueues one kernel; its parameters are one struct, copied by the call.
template <typename P>
int launch(void (*kernel)(P), int64_t groups, int threads, const P& params, hipStream_t s) {
    P copy = params;
    void* args[] = {&copy};
    const hipError_t e =
        hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3((uint32_t)groups),
                        dim3((uint32_t)threads), args, 0, s);
    return e == hipSuccess ? WS_OK : WS_E_HIP;
}

template <typename L>
int run_logprobs(const ws_rows& r, const LogprobsPlan& plan, const LogprobsParams& p,
                 hipStream_t s) {
    const bool ent = p.entropy != nullptr, top = p.k > 0;
    const auto wide = top ? (ent ? logprobs_kernel<L, 256, true, true>
                                 : logprobs_kernel<L, 256, false, true>)
                          : (ent ? logprobs_kernel<L, 256, true, false>
                                 : logprobs_kernel<L, 256, false, false>);
    const auto wave = top ? (ent ? logprobs_kernel<L, 64, true, true>
                                 : logprobs_kernel<L, 64, false, true>)
                          : (ent ? logprobs_kernel<L, 64, true, false>
                                 : logprobs_kernel<L, 64, false, false>);
    int v = launch(plan.threads == 64 ? wave : wide, (int64_t)r.rows * plan.parts, plan.threads, p,
                   s);
    if (v != WS_OK || plan.parts == 1) return v;
    return launch(ent ? logprobs_join_kernel<L, true> : logprobs_join_kernel<L, false>, r.rows, 64,
                  p, s);
}

float scale_c(const ws_rows& r) { return (float)(1.4426950408889634074 / (double)r.temperature); }
float scale_inv(const ws_rows& r) { return (float)(1.0 / (double)r.temperature); }

int run_distill_grad(const ws_rows& r, const GradParams& g, hipStream_t s) {
#define CALL(L) return launch(grad_kernel<L, true>, r.rows, kThreads, g, s)
    WS_BY_DTYPE(r.dtype, CALL);
#undef CALL
}

}  // namespace
}  // namespace ws

extern "C" int ws_logprobs_workspace(const ws_rows* rows, int32_t top_k, size_t* bytes) {
    const int v = ws::validate_rows(rows);
    if (v != WS_OK) return v;
    if (!bytes || ws::validate_top_k(*rows, top_k) != WS_OK) return WS_E_INVALID_ARG;
    *bytes = ws::plan_logprobs(*rows, top_k).workspace;
    return WS_OK;
}

extern "C" int ws_logprobs(const ws_rows* rows, const ws_logprobs_args* args, void* stream) {
    int v = ws::validate_logprobs(rows, args);
    if (v != WS_OK) return v;
    const ws_rows& r = *rows;
    if (r.rows == 0) return WS_OK;
    const ws::LogprobsPlan plan = ws::plan_logprobs(r, args->top_k);
    v = ws::validate_workspace(args->workspace, args->workspace_bytes, plan.workspace);
    if (v != WS_OK) return v;
    v = ws::device_ready(r.device);
    if (v != WS_OK) return v;
    ws::LogprobsParams p{};
    p.logits = args->logits;
    p.stride = r.row_stride;
    p.targets = args->targets;
    p.logprob = args->logprob;
    p.entropy = args->entropy;
    p.top = args->top;
    p.stats = args->stats;
    p.vocab = r.vocab;
    p.k = args->top_k;
    p.chunk = plan.chunk;
    p.parts = plan.parts;
    p.c = ws::scale_c(r);
    p.inv_tau = ws::scale_inv(r);
    if (plan.parts > 1) {
        p.keys = static_cast<uint64_t*>(args->workspace);
        p.sums = reinterpret_cast<ws::Sums*>(p.keys + (int64_t)r.rows * plan.parts * p.k);
    }
    const hipStream_t s = static_cast<hipStream_t>(stream);
#define CALL(L) return ws::run_logprobs<ws::L>(r, plan, p, s)
    WS_BY_DTYPE(r.dtype, CALL);
#undef CALL
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
#define CALL(L) return ws::launch(ws::grad_kernel<ws::L, false>, r.rows, ws::kThreads, g, s)
    WS_BY_DTYPE(r.dtype, CALL);
#undef CALL
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
#define CALL(L) v = ws::launch(ws::distill_kernel<ws::L>, r.rows, ws::kThreads, p, s)
    WS_BY_DTYPE(r.dtype, CALL);
#undef CALL
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
