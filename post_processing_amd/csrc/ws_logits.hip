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

// ---------------------------------------------------------------------------
// Forward: one pass over the row.
//
// Each thread keeps running sums of its own slots against its own running
// maximum (raised once per batch of slots), joined across lanes, waves and, for
// a row split over several workgroups, parts.  A row is read once (counted:
// 1.0745e9 bytes for 4,096 x 131,072 BF16, 1.0737e9 of them logits), and HBM
// bounds it: 169 us for that with entropy (6.4 TB/s; a plain copy moves 4.84
// TB/s read and written).  The vector unit is close behind with 9.3
// instructions an element, one of them an exponential at a quarter of the rate;
// one instruction fewer (16-bit exponents in one fused multiply-add) changed
// nothing.
//
// Best K: a thread also keeps its best slot (largest slot maximum, the first
// one) and the second largest slot maximum, four instructions a slot.  The K-th
// largest of 64 groups of threads' best values is a lower bound t on the row's
// K-th best: K threads reach it, so every element of the best K lies at or above
// t in the slots of a thread that reaches it - in its best slot, or, only if its
// second largest slot maximum reaches t as well, in any of its slots.  So after
// the pass about K slots are read again, element by element, instead of a
// selection running inside the pass.  What follows the pass is a chain of
// latencies: 0.5 us to the bound, 0.3 to the list of slots, 1.3 for reading them
// again and 0.8 for ordering and storing (one row of 131,072 BF16 in 16 parts, K
// = 20, 5.5 us in all, and 3.6 for the join); 2,048 rows of 50,001 take 42 us
// (4.9 TB/s): one round of workgroups, so the chain at its end stays visible.

constexpr int kBatch = kBatchSlots;   // slots a thread has in flight

template <int VEC>
__device__ __forceinline__ float slot_max(const float (&v)[VEC]) {
    float m = fmaxf(v[0], v[1]);
#pragma unroll
    for (int j = 2; j < VEC; ++j) m = fmaxf(m, v[j]);
    return m;
}

// Takes the tokens a slot's mark names out of its values.
template <int VEC>
__device__ __forceinline__ void hide_listed(uint32_t mark, float (&v)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = mark >> j & 1u ? -INFINITY : v[j];
}

// What a thread remembers of its slots for the best K.
struct SlotTrack {
    float best, second;   // largest and second largest slot maximum
    int slot;             // first slot of the largest
};

// Takes U slots of values, the first at `slot` and NT apart, into a thread's
// running sums.  ENT: the entropy's sum as well; TOPK: the slot maxima; MASK:
// without the marked tokens.
template <typename L, int NT, bool ENT, bool TOPK, bool MASK, int U>
__device__ __forceinline__ void take_slots(float (&v)[U][L::VEC], int slot, float c,
                                           const uint8_t* marks, Sums& a, SlotTrack& t) {
    constexpr int VEC = L::VEC;
    if constexpr (MASK) {
#pragma unroll
        for (int i = 0; i < U; ++i)   // rare
            if (const uint32_t mark = marks[slot + i * NT]) hide_listed<VEC>(mark, v[i]);
    }
    float top = a.m;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const float m = slot_max<VEC>(v[i]);
        top = fmaxf(top, m);
        if constexpr (TOPK) {
            t.second = __builtin_amdgcn_fmed3f(m, t.best, t.second);
            t.slot = m > t.best ? slot + i * NT : t.slot;
            t.best = fmaxf(t.best, m);
        }
    }
    a.raise<ENT>(top, c);
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float d = v[i][j] - a.m;
            const float e = __builtin_amdgcn_exp2f(d * c);
            a.s += e;
            if constexpr (ENT) a.u = fmaf(e, fmaxf(d, kFar), a.u);
        }
}

// A thread's running sums over its slots of a part.
template <typename L, int NT, bool ENT, bool TOPK, bool MASK>
__device__ __forceinline__ void stream_part(const Part<L>& part, float c, const uint8_t* marks,
                                            Sums& a, SlotTrack& t) {
    constexpr int VEC = L::VEC;
    const int tid = threadIdx.x;
    a.init();
    t = {-INFINITY, -INFINITY, tid};
    int s = tid;
    if (s < part.full_from) {   // the slot that sticks out in front
        float v[1][VEC];
        part.load_edge(s, v[0]);
        take_slots<L, NT, ENT, TOPK, MASK>(v, s, c, marks, a, t);
        s += NT;
    }
    for (; s < part.full_to; s += kBatch * NT) {
        float v[kBatch][VEC];
        uint4 w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) w[i] = part.load_near(s + i * NT);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) L::unpack(w[i], v[i]);
        if (s + (kBatch - 1) * NT >= part.full_to) {
#pragma unroll
            for (int i = 1; i < kBatch; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    v[i][j] = s + i * NT < part.full_to ? v[i][j] : -INFINITY;
        }
        take_slots<L, NT, ENT, TOPK, MASK>(v, s, c, marks, a, t);
    }
    // The slot that sticks out behind belongs to the thread next in turn.
    const int tail = part.full_to > part.full_from ? part.full_to : part.full_from;
    if (tail < part.n && tail % NT == tid) {
        float v[1][VEC];
        part.load_edge(tail, v[0]);
        take_slots<L, NT, ENT, TOPK, MASK>(v, tail, c, marks, a, t);
    }
}

template <int NT, bool ENT>
__device__ __forceinline__ Sums join_waves(Sums a, float c, const Sums* wave_sums) {
    if constexpr (NT > 64) {
        const int lane = threadIdx.x & 63;
        if (threadIdx.x < 64) {
            a.init();
            if (lane < NT / 64) a = wave_sums[lane];
            a = wave_join<ENT>(a, c, lane);
        }
    }
    return a;
}

// The sums of a workgroup's threads, in wave 0: each wave's across its lanes,
// then the waves' the same way.  FENCE: with the barrier between the two.
template <int NT, bool ENT, bool FENCE = true>
__device__ __forceinline__ Sums group_join(Sums a, float c, Sums* wave_sums) {
    const int lane = threadIdx.x & 63;
    a = wave_join<ENT>(a, c, lane);
    if constexpr (NT > 64) {
        if (lane == 0) wave_sums[threadIdx.x >> 6] = a;
        if constexpr (FENCE) {
            __syncthreads();
            a = join_waves<NT, ENT>(a, c, wave_sums);
        }
    }
    return a;
}

// A row's best keys as they are collected, in LDS.
template <typename L, int NT>
struct Best {
    static constexpr int kListed = 64;                  // threads looked at
    static constexpr int kEach = 4;                     // elements a thread reads again
    static constexpr int kScan = NT * kEach;
    static constexpr int kFound = kScan + WS_MAX_K;
    static constexpr int kRoom = kFound > NT ? kFound : NT;   // or a pair a thread
    uint64_t keys[kRoom];
    uint64_t sorted[WS_MAX_K];
    uint32_t groups[64];
    int single[kListed];           // slots to read again
    int thread[kListed];           // threads all of whose slots are read again
    uint32_t bound;
    int last, singles, threads, count;
    bool all;
};

// The K best of the collected keys into b.sorted, in order; returns how many
// (K, or all there are).
template <typename L, int NT>
__device__ __forceinline__ int sort_best(Best<L, NT>& b, int k) {
    const int n = b.count;
    for (int i = threadIdx.x; i < n; i += NT) {
        const uint64_t x = b.keys[i];
        const int r = keys_above(b.keys, n, x);
        if (r < k) b.sorted[r] = x;
    }
    __syncthreads();
    return n < k ? n : k;
}

// The largest of a group of NT / 64 neighbouring lanes, in each of them.
template <int NT>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int lane) {
    const auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    if constexpr (NT >= 128) v = larger(v, xor_lane32<1>(v, lane));
    if constexpr (NT >= 256) v = larger(v, xor_lane32<2>(v, lane));
    if constexpr (NT >= 512) v = larger(v, xor_lane32<4>(v, lane));
    if constexpr (NT >= 1024) v = larger(v, xor_lane32<8>(v, lane));
    return v;
}

// The K best keys of a part of a row into b.sorted; returns how many there are
// (K, or the part's elements if fewer).  Joins the sums on the way: in wave 0
// afterwards.
template <typename L, int NT, bool ENT>
__device__ __forceinline__ int select_best(const Part<L>& part, SlotTrack t, Sums& a, float c,
                                           Sums* wave_sums, int k, Best<L, NT>& b) {
    using B = Best<L, NT>;
    constexpr int kGroup = NT / 64;               // threads of a group
    constexpr int kSorter = NT > 64 ? 64 : 0;     // first thread of the wave that sorts
    const int tid = threadIdx.x, lane = tid & 63;
    const bool has = tid < part.n;
    const uint32_t best = has ? value_image(t.best) : 0;
    const uint32_t second = value_image(t.second);
    // The bound from 64 groups of threads: the K-th largest of their bests,
    // by one wave (a few more threads reach it than with every thread a group)
    // while wave 0 joins the sums.
    const uint32_t group = lanes_max<NT>(best, lane);
    if (lane % kGroup == 0) b.groups[tid / kGroup] = group;
    if (tid == 0) {
        b.last = 0x7fffffff;
        b.singles = b.threads = b.count = 0;
    }
    a = group_join<NT, ENT, false>(a, c, wave_sums);
    __syncthreads();
    if (tid < 64) {
        a = join_waves<NT, ENT>(a, c, wave_sums);
        if (tid == 0) b.all = a.s != a.s;   // a NaN in the row, which the maxima skip
    }
    if (tid >= kSorter && tid < kSorter + 64) {
        const uint32_t sorted = wave_sort<true>(b.groups[lane], lane);
        if (lane == k - 1) b.bound = sorted;
    }
    __syncthreads();
    const bool all = b.all;
    uint32_t bound = b.bound;
    uint64_t least = all ? 0 : (uint64_t)bound << 32;
    // A thread's slots that may hold elements at the bound: its best, or, if
    // its second largest slot maximum is there too, any.  (With equal bests
    // cut off behind slot `last`: a second slot at the bound comes at least NT
    // slots after the first when both are.)
    const auto list_slots = [&](bool chosen, int last) {
        if (chosen) {
            const bool more = second > bound ||
                              (second == bound && (best > bound || (int64_t)t.slot + NT <= last));
            int* list = more ? b.thread : b.single;
            const int at = atomicAdd(more ? &b.threads : &b.singles, 1);
            if (at < B::kListed) list[at] = more ? tid : t.slot;
        }
    };
    const bool chosen = has && !all && best >= bound;
    list_slots(chosen, 0x7fffffff);
    __syncthreads();
    if (b.singles > B::kListed || b.threads > B::kListed) {
        // Many reach the bound (equal values): exactly K threads then, by best
        // and slot; of elements equal to the K-th's best, those up to its slot.
        __syncthreads();
        const uint64_t pair = has ? ((uint64_t)best << 32) | (uint32_t)~t.slot : 0;
        b.keys[tid] = pair;
        if (tid == 0) b.singles = b.threads = b.count = 0;
        __syncthreads();
        const bool among = has && best >= bound && keys_above(b.keys, NT, pair) < k;
        if (among && keys_above(b.keys, NT, pair) == k - 1) {
            b.bound = best;
            b.last = t.slot;
        }
        __syncthreads();
        bound = b.bound;
        const int last = b.last;
        least = ((uint64_t)bound << 32) | (uint32_t)~(part.e0 + last * L::VEC + L::VEC - 1);
        list_slots(among, last);
        __syncthreads();
    }
    // Element by element: little code, as it runs once a row, and few rounds.
    const int each = (part.n + NT - 1) / NT * L::VEC;   // elements of a thread's slots
    const int singles = b.singles * L::VEC;
    const int items = all ? part.n * L::VEC : singles + b.threads * each;
    for (int from = 0;; from += B::kScan) {
        typename L::Elem x[B::kEach];
        int e[B::kEach];
#pragma unroll
        for (int i = 0; i < B::kEach; ++i) {
            const int item = from + tid + i * NT;
            e[i] = -1;
            if (item < items) {
                int at = item;   // element of the part
                if (!all) {
                    if (item < singles) {
                        at = b.single[item / L::VEC] * L::VEC + item % L::VEC;
                    } else {
                        const int j = item - singles;
                        const int slot = b.thread[j / each] + j % each / L::VEC * NT;
                        at = slot < part.n ? slot * L::VEC + j % L::VEC : part.vocab - part.e0;
                    }
                }
                e[i] = part.e0 + at;
            }
            x[i] = part.row[e[i] < 0 ? 0 : e[i] < part.vocab ? e[i] : part.vocab - 1];
        }
#pragma unroll
        for (int i = 0; i < B::kEach; ++i) {
            const uint64_t key = value_key(L::up(x[i]), (uint32_t)e[i]);
            if (key >= least && e[i] >= 0 && e[i] < part.vocab) b.keys[atomicAdd(&b.count, 1)] = key;
        }
        __syncthreads();
        if (from + B::kScan >= items) return sort_best(b, k);
        const int found = b.count;
        __syncthreads();   // everyone has read it before anyone adds to it
        if (found <= WS_MAX_K) continue;
        const int kept = sort_best(b, k);
        // Room for the next round: the K best so far, and a higher bound.
        if (tid < kept) b.keys[tid] = b.sorted[tid];
        if (tid == 0) b.count = kept;
        if (kept == k) least = umax64(least, b.sorted[k - 1]);
        __syncthreads();
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

// The token a row is asked for.  Its index is read before the pass and its logit
// after it, so that neither is waited for at the end.
struct Asked {
    int32_t index;   // -1: none
    float z;

    __device__ __forceinline__ void read_index(const LogprobsParams& p, int64_t row) {
        index = p.targets ? p.targets[row] : -1;
    }
    template <typename L>
    __device__ __forceinline__ void read_logit(const LogprobsParams& p, int64_t row) {
        const typename L::Elem* at =
            static_cast<const typename L::Elem*>(p.logits) + row * p.stride;
        z = L::up(at[index >= 0 && index < p.vocab ? index : 0]);
    }
};

// Row outputs from its sums; `sorted` holds its best keys.  Called by wave 0.
template <typename L>
__device__ __forceinline__ void write_logprobs(const LogprobsParams& p, int64_t row, Sums t,
                                               const Asked& asked, const uint64_t* sorted) {
    const bool empty = t.s == 0.0f;
    const float logsum = empty ? -INFINITY : logf(t.s);
    if (threadIdx.x == 0) {
        if (p.stats) p.stats[row] = {empty ? -INFINITY : t.m, logsum};
        if (p.entropy) p.entropy[row] = empty ? 0.0f : logsum - t.u * p.inv_tau / t.s;
        if (p.logprob) {
            float v = 0.0f;
            if (asked.index >= 0 && asked.index < p.vocab)
                v = empty ? -INFINITY : (asked.z - t.m) * p.inv_tau - logsum;
            else if (asked.index != -1)
                v = NAN;
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
    __shared__ Sums wave_sums[NT / 64];
    __shared__ typename Select<TOPK, Best<L, NT>>::Type best;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / (uint32_t)p.parts;
    const int index = (int)(blockIdx.x % (uint32_t)p.parts);
    Part<L> part;
    part.init(p.logits, row * p.stride, p.vocab, p.chunk, p.parts, index);

    Asked asked;
    asked.read_index(p, row);
    Sums a;
    SlotTrack t;
    stream_part<L, NT, ENT, TOPK, false>(part, p.c, nullptr, a, t);
    if (p.parts == 1) asked.read_logit<L>(p, row);
    int kept = 0;
    if constexpr (TOPK) {
        kept = select_best<L, NT, ENT>(part, t, a, p.c, wave_sums, p.k, best);
    } else {
        a = group_join<NT, ENT>(a, p.c, wave_sums);
    }
    if (tid >= 64) return;
    if (p.parts == 1) {
        write_logprobs<L>(p, row, a, asked, best.sorted);
    } else {
        if (tid == 0) p.sums[blockIdx.x] = a;
        if constexpr (TOPK) {
            if (tid < p.k)
                p.keys[(int64_t)blockIdx.x * p.k + tid] = tid < kept ? best.sorted[tid] : 0;
        }
    }
}

// Joins the parts of a row (at most 64): every key asked for at once, then the
// bound, the keys that reach it and their order (3.6 us for 16 lists of 20 keys,
// 2.1 us for sums alone; reading the lists in turn took 8.0 us for 64 of them).
constexpr int kJoin = 256;

template <typename L, bool ENT>
__global__ void __launch_bounds__(kJoin) logprobs_join_kernel(LogprobsParams p) {
    constexpr int kEach = kMaxRowParts * WS_MAX_K / kJoin;   // keys a thread
    __shared__ uint64_t keys[WS_MAX_K * WS_MAX_K + WS_MAX_K];
    __shared__ uint64_t sorted[WS_MAX_K];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x;
    Asked asked;
    asked.read_index(p, row);
    Sums a;
    a.init();
    if (lane < p.parts) a = p.sums[row * p.parts + lane];
    asked.read_logit<L>(p, row);
    if (p.k > 0) {
        const uint64_t* in = p.keys + row * p.parts * p.k;
        const int all = p.parts * p.k;
        // The K-th largest of the lists' leading keys, as many from each as
        // fill a wave, bounds the K-th best from below.
        const int lead = 64 / p.parts < p.k ? 64 / p.parts : p.k;
        const int from = lane < p.parts * lead ? lane / lead * p.k + lane % lead : 0;
        uint64_t x = in[from];
        uint64_t mine[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            mine[i] = in[tid + i * kJoin < all ? tid + i * kJoin : 0];
        if (lane >= p.parts * lead) x = 0;
        if (tid == 0) count = 0;
        __syncthreads();
        x = wave_sort<true>(x, lane);
        const uint64_t least = umax64(readlane64(x, p.k - 1), 1);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (tid + i * kJoin < all && mine[i] >= least) keys[atomicAdd(&count, 1)] = mine[i];
        __syncthreads();
        const int n = count;
        for (int i = tid; i < n; i += kJoin) {
            const uint64_t key = keys[i];
            const int r = keys_above(keys, n, key);
            if (r < p.k) sorted[r] = key;
        }
        __syncthreads();
    }
    if (tid >= 64) return;
    write_logprobs<L>(p, row, wave_join<ENT>(a, p.c, lane), asked, sorted);
}

// ---------------------------------------------------------------------------
// Tokens a row names: teacher entries, alternatives, the target.
//
// Wave 0 of a workgroup holds them, entries lane and lane + 64.  They are few,
// so what they need in FP64 (a teacher's probabilities, the small difference 1 -
// sum q, the loss's near-cancelling terms) costs a wave a few hundred
// instructions a row.

constexpr uint32_t kAbsent = 0xffffffffu;

struct Named {
    uint32_t id[2];    // kAbsent: none
    float z[2];        // its logit
    float add[2];      // what a gradient adds for the token, all its entries together
    bool first[2];     // the token's first entry
    float score[2];    // a teacher's
    bool bad;          // some index lies outside the row (wave-uniform)
};

// The logits of the tokens in [from, to), and whether any index lies outside
// the row.  Read before any thread writes a gradient over the logits (other
// workgroups may be writing theirs outside that range).
template <typename L>
__device__ __forceinline__ void read_named(Named& n, const typename L::Elem* row, int V, int from,
                                           int to) {
    bool bad = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        n.z[h] = -INFINITY;
        if (n.id[h] >= (uint32_t)from && n.id[h] < (uint32_t)to) n.z[h] = L::up(row[n.id[h]]);
        bad |= n.id[h] >= (uint32_t)V && n.id[h] != kAbsent;
    }
    n.bad = __ballot(bad) != 0;
}

// Finds tokens named more than once among `count` entries and gathers what
// their entries add at the first.  ids and adds: LDS scratch of wave 0.
__device__ __forceinline__ void merge_named(Named& n, int count, uint32_t* ids, float* adds,
                                            int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        ids[lane + 64 * h] = n.id[h];
        adds[lane + 64 * h] = n.add[h];
    }
    wave_lds_sync();
    n.first[0] = n.id[0] != kAbsent;
    n.first[1] = n.id[1] != kAbsent;
    bool again[2] = {false, false};
    const int padded = (count + 3) & ~3;   // entries past count are kAbsent
    for (int j = 0; j < padded; j += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(ids + j);
        const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            again[0] |= q[i] == n.id[0] && j + i < lane;
            again[1] |= q[i] == n.id[1] && j + i < lane + 64;
        }
    }
    if (__ballot((again[0] && n.first[0]) || (again[1] && n.first[1])) == 0) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (n.id[h] == kAbsent) continue;
        float sum = 0.0f;
        for (int j = 0; j < count; ++j) {
            if (ids[j] != n.id[h]) continue;
            if (j < lane + 64 * h) n.first[h] = false;
            sum += adds[j];
        }
        n.add[h] = sum;
    }
}

// A distillation row's teacher, in wave 0.
struct Teacher {
    double q[2], logq[2];
    double mass;   // sum of q, q_t included
    double rest;   // q_t
};

// A lane's two entries of a teacher's k, as they lie in memory (another's
// where there are fewer): loaded first and looked at later.
struct RawEntries {
    uint2 e[2];

    __device__ __forceinline__ void load(const ws_topk_entry* entries, int k, int lane) {
        const uint2* p = reinterpret_cast<const uint2*>(entries);
#pragma unroll
        for (int h = 0; h < 2; ++h) e[h] = p[lane + 64 * h < k ? lane + 64 * h : k - 1];
    }
    __device__ __forceinline__ void into(Named& n, int k, int lane) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            n.id[h] = lane + 64 * h < k ? e[h].y : kAbsent;
            n.score[h] = n.id[h] != kAbsent ? __uint_as_float(e[h].x) : -INFINITY;
        }
    }
};

__device__ __forceinline__ void read_entries(Named& n, const ws_topk_entry* entries, int k,
                                             int lane) {
    RawEntries raw;
    raw.load(entries, k, lane);
    raw.into(n, k, lane);
}

__device__ __forceinline__ Teacher weigh_teacher(Named& n, int k, int mode, int lane) {
    Teacher t;
    double shift = 0.0;
    if (mode == WS_DISTILL_RENORM) {
        const float high = wave_max(fmaxf(n.score[0], n.score[1]), lane);
        if (high != -INFINITY) shift = (double)high;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        t.logq[h] = (double)n.score[h] - shift;
        t.q[h] = h == 0 || k > 64 ? small_exp(t.logq[h]) : 0.0;
    }
    const double sum = wave_sum_d(t.q[0] + t.q[1], lane);
    t.mass = sum;
    t.rest = 0.0;
    if (mode == WS_DISTILL_RENORM) {
        if (sum != 0.0) {
            const double logsum = small_log(sum);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                t.q[h] /= sum;
                t.logq[h] -= logsum;
            }
            t.mass = sum / sum;   // 1, or NaN
        }
    } else {
        t.rest = sum < 1.0 ? 1.0 - sum : 0.0;
    }
    n.add[0] = -(float)t.q[0];
    n.add[1] = -(float)t.q[1];
    return t;
}

// Wave 0's teacher and named tokens (but for their logits) put aside in LDS
// while it streams its share of the row.
struct Aside {
    double q[WS_DISTILL_MAX_K], logq[WS_DISTILL_MAX_K];
    float add[WS_DISTILL_MAX_K];
    uint32_t id[WS_DISTILL_MAX_K];
    uint32_t first[WS_DISTILL_MAX_K];
    double mass, rest;
    uint32_t bad;

    __device__ __forceinline__ void put(const Named& n, const Teacher& t, int lane) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = lane + 64 * h;
            q[i] = t.q[h];
            logq[i] = t.logq[h];
            add[i] = n.add[h];
            id[i] = n.id[h];
            first[i] = n.first[h];
        }
        if (lane == 0) {
            mass = t.mass;
            rest = t.rest;
            bad = n.bad;
        }
        wave_lds_sync();
    }
    __device__ __forceinline__ void get(Named& n, Teacher& t, int lane) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = lane + 64 * h;
            t.q[h] = q[i];
            t.logq[h] = logq[i];
            n.add[h] = add[i];
            n.id[h] = id[i];
            n.first[h] = first[i] != 0;
        }
        t.mass = mass;
        t.rest = rest;
        n.bad = bad != 0;
    }
};

// With WS_DISTILL_TAIL, once merge_named has run: a list that names every
// token leaves no rest.
__device__ __forceinline__ void settle_rest(Teacher& t, const Named& n, int k, int V) {
    if (V <= k && __popcll(__ballot(n.first[0])) + __popcll(__ballot(n.first[1])) >= V)
        t.rest = 0.0;
    t.mass += t.rest;
}

// With WS_DISTILL_TAIL, once log p_t is known: a q_t that the scores' rounding
// may have left counts as 0 where the student has no p_t for it.
constexpr float kNoTail = -103.972077f;   // log 2^-150
__device__ __forceinline__ void drop_rounding(Teacher& t, double tail) {
    if (t.rest <= (double)WS_DISTILL_ROUNDING && (float)tail < kNoTail) {
        t.mass -= t.rest;
        t.rest = 0.0;
    }
}

// ---------------------------------------------------------------------------
// Distillation: the loss.
//
// With WS_DISTILL_TAIL the pass sums the unlisted tokens only (a byte a slot in
// LDS marks the listed ones), and the few listed ones are added at the end: a
// tail far below the listed tokens keeps its own maximum and its full
// precision, which the difference of two sums near 1 would not.  Bound as the
// forward pass above: 1,024 rows of 131,072 BF16 with 32 entries 50 us (5.4
// TB/s), in two rounds of workgroups whose starts and ends show.

struct DistillParams {
    const void* logits;
    int64_t stride;
    const ws_topk_entry* teacher;
    float* loss;
    ws_row_stats* stats;
    float* tail;
    Sums* sums;          // [rows][parts], when a row has several parts
    const float* grad_loss;
    void* grad;
    int64_t grad_stride;
    int32_t vocab, k, mode;
    int32_t chunk, parts;
    int32_t mark_words;   // LDS words of marks
    float c, inv_tau;
};

// What the gradient of a row is made of: dz_j = scale 2^((z_j - max) c - base)
// a, and for the listed tokens scale (2^((z_j - max) c - base_listed) a_listed +
// add).  An unlisted token of a row with a tail is measured against the unlisted
// tokens' own sum, so that a tail too small for FP32 still divides:
//   p_j (M - q_t / p_t) = (p_j / p_t) (M p_t - q_t).
struct Slope {
    float max, base, base_listed;
    float a, a_listed;
    float b;       // entropy: a + b log2 p_j in a's place
    float scale;
    bool none;     // a row without a distribution: no gradient

    // Its logits are all -inf, so every power of two comes out 0.
    __device__ __forceinline__ void clear() {
        max = a = a_listed = b = 0.0f;
        base = base_listed = INFINITY;
        none = true;
    }
};

__device__ __forceinline__ Slope distill_slope(const Teacher& t, bool bad, float max,
                                               double logsum, double tail, float scale) {
    constexpr double kLog2e64 = 1.4426950408889634074;
    Slope s;
    s.none = false;
    s.max = max;
    s.base = s.base_listed = (float)(logsum * kLog2e64);
    s.a = s.a_listed = bad ? NAN : (float)t.mass;
    s.b = 0.0f;
    if (t.rest > 0.0 && !bad) {
        s.a = 0.0f;
        if (tail != -(double)INFINITY) {
            s.a = (float)(t.mass * small_exp(tail) - t.rest);
            s.base = (float)((logsum + tail) * kLog2e64);
        }
    }
    s.scale = scale;
    if (logsum == -(double)INFINITY && !bad) s.clear();
    return s;
}

// Row outputs from its sums, by wave 0; the slope for a gradient that follows.
__device__ __forceinline__ Slope finish_distill(const DistillParams& p, int64_t row, Sums sums,
                                                const Named& n, Teacher t, int lane) {
    float m = sums.m, s = sums.s;
    if (p.mode == WS_DISTILL_TAIL) {
        m = fmaxf(m, wave_max(fmaxf(n.z[0], n.z[1]), lane));
        float e = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (n.first[h]) e += __builtin_amdgcn_exp2f((n.z[h] - m) * p.c);
        s = (s == 0.0f ? 0.0f : s * __builtin_amdgcn_exp2f((sums.m - m) * p.c)) + wave_sum(e, lane);
    }
    const bool empty = s == 0.0f;
    // The three logarithms a row needs, in three lanes at once.
    const double logs = small_log(lane == 0 ? (double)s : lane == 1 ? (double)sums.s : t.rest);
    const double logsum = empty ? -(double)INFINITY : lane_d(logs, 0);
    double tail = -(double)INFINITY;
    if (p.mode == WS_DISTILL_TAIL && sums.s != 0.0f)
        tail = ((double)sums.m - (double)m) * p.inv_tau + lane_d(logs, 1) - logsum;
    if (p.mode == WS_DISTILL_TAIL) drop_rounding(t, tail);
    double loss = 0.0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (t.q[h] == 0.0) continue;
        const double logp = empty ? -(double)INFINITY
                                  : ((double)n.z[h] - (double)m) * p.inv_tau - logsum;
        loss += t.q[h] * (t.logq[h] - logp);
    }
    loss = wave_sum_d(loss, lane);
    if (t.rest > 0.0) loss += t.rest * (lane_d(logs, 2) - tail);
    if (lane == 0) {
        // A NaN or +inf in the row reaches its sum, but not a loss without terms.
        p.loss[row] = n.bad || s != s ? NAN : (float)loss;
        if (p.stats) p.stats[row] = {empty ? -INFINITY : m, (float)logsum};
        if (p.tail) p.tail[row] = (float)tail;
    }
    return distill_slope(t, n.bad, m, logsum, tail,
                         p.grad_loss ? p.grad_loss[row] * p.inv_tau : 0.0f);
}

// Marks the listed tokens of a part, one bit an element, one byte a slot, in
// `words` words of LDS.  EACH = 1: slot s at byte s; the marks reach past the
// part's slots as far as a batch of the pass does.  Otherwise a thread's EACH
// slots (s, s + NT, ...) lie side by side, to be read at once.
template <typename L, int NT, int EACH>
__device__ __forceinline__ void mark_listed(const Part<L>& part, const Named& n, uint32_t* mask,
                                            int words) {
    for (int i = threadIdx.x; i < words; i += NT) mask[i] = 0;
    __syncthreads();
    if (threadIdx.x < 64) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (n.id[h] >= (uint32_t)part.vocab) continue;
            const int e = (int)n.id[h] - part.e0;
            if (e < 0 || e >= part.n * L::VEC) continue;
            const int slot = e / L::VEC;
            const int at = EACH == 1 ? slot : slot % NT * EACH + slot / NT;
            atomicOr(&mask[at >> 2], 1u << ((at & 3) * 8 + e % L::VEC));
        }
    }
    __syncthreads();
}

// Dynamic LDS of a part with `slots` slots: its marks.
extern __shared__ __align__(16) uint32_t listed_marks[];

template <typename L, int NT, bool TAIL>
__global__ void __launch_bounds__(NT) distill_kernel(DistillParams p) {
    __shared__ Sums wave_sums[NT / 64];
    __shared__ __align__(16) uint32_t ids[WS_DISTILL_MAX_K];
    __shared__ float adds[WS_DISTILL_MAX_K];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x / (uint32_t)p.parts;
    Part<L> part;
    part.init(p.logits, row * p.stride, p.vocab, p.chunk, p.parts,
              (int)(blockIdx.x % (uint32_t)p.parts));
    Named n;
    Teacher t;
    if (tid < 64) {
        read_entries(n, p.teacher + row * p.k, p.k, lane);
        if (p.parts == 1) {
            read_named<L>(n, part.row, p.vocab, 0, p.vocab);
            t = weigh_teacher(n, p.k, p.mode, lane);
        }
    }
    if constexpr (TAIL) mark_listed<L, NT, 1>(part, n, listed_marks, p.mark_words);
    Sums a;
    SlotTrack unused;
    stream_part<L, NT, false, false, TAIL>(part, p.c, reinterpret_cast<const uint8_t*>(listed_marks),
                                           a, unused);
    a = group_join<NT, false>(a, p.c, wave_sums);
    if (p.parts > 1) {
        if (tid == 0) p.sums[blockIdx.x] = a;
    } else if (tid < 64) {
        if constexpr (TAIL) {
            merge_named(n, p.k, ids, adds, lane);
            settle_rest(t, n, p.k, p.vocab);
        }
        finish_distill(p, row, a, n, t, lane);
    }
}

template <typename L>
__global__ void __launch_bounds__(64) distill_join_kernel(DistillParams p) {
    __shared__ __align__(16) uint32_t ids[WS_DISTILL_MAX_K];
    __shared__ float adds[WS_DISTILL_MAX_K];
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    Sums a;
    a.init();
    for (int i = lane; i < p.parts; i += 64) a.add<false>(p.sums[row * p.parts + i], p.c);
    Named n;
    read_entries(n, p.teacher + row * p.k, p.k, lane);
    Teacher t = weigh_teacher(n, p.k, p.mode, lane);
    read_named<L>(n, static_cast<const typename L::Elem*>(p.logits) + row * p.stride, p.vocab, 0,
                  p.vocab);
    if (p.mode == WS_DISTILL_TAIL) {
        merge_named(n, p.k, ids, adds, lane);
        settle_rest(t, n, p.k, p.vocab);
    }
    finish_distill(p, row, wave_join<false>(a, p.c, lane), n, t, lane);
}

// ---------------------------------------------------------------------------
// Gradients.
//
// One pass that reads a slot, forms p from the row's statistics and stores the
// gradient; the few named tokens are written over afterwards.  Bound by HBM:
// 4,096 x 65,536 BF16 with entropy 175 us (6.1 TB/s read and written), 2,048 x
// 65,536 FP16 with 32 teacher entries 98 us (5.5 TB/s); a copy of the same
// bytes at 4.84 TB/s would take 222 and 111 us.  255 rows of 50,001 FP16, which
// fit the last-level cache, 13 us.

// Where a part's gradient goes: slots at the same place as the logits' slots
// when both rows start alike relative to 16 bytes, else element by element.
template <typename L>
struct PartOut {
    typename L::Elem* row;
    char* base;
    bool slots;

    __device__ __forceinline__ void init(const Part<L>& part, void* grad, int64_t at) {
        row = static_cast<typename L::Elem*>(grad) + at;
        slots = (((uintptr_t)row ^ (uintptr_t)part.row) & 15u) == 0;
        base = reinterpret_cast<char*>(row + part.e0);
    }
    // A slot that lies in the row whole.
    __device__ __forceinline__ void store(const Part<L>& part, int s,
                                          const float (&v)[L::VEC]) const {
        if (slots) {
            store_slot<L>(base + (uint32_t)s * 16u, L::pack(v));
            return;
        }
        typename L::Elem* to = row + (part.e0 + s * L::VEC);
#pragma unroll
        for (int j = 0; j < L::VEC; ++j) to[j] = L::down(v[j]);
    }
    __device__ __forceinline__ void store_edge(const Part<L>& part, int s,
                                               const float (&v)[L::VEC]) const {
#pragma unroll
        for (int j = 0; j < L::VEC; ++j) {
            const int e = part.e0 + s * L::VEC + j;
            if (e >= 0 && e < part.vocab) row[e] = L::down(v[j]);
        }
    }
};

template <typename L, bool ENT>
__device__ __forceinline__ void slope_values(const Slope& g, float c, float (&v)[L::VEC]) {
    const float a = g.a * g.scale, b = g.b * g.scale;
#pragma unroll
    for (int j = 0; j < L::VEC; ++j) {
        const float t = fmaf(v[j] - g.max, c, -g.base);
        const float prob = __builtin_amdgcn_exp2f(t);
        if constexpr (ENT) v[j] = prob * fmaf(b, fmaxf(t, kFar), a);
        else v[j] = prob * a;
    }
}

// The named tokens' values, written over what the pass left for them.
template <typename L, bool ENT, bool DISTILL>
__device__ __forceinline__ void store_named(const Slope& g, const Named& n, float c, int from,
                                            int to, typename L::Elem* row) {
    if (g.none) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (!n.first[h] || n.id[h] < (uint32_t)from || n.id[h] >= (uint32_t)to) continue;
        const float t = fmaf(n.z[h] - g.max, c, -(DISTILL ? g.base_listed : g.base));
        float a = DISTILL ? g.a_listed : g.a;
        if constexpr (ENT) a = fmaf(g.b, fmaxf(t, kFar), a);
        row[n.id[h]] = L::down((__builtin_amdgcn_exp2f(t) * a + n.add[h]) * g.scale);
    }
}

struct GradParams {
    const void* logits;
    void* grad;
    int64_t stride, grad_stride;
    const ws_row_stats* stats;
    const ws_topk_entry* entries;   // alternatives, or the teacher's entries
    const float* grad_entries;      // [rows][k], upstream of the alternatives
    const int32_t* targets;
    const float* grad_target;
    const float* entropy;
    const float* grad_entropy;
    const float* tail;              // distillation
    const float* grad_loss;
    int32_t vocab, k, mode;
    int32_t chunk, parts;
    float c, inv_tau;
};

// The row's slope and named tokens, by wave 0.
template <typename L, bool DISTILL>
__device__ __forceinline__ Slope grad_slope(const GradParams& p, int64_t row,
                                            const typename L::Elem* z, int from, int to, Named& n,
                                            uint32_t* ids, float* adds, int lane) {
    const ws_row_stats st = p.stats[row];
    if constexpr (DISTILL) {
        read_entries(n, p.entries + row * p.k, p.k, lane);
        read_named<L>(n, z, p.vocab, from, to);
        Teacher t = weigh_teacher(n, p.k, p.mode, lane);
        merge_named(n, p.k, ids, adds, lane);
        double tail = 0.0;
        if (p.mode == WS_DISTILL_TAIL) {
            settle_rest(t, n, p.k, p.vocab);
            tail = (double)p.tail[row];
            drop_rounding(t, tail);
        }
        return distill_slope(t, n.bad, st.max, (double)st.logsum, tail,
                             p.grad_loss[row] * p.inv_tau);
    } else {
        n.id[0] = n.id[1] = kAbsent;
        n.add[0] = n.add[1] = 0.0f;
        if (lane < p.k) {
            n.id[0] = (uint32_t)p.entries[row * p.k + lane].index;
            if (n.id[0] != kAbsent) n.add[0] = p.grad_entries[row * p.k + lane];
        } else if (lane == p.k && p.targets) {
            n.id[0] = (uint32_t)p.targets[row];
            if (n.id[0] != kAbsent) n.add[0] = p.grad_target[row];
        }
        read_named<L>(n, z, p.vocab, from, to);
        Slope s;
        s.none = false;
        s.max = st.max;
        s.base = s.base_listed = st.logsum * kLog2e;
        s.a = -wave_sum(n.add[0], lane);
        s.b = 0.0f;
        if (p.entropy) {
            // log p_j = log2 p_j log 2
            const float gh = p.grad_entropy[row];
            s.b = -gh * 0.69314718055994530942f;
            s.a -= gh * p.entropy[row];
        }
        if (n.bad) s.a = NAN;
        s.a_listed = s.a;
        s.scale = p.inv_tau;
        if (st.logsum == -INFINITY && !n.bad) s.clear();
        merge_named(n, p.k + 1, ids, adds, lane);
        return s;
    }
}

template <typename L, bool ENT, bool DISTILL>
__global__ void __launch_bounds__(256) grad_kernel(GradParams p) {
    constexpr int NT = 256, VEC = L::VEC;
    __shared__ __align__(16) uint32_t ids[WS_DISTILL_MAX_K];
    __shared__ float adds[WS_DISTILL_MAX_K];
    __shared__ Slope slope;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / (uint32_t)p.parts;
    Part<L> part;
    part.init(p.logits, row * p.stride, p.vocab, p.chunk, p.parts,
              (int)(blockIdx.x % (uint32_t)p.parts));
    PartOut<L> out;
    out.init(part, p.grad, row * p.grad_stride);
    const int from = part.e0 < 0 ? 0 : part.e0;
    const int to = part.e0 + part.n * VEC < p.vocab ? part.e0 + part.n * VEC : p.vocab;
    Named n;
    if (tid < 64) {
        const Slope s = grad_slope<L, DISTILL>(p, row, part.row, from, to, n, ids, adds, tid);
        if (tid == 0) slope = s;
    }
    __syncthreads();   // every named logit is read before any is overwritten
    const Slope g = slope;
    const int whole_to = part.full_from < part.full_to ? part.full_to : 0;
    for (int s = tid; s < whole_to; s += kBatch * NT) {
        uint4 w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) w[i] = part.load_near(s + i * NT);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (!part.whole(s + i * NT)) continue;
            float v[VEC];
            L::unpack(w[i], v);
            slope_values<L, ENT>(g, p.c, v);
            out.store(part, s + i * NT, v);
        }
    }
    // The slots that stick out of the row.
    if (tid < 2) {
        const int s = tid == 0 ? 0 : part.n - 1;
        if (!part.whole(s) && (tid == 0 || s > 0)) {
            float v[VEC];
            part.load_edge(s, v);
            slope_values<L, ENT>(g, p.c, v);
            out.store_edge(part, s, v);
        }
    }
    __syncthreads();
    if (tid < 64) store_named<L, ENT, DISTILL>(g, n, p.c, from, to, out.row);
}

// Loss and gradient of a row in one pass: the row stays in the registers of
// its workgroup (sixteen slots a thread), so it is read once and the gradient
// written once (counted for 2,048 x 131,072 BF16: 542 MB and 543 MB, the logits
// being 537), where a loss kernel and a gradient kernel read it twice.  At most
// 128 registers a thread, so that a CU holds sixteen waves: one row of up to
// 131,072 16-bit logits, two of up to 65,536 or four of up to 32,768.
//
// Measured (MI355X, 64 entries, 1.07 GB read and written): 4,096 x 65,536 198 us
// (5.4 TB/s), 2,048 x 131,072 217 us (5.0 TB/s).  With one row to a CU its
// phases follow one another: loads and the sums, the join and FP64 finish by one
// wave (some 2 us a row), then exponentials and stores.  777 rows of 50,001 FP32
// take 71.6 us (4.3 TB/s): three full rounds over 256 CUs and a fourth of nine
// rows.  Tried when this took 253 us and not kept: walking the rows with the
// next row's loads issued as registers come free (280 us; loads and stores
// return in order), and reading the row a second time from the last-level cache
// with two rows to a CU (266 us).
constexpr int kHeld = kHeldSlots;
// With marks, slots asked for before the workgroup waits for them: a CU takes
// so many loads at once, so a barrier behind all of a row's loads waits for
// most of their data (2,048 x 131,072 BF16: 254 us with all 16 slots asked for
// before it, 249 with 8, 243 with 4, 234 with 2).
constexpr int kAhead = 2;

// Has the compiler work a value out again where it is used again, rather than
// hold what it derived the first time (a slot's elements, sixteen lane masks).
__device__ __forceinline__ void forget(uint4& w) {
    asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
}
__device__ __forceinline__ int forget(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

template <typename L, int NT, bool TAIL>
__global__ void __launch_bounds__(NT, 4) distill_step_kernel(DistillParams p) {
    constexpr int VEC = L::VEC, R = kHeld, B = 2;
    __shared__ Sums wave_sums[NT / 64];
    __shared__ __align__(16) uint32_t ids[WS_DISTILL_MAX_K];
    __shared__ float adds[WS_DISTILL_MAX_K];
    __shared__ Slope slope;
    __shared__ Aside aside;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x;
    Part<L> part;
    part.init(p.logits, row * p.stride, p.vocab, p.chunk, 1, 0);
    float v[VEC];
    // The teacher's entries before the row, as loads return in order.
    Named n;
    Teacher t;
    RawEntries raw;
    if (tid < 64) raw.load(p.teacher + row * p.k, p.k, lane);
    uint4 w[R];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) w[i] = part.load_near(tid + i * NT);
    if (tid < 64) raw.into(n, p.k, lane);
    if constexpr (TAIL) mark_listed<L, NT, R>(part, n, listed_marks, R * NT / 4);
#pragma unroll
    for (int i = kAhead; i < R; ++i) w[i] = part.load_near(tid + i * NT);
    if (tid < 64) {   // while the row is on its way
        read_named<L>(n, part.row, p.vocab, 0, p.vocab);
        t = weigh_teacher(n, p.k, p.mode, lane);
        merge_named(n, p.k, ids, adds, lane);
        if constexpr (TAIL) settle_rest(t, n, p.k, p.vocab);
        aside.put(n, t, lane);
    }
    uint4 marks = make_uint4(0, 0, 0, 0);   // this thread's, a byte a slot
    static_assert(R == sizeof(marks), "sixteen slots a thread");
    if constexpr (TAIL) marks = *reinterpret_cast<const uint4*>(listed_marks + tid * (R / 4));
    Sums a;
    SlotTrack unused;
    a.init();
#pragma unroll
    for (int i = 0; i < R; i += B) {
        float x[B][VEC];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int slot = forget(tid) + (i + j) * NT;
            if (__ballot(!part.whole(slot)) != 0) {
                if (!part.whole(slot)) w[i + j] = L::none();   // beyond the row
                if (!part.whole(slot) && slot < part.n) {      // sticks out of it
                    part.load_edge(slot, v);
                    w[i + j] = L::pack(v);
                }
            }
            if constexpr (TAIL) {
                // Listed tokens leave the held row for good: store_named
                // writes theirs.
                const uint32_t word = i + j < 4 ? marks.x : i + j < 8 ? marks.y
                                    : i + j < 12 ? marks.z : marks.w;
                const uint32_t mark = word >> (i + j) % 4 * 8 & 0xffu;
                if (__ballot(mark != 0) != 0) {
                    L::unpack(w[i + j], v);
                    hide_listed<VEC>(mark, v);
                    w[i + j] = L::pack(v);
                }
            }
            forget(w[i + j]);
            L::unpack(w[i + j], x[j]);
        }
        take_slots<L, NT, false, false, false>(x, 0, p.c, nullptr, a, unused);
        __builtin_amdgcn_sched_barrier(0);
    }
    a = group_join<NT, false>(a, p.c, wave_sums);
    if (tid < 64) {
        aside.get(n, t, lane);
        const Slope s = finish_distill(p, row, a, n, t, lane);
        if (lane == 0) slope = s;
    }
    __syncthreads();   // every named logit is read before any is overwritten
    const Slope g = slope;
    PartOut<L> out;
    out.init(part, p.grad, row * p.grad_stride);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int s = forget(tid) + i * NT;
        forget(w[i]);
        if (s < part.n) {
            L::unpack(w[i], v);
            slope_values<L, false>(g, p.c, v);
            if (part.whole(s)) out.store(part, s, v);
            else out.store_edge(part, s, v);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
    if (tid < 64) store_named<L, false, true>(g, n, p.c, 0, p.vocab, out.row);
}

// ---------------------------------------------------------------------------

int device_ready(int32_t device) {
    int ndev = 0;
    if (hipGetDeviceCount(&ndev) != hipSuccess || device >= ndev) return WS_E_NO_DEVICE;
    int cur = -1;
    if (hipGetDevice(&cur) != hipSuccess) return WS_E_HIP;
    return cur == device ? WS_OK : WS_E_INVALID_ARG;
}

// CALL(type) for the matrix's element type and way through the caches.
#define WS_BY_TYPE(r, CALL)                                        \
    do {                                                           \
        const bool stream = streams(r);                            \
        if ((r).dtype == WS_DTYPE_F32) {                           \
            if (stream) { CALL(Streamed<F32>); }                   \
            else { CALL(F32); }                                    \
        } else if ((r).dtype == WS_DTYPE_F16) {                    \
            if (stream) { CALL(Streamed<F16>); }                   \
            else { CALL(F16); }                                    \
        } else {                                                   \
            if (stream) { CALL(Streamed<BF16>); }                  \
            else { CALL(BF16); }                                   \
        }                                                          \
    } while (0)

// Enqueues one kernel; its parameters are one struct, copied by the call.
template <typename P>
int launch(void (*kernel)(P), int64_t groups, int threads, const P& params, hipStream_t s,
           size_t lds = 0) {
    P copy = params;
    void* args[] = {&copy};
    const hipError_t e =
        hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3((uint32_t)groups),
                        dim3((uint32_t)threads), args, lds, s);
    return e == hipSuccess ? WS_OK : WS_E_HIP;
}

template <typename L>
int run_logprobs(const ws_rows& r, const LogprobsPlan& plan, const LogprobsParams& p,
                 hipStream_t s) {
    const bool ent = p.entropy != nullptr, top = p.k > 0;
#define PICK(NT)                                                                           \
    (top ? (ent ? logprobs_kernel<L, NT, true, true> : logprobs_kernel<L, NT, false, true>) \
         : (ent ? logprobs_kernel<L, NT, true, false> : logprobs_kernel<L, NT, false, false>))
    const auto kernel = plan.threads == 64 ? PICK(64) : plan.threads == 256 ? PICK(256) : PICK(1024);
#undef PICK
    const int v = launch(kernel, (int64_t)r.rows * plan.parts, plan.threads, p, s);
    if (v != WS_OK || plan.parts == 1) return v;
    return launch(ent ? logprobs_join_kernel<L, true> : logprobs_join_kernel<L, false>, r.rows,
                  kJoin, p, s);
}

float scale_c(const ws_rows& r) { return (float)(1.4426950408889634074 / (double)r.temperature); }
float scale_inv(const ws_rows& r) { return (float)(1.0 / (double)r.temperature); }

template <typename L>
int run_grad(const ws_rows& r, GradParams g, bool distill, hipStream_t s) {
    const GradPlan plan = plan_grad(r);
    g.chunk = plan.chunk;
    g.parts = plan.parts;
    const auto kernel = distill ? grad_kernel<L, false, true>
                                : (g.entropy ? grad_kernel<L, true, false>
                                             : grad_kernel<L, false, false>);
    return launch(kernel, (int64_t)r.rows * plan.parts, 256, g, s);
}

template <typename L, bool TAIL>
int run_distill(const ws_rows& r, const DistillPlan& plan, const DistillParams& p, hipStream_t s) {
    const size_t lds = TAIL ? (size_t)plan.mark_bytes : 0;
    if (plan.held > 0) {
        const auto kernel = plan.threads == 256   ? distill_step_kernel<L, 256, TAIL>
                            : plan.threads == 512 ? distill_step_kernel<L, 512, TAIL>
                                                  : distill_step_kernel<L, 1024, TAIL>;
        return launch(kernel, r.rows, plan.threads, p, s, lds);
    }
    const int v = launch(plan.threads == 64    ? distill_kernel<L, 64, TAIL>
                         : plan.threads == 256 ? distill_kernel<L, 256, TAIL>
                                               : distill_kernel<L, 1024, TAIL>,
                         (int64_t)r.rows * plan.parts, plan.threads, p, s, lds);
    if (v != WS_OK || plan.parts == 1) return v;
    return launch(distill_join_kernel<L>, r.rows, 64, p, s);
}

int enqueue_distill_grad(const ws_rows& r, const ws_distill_grad_args& a, hipStream_t s) {
    GradParams g{};
    g.logits = a.logits;
    g.grad = a.grad_logits;
    g.stride = r.row_stride;
    g.grad_stride = a.grad_stride;
    g.stats = a.stats;
    g.entries = a.teacher;
    g.tail = a.tail;
    g.grad_loss = a.grad_loss;
    g.vocab = r.vocab;
    g.k = a.teacher_k;
    g.mode = a.mode;
    g.c = scale_c(r);
    g.inv_tau = scale_inv(r);
#define CALL(L) return run_grad<L>(r, g, true, s)
    WS_BY_TYPE(r, CALL);
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
    using namespace ws;
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
#define CALL(L) return run_logprobs<L>(r, plan, p, s)
    WS_BY_TYPE(r, CALL);
#undef CALL
}

extern "C" int ws_logprobs_grad(const ws_rows* rows, const ws_logprobs_grad_args* args,
                                void* stream) {
    using namespace ws;
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
#define CALL(L) return run_grad<L>(r, g, false, s)
    WS_BY_TYPE(r, CALL);
#undef CALL
}

extern "C" int ws_distill_workspace(const ws_rows* rows, int32_t mode, int32_t gradient,
                                    size_t* bytes) {
    const int v = ws::validate_rows(rows);
    if (v != WS_OK) return v;
    if (!bytes || ws::validate_teacher(1, mode) != WS_OK || (gradient != 0 && gradient != 1))
        return WS_E_INVALID_ARG;
    *bytes = ws::plan_distill(*rows, mode, gradient == 1, false).workspace;
    return WS_OK;
}

extern "C" int ws_distill(const ws_rows* rows, const ws_distill_args* args, void* stream) {
    using namespace ws;
    int v = ws::validate_distill(rows, args);
    if (v != WS_OK) return v;
    const ws_rows& r = *rows;
    if (r.rows == 0) return WS_OK;
    const bool gradient = args->grad_logits != nullptr;
    const ws::DistillPlan plan =
        ws::plan_distill(r, args->mode, gradient, ws::rows_aligned(r, args->logits));
    v = ws::validate_workspace(args->workspace, args->workspace_bytes, plan.workspace);
    if (v != WS_OK) return v;
    v = ws::device_ready(r.device);
    if (v != WS_OK) return v;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    ws::DistillParams p{};
    p.logits = args->logits;
    p.stride = r.row_stride;
    p.teacher = args->teacher;
    p.loss = args->loss;
    p.stats = args->stats;
    p.tail = args->tail;
    p.vocab = r.vocab;
    p.k = args->teacher_k;
    p.mode = args->mode;
    p.chunk = plan.chunk;
    p.parts = plan.parts;
    p.mark_words = plan.mark_bytes / 4;
    p.c = ws::scale_c(r);
    p.inv_tau = ws::scale_inv(r);
    char* space = static_cast<char*>(args->workspace);
    if (plan.parts > 1) p.sums = reinterpret_cast<ws::Sums*>(space + plan.sums_at);
    if (plan.held > 0) {
        p.grad_loss = args->grad_loss;
        p.grad = args->grad_logits;
        p.grad_stride = args->grad_stride;
    } else if (gradient) {
        // The loss first, then its gradient from the statistics it leaves.
        if (!p.stats) p.stats = reinterpret_cast<ws_row_stats*>(space);
        if (!p.tail) p.tail = reinterpret_cast<float*>(space + plan.tail_at);
    }
#define CALL(L)                                                                       \
    v = args->mode == WS_DISTILL_TAIL ? run_distill<L, true>(r, plan, p, s)   \
                                      : run_distill<L, false>(r, plan, p, s)
    WS_BY_TYPE(r, CALL);
#undef CALL
    if (v != WS_OK || !gradient || plan.held > 0) return v;
    ws_distill_grad_args g{};
    g.logits = args->logits;
    g.teacher = args->teacher;
    g.stats = p.stats;
    g.tail = p.tail;
    g.grad_loss = args->grad_loss;
    g.grad_logits = args->grad_logits;
    g.grad_stride = args->grad_stride;
    g.teacher_k = args->teacher_k;
    g.mode = args->mode;
    return ws::enqueue_distill_grad(r, g, s);
}

extern "C" int ws_distill_grad(const ws_rows* rows, const ws_distill_grad_args* args,
                               void* stream) {
    int v = ws::validate_distill_grad(rows, args);
    if (v != WS_OK) return v;
    if (rows->rows == 0) return WS_OK;
    v = ws::device_ready(rows->device);
    if (v != WS_OK) return v;
    return ws::enqueue_distill_grad(*rows, *args, static_cast<hipStream_t>(stream));
}
