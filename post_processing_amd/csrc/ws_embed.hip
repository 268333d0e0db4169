// ws_embed.hip -- embedding lookup with scaling and its gradient by sorted
// tokens (ws_states.h), written for gfx950 (CDNA4, wave64).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ws_enqueue.h"
#include "ws_lanes.h"
#include "ws_state_slots.h"
#include "ws_states.h"
#include "ws_states_plan.h"

namespace ws {
namespace {

struct EmbedParams {
    const void* table;
    const int32_t* ids;
    void* out;
    int64_t table_stride, out_stride;
    int32_t rows;
    int32_t width;
    int32_t vocab;
    int32_t lanes;   // threads to a row
    float scale;
};

// A copy: bound by HBM, or for few rows by the index's and the row's latency
// one after the other.
template <typename L>
__global__ void __launch_bounds__(kLookupThreads) embed_kernel(EmbedParams p) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC;
    const int lane = threadIdx.x & (p.lanes - 1);
    const int64_t row =
        (int64_t)blockIdx.x * (kLookupThreads / p.lanes) + threadIdx.x / (uint32_t)p.lanes;
    if (row >= p.rows) return;
    const int32_t id = p.ids[row];
    const bool named = (uint32_t)id < (uint32_t)p.vocab;
    const Elem* from = static_cast<const Elem*>(p.table) + (int64_t)(named ? id : 0) * p.table_stride;
    Elem* to = static_cast<Elem*>(p.out) + row * p.out_stride;
    const float other = id == -1 ? 0.0f : NAN;
    for (int c = lane * VEC; c < p.width; c += p.lanes * VEC) {
        float v[VEC];
        L::unpack(load_columns<L>(from, c, p.width), v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = named ? v[j] * p.scale : other;
        store_columns<L>(to, c, p.width, v);
    }
}

// ---------------------------------------------------------------------------
// Gradient.
//
// Tokens are sorted by a stable radix sort, a digit of kDigitBits a pass: every
// tile counts its digits, the counts are summed, every tile puts its tokens
// where they belong.  Then blocks of sorted rows are added, each thread its
// columns: a token whose rows lie in one block is written at once; of a token
// that goes over a border each block leaves a partial sum, and the block where
// the token begins has them added in order.  So no sum depends on timing, and
// one token that half the rows name is as many blocks' work as half the rows.

constexpr int kSortThreads = 256;
constexpr int kSortEach = kSortTile / kSortThreads;
constexpr int kSortWaves = kSortThreads / 64;

struct SortParams {
    const int32_t* ids;        // the first pass reads these
    const uint32_t* keys_in;
    const uint32_t* rows_in;
    uint32_t* keys_out;
    uint32_t* rows_out;
    uint32_t* counts;          // [tiles][kDigits]
    int32_t n;
    int32_t vocab;
    int32_t tiles;
    int32_t shift;
};

__device__ __forceinline__ uint32_t key_of(const SortParams& p, int i) {
    if (p.shift > 0) return p.keys_in[i];
    const uint32_t id = (uint32_t)p.ids[i];
    return id < (uint32_t)p.vocab ? id : (uint32_t)p.vocab;
}

__device__ __forceinline__ uint32_t digit_of(uint32_t key, int shift) {
    return key >> shift & (kDigits - 1);
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortParams p) {
    __shared__ uint32_t count[kDigits];
    for (int d = threadIdx.x; d < kDigits; d += kSortThreads) count[d] = 0;
    __syncthreads();
    const int from = blockIdx.x * kSortTile;
#pragma unroll
    for (int i = 0; i < kSortEach; ++i) {
        const int at = from + i * kSortThreads + (int)threadIdx.x;
        if (at < p.n) atomicAdd(&count[digit_of(key_of(p, at), p.shift)], 1u);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < kDigits; d += kSortThreads)
        p.counts[(int64_t)blockIdx.x * kDigits + d] = count[d];
}

// The exclusive sum across a workgroup of one value a thread.
template <int NT>
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t* waves) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t upto = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t other = __shfl_up(upto, d);
        if (lane >= d) upto += other;
    }
    if (lane == 63) waves[wave] = upto;
    __syncthreads();
    uint32_t before = upto - v;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) before += i < wave ? waves[i] : 0;
    return before;
}

// counts[tile][digit] becomes where the tile's tokens of that digit go: one
// digit a thread.
__global__ void __launch_bounds__(kDigits) sort_scan_kernel(SortParams p) {
    __shared__ uint32_t waves[kDigits / 64];
    uint32_t total = 0;
    for (int t = 0; t < p.tiles; ++t) total += p.counts[(int64_t)t * kDigits + threadIdx.x];
    uint32_t at = sum_before<kDigits>(total, waves);
    for (int t = 0; t < p.tiles; ++t) {
        uint32_t* c = p.counts + (int64_t)t * kDigits + threadIdx.x;
        const uint32_t n = *c;
        *c = at;
        at += n;
    }
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortParams p) {
    __shared__ uint32_t next[kSortWaves][kDigits];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < kSortWaves * kDigits; i += kSortThreads) (&next[0][0])[i] = 0;
    __syncthreads();
    // A wave takes 64 neighbouring tokens at a time: lanes of the same digit
    // find each other bit by bit, so equal digits keep their order.
    const int from = blockIdx.x * kSortTile + wave * (kSortTile / kSortWaves) + lane;
    uint32_t key[kSortEach], rank[kSortEach];
#pragma unroll
    for (int i = 0; i < kSortEach; ++i) {
        const int at = from + i * 64;
        key[i] = at < p.n ? key_of(p, at) : 0;
    }
#pragma unroll
    for (int i = 0; i < kSortEach; ++i) {
        const uint32_t d = digit_of(key[i], p.shift);
        uint64_t same = __ballot(from + i * 64 < p.n);
#pragma unroll
        for (int b = 0; b < kDigitBits; ++b) {
            const uint64_t set = __ballot(d >> b & 1u);
            same &= d >> b & 1u ? set : ~set;
        }
        const int before = lanes_below(same);
        rank[i] = next[wave][d] + (uint32_t)before;
        wave_lds_sync();
        if (from + i * 64 < p.n && before == 0) next[wave][d] += (uint32_t)__popcll(same);
        wave_lds_sync();
    }
    __syncthreads();
    for (int d = tid; d < kDigits; d += kSortThreads) {
        uint32_t at = p.counts[(int64_t)blockIdx.x * kDigits + d];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t n = next[w][d];
            next[w][d] = at;
            at += n;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortEach; ++i) {
        const int at = from + i * 64;
        if (at >= p.n) continue;
        const uint32_t to = next[wave][digit_of(key[i], p.shift)] + rank[i];
        p.keys_out[to] = key[i];
        p.rows_out[to] = p.shift > 0 ? p.rows_in[at] : (uint32_t)at;
    }
}

struct SumParams {
    const void* grad_out;
    const uint32_t* keys;   // sorted
    const uint32_t* rows;
    void* grad_table;
    float* partial;         // [blocks][2][partial_stride]
    int64_t stride, grad_stride, partial_stride;
    int32_t n;
    int32_t width;
    int32_t vocab;
    int32_t block, blocks;
    int32_t columns;
    int32_t grad_f32;
    int32_t accumulate;
    float scale;
};

template <typename L>
__device__ __forceinline__ void write_sum(const SumParams& p, uint32_t key, int c,
                                          float (&sum)[L::VEC]) {
    constexpr int VEC = L::VEC;
    char* at = static_cast<char*>(p.grad_table) +
               (int64_t)key * p.grad_stride * (p.grad_f32 ? 4 : (int)sizeof(typename L::Elem));
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] *= p.scale;
    if (p.accumulate) {
        float old[VEC];
        load_either<L>(at, p.grad_f32, c, p.width, old);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[j] += old[j];
    }
    store_either<L>(at, p.grad_f32, c, p.width, sum);
}

// The rows of one block of the sorted tokens.
template <typename L>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(SumParams p) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC;
    const int tile = blockIdx.x % (uint32_t)p.columns;
    const int64_t block = blockIdx.x / (uint32_t)p.columns;
    const int c = (tile * kSumThreads + (int)threadIdx.x) * VEC;
    if (c >= p.width) return;
    const int from = (int)block * p.block;
    const int to = p.n - from < p.block ? p.n : from + p.block;
    float sum[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
    bool began = from > 0 && p.keys[from - 1] == p.keys[from];   // in an earlier block
    for (int i = from; i < to; ++i) {
        const uint32_t key = p.keys[i];
        if (key >= (uint32_t)p.vocab) return;   // no token: all behind are
        float v[VEC];
        const Elem* row = static_cast<const Elem*>(p.grad_out) + (int64_t)p.rows[i] * p.stride;
        L::unpack(load_columns<L>(row, c, p.width), v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[j] += v[j];
        const bool last = i + 1 == p.n || p.keys[i + 1] != key;
        if (!last && i + 1 < to) continue;
        if (last && !began) {
            write_sum<L>(p, key, c, sum);
        } else {
            float* out = p.partial + (block * 2 + (began ? 0 : 1)) * p.partial_stride;
            store_either<L>(out, true, c, p.width, sum);
        }
        began = false;
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
    }
}

// A token that begins in this block and goes on: its partial sums in order.
template <typename L>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(SumParams p) {
    constexpr int VEC = L::VEC;
    const int tile = blockIdx.x % (uint32_t)p.columns;
    const int64_t block = blockIdx.x / (uint32_t)p.columns;
    const int from = (int)block * p.block;
    if (p.n - from <= p.block) return;   // the last block
    const int end = from + p.block;      // behind it
    const uint32_t key = p.keys[end];
    if (key >= (uint32_t)p.vocab || p.keys[end - 1] != key) return;
    if (from > 0 && p.keys[from - 1] == key) return;   // began earlier
    const int c = (tile * kSumThreads + (int)threadIdx.x) * VEC;
    if (c >= p.width) return;
    float sum[VEC];
    load_either<L>(p.partial + (block * 2 + 1) * p.partial_stride, true, c, p.width, sum);
    for (int64_t b = block + 1; b < p.blocks; ++b) {
        const int first = (int)b * p.block;
        if (p.keys[first] != key) break;
        float v[VEC];
        load_either<L>(p.partial + b * 2 * p.partial_stride, true, c, p.width, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[j] += v[j];
    }
    write_sum<L>(p, key, c, sum);
}

struct ClearParams {
    void* grad_table;
    int64_t grad_stride;
    int32_t vocab;
    int32_t width;
    int32_t lanes;
};

// Zeros, as embed_kernel lays its rows over a workgroup.
template <typename L>
__global__ void __launch_bounds__(kLookupThreads) clear_kernel(ClearParams p) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC;
    const int lane = threadIdx.x & (p.lanes - 1);
    const int64_t row =
        (int64_t)blockIdx.x * (kLookupThreads / p.lanes) + threadIdx.x / (uint32_t)p.lanes;
    if (row >= p.vocab) return;
    Elem* to = static_cast<Elem*>(p.grad_table) + row * p.grad_stride;
    const float v[VEC] = {};
    for (int c = lane * VEC; c < p.width; c += p.lanes * VEC) store_columns<L>(to, c, p.width, v);
}

// ---------------------------------------------------------------------------

#define WS_BY_DTYPE(dtype, CALL)                             \
    do {                                                     \
        if ((dtype) == WS_DTYPE_F32) { CALL(F32); }          \
        else if ((dtype) == WS_DTYPE_F16) { CALL(F16); }     \
        else { CALL(BF16); }                                 \
    } while (0)

int clear_table(const ws_states& t, const ws_embed_grad_args& a, hipStream_t s) {
    ws_states rows = t;
    rows.rows = a.vocab;
    rows.dtype = a.grad_dtype;
    const EmbedPlan plan = plan_embed(rows);
    ClearParams p{};
    p.grad_table = a.grad_table;
    p.grad_stride = a.grad_stride;
    p.vocab = a.vocab;
    p.width = t.width;
    p.lanes = plan.lanes;
#define CALL(L) return launch(clear_kernel<L>, plan.groups, kLookupThreads, p, s)
    WS_BY_DTYPE(a.grad_dtype, CALL);
#undef CALL
}

// Sorted keys and rows; returns which of the two buffers holds them.
int sort_tokens(const ws_states& t, const ws_embed_grad_args& a, const EmbedGradPlan& plan,
                hipStream_t s, int* where) {
    char* space = static_cast<char*>(a.workspace);
    uint32_t* keys[2], *rows[2];
    for (int i = 0; i < 2; ++i) {
        keys[i] = reinterpret_cast<uint32_t*>(space + plan.keys_at[i]);
        rows[i] = reinterpret_cast<uint32_t*>(space + plan.rows_at[i]);
    }
    SortParams p{};
    p.ids = a.ids;
    p.counts = reinterpret_cast<uint32_t*>(space + plan.counts_at);
    p.n = t.rows;
    p.vocab = a.vocab;
    p.tiles = plan.tiles;
    for (int pass = 0; pass < plan.passes; ++pass) {
        const int to = pass & 1;
        p.keys_in = keys[to ^ 1];
        p.rows_in = rows[to ^ 1];
        p.keys_out = keys[to];
        p.rows_out = rows[to];
        p.shift = pass * kDigitBits;
        int v = launch(sort_count_kernel, plan.tiles, kSortThreads, p, s);
        if (v == WS_OK) v = launch(sort_scan_kernel, 1, kDigits, p, s);
        if (v == WS_OK) v = launch(sort_place_kernel, plan.tiles, kSortThreads, p, s);
        if (v != WS_OK) return v;
        *where = to;
    }
    return WS_OK;
}

template <typename L>
int run_sum(const EmbedGradPlan& plan, const SumParams& p, hipStream_t s) {
    const int64_t groups = (int64_t)plan.blocks * plan.columns;
    const int v = launch(embed_sum_kernel<L>, groups, kSumThreads, p, s);
    if (v != WS_OK || plan.blocks == 1) return v;
    return launch(embed_join_kernel<L>, groups, kSumThreads, p, s);
}

}  // namespace
}  // namespace ws

extern "C" int ws_embed(const ws_states* states, const ws_embed_args* args, void* stream) {
    using namespace ws;
    int v = ws::validate_embed(states, args);
    if (v != WS_OK) return v;
    if (states->rows == 0) return WS_OK;
    v = ws::device_ready(states->device);
    if (v != WS_OK) return v;
    const ws::EmbedPlan plan = ws::plan_embed(*states);
    ws::EmbedParams p{};
    p.table = args->table;
    p.ids = args->ids;
    p.out = args->out;
    p.table_stride = args->table_stride;
    p.out_stride = states->row_stride;
    p.rows = states->rows;
    p.width = states->width;
    p.vocab = args->vocab;
    p.lanes = plan.lanes;
    p.scale = args->scale;
    const hipStream_t s = static_cast<hipStream_t>(stream);
#define CALL(L) return launch(embed_kernel<L>, plan.groups, kLookupThreads, p, s)
    WS_BY_DTYPE(states->dtype, CALL);
#undef CALL
}

extern "C" int ws_embed_grad_workspace(const ws_states* states, int32_t vocab, size_t* bytes) {
    const int v = ws::validate_states(states);
    if (v != WS_OK) return v;
    if (!bytes || vocab < 1 || vocab > WS_MAX_TOKENS) return WS_E_INVALID_ARG;
    *bytes = ws::plan_embed_grad(*states, vocab).workspace;
    return WS_OK;
}

extern "C" int ws_embed_grad(const ws_states* states, const ws_embed_grad_args* args,
                             void* stream) {
    using namespace ws;
    int v = ws::validate_embed_grad(states, args);
    if (v != WS_OK) return v;
    const ws::EmbedGradPlan plan = ws::plan_embed_grad(*states, args->vocab);
    v = ws::validate_workspace(args->workspace, args->workspace_bytes, plan.workspace);
    if (v != WS_OK) return v;
    if (states->rows == 0 && args->accumulate) return WS_OK;
    v = ws::device_ready(states->device);
    if (v != WS_OK) return v;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (!args->accumulate) {
        v = ws::clear_table(*states, *args, s);
        if (v != WS_OK || states->rows == 0) return v;
    }
    int where = 0;
    v = ws::sort_tokens(*states, *args, plan, s, &where);
    if (v != WS_OK) return v;
    char* space = static_cast<char*>(args->workspace);
    ws::SumParams p{};
    p.grad_out = args->grad_out;
    p.keys = reinterpret_cast<const uint32_t*>(space + plan.keys_at[where]);
    p.rows = reinterpret_cast<const uint32_t*>(space + plan.rows_at[where]);
    p.grad_table = args->grad_table;
    p.partial = reinterpret_cast<float*>(space + plan.partial_at);
    p.stride = states->row_stride;
    p.grad_stride = args->grad_stride;
    p.partial_stride = (int64_t)(ws::round16((size_t)states->width * 4) / 4);
    p.n = states->rows;
    p.width = states->width;
    p.vocab = args->vocab;
    p.block = plan.block;
    p.blocks = plan.blocks;
    p.columns = plan.columns;
    p.grad_f32 = args->grad_dtype == WS_DTYPE_F32;
    p.accumulate = args->accumulate;
    p.scale = args->scale;
#define CALL(L) return run_sum<L>(plan, p, s)
    WS_BY_DTYPE(states->dtype, CALL);
#undef CALL
}
