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

// A copy: bound by HBM and the caches, or for few rows by the index's and the row's
// latency one after the other (64 x 4,096 BF16 3.2 us; 16,384 x 4,096 from 32,768
// rows 42 us: 134.2 MB written and 78.6 read, tokens that repeat come from the
// caches).
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
// tile counts its digits, and from all tiles' counts puts its tokens where they
// belong (two tiles count all tokens for themselves, a launch less); up to kSortTile
// tokens are sorted by one workgroup in LDS.  (Counting a pass's digits while the pass
// before places them saves a launch, but its atomics wait behind the zeros: 16,384
// tokens 27 us instead of 16.)  Then blocks of sorted
// rows are added, each thread its columns: a token whose rows lie in one block is
// written at once; of a token that goes over a border each block leaves a partial
// sum, and the block where the token begins has them added in order.  So no sum
// depends on timing, and one token that half the rows name is as many blocks' work
// as half the rows.  Rows of few slots have their blocks side by side in a workgroup
// (200,000 x 64 BF16 into 50,000 rows 178 us with a block a workgroup and one
// workgroup that sums the tiles' counts, 59 with this and a wave a digit; 1,000,000
// rows 552 and 134).  The table's zeros are written by workgroups beside the sort's,
// whose few workgroups wait on latency.
//
// Bytes bound it: 16,384 rows into 32,768 x 4,096 BF16, 114 us for 268 MB of zeros,
// 134 of rows and 47 of sums written (4.0 TB/s): the sort with the zeros 46, the sums 58
// (while the zeros still drain), the join 10; added to what the table holds, without
// zeros, 68; into FP32 183.  Leaving out the zeros of rows that are named would save
// 45 MB; clearing workgroups that read all tokens for it cost as much (129 us), ones
// behind the sort that search its tokens have not been tried.  Sorted, 777 x 1,000 FP32
// rows take 18 us: three launches, each a chain of latencies (sort 7.8, sums 5.7, join
// 3.6); few rows go without (embed_few_kernel).

struct ClearParams {
    void* table;
    int64_t stride;
    int32_t from, to;   // rows
    int32_t width;
    int32_t lanes;      // threads to a row
    int32_t f32;
};

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
    int32_t passes;            // of sort_few_kernel
    ClearParams clear;         // by the workgroups behind the tiles
};

// Zeros: rows of the table, kClearRows a workgroup, but for those whose bits `skip` has.
template <typename L, int NT>
__device__ __forceinline__ void clear_rows(const ClearParams& p, int group, uint32_t skip = 0) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC;
    const int lane = threadIdx.x & (p.lanes - 1), each = NT / p.lanes;
    const int first = p.from + group * kClearRows;
    const int end = first + kClearRows < p.to ? first + kClearRows : p.to;
    const float v[VEC] = {};
    for (int row = first + (int)(threadIdx.x / (uint32_t)p.lanes); row < end; row += each) {
        if (skip >> (row - first) & 1u) continue;
        Elem* to = static_cast<Elem*>(p.table) + (int64_t)row * p.stride;
        for (int c = lane * VEC; c < p.width; c += p.lanes * VEC)
            store_columns<L>(to, c, p.width, v);
    }
}

__device__ __forceinline__ void clear_part(const ClearParams& p, int group) {
    // (zeros are the same bits in FP16 and BF16)
    if (p.f32) clear_rows<F32, kSortThreads>(p, group);
    else clear_rows<BF16, kSortThreads>(p, group);
}

__global__ void __launch_bounds__(kSortThreads) clear_kernel(ClearParams p) {
    clear_part(p, blockIdx.x);
}

__device__ __forceinline__ uint32_t key_of(const SortParams& p, int i) {
    if (p.shift > 0) return p.keys_in[i];
    const uint32_t id = (uint32_t)p.ids[i];
    return id < (uint32_t)p.vocab ? id : (uint32_t)p.vocab;
}

__device__ __forceinline__ uint32_t digit_of(uint32_t key, int shift) {
    return key >> shift & (kDigits - 1);
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortParams p) {
    if ((int)blockIdx.x >= p.tiles) {
        clear_part(p.clear, blockIdx.x - p.tiles);
        return;
    }
    __shared__ uint32_t count[kDigits];
    const int tid = threadIdx.x;
    if (tid < kDigits) count[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortEach; ++i) {
        const int at = (int)blockIdx.x * kSortTile + i * kSortThreads + tid;
        if (at < p.n) atomicAdd(&count[digit_of(key_of(p, at), p.shift)], 1u);
    }
    __syncthreads();
    if (tid < kDigits) p.counts[(int64_t)blockIdx.x * kDigits + tid] = count[tid];
}

// The exclusive sum over the first kDigits threads of one value each, which the
// others take part in with 0.
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t* waves) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t upto = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t other = __shfl_up(upto, d);
        if (lane >= d) upto += other;
    }
    if (lane == 63 && wave < kDigits / 64) waves[wave] = upto;
    __syncthreads();
    uint32_t before = upto - v;
#pragma unroll
    for (int i = 0; i < kDigits / 64; ++i) before += i < wave ? waves[i] : 0;
    return before;
}

// Many tiles: counts[tile][digit] becomes how many tokens of the digit are in the
// tiles before, and counts[tiles][digit] how many there are: a digit a wave, whose
// lanes take neighbouring tiles.
__global__ void __launch_bounds__(kScanDigits * 64) sort_scan_kernel(SortParams p) {
    const int lane = threadIdx.x & 63;
    uint32_t* c = p.counts + blockIdx.x * kScanDigits + (threadIdx.x >> 6);
    const int each = (p.tiles + 63) / 64;
    const int first = lane * each, end = first + each < p.tiles ? first + each : p.tiles;
    uint32_t total = 0;
#pragma unroll 4
    for (int t = first; t < end; ++t) total += c[(int64_t)t * kDigits];
    uint32_t upto = total;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t other = __shfl_up(upto, d);
        if (lane >= d) upto += other;
    }
    if (lane == 63) c[(int64_t)p.tiles * kDigits] = upto;
    uint32_t at = upto - total;
    for (int t = first; t < end; ++t) {
        const uint32_t n = c[(int64_t)t * kDigits];
        c[(int64_t)t * kDigits] = at;
        at += n;
    }
}

struct SortTile {
    uint32_t next[kSortWaves][kDigits];
    uint32_t waves[kDigits / 64];
};

// Ranks of a tile's tokens among those of their digit in their wave, whose
// counts are left in next[wave].  A wave has 64 * kSortEach neighbouring tokens,
// 64 at a time: lanes of the same digit find each other bit by bit, so equal digits
// keep their order.
__device__ __forceinline__ void rank_tile(const uint32_t (&key)[kSortEach], int first, int n,
                                          int shift, SortTile& t, uint32_t (&rank)[kSortEach]) {
    const int tid = threadIdx.x, wave = tid >> 6;
    for (int i = tid; i < kSortWaves * kDigits; i += kSortThreads) (&t.next[0][0])[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortEach; ++i) {
        const uint32_t d = digit_of(key[i], shift);
        const bool there = first + i * 64 < n;
        uint64_t same = __ballot(there);
#pragma unroll
        for (int b = 0; b < kDigitBits; ++b) {
            const uint64_t set = __ballot(d >> b & 1u);
            same &= d >> b & 1u ? set : ~set;
        }
        const int before = lanes_below(same);
        rank[i] = t.next[wave][d] + (uint32_t)before;
        wave_lds_sync();
        if (there && before == 0) t.next[wave][d] += (uint32_t)__popcll(same);
        wave_lds_sync();
    }
    __syncthreads();
}

// next[wave][digit] from counts to places, the tile's tokens of a digit going to
// `at` and behind: one digit a thread.
__device__ __forceinline__ void place_tile(SortTile& t, uint32_t at) {
    const int d = threadIdx.x;
    if (d < kDigits) {
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t n = t.next[w][d];
            t.next[w][d] = at;
            at += n;
        }
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortParams p) {
    if ((int)blockIdx.x >= p.tiles) {
        clear_part(p.clear, blockIdx.x - p.tiles);
        return;
    }
    __shared__ SortTile tile;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int first = (int)blockIdx.x * kSortTile + wave * 64 * kSortEach + lane;
    uint32_t key[kSortEach], row[kSortEach], rank[kSortEach];
#pragma unroll
    for (int i = 0; i < kSortEach; ++i) {
        const int at = first + i * 64 < p.n ? first + i * 64 : p.n - 1;
        key[i] = key_of(p, at);
        row[i] = p.shift > 0 ? p.rows_in[at] : (uint32_t)at;
    }
    // Where the tile's tokens of a digit go.
    uint32_t at = 0, total = 0;
    if (p.tiles <= kOwnTiles) {   // counted here, all tiles
        uint32_t* all = tile.next[0];
        uint32_t* earlier = tile.next[1];
        if (tid < kDigits) all[tid] = earlier[tid] = 0;
        __syncthreads();
        for (int i = tid; i < p.n; i += kSortThreads) {
            const uint32_t d = digit_of(key_of(p, i), p.shift);
            atomicAdd(&all[d], 1u);
            if (i < (int)blockIdx.x * kSortTile) atomicAdd(&earlier[d], 1u);
        }
        __syncthreads();
        if (tid < kDigits) {
            total = all[tid];
            at = earlier[tid];
        }
        __syncthreads();   // read before rank_tile clears them
    } else if (tid < kDigits && p.tiles > kScanTiles) {
        at = p.counts[(int64_t)blockIdx.x * kDigits + tid];
        total = p.counts[(int64_t)p.tiles * kDigits + tid];
    } else if (tid < kDigits) {
#pragma unroll 8
        for (int t = 0; t < p.tiles; ++t) {
            const uint32_t c = p.counts[t * kDigits + tid];
            total += c;
            at += t < (int)blockIdx.x ? c : 0;
        }
    }
    at += sum_before(total, tile.waves);
    rank_tile(key, first, p.n, p.shift, tile, rank);
    place_tile(tile, at);
#pragma unroll
    for (int i = 0; i < kSortEach; ++i) {
        if (first + i * 64 >= p.n) continue;
        const uint32_t to = tile.next[wave][digit_of(key[i], p.shift)] + rank[i];
        p.keys_out[to] = key[i];
        p.rows_out[to] = row[i];
    }
}

// All passes over at most kSortTile tokens.
__global__ void __launch_bounds__(kSortThreads) sort_few_kernel(SortParams p) {
    if (blockIdx.x >= 1) {
        clear_part(p.clear, blockIdx.x - 1);
        return;
    }
    __shared__ SortTile tile;
    __shared__ uint32_t keys[kSortTile], rows[kSortTile];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int first = wave * 64 * kSortEach + lane;
    uint32_t key[kSortEach], row[kSortEach], rank[kSortEach];
#pragma unroll
    for (int i = 0; i < kSortEach; ++i) {
        const int at = first + i * 64 < p.n ? first + i * 64 : p.n - 1;
        row[i] = (uint32_t)at;
        key[i] = key_of(p, at);
    }
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * kDigitBits;
        rank_tile(key, first, p.n, shift, tile, rank);
        uint32_t total = 0;
        if (tid < kDigits) {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) total += tile.next[w][tid];
        }
        place_tile(tile, sum_before(total, tile.waves));
#pragma unroll
        for (int i = 0; i < kSortEach; ++i) {
            if (first + i * 64 >= p.n) continue;
            const uint32_t to = tile.next[wave][digit_of(key[i], shift)] + rank[i];
            keys[to] = key[i];
            rows[to] = row[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortEach; ++i) {
            const int at = first + i * 64 < p.n ? first + i * 64 : p.n - 1;
            key[i] = keys[at];
            row[i] = rows[at];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kSortEach; ++i) {
        if (first + i * 64 >= p.n) continue;
        p.keys_out[first + i * 64] = key[i];
        p.rows_out[first + i * 64] = row[i];
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
    int32_t lanes;          // threads to a block
    int32_t grad_f32;
    int32_t accumulate;
    float scale;
};

// A thread's columns of every row: `at` and the VEC - 1 behind, of which those
// from at + own on are its own.  A last slot that would end behind the row begins
// earlier (its first columns are its neighbour's too), so that loads hang on no
// condition; rows of less than a slot are read column by column.
template <typename L>
struct Columns {
    int at, own, width;

    __device__ __forceinline__ Columns(int c, int row_width) : at(c), own(0), width(row_width) {
        if (c + L::VEC > width && width >= L::VEC) {
            at = width - L::VEC;
            own = c - at;
        }
    }
    __device__ __forceinline__ bool short_row() const { return width < L::VEC; }
    __device__ __forceinline__ uint4 load(const typename L::Elem* row) const {
        return load_loose<L>(row + at);
    }
    __device__ __forceinline__ void load_sum(const float* row, float (&v)[L::VEC]) const {
        load_either<L>(row, true, at, width, v);
    }
    __device__ __forceinline__ void store_sum(float* row, const float (&v)[L::VEC]) const {
        store_either<L>(row, true, at, width, v);   // shared columns hold the same
    }
};

template <typename L>
__device__ __forceinline__ void write_sum(const SumParams& p, uint32_t key, const Columns<L>& c,
                                          float (&sum)[L::VEC]) {
    constexpr int VEC = L::VEC;
    char* row = static_cast<char*>(p.grad_table) +
                (int64_t)key * p.grad_stride * (p.grad_f32 ? 4 : (int)sizeof(typename L::Elem));
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] *= p.scale;
    if (c.own == 0) {
        if (p.accumulate) {
            float old[VEC];
            load_either<L>(row, p.grad_f32, c.at, p.width, old);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum[j] += old[j];
        }
        store_either<L>(row, p.grad_f32, c.at, p.width, sum);
        return;
    }
    // Its own columns only: the others are their thread's to add to.
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        if (j < c.own) continue;
        if (p.grad_f32) {
            float* to = reinterpret_cast<float*>(row) + c.at + j;
            *to = p.accumulate ? sum[j] + *to : sum[j];
        } else {
            typename L::Elem* to = reinterpret_cast<typename L::Elem*>(row) + c.at + j;
            *to = L::down(p.accumulate ? sum[j] + L::up(*to) : sum[j]);
        }
    }
}

// A value that WAVES says is the same in a whole wave.
template <bool WAVES>
__device__ __forceinline__ uint32_t same(uint32_t v) {
    return WAVES ? __builtin_amdgcn_readfirstlane(v) : v;
}

// The rows of blocks of the sorted tokens, kSumAhead at a time on their way; rows of
// few slots have several blocks side by side, WAVES: each of whole waves.
constexpr int kSumAhead = 8;

template <typename L, bool WAVES>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(SumParams p) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC, U = kSumAhead;
    __shared__ uint32_t all_keys[kMostRows + 2], all_rows[kMostRows];
    const int tile = blockIdx.x % (uint32_t)p.columns;
    const int side = threadIdx.x / (uint32_t)p.lanes, beside = kSumThreads / p.lanes;
    const int64_t first = blockIdx.x / (uint32_t)p.columns * (int64_t)beside;
    const int from = (int)first * p.block;
    const int n_all = p.n - from < beside * p.block ? p.n - from : beside * p.block;
    // The blocks' tokens, and the ones before and behind (none: no token's key).
    for (int i = threadIdx.x; i < n_all + 2; i += kSumThreads) {
        const int at = from + i - 1;
        all_keys[i] = at >= 0 && at < p.n ? p.keys[at] : 0xffffffffu;
        if (i < n_all) all_rows[i] = p.rows[from + i];
    }
    __syncthreads();
    const int64_t block = first + side;
    const uint32_t* keys = all_keys + side * p.block;
    const uint32_t* rows = all_rows + side * p.block;
    const int left = n_all - side * p.block, n = left < p.block ? left : p.block;
    const int column = (tile * p.lanes + (int)threadIdx.x % p.lanes) * VEC;
    if (n <= 0 || column >= p.width) return;
    const Columns<L> c(column, p.width);
    float sum[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
    bool began = keys[0] == keys[1];   // in an earlier block
    const Elem* grad = static_cast<const Elem*>(p.grad_out);
    for (int base = 0; base < n; base += U) {
        uint4 w[U];
        if (c.short_row()) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                w[i] = load_columns<L>(grad + (int64_t)rows[base + i < n ? base + i : n - 1] * p.stride,
                                       0, p.width);
        } else {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const uint32_t row = same<WAVES>(rows[base + i < n ? base + i : n - 1]);
                w[i] = c.load(grad + (int64_t)row * p.stride);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (base + i >= n) return;
            const uint32_t key = same<WAVES>(keys[base + i + 1]);
            if (key >= (uint32_t)p.vocab) return;   // no token: all behind are
            float v[VEC];
            L::unpack(w[i], v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum[j] += v[j];
            const bool last = same<WAVES>(keys[base + i + 2]) != key;
            if (!last && base + i + 1 < n) continue;
            if (last && !began) {
                write_sum<L>(p, key, c, sum);
            } else {
                float* out = p.partial + (block * 2 + (began ? 0 : 1)) * p.partial_stride;
                c.store_sum(out, sum);
            }
            began = false;
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
        }
    }
}

// The sum of the token's partial sums of blocks from `b` on, kJoinAhead of them at a
// time and `step` from one time to the next, until the token ends (true) or the
// block `until`.
constexpr int kJoinAhead = 16;

template <typename L>
__device__ __forceinline__ bool add_partials(const SumParams& p, uint32_t key, int64_t b,
                                             int64_t step, int64_t until, const Columns<L>& c,
                                             float (&sum)[L::VEC]) {
    constexpr int VEC = L::VEC, U = kJoinAhead;
    for (; b < until; b += step) {
        uint32_t found[U];
        float v[U][VEC];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t at = b + i < p.blocks ? b + i : b;
            found[i] = p.keys[at * p.block];
            c.load_sum(p.partial + at * 2 * p.partial_stride, v[i]);
        }
        bool over = false;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            over = over || b + i >= p.blocks || found[i] != key;
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum[j] += over ? 0.0f : v[i][j];
        }
        if (over) return true;
    }
    return until >= p.blocks;
}

// Tokens that begin in one of the workgroup's blocks and go on: their partial sums
// in order.  Of a token that goes on for more than kJoinShort blocks the rest is
// added by all threads, the sums of blocks side by side taking turns, and theirs
// joined in order.
constexpr int kJoinShort = kJoinAhead;

template <typename L>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(SumParams p) {
    constexpr int VEC = L::VEC;
    __shared__ uint32_t goes_on;
    __shared__ float sums[kSumThreads][VEC];
    const int tile = blockIdx.x % (uint32_t)p.columns;
    const int side = threadIdx.x / (uint32_t)p.lanes, beside = kSumThreads / p.lanes;
    const int64_t first = blockIdx.x / (uint32_t)p.columns * (int64_t)beside;
    const int column = (tile * p.lanes + (int)threadIdx.x % p.lanes) * VEC;
    const Columns<L> c(column < p.width ? column : 0, p.width);
    if (threadIdx.x == 0) goes_on = 0;
    __syncthreads();

    const auto begins = [&](int64_t block, uint32_t* key) {
        const int64_t from = block * p.block, end = from + p.block;
        if (end >= p.n) return false;   // the last block
        *key = p.keys[end];
        return *key < (uint32_t)p.vocab && p.keys[end - 1] == *key &&
               !(from > 0 && p.keys[from - 1] == *key);   // began earlier
    };
    const int64_t block = first + side;
    uint32_t key;
    float sum[VEC];
    if (begins(block, &key) && column < p.width) {
        c.load_sum(p.partial + (block * 2 + 1) * p.partial_stride, sum);
        const int64_t until = block + 1 + kJoinShort;
        if (add_partials<L>(p, key, block + 1, kJoinAhead, until < p.blocks ? until : p.blocks, c, sum))
            write_sum<L>(p, key, c, sum);
        else if (threadIdx.x % p.lanes == 0)
            atomicOr(&goes_on, 1u << side);
    }
    __syncthreads();
    uint32_t rest = goes_on;   // bits in ascending order, the same in every thread
    while (rest != 0) {
        const int at = __ffs(rest) - 1;
        rest &= rest - 1;
        const int64_t from = first + at;
        begins(from, &key);
        float more[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) more[j] = 0.0f;
        if (column < p.width)
            add_partials<L>(p, key, from + 1 + kJoinShort + side * kJoinAhead, beside * kJoinAhead,
                            p.blocks, c, more);
        if (beside > 1) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) sums[threadIdx.x][j] = more[j];
            __syncthreads();
        }
        if (side == at && column < p.width) {
            if (beside > 1)
                for (int i = 0; i < beside; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        sum[j] += sums[i * p.lanes + threadIdx.x % p.lanes][j];
            else
#pragma unroll
                for (int j = 0; j < VEC; ++j) sum[j] += more[j];
            write_sum<L>(p, key, c, sum);
        }
        __syncthreads();
    }
}

// Few rows, without a sort, in one launch.  A workgroup a row (and a tile of the
// columns) reads all tokens and lists the rows of its own row's; if its row is the
// first of them, it adds them: p.lanes threads a row, and the shares of the rows that
// lie side by side joined in order.  Further workgroups write zeros into the rows that
// no token names, and read all tokens for that.  Two latencies one after the other
// (tokens, rows) and the workgroups' turns bound it (777 x 1,000 FP32 into 5,003 rows
// 9.4 us; with 1,024 threads a workgroup 8.8, but 13.2 instead of 7.6 for 1,000 x 64
// into 50,000, whose many clearing workgroups then wait for room).
struct FewParams {
    SumParams sum;
    const int32_t* ids;
    ClearParams clear;
    int32_t groups;   // of sums
};

constexpr int kFewEach = kFewRows / kSumThreads;   // tokens a thread reads

template <typename L>
__device__ __forceinline__ void clear_unnamed(const FewParams& few, int group) {
    __shared__ uint32_t named;
    const int first = few.clear.from + group * kClearRows;
    if (threadIdx.x == 0) named = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kFewEach; ++k) {
        const int i = k * kSumThreads + (int)threadIdx.x;
        const uint32_t at = i < few.sum.n ? (uint32_t)few.ids[i] - (uint32_t)first : ~0u;
        if (at < (uint32_t)kClearRows) atomicOr(&named, 1u << at);
    }
    __syncthreads();
    clear_rows<L, kSumThreads>(few.clear, group, named);
}

template <typename L>
__global__ void __launch_bounds__(kSumThreads) embed_few_kernel(FewParams few) {
    using Elem = typename L::Elem;
    constexpr int VEC = L::VEC, U = 8;
    if ((int)blockIdx.x >= few.groups) {
        if (few.clear.f32) clear_unnamed<F32>(few, blockIdx.x - few.groups);
        else clear_unnamed<BF16>(few, blockIdx.x - few.groups);
        return;
    }
    const SumParams& p = few.sum;
    __shared__ uint64_t found[kFewRows / 64];   // bit by bit, the rows of the token
    __shared__ uint32_t rows[kFewRows];
    __shared__ float sums[kSumThreads][VEC];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int tile = blockIdx.x % (uint32_t)p.columns;
    const int own = blockIdx.x / (uint32_t)p.columns;
    const uint32_t key = (uint32_t)few.ids[own];
    if (key >= (uint32_t)p.vocab) return;
#pragma unroll
    for (int k = 0; k < kFewEach; ++k) {
        const int i = k * kSumThreads + tid;
        const uint64_t set = __ballot(i < p.n && (uint32_t)few.ids[i < p.n ? i : own] == key);
        if (lane == 0) found[i >> 6] = set;
    }
    __syncthreads();
    int n = 0, before[kFewEach];
    bool earlier = false;
#pragma unroll
    for (int w = 0; w < kFewRows / 64; ++w) {
        const uint64_t set = found[w];
#pragma unroll
        for (int k = 0; k < kFewEach; ++k)
            if (w == k * (kSumThreads / 64) + wave) before[k] = n + lanes_below(set);
        n += __popcll(set);
        const int upto = own - w * 64;   // bits of rows before its own
        earlier |= upto >= 64 ? set != 0 : upto > 0 && (set & ((1ull << upto) - 1)) != 0;
    }
    if (earlier) return;   // another row's
    if (n == 1) {
        if (tid == 0) rows[0] = (uint32_t)own;
    } else {
#pragma unroll
        for (int k = 0; k < kFewEach; ++k) {
            const int w = k * (kSumThreads / 64) + wave;
            if (found[w] >> lane & 1u) rows[before[k]] = (uint32_t)(w * 64 + lane);
        }
    }
    __syncthreads();

    const int side = tid / (uint32_t)p.lanes, beside = kSumThreads / p.lanes;
    const int column = (tile * p.lanes + tid % p.lanes) * VEC;
    const Columns<L> c(column < p.width ? column : 0, p.width);
    const Elem* grad = static_cast<const Elem*>(p.grad_out);
    float sum[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
    if (column < p.width) {
        for (int base = side; base < n; base += U * beside) {
            uint4 w[U];
            uint32_t r[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                r[i] = rows[base + i * beside < n ? base + i * beside : base];
            if (c.short_row()) {
#pragma unroll
                for (int i = 0; i < U; ++i)
                    w[i] = load_columns<L>(grad + (int64_t)r[i] * p.stride, 0, p.width);
            } else {
#pragma unroll
                for (int i = 0; i < U; ++i) w[i] = c.load(grad + (int64_t)r[i] * p.stride);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (base + i * beside >= n) break;
                float v[VEC];
                L::unpack(w[i], v);
#pragma unroll
                for (int j = 0; j < VEC; ++j) sum[j] += v[j];
            }
        }
    }
    const int shares = n < beside ? n : beside;
    if (shares > 1) {
        if (side < shares) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) sums[tid][j] = sum[j];
        }
        __syncthreads();
        if (side == 0)
            for (int i = 1; i < shares; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) sum[j] += sums[i * p.lanes + tid][j];
    }
    if (side == 0 && column < p.width) write_sum<L>(p, key, c, sum);
}

// ---------------------------------------------------------------------------

// Rows [from, to) of the table as a kernel clears them; `groups` workgroups.
ClearParams clear_of(const ws_states& t, const ws_embed_grad_args& a, int from, int to,
                     int64_t* groups) {
    ws_states rows = t;
    rows.dtype = a.grad_dtype;
    ClearParams p{};
    p.table = a.grad_table;
    p.stride = a.grad_stride;
    p.from = from;
    p.to = to;
    p.width = t.width;
    p.lanes = plan_embed(rows).lanes;
    p.f32 = a.grad_dtype == WS_DTYPE_F32;
    *groups = (to - from + kClearRows - 1) / kClearRows;
    return p;
}

// Sorted keys and rows, and beside that zeros in the table; `where` becomes the
// one of the two buffers that holds them.
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
    p.keys_out = keys[0];
    p.rows_out = rows[0];
    p.counts = reinterpret_cast<uint32_t*>(space + plan.counts_at);
    p.n = t.rows;
    p.vocab = a.vocab;
    p.tiles = plan.tiles;
    p.passes = plan.passes;
    const bool counted = plan.tiles > kOwnTiles;
    const int64_t steps = plan.tiles == 1 ? 1 : (counted ? 2 : 1) * plan.passes;
    int64_t clears = 0, step = 0;
    const auto share = [&] {
        if (!a.accumulate)
            p.clear = clear_of(t, a, (int)(a.vocab * step / steps),
                               (int)(a.vocab * (step + 1) / steps), &clears);
        ++step;
    };
    *where = 0;
    if (plan.tiles == 1) {
        share();
        return launch(sort_few_kernel, 1 + clears, kSortThreads, p, s);
    }
    int v = WS_OK;
    for (int pass = 0; pass < plan.passes && v == WS_OK; ++pass) {
        const int to = pass & 1;
        p.keys_in = keys[to ^ 1];
        p.rows_in = rows[to ^ 1];
        p.keys_out = keys[to];
        p.rows_out = rows[to];
        p.shift = pass * kDigitBits;
        if (counted) {
            share();
            v = launch(sort_count_kernel, plan.tiles + clears, kSortThreads, p, s);
        }
        if (v == WS_OK && plan.tiles > kScanTiles)
            v = launch(sort_scan_kernel, kDigits / kScanDigits, kScanDigits * 64, p, s);
        share();
        if (v == WS_OK) v = launch(sort_place_kernel, plan.tiles + clears, kSortThreads, p, s);
        *where = to;
    }
    return v;
}

template <typename L>
int run_few(const ws_states& t, const ws_embed_grad_args& a, const SumParams& sum, hipStream_t s) {
    FewParams p{};
    p.sum = sum;
    p.ids = a.ids;
    p.groups = t.rows * sum.columns;
    int64_t clears = 0;
    if (!a.accumulate) p.clear = clear_of(t, a, 0, a.vocab, &clears);
    return launch(embed_few_kernel<L>, p.groups + clears, kSumThreads, p, s);
}

template <typename L>
int run_sum(const EmbedGradPlan& plan, const SumParams& p, hipStream_t s) {
    const int64_t beside = kSumThreads / plan.lanes;
    const int64_t groups = (plan.blocks + beside - 1) / beside * plan.columns;
    const int v = plan.lanes >= 64 ? launch(embed_sum_kernel<L, true>, groups, kSumThreads, p, s)
                                   : launch(embed_sum_kernel<L, false>, groups, kSumThreads, p, s);
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
    v = ws::validate_embed_grad_workspace(*states, *args, plan.workspace);
    if (v != WS_OK) return v;
    if (states->rows == 0 && args->accumulate) return WS_OK;
    v = ws::device_ready(states->device);
    if (v != WS_OK) return v;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (states->rows == 0) {
        int64_t groups = 0;
        const ws::ClearParams p = ws::clear_of(*states, *args, 0, args->vocab, &groups);
        return ws::launch(ws::clear_kernel, groups, ws::kSortThreads, p, s);
    }
    char* space = static_cast<char*>(args->workspace);
    ws::SumParams p{};
    p.grad_out = args->grad_out;
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
    p.lanes = plan.lanes;
    p.grad_f32 = args->grad_dtype == WS_DTYPE_F32;
    p.accumulate = args->accumulate;
    p.scale = args->scale;
    if (plan.few) {
#define CALL(L) return run_few<L>(*states, *args, p, s)
        WS_BY_DTYPE(states->dtype, CALL);
#undef CALL
    }
    int where = 0;
    v = ws::sort_tokens(*states, *args, plan, s, &where);
    if (v != WS_OK) return v;
    p.keys = reinterpret_cast<const uint32_t*>(space + plan.keys_at[where]);
    p.rows = reinterpret_cast<const uint32_t*>(space + plan.rows_at[where]);
#define CALL(L) return run_sum<L>(plan, p, s)
    WS_BY_DTYPE(states->dtype, CALL);
#undef CALL
}
