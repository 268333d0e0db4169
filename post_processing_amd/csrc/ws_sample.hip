// ws_sample.hip -- tokens drawn from rows of logits (ws_logits.h), written for
// gfx950 (CDNA4, wave64).
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "ws_enqueue.h"
#include "ws_lanes.h"
#include "ws_logits.h"
#include "ws_logits_plan.h"
#include "ws_logits_rows.h"

namespace ws {
namespace {

// ---------------------------------------------------------------------------
// A row is cut into stretches of neighbouring slots, one a wave.  Each is read
// once: its lanes keep the largest logit of their slots, and where the draw needs
// the mass of the whole row, its sum.  From there
//
//   everything kept    the stretch that holds the target, read again
//   greedy             the first stretch that holds the largest logit, likewise
//   top-k, min-p, and  a bound t below which nothing is kept, from the lanes'
//   a peaked top-p     largest logits (K of them at or above t: so are the best K
//                      logits); the slots of the lanes that reach t are read
//                      again for the few logits at or above it, which are sorted,
//                      cut and drawn from exactly
//   otherwise          a histogram over the row finds the cut (many tokens kept:
//                      a flat row's nucleus, a large k, many equal logits), and
//                      another pass over it draws
//
// Few long rows have their stretches read by many workgroups, and a second
// kernel goes on from there.
//
// A pass with the mass is bound by the vector unit: FP64 runs at FP32's rate, so an
// element costs sixteen to twenty instructions, 15 us for 131,072 in a workgroup of
// 1,024 threads; without the mass HBM bounds it.  The rest is a chain of latencies,
// for a best 50 of 131,072: bound 1.3 us, the few logits 2.5, sorting and drawing
// 2.5; a nucleus of thousands takes 13 us for the histogram and 38 for the exact
// pass.  Whole calls: 1 x 131,072 BF16 with the best 50 12.8 us (3.6 and 9.5 in the
// two kernels), greedy 8.5, an undecided row's nucleus of 0.9 69; 64 x 32,768 FP16 with
// mixed settings 25-35, as the inputs have an undecided row or none; 300 x 50,001 FP32
// all kept 30.7; 1,024 x 131,072 BF16 mixed 104-136 by the inputs, best 50 78 (3.4
// TB/s), greedy 58, all undecided nuclei 354.  A sort of the whole row in elementary
// operations takes 350 us for the first and 16.8 ms for the mixed 1,024.

struct SampleParams {
    const void* logits;
    int64_t stride;
    const float* uniform;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* token;
    float* logprob;
    char* space;        // of split rows: [rows] of kStretchBytes * stretches
    int32_t rows;
    int32_t vocab;
    int32_t chunk;      // slots of a part
    int32_t parts;
    float tau;          // of every row, without `temperature`
    int32_t unit;       // sums in fixed point count units of 2^-unit
};

// A row's settings.
struct Settings {
    double inv_tau, uniform, least;   // least: log q
    double p;
    int k;                            // 1..V; V: all
    bool fine;

    __device__ __forceinline__ void read(const SampleParams& a, int64_t row) {
        const float u = a.uniform[row];
        const float t = a.temperature ? a.temperature[row] : a.tau;
        const int32_t top_k = a.top_k ? a.top_k[row] : 0;
        const float top_p = a.top_p ? a.top_p[row] : 1.0f;
        const float q = a.min_p ? a.min_p[row] : 0.0f;
        fine = u >= 0.0f && u < 1.0f && top_k >= 0 && top_p >= 0.0f && top_p <= 1.0f &&
               q >= 0.0f && q <= 1.0f &&
               (t == 0.0f || (t >= WS_MIN_TEMPERATURE && t <= WS_MAX_TEMPERATURE));
        const bool greedy = t == 0.0f;
        k = greedy ? 1 : top_k == 0 || top_k > a.vocab ? a.vocab : top_k;
        inv_tau = greedy ? 1.0 : 1.0 / (double)t;
        uniform = (double)u;
        p = (double)top_p;
        least = q > 0.0f ? log((double)q) : -INFINITY;
    }
    __device__ __forceinline__ bool cut_by_k(int vocab) const { return k < vocab; }
    // Whether the mass of the whole row decides.
    __device__ __forceinline__ bool needs_mass(int vocab) const {
        return k == vocab && (p < 1.0 || least == -INFINITY);
    }
};

// ---- weights -----------------------------------------------------------------

constexpr int kTable = 256;
constexpr double kNone = -200.0;   // exponents below count as weight 0

__device__ __forceinline__ void fill_table(double* table, int threads) {
    for (int i = threadIdx.x; i < kTable; i += threads)
        table[i] = small_exp((double)i * (0.6931471805599453 / kTable));
}

constexpr double kScale = 369.3299304675746;     // 256 / log 2

// e^(t / kScale) for t between -700 and 130 times kScale: t = n + r, 2 to the n / 256
// from a table (LDS) and a shift of its exponent, and the series of what is left (at
// most 1.4e-3) to the third power, whose next term leaves the result up to 1.4e-13
// too small, 1.6e-13 with the rounding of t down to e^-200.  Sums of such weights and
// their borders between tokens, as shares of the whole, are off by less than 2e-13, so
// a draw differs from the exact one only where the uniform number is that near a
// border: for at most V x 4e-13 of the numbers, 5e-8 at V = 131,072.  Sixteen
// instructions with the sum, half of the exponential the library has in FP64.
__device__ __forceinline__ double table_exp_scaled(double t, const double* table) {
    constexpr double kMagic = 6755399441055744.0;    // 1.5 x 2^52: adds to an integer
    constexpr double a1 = 0.0027076061740622863;     // log 2 / 256
    const double y = t + kMagic;
    const int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, y);
    const double r = t - (y - kMagic);
    const double q = r * fma(r, fma(r, a1 * a1 * a1 / 6.0, a1 * a1 / 2.0), a1);
    const uint64_t w = __builtin_bit_cast(uint64_t, table[n & (kTable - 1)]);
    const uint32_t hi = (uint32_t)(w >> 32) + ((uint32_t)(n & ~(kTable - 1)) << 12);
    const double s = __builtin_bit_cast(double, ((uint64_t)hi << 32) | (uint32_t)w);
    return fma(s, q, s);
}

__device__ __forceinline__ double table_exp(double x, const double* table) {
    return table_exp_scaled(x * kScale, table);
}

// ---- stretches -----------------------------------------------------------------

constexpr int kScanThreads = 256, kScanWaves = kScanThreads / 64;
constexpr int kMostStretches = kMaxSampleParts * kScanWaves;

struct Stretch {
    double sum;       // of weights against ref
    float ref;
    float top;        // largest logit; NaN or +inf: the row has none
    float low;        // smallest of the lanes' largest logits, finite ones
    float unused;
};
static_assert(sizeof(Stretch) + 64 * sizeof(float) == kStretchBytes, "workspace");

// Slots [from, to) of stretch i of a row: `waves` to a part.
template <typename L>
__device__ __forceinline__ void stretch_slots(const Part<L>& row, const SampleParams& p, int waves,
                                              int i, int& from, int& to) {
    const int part = i / waves;
    const int begin = part * p.chunk;
    const int end = part == p.parts - 1 ? row.n : begin + p.chunk;
    const int each = (end - begin + waves - 1) / waves;
    from = begin + i % waves * each;
    to = from + each < end ? from + each : end;
    if (from > to) from = to;
}

template <int VEC>
__device__ __forceinline__ float slot_maximum(const float (&v)[VEC]) {
    float m = __builtin_elementwise_maximum(v[0], v[1]);   // NaN if there is one
#pragma unroll
    for (int j = 2; j < VEC; ++j) m = __builtin_elementwise_maximum(m, v[j]);
    return m;
}

__device__ __forceinline__ float wave_maximum(float v, int lane) {
    v = __builtin_elementwise_maximum(v, xor_lane_f<32>(v, lane));
    v = __builtin_elementwise_maximum(v, xor_lane_f<16>(v, lane));
    v = __builtin_elementwise_maximum(v, xor_lane_f<8>(v, lane));
    v = __builtin_elementwise_maximum(v, xor_lane_f<4>(v, lane));
    v = __builtin_elementwise_maximum(v, xor_lane_f<2>(v, lane));
    return __builtin_elementwise_maximum(v, xor_lane_f<1>(v, lane));
}

__device__ __forceinline__ float wave_minimum(float v, int lane) {
    v = fminf(v, xor_lane_f<32>(v, lane));
    v = fminf(v, xor_lane_f<16>(v, lane));
    v = fminf(v, xor_lane_f<8>(v, lane));
    v = fminf(v, xor_lane_f<4>(v, lane));
    v = fminf(v, xor_lane_f<2>(v, lane));
    return fminf(v, xor_lane_f<1>(v, lane));
}

__device__ __forceinline__ int wave_least(int v, int lane) {
    const auto least = [](int a, uint32_t b) { return a < (int)b ? a : (int)b; };
    v = least(v, xor_lane32<32>((uint32_t)v, lane));
    v = least(v, xor_lane32<16>((uint32_t)v, lane));
    v = least(v, xor_lane32<8>((uint32_t)v, lane));
    v = least(v, xor_lane32<4>((uint32_t)v, lane));
    v = least(v, xor_lane32<2>((uint32_t)v, lane));
    return least(v, xor_lane32<1>((uint32_t)v, lane));
}

// Calls f(values of U slots, element of the first) for the slots that thread
// `lane` of LANES has of slots [from, to): its whole slots LANES apart, U loaded
// at a time, the next U while f runs if AHEAD, and in one more round, by threads 0
// and 1, what sticks out of the row's ends.  Elements outside the row or the range
// are -inf.  f is there once: code that runs once a row waits for its instructions.
template <typename L, int LANES, int U, bool AHEAD, typename F>
__device__ __forceinline__ void lane_batches(const Part<L>& row, int from, int to, int lane, F f) {
    constexpr int VEC = L::VEC;
    const int a = from > row.full_from ? from : row.full_from;
    const int b = to < row.full_to ? to : row.full_to;
    const int tail = row.full_to > row.full_from ? row.full_to : row.full_from;
    const bool front = row.full_from > 0 && from == 0 && to > 0;
    const bool back = tail < row.n && tail >= from && tail < to;
    const int rounds = b > a ? (b - a + U * LANES - 1) / (U * LANES) : 0;
    uint4 w[U];
    const auto load = [&](int base) {
        // (a load under a condition would be waited for before the next)
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int s = base + lane + i * LANES;
            w[i] = row.load(s < b ? s : b - 1);
        }
    };
    if (AHEAD && rounds > 0) load(a);
    for (int r = 0; r < rounds + (front || back ? 1 : 0); ++r) {
        float v[U][VEC];
        int e;
        if (r < rounds) {
            const int base = a + r * U * LANES;
            if constexpr (!AHEAD) load(base);
            if (base + U * LANES > b) {
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (base + lane + i * LANES >= b) w[i] = L::none();
            }
#pragma unroll
            for (int i = 0; i < U; ++i) L::unpack(w[i], v[i]);
            if (AHEAD && r + 1 < rounds) load(base + U * LANES);
            e = row.e0 + (base + lane) * VEC;
        } else {
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[i][j] = -INFINITY;
            const int s = lane == 0 ? 0 : tail;
            if ((lane == 0 && front) || (lane == 1 && back)) row.load_edge(s, v[0]);
            e = row.e0 + s * VEC;
        }
        f(v, e);
    }
}

// The same slot by slot: f(values, element of values[0]).
template <typename L, int LANES, typename F>
__device__ __forceinline__ void lane_slots(const Part<L>& row, int from, int to, int lane, F f) {
    lane_batches<L, LANES, 1, true>(row, from, to, lane,
                                    [&](const float (&v)[1][L::VEC], int e) { f(v[0], e); });
}

// One wave's pass over its stretch.  lane_top: the largest of the lane's logits.
template <typename L, bool MASS>
__device__ __forceinline__ Stretch scan_stretch(const Part<L>& row, int from, int to, double inv_tau,
                                                const double* table, float& lane_top) {
    constexpr int VEC = L::VEC;
    const int lane = threadIdx.x & 63;
    Stretch s;
    s.sum = 0.0;
    s.ref = -INFINITY;
    float top = -INFINITY;
    double ref = 0.0;
    const double steepness = inv_tau * kScale;
    // A logit 60 exponents above the reference makes it the new one.
    float limit = -INFINITY;
    const float reach = (float)(60.0 / inv_tau);
    lane_batches<L, 64, kBatchSlots, false>(row, from, to, lane,
                                            [&](const float (&v)[kBatchSlots][VEC], int) {
        float m = slot_maximum<VEC>(v[0]);
#pragma unroll
        for (int i = 1; i < kBatchSlots; ++i)
            m = __builtin_elementwise_maximum(m, slot_maximum<VEC>(v[i]));
        top = __builtin_elementwise_maximum(top, m);
        if constexpr (MASS) {
            if (m > limit) {   // rare
                const double x = ((double)s.ref - (double)m) * inv_tau;
                s.sum = x < -700.0 ? 0.0 : s.sum * table_exp(x, table);
                s.ref = m;
                ref = (double)m;
                limit = m + reach;
            }
            // (against the reference 0 while all are -inf: e^-700 each)
            double sum[kBatchSlots] = {};
#pragma unroll
            for (int i = 0; i < kBatchSlots; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    sum[i] += table_exp_scaled(
                        fmax(((double)v[i][j] - ref) * steepness, -700.0 * kScale), table);
#pragma unroll
            for (int i = 0; i < kBatchSlots; ++i) s.sum += sum[i];
        }
    });
    lane_top = top;
    s.top = wave_maximum(top, lane);
    s.low = wave_minimum(top > -INFINITY ? top : INFINITY, lane);
    s.unused = 0.0f;
    if constexpr (MASS) {
        // The lanes' references become one, the largest.
        const float high = wave_max(s.ref, lane);
        if (s.ref < high) {
            const double x = ((double)s.ref - (double)high) * inv_tau;
            s.sum = s.ref == -INFINITY || x < -700.0 ? 0.0 : s.sum * table_exp(x, table);
        }
        s.ref = high;
        s.sum = wave_sum_d(s.sum, lane);
    }
    return s;
}

template <typename L>
__device__ __forceinline__ Stretch scan_any(const Part<L>& row, int from, int to, const Settings& set,
                                            int vocab, const double* table, float& lane_top) {
    return set.fine && set.needs_mass(vocab)
               ? scan_stretch<L, true>(row, from, to, set.inv_tau, table, lane_top)
               : scan_stretch<L, false>(row, from, to, set.inv_tau, table, lane_top);
}

// ---- prefix sums of a wave --------------------------------------------------------

// v of the lanes that DPP control CTRL names, 0 where it names none.
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T dpp_or_zero(T v) {
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(
            T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
    } else {
        const uint64_t w = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = dpp_or_zero<CTRL, ROWS>((uint32_t)w);
        const uint32_t hi = dpp_or_zero<CTRL, ROWS>((uint32_t)(w >> 32));
        return __builtin_bit_cast(T, ((uint64_t)hi << 32) | lo);
    }
}

// The sum of the lanes up to and including one's own.
template <typename T>
__device__ __forceinline__ T wave_upto(T v) {
    v += dpp_or_zero<0x111, 0xf>(v);   // row_shr:1, 2, 4, 8: inside rows of 16 lanes
    v += dpp_or_zero<0x112, 0xf>(v);
    v += dpp_or_zero<0x114, 0xf>(v);
    v += dpp_or_zero<0x118, 0xf>(v);
    v += dpp_or_zero<0x142, 0xa>(v);   // row_bcast:15 into rows 1 and 3
    v += dpp_or_zero<0x143, 0xc>(v);   // row_bcast:31 into rows 2 and 3
    return v;
}

// ---- what a row's workgroup does with them --------------------------------------

// A value's rank as an integer of few bits: 16-bit types have images whose low
// bits all are the sign's.
template <typename L>
struct Image {
    static constexpr int kDrop = __is_same(typename L::Elem, float)      ? 0
                                 : __is_same(typename L::Elem, _Float16) ? 13
                                                                         : 16;
    static __device__ __forceinline__ uint32_t of(float v) { return value_image(v) >> kDrop; }
    static __device__ __forceinline__ float value(uint32_t i) {
        const uint32_t low = (1u << kDrop) - 1;
        const uint32_t w = i << kDrop;
        return image_value(w & 0x80000000u ? w : w | low);
    }
};

// Calls f(values, element of values[0]) for slots [from, to) in order; elements
// outside the row are -inf.
template <typename L, typename F>
__device__ __forceinline__ void walk(const Part<L>& row, int from, int to, F f) {
    const bool whole = row.full_to > row.full_from;
    uint4 next = L::none();
    if (whole) next = row.load_near(from);
    for (int s = from; s < to; ++s) {
        float v[L::VEC];
        L::unpack(next, v);
        if (whole) next = row.load_near(s + 1);   // on its way while f runs
        if (!row.whole(s)) row.load_edge(s, v);
        f(v, row.e0 + s * L::VEC);
    }
}

constexpr int kBins = 2048, kBounds = 1024;
// A lane sums 16 neighbouring bounds: one word more for every 16, so that the lanes
// read from different banks.
constexpr int kBoundsRoom = kBounds + kBounds / 16;
__device__ __forceinline__ int bound_at(int b) { return b + (b >> 4); }


// A prefix of the order: tokens above z, and those at it up to element `last`.
struct Cut {
    float z;
    int last;
    double ties;   // above 0: `last` is not known yet, but this many at z belong
    double mass;   // of the prefix, if it was asked for
};

template <typename L, int NT, int GROUPS>
struct Sampler {
    static constexpr int VEC = L::VEC;
    static constexpr int kWaves = NT / 64;
    static constexpr int kList = NT;

    struct Shared {
        double table[kTable];
        Stretch stretch[kMostStretches > kWaves ? kMostStretches : kWaves];
        union {
            uint32_t bounds[kBoundsRoom];
            struct {
                unsigned long long mass[kBins];
                uint32_t count[kBins];
            } bins;
            struct {
                uint64_t keys[kList];
                uint64_t sorted[kList];
                double weight[kList];
            } list;
        };
        uint64_t waves_mass[kWaves];
        double waves[kWaves], waves_above[kWaves];
        uint32_t waves_count[kWaves];
        double total, left;
        uint64_t before_mass;
        uint32_t before_count;
        float limit;
        int chosen, bin, first, last, token, count, active;
        uint32_t low, high;
    };

    Part<L> row;
    const SampleParams& p;
    Shared* sh;
    Settings set;
    int stretches, stretch_waves;
    float group[GROUPS];   // largest logits of groups of slots: this thread's
    float top32;
    double top, scale;
    Cut cut;               // what is kept, but for min-p

    __device__ __forceinline__ Sampler(const SampleParams& params, Shared* shared)
        : p(params), sh(shared) {}

    __device__ __forceinline__ double exponent(float z) const {
        return ((double)z - top) * set.inv_tau;
    }
    __device__ __forceinline__ double weight(float z) const {
        const double x = exponent(z);
        return x < kNone ? 0.0 : table_exp(x, sh->table);
    }
    __device__ __forceinline__ double kept(float v, int e) const {   // its weight, or 0
        const double x = exponent(v);
        const bool in = (v > cut.z || (v == cut.z && e <= cut.last)) && x >= set.least && x >= kNone;
        return in ? table_exp(fmax(x, kNone), sh->table) : 0.0;
    }
    __device__ __forceinline__ unsigned long long fixed(double w) const {
        return (unsigned long long)fma(w, scale, 0.5);
    }

    // Keeps what a loop derives from the row's place out of the registers of all
    // that comes before the loop.
    __device__ __forceinline__ void recompute() {
        asm volatile("" : "+v"(row.row), "+v"(row.base), "+v"(row.vocab), "+v"(row.e0));
    }

    // The log of the drawn token's share, in thread 0.
    __device__ __forceinline__ float log_share(double all) const {
        return threadIdx.x == 0 ? (float)log(sh->left / all) : 0.0f;
    }

    // Exclusive sums across the threads.  A barrier inside.
    template <typename T>
    __device__ __forceinline__ T before(T v, T* waves, T& total) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const T upto = wave_upto(v);
        if (lane == 63) waves[wave] = upto;
        __syncthreads();
        T at = upto - v;
        total = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            at += i < wave ? waves[i] : 0;
            total += waves[i];
        }
        return at;
    }

    // The first and the last thread of which `yes` holds, into sh->first and
    // sh->last (one atomic a wave: 64 lanes at one address take turns).
    __device__ __forceinline__ void note_first(bool yes) {
        const uint64_t all = __ballot(yes);
        if (all && (threadIdx.x & 63) == 0)
            atomicMin(&sh->first, (int)threadIdx.x + __ffsll((unsigned long long)all) - 1);
    }
    __device__ __forceinline__ void note_last(bool yes) {
        const uint64_t all = __ballot(yes);
        if (all && (threadIdx.x & 63) == 0)
            atomicMax(&sh->last, (int)threadIdx.x + 63 - __clzll(all));
    }

    // The first thread at whose end the threads' sums exceed `left`, or, where
    // rounding leaves `left` behind all of them, the last above 0; `at` is what
    // lies before one's own.
    __device__ __forceinline__ int find_thread(double sum, double left, double& at) {
        if (threadIdx.x == 0) {
            sh->first = NT;
            sh->last = -1;
        }
        double total;
        at = before(sum, sh->waves, total);
        note_first(sum > 0.0 && at + sum > left);
        note_last(sum > 0.0);
        __syncthreads();
        const int found = sh->first < NT ? sh->first : sh->last;
        __syncthreads();   // everyone has read it before it is cleared
        return found;
    }

    // The kept token at which the weights of slots [from, to) sum to more than
    // `left` in the order of the vocabulary, and its weight in sh->left.  Every sum's
    // order is fixed.
    __device__ __forceinline__ int locate(int from, int to, double left) {
        const int tid = threadIdx.x;
        for (;;) {
            recompute();
            const int each = (to - from + NT - 1) / NT;
            int mine = from + tid * each;
            if (mine > to) mine = to;
            const int end = mine + each < to ? mine + each : to;
            double w[VEC], sum = 0.0, at;   // w: of the last slot
            int element = 0;
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[j] = 0.0;
            walk(row, mine, end, [&](const float (&v)[VEC], int e) {
                element = e;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    w[j] = kept(v[j], e + j);
                    sum += w[j];
                }
            });
            const int found = find_thread(sum, left, at);
            if (found < 0) return -1;
            if (tid == found) {
                sh->total = at;
                bool done = false;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    if (!done && w[j] > 0.0) {
                        sh->token = element + j;
                        sh->left = w[j];
                    }
                    at += w[j];
                    done = done || (w[j] > 0.0 && at > left);
                }
            }
            __syncthreads();
            const double skipped = sh->total;
            const int token = sh->token;
            __syncthreads();   // everyone has read them before they change
            if (each == 1) return token;
            from += found * each;
            to = from + each < to ? from + each : to;
            left -= skipped;
        }
    }

    __device__ __forceinline__ int row_stretch() const { return (row.n + kWaves - 1) / kWaves; }

    // The kept weights of the row's stretches, one a wave, in sh->waves; returns
    // their sum.
    __device__ __forceinline__ double sum_row() {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, each = row_stretch();
        int from = wave * each;
        if (from > row.n) from = row.n;
        double sum = 0.0;
        lane_slots<L, 64>(row, from, from + each < row.n ? from + each : row.n, lane,
                          [&](const float (&v)[VEC], int e) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += kept(v[j], e + j);
        });
        sum = wave_sum_d(sum, lane);
        if (lane == 0) sh->waves[wave] = sum;
        __syncthreads();
        double total = 0.0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) total += sh->waves[i];
        return total;
    }

    // The stretch of sh->waves that holds the target, and what is left to go in it.
    __device__ __forceinline__ void find_stretch(double target, int& from, int& to, double& left) {
        int chosen = 0;
        left = 0.0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const double w = sh->waves[i];
            if (w > 0.0 && target >= 0.0) {
                chosen = i;
                left = target;
            }
            target -= w;
        }
        __syncthreads();
        const int each = row_stretch();
        from = chosen * each;
        to = from + each < row.n ? from + each : row.n;
    }

    // The element that is the n-th at z, by index: slots NT at a time.
    __device__ __forceinline__ int find_tie(float z, uint32_t n) {
        const int tid = threadIdx.x;
        uint32_t passed = 0;
        for (int base = 0; base < row.n; base += NT) {
            recompute();
            uint32_t hits = 0, total;   // a bit an element
            int e = 0;
            walk(row, base + tid, base + tid < row.n ? base + tid + 1 : 0,
                 [&](const float (&v)[VEC], int element) {
                e = element;
#pragma unroll
                for (int j = 0; j < VEC; ++j) hits |= v[j] == z ? 1u << j : 0u;
            });
            const uint32_t mine = __popc(hits);
            uint32_t at = passed + before(mine, sh->waves_count, total);
            if (at < n && at + mine >= n) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    at += hits >> j & 1u;
                    if ((hits >> j & 1u) && at == n) sh->token = e + j;
                }
            }
            __syncthreads();
            passed += total;
            if (passed >= n) break;
        }
        const int token = sh->token;
        __syncthreads();   // everyone has read it before it changes
        return token;
    }

    // The largest logit of the row.
    __device__ __forceinline__ void find_top() {
        const int lane = threadIdx.x & 63;
        float m = -INFINITY;
        for (int i = lane; i < stretches; i += 64)
            m = __builtin_elementwise_maximum(m, sh->stretch[i].top);
        top32 = wave_maximum(m, lane);
        top = (double)top32;
    }

    // The mass of the row in sh->total, and of the stretch that holds u times it
    // the number and what is left to go in it.
    __device__ __forceinline__ void sum_stretches() {
        constexpr int kEach = (kMostStretches + 63) / 64;
        const int lane = threadIdx.x & 63;
        if (threadIdx.x < 64) {
            double w[kEach], sum = 0.0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int at = lane * kEach + i;
                w[i] = 0.0;
                if (at < stretches) {
                    // A stretch with a weight above 0 has mass above 0.
                    const Stretch& s = sh->stretch[at];
                    if (exponent(s.top) >= kNone)
                        w[i] = s.sum * table_exp(fmax(exponent(s.ref), -600.0), sh->table);
                }
                sum += w[i];
            }
            const double upto = wave_upto(sum);
            const double total = lane_d(upto, 63);
            double rest = set.uniform * total - (upto - sum), left = 0.0;
            int chosen = -1;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (w[i] > 0.0 && rest >= 0.0) {
                    chosen = lane * kEach + i;
                    left = rest;
                }
                rest -= w[i];
            }
            const uint64_t some = __ballot(chosen >= 0);   // the last lane that has one
            if (some && lane == 63 - __clzll(some)) {
                sh->chosen = chosen;
                sh->left = left;
                sh->total = total;
            }
        }
        __syncthreads();
    }

    // Sorts one key a thread (0: none) in descending order into `to` (LDS, which
    // no one reads before this; a barrier at the end).  n: number of keys.
    __device__ __forceinline__ void sort_keys(uint64_t key, int n, uint64_t* lists, uint64_t* to) {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
        const int waves = (n + 63) / 64;
        if (wave < waves) {
            key = wave_sort<true>(key, lane);
            lists[tid] = key;
        }
        __syncthreads();
        if (wave < waves && key != 0) {
            // Keys above this one in the waves' lists, each sorted in descending
            // order: four searches at a time, each a chain of reads.
            constexpr int U = kWaves < 4 ? kWaves : 4;
            int rank = 0;
            for (int w = 0; w < waves; w += U) {
                const uint64_t* list[U];
                int above[U] = {};
#pragma unroll
                for (int i = 0; i < U; ++i) list[i] = lists + (w + i < waves ? w + i : wave) * 64;
#pragma unroll
                for (int step = 32; step > 0; step /= 2)
#pragma unroll
                    for (int i = 0; i < U; ++i)
                        above[i] += list[i][above[i] + step - 1] > key ? step : 0;
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (w + i < waves) rank += above[i] + (list[i][above[i]] > key);
            }
            to[rank] = key;
        }
        __syncthreads();
    }

    __device__ __forceinline__ bool among(float v, float steps, float limit) const {
        return v > -INFINITY && fminf(top32 - v, FLT_MAX) * steps < limit;
    }

    // The logits at most limit / steps below the largest, as keys in sh->list;
    // returns how many (more than kList: they are not all there).  The groups that
    // reach so far are listed, and their slots shared out over the threads.
    __device__ __forceinline__ int collect(float steps, float limit) {
        const int tid = threadIdx.x, lane = tid & 63;
        uint32_t* active = reinterpret_cast<uint32_t*>(sh->list.sorted);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int at = g * NT + tid;
            const bool on = at < stretches * 64 && among(group[g], steps, limit);
            const uint64_t all = __ballot(on);
            if (!all) continue;
            int base = 0;
            if (lane == 0) base = atomicAdd(&sh->active, (int)__popcll(all));
            const int i = __builtin_amdgcn_readfirstlane(base) + lanes_below(all);
            if (on && i < kList) active[i] = (uint32_t)at;
        }
        __syncthreads();
        const int groups = sh->active;
        if (groups > kList) return groups;   // each has a logit that reaches
        int from, to;
        int each = (row.n - (p.parts - 1) * p.chunk + stretch_waves - 1) / stretch_waves;
        each = (each + 63) / 64;   // slots of a group at most
        const int items = row.full_to > row.full_from ? groups * each : 0;
        const auto slot = [&](int item) {   // -1: none
            const int a = item < items ? item / each : 0;
            const int at = (int)active[a];
            stretch_slots(row, p, stretch_waves, at >> 6, from, to);
            from = from > row.full_from ? from : row.full_from;
            to = to < row.full_to ? to : row.full_to;
            const int s = from + (at & 63) + (item - a * each) * 64;
            return item < items && s < to ? s : -1;
        };
        const int tail = row.full_to > row.full_from ? row.full_to : row.full_from;
        const int rounds = (items + NT - 1) / NT;
        int next = -1;
        uint4 ahead = L::none();
        if (rounds > 0) {
            next = slot(tid);
            ahead = row.load_near(next < 0 ? row.full_from : next);
        }
        for (int r = 0; r <= rounds; ++r) {
            int s = next;
            float v[VEC];
            L::unpack(ahead, v);
            if (r + 1 < rounds) {
                next = slot((r + 1) * NT + tid);
                ahead = row.load_near(next < 0 ? row.full_from : next);
            } else if (r == rounds) {   // what sticks out of the row's ends
                s = tid == 0 && row.full_from > 0 ? 0 : tid == 1 && tail < row.n ? tail : -1;
                if (s >= 0) row.load_edge(s, v);
            }
            if (s >= 0) push<VEC>(v, row.e0 + s * VEC, steps, limit);
        }
        __syncthreads();
        return sh->count;
    }

    template <int N>
    __device__ __forceinline__ void push(const float (&v)[N], int e, float steps, float limit) {
        if (!among(slot_maximum<N>(v), steps, limit) || sh->count > kList) return;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (among(v[j], steps, limit)) {
                const int i = atomicAdd(&sh->count, 1);
                if (i < kList) sh->list.keys[i] = value_key(v[j], (uint32_t)(e + j));
            }
    }

    // A bound for `collect` from the groups' largest logits: as many of them at
    // or above it as make up `target` (their number, or their weights in units
    // of 2^-18, rounded down).  Infinite if they never do.
    __device__ __forceinline__ float bound(uint32_t target, bool mass, float steps) {
        const int tid = threadIdx.x, lane = tid & 63;
        const float c = (float)(set.inv_tau * 1.4426950408889634);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const float v = group[g];
            if (g * NT + tid >= stretches * 64 || !(v > -INFINITY)) continue;
            const float d = fminf(top32 - v, FLT_MAX);
            const float b = fminf(d * steps, (float)(kBounds - 1));
            const uint32_t amount =
                mass ? (uint32_t)(__builtin_amdgcn_exp2f(-d * c) * 262144.0f) : 1u;
            if (amount) atomicAdd(&sh->bounds[bound_at((int)b)], amount);
        }
        __syncthreads();
        if (tid < 64) {
            constexpr int kEach = kBounds / 64;
            uint32_t sum = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) sum += sh->bounds[bound_at(lane * kEach + i)];
            const uint32_t upto = wave_upto(sum);
            uint32_t at = upto - sum;
            if (lane == 63 && upto < target) sh->limit = INFINITY;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const uint32_t next = at + sh->bounds[bound_at(lane * kEach + i)];
                if (at < target && next >= target) sh->limit = (float)(lane * kEach + i + 1);
                at = next;
            }
        }
        __syncthreads();
        return sh->limit;
    }

    // Draws from n <= 64 collected logits, which hold everything kept: in one wave.
    __device__ __forceinline__ int draw_few(int n, bool by_k, double mass, float& logprob) {
        const int lane = threadIdx.x & 63;
        if (threadIdx.x < 64) {
            const uint64_t key = wave_sort<true>(lane < n ? sh->list.keys[lane] : 0, lane);
            const double x = exponent(image_value((uint32_t)(key >> 32)));
            double w = lane < n && x >= kNone ? table_exp(x, sh->table) : 0.0;
            if (by_k && lane >= set.k) w = 0.0;
            double upto = wave_upto(w);
            const double all = by_k ? lane_d(upto, 63) : mass;
            const bool kept = w > 0.0 && x >= set.least &&
                              (set.p == 1.0 || lane == 0 || upto - w < set.p * all);
            // Again in the order of the vocabulary.
            sh->list.weight[lane] = w;
            wave_lds_sync();
            const uint64_t there = wave_sort<true>(
                kept ? (uint64_t)(uint32_t)key << 32 | (uint32_t)lane : 0, lane);
            w = there != 0 ? sh->list.weight[(uint32_t)there] : 0.0;
            upto = wave_upto(w);
            const double total = lane_d(upto, 63);
            const uint64_t some = __ballot(w > 0.0);
            uint64_t past = __ballot(w > 0.0 && upto > set.uniform * total);
            if (!past) past = 1ull << (63 - __clzll(some));
            if (lane == __ffsll((unsigned long long)past) - 1) {
                sh->token = (int)~(uint32_t)(there >> 32);
                sh->left = w;
                sh->total = total;
            }
        }
        __syncthreads();
        logprob = log_share(sh->total);
        return sh->token;
    }

    // Draws from the n collected logits, which hold everything kept.
    __device__ __forceinline__ int draw_list(int n, bool by_k, double mass, float& logprob) {
        const int tid = threadIdx.x;
        sort_keys(tid < n ? sh->list.keys[tid] : 0, n, sh->list.keys, sh->list.sorted);
        const uint64_t key = tid < n ? sh->list.sorted[tid] : 0;
        const double x = exponent(image_value((uint32_t)(key >> 32)));
        double w = tid < n && x >= kNone ? table_exp(x, sh->table) : 0.0;
        if (by_k && tid >= set.k) w = 0.0;
        double all;
        const double upto = before(w, sh->waves, all);
        if (!by_k) all = mass;
        const bool kept = w > 0.0 && x >= set.least &&
                          (set.p == 1.0 || tid == 0 || upto < set.p * all);
        // Again in the order of the vocabulary.
        const uint32_t index = ~(uint32_t)key;
        if (tid < n) sh->list.weight[tid] = w;
        if (tid == 0) {
            sh->first = kList;
            sh->last = -1;
        }
        sort_keys(kept ? (uint64_t)~index << 32 | (uint32_t)tid : 0, n, sh->list.keys,
                  sh->list.sorted);
        const int many = __syncthreads_count(kept);
        double mine = 0.0;
        uint64_t here = 0;
        if (tid < many) {
            here = sh->list.sorted[tid];
            mine = sh->list.weight[(uint32_t)here];
        }
        const double at = before(mine, sh->waves, all);
        note_first(mine > 0.0 && at + mine > set.uniform * all);
        note_last(mine > 0.0);
        __syncthreads();
        const int found = sh->first < kList ? sh->first : sh->last;
        if (tid == found) {
            sh->token = (int)~(uint32_t)(here >> 32);
            sh->left = mine;
        }
        __syncthreads();
        logprob = log_share(all);
        return sh->token;
    }

    // The shortest prefix of the order whose count (or mass) reaches `target`:
    // the bin of a histogram over the values in which it ends, and that bin's
    // logits sorted, or, if they are many, bins of them again down to one value,
    // whose ties are counted.  reach: how far below the largest logit the bins
    // go; the last one holds what lies beyond.  Bins sum in fixed point, whose
    // order does not matter; inside a bin sums are FP64.
    __device__ __forceinline__ Cut select(bool by_mass, double target, bool masses, float reach) {
        const int tid = threadIdx.x, lane = tid & 63;
        const Cut everything{-INFINITY, 0x7fffffff, 0.0, 0.0};
        const double unit = 1.0 / scale;
        const uint64_t goal =
            by_mass ? (uint64_t)fmax(ceil(target * scale), 1.0) : (uint64_t)target;
        const float steps = fminf((float)(kBins - 1) / reach, 1e30f);
        const auto bin_of = [&](float v) {
            return (int)fminf(fminf(top32 - v, FLT_MAX) * steps, (float)(kBins - 1));
        };
        clear_bins();
        lane_slots<L, NT>(row, 0, row.n, tid, [&](const float (&v)[VEC], int) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (!(v[j] > -INFINITY)) continue;
                const int b = bin_of(v[j]);
                atomicAdd(&sh->bins.count[b], 1u);
                if (masses && (!by_mass || b < kBins - 1))
                    atomicAdd(&sh->bins.mass[b], fixed(weight(v[j])));
            }
        });
        uint32_t count = 0, here = 0;
        uint64_t mass = 0, here_mass = 0;
        int bin = find_bin(by_mass, goal, count, mass, here, here_mass);
        if (bin == kBins) return everything;
        if (here <= (uint32_t)kList) {
            if (tid == 0) sh->count = 0;
            __syncthreads();
            lane_slots<L, NT>(row, 0, row.n, tid, [&](const float (&v)[VEC], int e) {
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (v[j] > -INFINITY && bin_of(v[j]) == bin)
                        sh->list.keys[atomicAdd(&sh->count, 1)] =
                            value_key(v[j], (uint32_t)(e + j));
            });
            __syncthreads();
            sort_keys(tid < (int)here ? sh->list.keys[tid] : 0, (int)here, sh->list.keys,
                      sh->list.sorted);
            const uint64_t key = tid < (int)here ? sh->list.sorted[tid] : 0;
            const float z = image_value((uint32_t)(key >> 32));
            const double w = masses && tid < (int)here ? weight(z) : 0.0;
            double all;
            const double m = (double)mass * unit + before(w, sh->waves, all);
            const bool reached = by_mass ? m + w >= target : (double)count + tid + 1.0 >= target;
            if (tid == 0) sh->first = (int)here - 1;
            __syncthreads();
            note_first(tid < (int)here && reached);
            __syncthreads();
            if (tid == sh->first) {
                sh->limit = z;
                sh->last = (int)~(uint32_t)key;
                sh->total = m + w;
            }
            __syncthreads();
            const Cut found{sh->limit, sh->last, 0.0, sh->total};
            __syncthreads();
            return found;
        }
        // The images of the bin's logits, from smallest to largest.
        uint32_t lo = 0xffffffffu, hi = 0;
        lane_slots<L, NT>(row, 0, row.n, tid, [&](const float (&v)[VEC], int) {
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (v[j] > -INFINITY && bin_of(v[j]) == bin) {
                    const uint32_t i = Image<L>::of(v[j]);
                    lo = i < lo ? i : lo;
                    hi = i > hi ? i : hi;
                }
        });
        if (tid == 0) {
            sh->low = 0xffffffffu;
            sh->high = 0;
        }
        __syncthreads();
        lo = (uint32_t)wave_least((int)(lo ^ 0x80000000u), lane) ^ 0x80000000u;
        hi = ~((uint32_t)wave_least((int)(~hi ^ 0x80000000u), lane) ^ 0x80000000u);
        if (lane == 0 && lo <= hi) {
            atomicMin(&sh->low, lo);
            atomicMax(&sh->high, hi);
        }
        __syncthreads();
        lo = sh->low;
        hi = sh->high;
        for (;;) {
            recompute();
            int shift = 0;
            while ((hi - lo) >> shift >= (uint32_t)kBins) ++shift;
            clear_bins();
            lane_slots<L, NT>(row, 0, row.n, tid, [&](const float (&v)[VEC], int e) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const uint32_t i = Image<L>::of(v[j]);
                    if (i > hi || i < lo || !(v[j] > -INFINITY)) continue;
                    const uint32_t b = (hi - i) >> shift;
                    atomicAdd(&sh->bins.count[b], 1u);
                    if (masses)
                        atomicAdd(&sh->bins.mass[b], fixed(weight(v[j])));
                }
            });
            bin = find_bin(by_mass, goal, count, mass, here, here_mass);
            if (bin == kBins) return everything;
            const uint32_t last = hi - ((uint32_t)bin << shift);
            const uint32_t first = last - ((1u << shift) - 1);
            hi = last;
            lo = first < lo || first > last ? lo : first;
            if (shift == 0) break;
        }
        // One value: as many of its tokens as the target wants, by index.
        const float z = Image<L>::value(hi);
        const double w = masses ? weight(z) : 0.0, light = (double)mass * unit;
        double ties = by_mass ? ceil((target - light) / w) : target - (double)count;
        ties = fmin(fmax(ties, 1.0), (double)here);
        return {z, 0x7fffffff, ties < (double)here ? ties : 0.0, light + w * ties};
    }

    // The shortest prefix of the order that holds `target` of the mass, as select
    // finds it, in two passes: a histogram of weights in FP32, whose sums are sure
    // of the cut up to a few bins, then those bins' logits, sorted, on top of an
    // exact sum of what lies above them, by stretches of a wave each, which stays
    // in sh->waves with the kept ones added.  False if those logits are too many.
    __device__ __forceinline__ bool nucleus(double target, float reach, double& total) {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, each = row_stretch();
        constexpr float kUnit = 2147483648.0f;
        const float steps = fminf((float)(kBins - 1) / reach, 1e30f);
        const float c = (float)(set.inv_tau * 1.4426950408889634);
        clear_bins();
        lane_slots<L, NT>(row, 0, row.n, tid, [&](const float (&v)[VEC], int) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = fminf(top32 - v[j], FLT_MAX);
                const int b = (int)fminf(d * steps, (float)(kBins - 1));
                const uint32_t w = (uint32_t)(__builtin_amdgcn_exp2f(-d * c) * kUnit);
                if (w != 0 && b < kBins - 1)
                    atomicAdd(&sh->bins.mass[b], (unsigned long long)w);
            }
        });
        __syncthreads();
        // A weight is off by less than 1e-5 of itself and one unit.
        constexpr int kEach = kBins / NT;
        uint64_t m = 0, all;
#pragma unroll
        for (int i = 0; i < kEach; ++i) m += sh->bins.mass[tid * kEach + i];
        if (tid == 0) {
            sh->first = kBins;
            sh->last = kBins;
        }
        m = before(m, sh->waves_mass, all);
        const double goal = target * (double)kUnit;
        int most = kBins, least = kBins;
#pragma unroll
        for (int i = kEach - 1; i >= 0; --i) {
            uint64_t upto = m;
#pragma unroll
            for (int k = 0; k <= i; ++k) upto += sh->bins.mass[tid * kEach + k];
            if ((double)upto * (1.0 + 1e-5) + (double)p.vocab >= goal) least = tid * kEach + i;
            if ((double)upto * (1.0 - 1e-5) >= goal) most = tid * kEach + i;
        }
        // (the sums ascend: a wave's first lane that has one)
        const uint64_t some = __ballot(least < kBins), sure = __ballot(most < kBins);
        if (some && lane == __ffsll((unsigned long long)some) - 1) atomicMin(&sh->first, least);
        if (sure && lane == __ffsll((unsigned long long)sure) - 1) atomicMin(&sh->last, most);
        if (tid == 0) sh->count = 0;
        __syncthreads();
        const float low = (float)sh->first, high = (float)(sh->last + 1);
        __syncthreads();   // everyone has read them before they change
        if (high > (float)kBins) return false;
        int from = wave * each;
        if (from > row.n) from = row.n;
        double sum = 0.0;
        const double steepness = set.inv_tau * kScale;
        lane_slots<L, 64>(row, from, from + each < row.n ? from + each : row.n, lane,
                          [&](const float (&v)[VEC], int e) {
            bool some = false;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float b = fminf(top32 - v[j], FLT_MAX) * steps;
                // (what lies above the cut is far from weight 0)
                const double w = table_exp_scaled(
                    fmax(((double)v[j] - top) * steepness, -700.0 * kScale), sh->table);
                sum += b < low ? w : 0.0;
                some = some || (b >= low && b < high);
            }
            if (!some) return;   // one branch a slot
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float b = fminf(top32 - v[j], FLT_MAX) * steps;
                if (b >= low && b < high) {
                    const int i = atomicAdd(&sh->count, 1);
                    if (i < kList) sh->list.keys[i] = value_key(v[j], (uint32_t)(e + j));
                }
            }
        });
        sum = wave_sum_d(sum, lane);
        if (lane == 0) sh->waves_above[wave] = sum;
        if (tid == 0) sh->first = 0x7fffffff;
        __syncthreads();
        const int n = sh->count;
        if (n > kList || n == 0) return false;
        double above = 0.0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) above += sh->waves_above[i];
        sort_keys(tid < n ? sh->list.keys[tid] : 0, n, sh->list.keys, sh->list.sorted);
        const uint64_t key = tid < n ? sh->list.sorted[tid] : 0;
        const float z = image_value((uint32_t)(key >> 32));
        const double w = tid < n ? weight(z) : 0.0;
        sh->list.weight[tid] = w;
        double here;
        const double upto = above + before(w, sh->waves, here) + w;
        note_first(tid < n && upto >= target);
        __syncthreads();
        const int end = sh->first < n ? sh->first : n - 1;   // the last one kept
        if (tid == end) {
            sh->limit = z;
            sh->last = (int)~(uint32_t)key;
        }
        // The stretches' shares of the kept ones.
        sum = 0.0;
        for (int i = lane; i <= end; i += 64) {
            const int slot = ((int)~(uint32_t)sh->list.sorted[i] - row.e0) / VEC;
            if (slot / each == wave) sum += sh->list.weight[i];
        }
        sum = wave_sum_d(sum, lane);
        if (lane == 0) sh->waves[wave] = sh->waves_above[wave] + sum;
        __syncthreads();
        cut.z = sh->limit;
        cut.last = sh->last;
        cut.ties = 0.0;
        total = 0.0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) total += sh->waves[i];
        return true;
    }

    __device__ __forceinline__ void clear_bins() {
        for (int b = threadIdx.x; b < kBins; b += NT) {
            sh->bins.count[b] = 0;
            sh->bins.mass[b] = 0;
        }
        if (threadIdx.x == 0) sh->bin = kBins;
        __syncthreads();
    }

    // The first bin at whose end the count (or mass) reaches the target; count and
    // mass become what lies before it, here and here_mass its own.
    __device__ __forceinline__ int find_bin(bool by_mass, uint64_t target, uint32_t& count, uint64_t& mass,
                                            uint32_t& here, uint64_t& here_mass) {
        constexpr int kEach = kBins / NT;
        const int tid = threadIdx.x;
        __syncthreads();
        uint32_t c = 0, all_count;
        uint64_t m = 0, all_mass;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            c += sh->bins.count[tid * kEach + i];
            m += sh->bins.mass[tid * kEach + i];
        }
        c = count + before(c, sh->waves_count, all_count);
        m = mass + before(m, sh->waves_mass, all_mass);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int b = tid * kEach + i;
            const uint32_t c1 = c + sh->bins.count[b];
            const uint64_t m1 = m + sh->bins.mass[b];
            const uint64_t was = by_mass ? m : c, is = by_mass ? m1 : c1;
            if (was < target && is >= target) {   // one bin of all
                sh->bin = b;
                sh->before_count = c;
                sh->before_mass = m;
            }
            c = c1;
            m = m1;
        }
        __syncthreads();
        const int bin = sh->bin;
        if (bin < kBins) {
            count = sh->before_count;
            mass = sh->before_mass;
            here = sh->bins.count[bin];
            here_mass = sh->bins.mass[bin];
        }
        __syncthreads();
        return bin;
    }

    // From the stretches' sums in LDS to the token.  Every thread comes here.
    __device__ __forceinline__ int draw(float& logprob) {
        const int tid = threadIdx.x, vocab = p.vocab;
        logprob = NAN;
        find_top();
        if (!(top32 < INFINITY) || !set.fine) return -1;   // NaN, +inf
        if (top32 == -INFINITY) {
            logprob = -INFINITY;
            return -1;
        }
        const bool by_k = set.cut_by_k(vocab), by_p = set.p < 1.0;
        if (set.k == 1) {
            // The first stretch that holds the largest logit.
            int s = 0;
            while (sh->stretch[s].top != top32) ++s;
            int from, to;
            stretch_slots(row, p, stretch_waves, s, from, to);
            if (tid == 0) sh->first = 0x7fffffff;
            __syncthreads();
            int mine = 0x7fffffff;
            lane_slots<L, NT>(row, from, to, tid, [&](const float (&v)[VEC], int e) {
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (v[j] == top32 && e + j < mine) mine = e + j;
            });
            mine = wave_least(mine, tid & 63);
            if ((tid & 63) == 0 && mine != 0x7fffffff) atomicMin(&sh->first, mine);
            __syncthreads();
            logprob = 0.0f;
            return sh->first;
        }
        cut = {-INFINITY, 0x7fffffff, 0.0, 0.0};
        double mass = 0.0, left = 0.0;
        int from = 0, to = -1;   // the stretch to draw in, once it is known
        if (set.needs_mass(vocab)) {
            sum_stretches();
            mass = sh->total;
            if (!by_p) {
                stretch_slots(row, p, stretch_waves, sh->chosen, from, to);
                left = sh->left;
            }
        }
        if (to < 0) {
            // A bound, and the few logits at or above it.
            float low = INFINITY;
            for (int i = tid & 63; i < stretches; i += 64) low = fminf(low, sh->stretch[i].low);
            low = wave_minimum(low, tid & 63);
            const float steps = fminf((float)(kBounds - 1) / fminf(top32 - low, FLT_MAX), 1e30f);
            float limit = INFINITY;
            bool bounded = by_k && set.k <= kList / 2;
            // (the weights in FP32 are off by less than 1e-5)
            const double want = by_k ? (double)set.k : set.p * mass * (262144.0 * (1.0 + 1e-5)) + 2.0;
            if (bounded || (by_p && !by_k && want < 2e9))
                limit = bound((uint32_t)want, !by_k, steps);
            // Tokens under min-p matter to the mass of the first k alone.
            if (set.least > -INFINITY && !(by_k && by_p))
                limit = fminf(limit, fmaxf((float)(-set.least / set.inv_tau * (1.0 + 2e-5)) * steps,
                                           FLT_MIN));
            bounded = bounded || limit < INFINITY;
            if (tid == 0) sh->count = sh->active = 0;
            __syncthreads();
            if (bounded) {
                const int n = collect(steps, limit);
                if (n <= 64) return draw_few(n, by_k, mass, logprob);
                if (n <= kList) return draw_list(n, by_k, mass, logprob);
                __syncthreads();
            }
            // Many: by a histogram of the row, by k and then by p.
            const float octave = (float)(0.6931471805599453 / set.inv_tau);
            bool summed = false;   // the stretches of what is kept
            double all = 0.0;
            if (by_k) {
                cut = select(false, (double)set.k, by_p, 64.0f * octave);
                mass = cut.mass;
                if (by_p && cut.z == -INFINITY) {
                    // Fewer finite logits than k: all of them, min-p or not.
                    const double least = set.least;
                    set.least = -INFINITY;
                    mass = sum_row();
                    set.least = least;
                    __syncthreads();
                }
            }
            if (by_p) {
                // Tokens too light to make up 1 - p of the mass all together are
                // not in the shortest prefix.
                const float light = log2f((float)(3.0 * (double)vocab / ((1.0 - set.p) * mass)));
                const float reach = fminf(fmaxf(light, 1.0f), 64.0f) * octave;
                summed = nucleus(set.p * mass, reach, all);
                if (!summed) {
                    // The finest steps in which a row of this mass stays below 2^62.
                    if (!by_k) scale = ldexp(1.0, 61 - ilogb(mass));
                    cut = select(true, set.p * mass, true, reach);
                }
            }
            if (cut.ties > 0.0) cut.last = find_tie(cut.z, (uint32_t)cut.ties);
            if (!summed || exponent(cut.z) < set.least) all = sum_row();
            mass = all;
            find_stretch(set.uniform * all, from, to, left);
        }
        const int token = locate(from, to, left);
        logprob = log_share(mass);
        return token;
    }

    __device__ __forceinline__ void finish(int64_t r) {
        float logprob;
        const int token = draw(logprob);
        if (threadIdx.x == 0) {
            p.token[r] = token;
            if (p.logprob) p.logprob[r] = logprob;
        }
    }
};

// Where there are more rows than workgroups at work at a time, those whose whole
// mass is needed go first, among kOrdered neighbouring rows: a flat row's nucleus
// takes a workgroup ten times as long as a best-50, and one that began last would
// be waited for alone (1,024 rows of 131,072 BF16 with mixed settings 163 us in
// their own order).  Every workgroup finds its row from the settings.
constexpr int kOrdered = 1024;

template <int NT>
__device__ __forceinline__ int64_t ordered_row(const SampleParams& p, uint32_t* counts) {
    constexpr int kEach = kOrdered / NT;   // neighbouring rows of a thread
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t base = (int64_t)(blockIdx.x / kOrdered) * kOrdered;
    const int n = p.rows - base < kOrdered ? (int)(p.rows - base) : kOrdered;
    const uint32_t want = blockIdx.x % kOrdered;
    uint32_t heavy[kEach], mine = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t r = base + (tid * kEach + i < n ? tid * kEach + i : 0);
        const float t = p.temperature ? p.temperature[r] : p.tau;
        const int32_t k = p.top_k ? p.top_k[r] : 0;
        const float top_p = p.top_p ? p.top_p[r] : 1.0f, q = p.min_p ? p.min_p[r] : 0.0f;
        heavy[i] = tid * kEach + i < n && t != 0.0f && (k <= 0 || k >= p.vocab) &&
                   (top_p < 1.0f || !(q > 0.0f));
        mine += heavy[i];
    }
    const uint32_t upto = wave_upto(mine);
    if (lane == 63) counts[wave] = upto;
    __syncthreads();
    uint32_t before = upto - mine, all = 0;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
        before += i < wave ? counts[i] : 0;
        all += counts[i];
    }
    // The row that lands on this workgroup's place.
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t r = tid * kEach + i;
        const uint32_t place = heavy[i] ? before : all + r - before;
        if ((int)r < n && place == want) counts[NT / 64] = r;
        before += heavy[i];
    }
    __syncthreads();
    return base + counts[NT / 64];
}

// A row a workgroup.
template <typename L, int NT>
__global__ void __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(4)))
sample_kernel(SampleParams p) {
    using S = Sampler<L, NT, 1>;
    __shared__ typename S::Shared shared;
    __shared__ uint32_t counts[NT / 64 + 1];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int64_t r = p.rows > kSampleGroups * (1024 / NT) ? ordered_row<NT>(p, counts) : blockIdx.x;
    S s(p, &shared);
    s.set.read(p, r);
    s.row.init(p.logits, r * p.stride, p.vocab, p.chunk, 1, 0);
    s.scale = ldexp(1.0, p.unit);
    s.stretches = s.stretch_waves = NT / 64;
    fill_table(shared.table, NT);
    for (int i = tid; i < kBoundsRoom; i += NT) shared.bounds[i] = 0;
    __syncthreads();
    int from, to;
    stretch_slots(s.row, p, NT / 64, wave, from, to);
    const Stretch got = scan_any<L>(s.row, from, to, s.set, p.vocab, shared.table, s.group[0]);
    if ((tid & 63) == 0) shared.stretch[wave] = got;
    __syncthreads();
    s.finish(r);
}

// A part of a row a workgroup: its stretches, left in the workspace.
template <typename L>
__global__ void __launch_bounds__(kScanThreads) sample_scan_kernel(SampleParams p) {
    __shared__ double table[kTable];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int64_t r = blockIdx.x / (uint32_t)p.parts;
    const int part = (int)(blockIdx.x % (uint32_t)p.parts);
    Settings set;
    set.read(p, r);
    Part<L> row;
    row.init(p.logits, r * p.stride, p.vocab, p.chunk, 1, 0);
    fill_table(table, kScanThreads);
    __syncthreads();
    const int i = part * kScanWaves + wave;
    int from, to;
    stretch_slots(row, p, kScanWaves, i, from, to);
    float lane_top;
    const Stretch got = scan_any<L>(row, from, to, set, p.vocab, table, lane_top);
    const int stretches = p.parts * kScanWaves;
    char* space = p.space + r * stretches * kStretchBytes;
    if ((tid & 63) == 0) reinterpret_cast<Stretch*>(space)[i] = got;
    reinterpret_cast<float*>(space + stretches * sizeof(Stretch))[part * kScanThreads + tid] =
        lane_top;
}

constexpr int kDrawThreads = 1024;

template <typename L>
__global__ void __launch_bounds__(kDrawThreads) sample_draw_kernel(SampleParams p) {
    constexpr int NT = kDrawThreads;
    constexpr int kGroups = kMostStretches * 64 / NT;
    using S = Sampler<L, NT, kGroups>;
    __shared__ typename S::Shared shared;
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x;
    S s(p, &shared);
    s.stretches = p.parts * kScanWaves;
    s.stretch_waves = kScanWaves;
    const char* space = p.space + r * s.stretches * kStretchBytes;
    const float* tops = reinterpret_cast<const float*>(space + s.stretches * sizeof(Stretch));
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
        s.group[g] = g * NT + tid < s.stretches * 64 ? tops[g * NT + tid] : -INFINITY;
    if (tid < s.stretches) shared.stretch[tid] = reinterpret_cast<const Stretch*>(space)[tid];
    s.set.read(p, r);
    s.row.init(p.logits, r * p.stride, p.vocab, p.chunk, 1, 0);
    s.scale = ldexp(1.0, p.unit);
    fill_table(shared.table, NT);
    for (int i = tid; i < kBoundsRoom; i += NT) shared.bounds[i] = 0;
    __syncthreads();
    s.finish(r);
}

template <typename L>
int run_sample(const ws_rows& r, const SamplePlan& plan, const SampleParams& p, hipStream_t s) {
    if (plan.parts > 1) {
        const int v = launch(sample_scan_kernel<L>, (int64_t)r.rows * plan.parts, kScanThreads, p, s);
        return v != WS_OK ? v : launch(sample_draw_kernel<L>, r.rows, kDrawThreads, p, s);
    }
    const auto kernel = plan.threads == 256   ? sample_kernel<L, 256>
                        : plan.threads == 512 ? sample_kernel<L, 512>
                                              : sample_kernel<L, 1024>;
    return launch(kernel, r.rows, plan.threads, p, s);
}

}  // namespace
}  // namespace ws

extern "C" int ws_sample_workspace(const ws_rows* rows, size_t* bytes) {
    const int v = ws::validate_rows(rows);
    if (v != WS_OK) return v;
    if (!bytes) return WS_E_INVALID_ARG;
    *bytes = ws::plan_sample(*rows).workspace;
    return WS_OK;
}

extern "C" int ws_sample(const ws_rows* rows, const ws_sample_args* args, void* stream) {
    using namespace ws;
    int v = ws::validate_sample(rows, args);
    if (v != WS_OK) return v;
    const ws_rows& r = *rows;
    if (r.rows == 0) return WS_OK;
    const ws::SamplePlan plan = ws::plan_sample(r);
    v = ws::validate_sample_workspace(r, *args, plan.workspace);
    if (v != WS_OK) return v;
    v = ws::device_ready(r.device);
    if (v != WS_OK) return v;
    ws::SampleParams p{};
    p.logits = args->logits;
    p.stride = r.row_stride;
    p.uniform = args->uniform;
    p.temperature = args->temperature;
    p.top_k = args->top_k;
    p.top_p = args->top_p;
    p.min_p = args->min_p;
    p.token = args->token;
    p.logprob = args->logprob;
    p.space = static_cast<char*>(args->workspace);
    p.rows = r.rows;
    p.vocab = r.vocab;
    p.chunk = plan.chunk;
    p.parts = plan.parts;
    p.tau = r.temperature;
    p.unit = plan.unit;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (r.dtype == WS_DTYPE_F32) return ws::run_sample<F32>(r, plan, p, s);
    if (r.dtype == WS_DTYPE_F16) return ws::run_sample<F16>(r, plan, p, s);
    return ws::run_sample<BF16>(r, plan, p, s);
}
