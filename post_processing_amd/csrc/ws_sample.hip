// ws_sample.hip -- tokens drawn from rows of logits (ws_logits.h), written for
// gfx950 (CDNA4, wave64).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ws_enqueue.h"
#include "ws_lanes.h"
#include "ws_logits.h"
#include "ws_logits_plan.h"
#include "ws_logits_rows.h"

namespace ws {
namespace {

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
    int32_t vocab;
    int32_t slots;      // of an aligned row
    float tau;          // of every row, without `temperature`
    int32_t unit;       // sums in fixed point count units of 2^-unit
};

// A row's settings as its workgroup reads them.
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
};

// Calls f(values, element of values[0]) for slots from, from + step, ... below
// `to` of a part; elements outside the row are -inf.
template <typename L, typename F>
__device__ __forceinline__ void walk(const Part<L>& part, int from, int to, int step, F f) {
    for (int s = from; s < to; s += step) {
        float v[L::VEC];
        if (part.whole(s)) L::unpack(part.load(s), v);
        else part.load_edge(s, v);
        f(v, part.e0 + s * L::VEC);
    }
}

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

constexpr int kBins = 2048;

struct Histogram {
    uint32_t count[kBins];
    unsigned long long mass[kBins];
};

// A prefix of the order: the tokens above z, and the first `ties` at it.
struct Cut {
    float z;
    int ties;             // as many as there are: all
    bool all;             // every token at z
    uint32_t above;       // how many before z
    uint64_t mass;        // of the prefix, in fixed point
};

template <typename L, int NT>
struct Sampler {
    static constexpr int VEC = L::VEC;
    static constexpr int kWaves = NT / 64;

    struct Shared {
        Histogram h;
        uint64_t waves_mass[kWaves];
        uint32_t waves_count[kWaves];
        double waves[kWaves];
        float top[kWaves];
        int flags[kWaves];
        int bin;
        int first, last;
        uint32_t before_count;
        uint64_t before_mass;
        int token;
    };

    Part<L> part;
    Shared* sh;
    Settings set;
    double top;       // largest logit
    double scale;     // 2^unit

    __device__ __forceinline__ double weight(float z) const {
        return small_exp(((double)z - top) * set.inv_tau);
    }
    __device__ __forceinline__ uint64_t fixed(double w) const { return (uint64_t)(w * scale + 0.5); }

    // The largest logit; false if the row holds a NaN or +inf.
    __device__ __forceinline__ bool find_top() {
        float m = -INFINITY;
        bool bad = false;
        walk(part, threadIdx.x, part.n, NT, [&](const float (&v)[VEC], int) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                m = fmaxf(m, v[j]);
                bad |= !(v[j] < INFINITY);
            }
        });
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        m = wave_max(m, lane);
        const bool any = __ballot(bad) != 0;
        if (lane == 0) {
            sh->top[wave] = m;
            sh->flags[wave] = any;
        }
        __syncthreads();
        bad = false;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            m = fmaxf(m, sh->top[i]);
            bad |= sh->flags[i] != 0;
        }
        top = (double)m;
        return !bad;
    }

    // The shortest prefix of the order whose count (or mass) reaches `target`,
    // narrowed down bin by bin over the values' images.
    template <bool MASS>
    __device__ Cut select(uint64_t target, bool masses) {
        const int tid = threadIdx.x;
        uint32_t hi = Image<L>::of((float)top), lo = 0;
        Cut cut{-INFINITY, 0, true, 0, 0};
        uint32_t count = 0;       // before hi
        uint64_t mass = 0;
        for (;;) {
            int shift = 0;
            while ((hi - lo) >> shift >= (uint32_t)kBins) ++shift;
            for (int b = tid; b < kBins; b += NT) {
                sh->h.count[b] = 0;
                sh->h.mass[b] = 0;
            }
            if (tid == 0) sh->bin = kBins;
            __syncthreads();
            walk(part, tid, part.n, NT, [&](const float (&v)[VEC], int e) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const uint32_t i = Image<L>::of(v[j]);
                    if (i > hi || i < lo || e + j < 0 || e + j >= part.vocab) continue;
                    const uint32_t b = (hi - i) >> shift;
                    atomicAdd(&sh->h.count[b], 1u);
                    if (masses) atomicAdd(&sh->h.mass[b], (unsigned long long)fixed(weight(v[j])));
                }
            });
            __syncthreads();
            // Sums of a thread's neighbouring bins, then across the threads.
            constexpr int kEach = kBins / NT;
            uint32_t c = 0;
            uint64_t m = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                c += sh->h.count[tid * kEach + i];
                m += sh->h.mass[tid * kEach + i];
            }
            scan(c, m, count, mass);
            // The first bin whose end reaches the target.
            uint32_t cc = c;
            uint64_t mm = m;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int b = tid * kEach + i;
                const uint32_t c1 = cc + sh->h.count[b];
                const uint64_t m1 = mm + sh->h.mass[b];
                const uint64_t was = MASS ? mm : cc, is = MASS ? m1 : c1;
                if (was < target && is >= target) {   // one bin of all
                    sh->bin = b;
                    sh->before_count = cc;
                    sh->before_mass = mm;
                }
                cc = c1;
                mm = m1;
            }
            __syncthreads();
            const int bin = sh->bin;
            count = sh->before_count;
            mass = sh->before_mass;
            const uint32_t here = sh->h.count[bin < kBins ? bin : 0];
            const uint64_t here_mass = sh->h.mass[bin < kBins ? bin : 0];
            __syncthreads();
            if (bin == kBins) return cut;   // all of them do not
            const uint32_t last = hi - ((uint32_t)bin << shift);
            const uint32_t first = last - ((1u << shift) - 1);
            hi = last;
            lo = first < lo || first > last ? lo : first;
            if (shift > 0) continue;
            cut.z = Image<L>::value(hi);
            cut.above = count;
            uint32_t ties = here;
            if (MASS) {
                const uint64_t each = here_mass / here;
                ties = (uint32_t)((target - mass + each - 1) / each);
            } else {
                ties = (uint32_t)target - count;
            }
            cut.all = ties >= here;
            cut.ties = (int)(cut.all ? here : ties);
            cut.mass = mass + here_mass / here * (uint64_t)cut.ties;
            return cut;
        }
    }

    // Exclusive sums across the threads, on top of what came before.
    __device__ __forceinline__ void scan(uint32_t& c, uint64_t& m, uint32_t count, uint64_t mass) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        uint32_t ci = c;
        uint64_t mi = m;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t co = __shfl_up(ci, d);
            const uint64_t mo = __shfl_up((unsigned long long)mi, d);
            if (lane >= d) {
                ci += co;
                mi += mo;
            }
        }
        if (lane == 63) {
            sh->waves_count[wave] = ci;
            sh->waves_mass[wave] = mi;
        }
        __syncthreads();
        c = count + ci - c;
        m = mass + mi - m;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            c += i < wave ? sh->waves_count[i] : 0;
            m += i < wave ? sh->waves_mass[i] : 0;
        }
    }

    // Over the amounts f(value, element) >= 0 of the row in the order of the
    // vocabulary: the first element up to which they sum to more than
    // target(all of them); -1 if all are 0.  A workgroup's waves sum
    // neighbouring stretches; the threads then share out the stretch that holds
    // the target; one thread walks its part of that.  Every sum's order is
    // fixed; where rounding leaves the target behind a stretch's end, its last
    // element above 0 is taken.
    template <typename F, typename T>
    __device__ int locate(F f, T target, double& total) {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
        const int stretch = (part.n + kWaves - 1) / kWaves;
        const int from = wave * stretch;
        const int to = from + stretch < part.n ? from + stretch : part.n;
        double sum = 0.0;
        walk(part, from + lane, to, 64, [&](const float (&v)[VEC], int e) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += f(v[j], e + j);
        });
        sum = wave_sum_d(sum, lane);
        if (lane == 0) sh->waves[wave] = sum;
        if (tid == 0) {
            sh->first = NT;
            sh->last = -1;
            sh->token = -1;
        }
        __syncthreads();
        total = 0.0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) total += sh->waves[i];
        double rest = target(total);
        int chosen = -1;
        double left = 0.0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const double w = sh->waves[i];
            if (w > 0.0 && rest >= 0.0) {
                chosen = i;
                left = rest;
            }
            rest -= w;
        }
        __syncthreads();
        if (chosen < 0) return -1;
        const int begin = chosen * stretch;
        const int end = begin + stretch < part.n ? begin + stretch : part.n;
        const int each = (end - begin + NT - 1) / NT;
        const int mine = begin + tid * each;
        const int mine_end = mine + each < end ? mine + each : end;
        sum = 0.0;
        walk(part, mine, mine_end, 1, [&](const float (&v)[VEC], int e) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += f(v[j], e + j);
        });
        double upto = sum;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const double other = __shfl_up(upto, d);
            if (lane >= d) upto += other;
        }
        if (lane == 63) sh->waves[wave] = upto;
        __syncthreads();
        double before = 0.0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) before += i < wave ? sh->waves[i] : 0.0;
        upto += before;
        if (sum > 0.0) {
            if (upto > left) atomicMin(&sh->first, tid);
            atomicMax(&sh->last, tid);
        }
        __syncthreads();
        if (tid == (sh->first < NT ? sh->first : sh->last)) {
            double at = upto - sum;
            int found = -1;
            bool done = false;
            walk(part, mine, mine_end, 1, [&](const float (&v)[VEC], int e) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const double w = f(v[j], e + j);
                    if (!done && w > 0.0) {
                        found = e + j;
                        at += w;
                        done = at > left;
                    }
                }
            });
            sh->token = found;
        }
        __syncthreads();
        const int token = sh->token;
        __syncthreads();   // everyone has read it before the next call clears it
        return token;
    }
};

template <typename L, int NT>
__global__ void __launch_bounds__(NT) sample_kernel(SampleParams p) {
    using S = Sampler<L, NT>;
    __shared__ typename S::Shared shared;
    const int64_t row = blockIdx.x;
    S s;
    s.sh = &shared;
    s.part.init(p.logits, row * p.stride, p.vocab, p.slots, 1, 0);
    s.set.read(p, row);
    s.scale = ldexp(1.0, p.unit);
    const bool clean = s.find_top();
    int token = -1;
    float logprob = NAN;
    if (clean && s.set.fine) {
        if (s.top == -INFINITY) {
            logprob = -INFINITY;
        } else {
            // The cut: of the first k, then of their mass.
            Cut cut{-INFINITY, 0, true, 0, 0};
            const bool by_mass = s.set.p < 1.0;
            uint64_t mass = 0;
            if (s.set.k < p.vocab) {
                cut = s.template select<false>((uint64_t)s.set.k, by_mass);
                mass = cut.mass;
            } else if (by_mass) {
                // All of it: the mass no prefix can exceed.
                double all;
                s.locate([&](float z, int) { return (double)s.fixed(s.weight(z)); },
                         [](double) { return 0.0; }, all);
                mass = (uint64_t)all;
            }
            if (by_mass) {
                const double want = ceil(s.set.p * (double)mass);
                cut = s.template select<true>(want < 1.0 ? 1 : (uint64_t)want, true);
            }
            // The last of the ties at the cut that belongs to it.
            int last = 0x7fffffff;
            double all;
            if (!cut.all) {
                const float z = cut.z;
                last = s.locate([&](float v, int) { return v == z ? 1.0 : 0.0; },
                                [&](double) { return (double)cut.ties - 0.5; }, all);
            }
            const float z = cut.z;
            const auto kept = [&](float v, int e) {
                if (!(v > z || (v == z && e <= last)) || v == -INFINITY) return 0.0;
                const double x = ((double)v - s.top) * s.set.inv_tau;
                return x >= s.set.least ? small_exp(x) : 0.0;
            };
            token = s.locate(kept, [&](double w) { return s.set.uniform * w; }, all);
            if (token >= 0) {
                const double x = ((double)L::up(s.part.row[token]) - s.top) * s.set.inv_tau;
                logprob = (float)(x - small_log(all));
            }
        }
    }
    if (threadIdx.x == 0) {
        p.token[row] = token;
        if (p.logprob) p.logprob[row] = logprob;
    }
}

template <typename L>
int run_sample(const ws_rows& r, const SamplePlan& plan, const SampleParams& p, hipStream_t s) {
    return launch(plan.threads == 256 ? sample_kernel<L, 256> : sample_kernel<L, 1024>, r.rows,
                  plan.threads, p, s);
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
    v = ws::validate_workspace(args->workspace, args->workspace_bytes, plan.workspace);
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
    p.vocab = r.vocab;
    p.slots = (int32_t)ws::slots_of(r);
    p.tau = r.temperature;
    int bits = 10;
    while ((1ll << bits) < r.vocab) ++bits;
    p.unit = 62 - bits;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (r.dtype == WS_DTYPE_F32) return ws::run_sample<F32>(r, plan, p, s);
    if (r.dtype == WS_DTYPE_F16) return ws::run_sample<F16>(r, plan, p, s);
    return ws::run_sample<BF16>(r, plan, p, s);
}
