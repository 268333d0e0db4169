// ws_logits_rows.h -- device code shared by the kernels over rows of logits:
// a row as 16-byte slots, running softmax sums, and reductions of a workgroup.
// Internal to the library.
//
// A row may start at any element address.  It is read as 16-byte slots at
// aligned addresses: slot s holds the VEC elements from s * VEC - off on,
// where off is the row start's distance, in elements, from the aligned
// address at or below it.  Slots that lie in the row whole are one 16-byte
// load; the first and last, where they stick out, are read element by element.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "ws_fp64.h"
#include "ws_lanes.h"
#include "ws_logits.h"

namespace ws {

constexpr float kLog2e = 1.44269504088896340736f;
// A finite stand-in below every difference z - max that matters: at the
// highest temperature exp((z - max) / tau) is 0 from -1.04e5 on, and 0 times a
// finite number is 0 where 0 times -inf would be NaN.
constexpr float kFar = -1.0e6f;

// ---- element types ---------------------------------------------------------

// kStream: slots are read and written past the caches, for matrices too large
// to find or leave anything there.
struct F32 {
    using Elem = float;
    static constexpr bool kStream = false;
    static constexpr int VEC = 4;
    static __device__ __forceinline__ uint4 none() {   // -inf
        return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
    }
    static __device__ __forceinline__ float up(float v) { return v; }
    static __device__ __forceinline__ float down(float v) { return v; }
    static __device__ __forceinline__ void unpack(uint4 w, float (&v)[VEC]) {
        v[0] = __uint_as_float(w.x);
        v[1] = __uint_as_float(w.y);
        v[2] = __uint_as_float(w.z);
        v[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[VEC]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
};

struct F16 {
    using Elem = _Float16;
    static constexpr bool kStream = false;
    static constexpr int VEC = 8;
    typedef _Float16 Pair __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ uint4 none() {   // -inf
        return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u);
    }
    static __device__ __forceinline__ float up(_Float16 v) { return (float)v; }
    static __device__ __forceinline__ _Float16 down(float v) { return (_Float16)v; }
    static __device__ __forceinline__ void unpack(uint4 w, float (&v)[VEC]) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Pair p = __builtin_bit_cast(Pair, x[i]);
            v[2 * i] = (float)p.x;
            v[2 * i + 1] = (float)p.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[VEC]) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Pair p;
            p.x = (_Float16)v[2 * i];
            p.y = (_Float16)v[2 * i + 1];
            x[i] = __builtin_bit_cast(uint32_t, p);
        }
        return make_uint4(x[0], x[1], x[2], x[3]);
    }
};

struct BF16 {
    using Elem = __bf16;
    static constexpr bool kStream = false;
    static constexpr int VEC = 8;
    typedef __bf16 Pair __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ uint4 none() {   // -inf
        return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
    }
    static __device__ __forceinline__ float up(__bf16 v) {
        return __uint_as_float((uint32_t)__builtin_bit_cast(uint16_t, v) << 16);
    }
    static __device__ __forceinline__ __bf16 down(float v) { return (__bf16)v; }   // nearest even
    static __device__ __forceinline__ void unpack(uint4 w, float (&v)[VEC]) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(x[i] << 16);
            v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[VEC]) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Pair p;
            p.x = (__bf16)v[2 * i];
            p.y = (__bf16)v[2 * i + 1];
            x[i] = __builtin_bit_cast(uint32_t, p);
        }
        return make_uint4(x[0], x[1], x[2], x[3]);
    }
};

template <typename B>
struct Streamed : B {
    static constexpr bool kStream = true;
};

typedef uint32_t Slot16 __attribute__((ext_vector_type(4)));

template <typename L>
__device__ __forceinline__ uint4 load_slot(const void* p) {
    if constexpr (L::kStream) {
        const Slot16 v = __builtin_nontemporal_load(static_cast<const Slot16*>(p));
        return make_uint4(v.x, v.y, v.z, v.w);
    } else {
        return *static_cast<const uint4*>(p);
    }
}

template <typename L>
__device__ __forceinline__ void store_slot(void* p, uint4 w) {
    if constexpr (L::kStream) {
        const Slot16 v = {w.x, w.y, w.z, w.w};
        __builtin_nontemporal_store(v, static_cast<Slot16*>(p));
    } else {
        *static_cast<uint4*>(p) = w;
    }
}

// ---- a workgroup's part of a row ---------------------------------------------

// Slots [first, first + n) of a row; slot numbers below are relative to first.
template <typename L>
struct Part {
    static constexpr int VEC = L::VEC;
    const typename L::Elem* row;   // element 0 of the row
    const char* base;              // address of relative slot 0 (16-byte aligned)
    int vocab;
    int e0;                        // element at relative slot 0's start (may be < 0)
    int n;                         // slots
    int full_from, full_to;        // relative slots that lie in the row whole

    // chunk: slots of a part; index: which of `parts`.  The last takes the rest.
    __device__ __forceinline__ void init(const void* logits, int64_t at, int V, int chunk,
                                         int parts, int index) {
        row = static_cast<const typename L::Elem*>(logits) + at;
        vocab = V;
        const int off = (int)(((uintptr_t)row & 15u) / sizeof(typename L::Elem));
        const int slots = (V + off + VEC - 1) / VEC;
        const int first = index * chunk;
        n = index == parts - 1 ? slots - first : chunk;
        e0 = first * VEC - off;
        base = reinterpret_cast<const char*>(row - off) + (int64_t)first * 16;
        full_from = first == 0 && off != 0 ? 1 : 0;
        const int whole = (V + off) / VEC - first;
        full_to = whole < n ? whole : n;
    }
    __device__ __forceinline__ uint4 load(int s) const {
        return load_slot<L>(base + (uint32_t)s * 16u);
    }
    // The nearest whole slot's content (there is one), whatever s: a load under
    // a condition would be waited for before the next is issued.
    __device__ __forceinline__ uint4 load_near(int s) const {
        const int last = full_to - 1;
        return load(s < full_from ? full_from : s < last ? s : last);
    }
    // Element by element; -inf outside the row.
    __device__ __forceinline__ void load_edge(int s, float (&v)[VEC]) const {
        typename L::Elem x[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int e = e0 + s * VEC + j;
            x[j] = row[e < 0 ? 0 : e < vocab ? e : vocab - 1];
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int e = e0 + s * VEC + j;
            v[j] = e >= 0 && e < vocab ? L::up(x[j]) : -INFINITY;
        }
    }
    __device__ __forceinline__ bool whole(int s) const { return s >= full_from && s < full_to; }
};

// ---- running sums --------------------------------------------------------------

// With respect to a running maximum m (-FLT_MAX or more, so that a difference
// from it is never inf - inf in a row without +inf):
//   s = sum e_j, u = sum e_j (z_j - m), e_j = 2^((z_j - m) c), c = log2(e) / tau.
struct Sums {
    float m, s, u;

    __device__ __forceinline__ void init() {
        m = -FLT_MAX;
        s = 0.0f;
        u = 0.0f;
    }
    // Moves to a maximum of at least m.
    template <bool ENT>
    __device__ __forceinline__ void raise(float to, float c) {
        const float d = m - to;
        const float a = __builtin_amdgcn_exp2f(d * c);
        if constexpr (ENT) u = a * (u + fmaxf(d, kFar) * s);
        s *= a;
        m = to;
    }
    template <bool ENT>
    __device__ __forceinline__ void add(Sums b, float c) {
        const float to = fmaxf(m, b.m);
        raise<ENT>(to, c);
        b.raise<ENT>(to, c);
        s += b.s;
        if constexpr (ENT) u += b.u;
    }
};

template <int J>
__device__ __forceinline__ float xor_lane_f(float v, int lane) {
    return __uint_as_float(xor_lane32<J>(__float_as_uint(v), lane));
}

__device__ __forceinline__ float wave_max(float v, int lane) {
    v = fmaxf(v, xor_lane_f<32>(v, lane));
    v = fmaxf(v, xor_lane_f<16>(v, lane));
    v = fmaxf(v, xor_lane_f<8>(v, lane));
    v = fmaxf(v, xor_lane_f<4>(v, lane));
    v = fmaxf(v, xor_lane_f<2>(v, lane));
    return fmaxf(v, xor_lane_f<1>(v, lane));
}

__device__ __forceinline__ float wave_sum(float v, int lane) {
    v += xor_lane_f<32>(v, lane);
    v += xor_lane_f<16>(v, lane);
    v += xor_lane_f<8>(v, lane);
    v += xor_lane_f<4>(v, lane);
    v += xor_lane_f<2>(v, lane);
    return v + xor_lane_f<1>(v, lane);
}

template <int J>
__device__ __forceinline__ double xor_lane_d(double v, int lane) {
    return __builtin_bit_cast(double, xor_lane64<J>(__builtin_bit_cast(uint64_t, v), lane));
}

__device__ __forceinline__ double lane_d(double v, int lane) {
    return __builtin_bit_cast(double, readlane64(__builtin_bit_cast(uint64_t, v), lane));
}

__device__ __forceinline__ double wave_sum_d(double v, int lane) {
    v += xor_lane_d<32>(v, lane);
    v += xor_lane_d<16>(v, lane);
    v += xor_lane_d<8>(v, lane);
    v += xor_lane_d<4>(v, lane);
    v += xor_lane_d<2>(v, lane);
    return v + xor_lane_d<1>(v, lane);
}

// log x in FP64 for x between 1e-30 and 1e30: the FP32 logarithm L, and what
// x e^-L leaves of 1.
__device__ __forceinline__ double small_log(double x) {
    const double l = (double)__logf((float)x);
    const double r = fma(x, small_exp(-l), -1.0);
    return l + r * fma(r, fma(r, 1.0 / 3.0, -0.5), 1.0);
}

// The sums of a wave's lanes, in every lane.
template <bool ENT>
__device__ __forceinline__ Sums wave_join(Sums a, float c, int lane) {
    a.raise<ENT>(wave_max(a.m, lane), c);
    a.s = wave_sum(a.s, lane);
    if constexpr (ENT) a.u = wave_sum(a.u, lane);
    return a;
}

// ---- order keys ------------------------------------------------------------------

// Order-preserving unsigned image of an FP32 value: NaN -> -inf and -0 -> +0
// first, then larger values have larger images; 0 is below every image.
__device__ __forceinline__ uint32_t value_image(float v) {
    uint32_t b = __float_as_uint(v);
    b = (b & 0x7fffffffu) > 0x7f800000u ? 0xff800000u : b;
    b = b == 0x80000000u ? 0u : b;
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float image_value(uint32_t i) {
    return __uint_as_float(i & 0x80000000u ? i ^ 0x80000000u : ~i);
}

// (value descending, index ascending) as one integer, larger = better.
__device__ __forceinline__ uint64_t value_key(float v, uint32_t index) {
    return ((uint64_t)value_image(v) << 32) | (uint32_t)~index;
}

// Number of the n keys of v (LDS) greater than x.
__device__ __forceinline__ int keys_above(const uint64_t* v, int n, uint64_t x) {
    int r = 0, j = 0;
    for (; j + 8 <= n; j += 8) {
        uint64_t t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = v[j + i];
#pragma unroll
        for (int i = 0; i < 8; ++i) r += t[i] > x ? 1 : 0;
    }
    for (; j < n; ++j) r += v[j] > x ? 1 : 0;
    return r;
}

}  // namespace ws
