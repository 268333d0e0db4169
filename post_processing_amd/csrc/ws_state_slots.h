// ws_state_slots.h -- device code shared by the kernels over rows of hidden
// states: 16-byte slots of a row at any element address, and a workgroup's
// sums.  Internal to the library.
//
// Slot s of a row is its elements s * VEC .. s * VEC + VEC - 1, read and
// written as one 16-byte access wherever the row starts: gfx950 takes global
// accesses of dwords at any byte address (a row that starts off 16 bytes
// straddles a cache line in every fourth slot or so).  The elements of a last
// slot that ends behind the row are read and written one by one.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ws_logits_rows.h"

// CALL(type) for the rows' element type.
#define WS_BY_DTYPE(dtype, CALL)                             \
    do {                                                     \
        if ((dtype) == WS_DTYPE_F32) { CALL(F32); }          \
        else if ((dtype) == WS_DTYPE_F16) { CALL(F16); }     \
        else { CALL(BF16); }                                 \
    } while (0)

namespace ws {

typedef uint32_t Slot2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t Slot4 __attribute__((ext_vector_type(4), aligned(4)));

template <typename L>
using LooseSlot = std::conditional_t<sizeof(typename L::Elem) == 2, Slot2, Slot4>;

template <typename L>
__device__ __forceinline__ uint4 load_loose(const typename L::Elem* p) {
    const Slot16 v = *reinterpret_cast<const LooseSlot<L>*>(p);
    return make_uint4(v.x, v.y, v.z, v.w);
}

template <typename L>
__device__ __forceinline__ void store_loose(typename L::Elem* p, uint4 w) {
    const Slot16 v = {w.x, w.y, w.z, w.w};
    *reinterpret_cast<LooseSlot<L>*>(p) = v;
}

// Elements c .. c + VEC - 1 of a row of `width`, 0 behind it.
template <typename L>
__device__ __forceinline__ uint4 load_columns(const typename L::Elem* row, int c, int width) {
    if (c + L::VEC <= width) return load_loose<L>(row + c);
    float v[L::VEC];
#pragma unroll
    for (int j = 0; j < L::VEC; ++j) v[j] = c + j < width ? L::up(row[c + j]) : 0.0f;
    return L::pack(v);
}

template <typename L>
__device__ __forceinline__ void store_columns(typename L::Elem* row, int c, int width,
                                              const float (&v)[L::VEC]) {
    if (c + L::VEC <= width) {
        store_loose<L>(row + c, L::pack(v));
        return;
    }
#pragma unroll
    for (int j = 0; j < L::VEC; ++j)
        if (c + j < width) row[c + j] = L::down(v[j]);
}

// The same of a row of N FP32 or L values (a weight, a sum), as `f32` says.
template <typename L>
__device__ __forceinline__ void load_either(const void* row, bool f32, int c, int width,
                                            float (&v)[L::VEC]) {
    if (f32) {
        const float* p = static_cast<const float*>(row);
        if (c + L::VEC <= width) {
#pragma unroll
            for (int j = 0; j < L::VEC; j += 4) {
                float part[4];
                F32::unpack(load_loose<F32>(p + c + j), part);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j + i] = part[i];
            }
        } else {
#pragma unroll
            for (int j = 0; j < L::VEC; ++j) v[j] = c + j < width ? p[c + j] : 0.0f;
        }
    } else {
        L::unpack(load_columns<L>(static_cast<const typename L::Elem*>(row), c, width), v);
    }
}

template <typename L>
__device__ __forceinline__ void store_either(void* row, bool f32, int c, int width,
                                             const float (&v)[L::VEC]) {
    if (f32) {
        float* p = static_cast<float*>(row);
        if (c + L::VEC <= width) {
#pragma unroll
            for (int j = 0; j < L::VEC; j += 4) {
                const float part[4] = {v[j], v[j + 1], v[j + 2], v[j + 3]};
                store_loose<F32>(p + c + j, F32::pack(part));
            }
        } else {
#pragma unroll
            for (int j = 0; j < L::VEC; ++j)
                if (c + j < width) p[c + j] = v[j];
        }
    } else {
        store_columns<L>(static_cast<typename L::Elem*>(row), c, width, v);
    }
}

// The sum over the LANES neighbouring lanes (a power of two) one's own is among,
// in each of them.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v, int lane) {
    if constexpr (LANES > 32) v += xor_lane_f<32>(v, lane);
    if constexpr (LANES > 16) v += xor_lane_f<16>(v, lane);
    if constexpr (LANES > 8) v += xor_lane_f<8>(v, lane);
    v += xor_lane_f<4>(v, lane);
    v += xor_lane_f<2>(v, lane);
    return v + xor_lane_f<1>(v, lane);
}

// The sums of two values over NT threads, in each of them: neighbouring lanes of a
// wave, or the workgroup.  `waves` (LDS) must not be written again before every
// thread has read it: two sums in turn take two.
template <int NT>
__device__ __forceinline__ float2 group_sums(float2 v, float2* waves) {
    const int lane = threadIdx.x & 63;
    v.x = lanes_sum<NT < 64 ? NT : 64>(v.x, lane);
    v.y = lanes_sum<NT < 64 ? NT : 64>(v.y, lane);
    if constexpr (NT > 64) {
        if (lane == 0) waves[threadIdx.x >> 6] = v;
        __syncthreads();
        v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) {
            v.x += waves[i].x;
            v.y += waves[i].y;
        }
    }
    return v;
}

template <int NT>
__device__ __forceinline__ float group_sum(float v, float* waves) {
    const int lane = threadIdx.x & 63;
    v = lanes_sum<NT < 64 ? NT : 64>(v, lane);
    if constexpr (NT > 64) {
        if (lane == 0) waves[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) v += waves[i];
    }
    return v;
}

// Slots a thread holds of every row of its NT threads: i * NT + thread.  All are full, so that no
// load hangs on a condition: a last slot that would end behind the row begins
// earlier instead and has its first elements in common with the one before, and
// threads without a slot hold the row's end too.  Needs rows of VEC elements.
template <typename L, int NT, int R>
struct HeldSlots {
    static constexpr int VEC = L::VEC;
    int at[R];      // first column
    int own[R];     // the thread's own elements are own[i] and behind

    __device__ __forceinline__ explicit HeldSlots(int width) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (i * NT + (int)threadIdx.x % NT) * VEC;
            at[i] = c + VEC <= width ? c : width - VEC;
            own[i] = c - at[i];
        }
    }
    __device__ __forceinline__ bool mine(int i, int j) const { return j >= own[i]; }
    // Whether the slot holds elements of its own, and so is written whole: what
    // two threads write twice is the same.
    __device__ __forceinline__ bool any(int i) const { return own[i] < VEC; }
    __device__ __forceinline__ void load(const typename L::Elem* row, uint4 (&w)[R]) const {
#pragma unroll
        for (int i = 0; i < R; ++i) w[i] = load_loose<L>(row + at[i]);
    }
    // A weight's values for the slots, FP32 or L; `none` without one.
    __device__ __forceinline__ void weights(const void* row, bool f32, float none,
                                            float (&v)[R][VEC]) const {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (row) {
                load_either<L>(row, f32, at[i], at[i] + VEC, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[i][j] = none;
            }
        }
    }
};

}  // namespace ws
