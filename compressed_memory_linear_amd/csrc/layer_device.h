// layer_device.h -- device helpers shared by the layer operators' kernels:
// vectors of V consecutive elements, and the gates.
#pragma once

#include <type_traits>

#include "osr_device.h"

namespace layer {

// V consecutive elements as stored: V floats, or V bf16 bit patterns.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p, int64_t i) {
    return *reinterpret_cast<const Vec<T, V>*>(p + i);
}
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return osr::bf16_bits_to_f32(x); }

// V values stored as fp32, or as bf16 (the one rounding, to nearest even).
template <int V>
__device__ __forceinline__ void store_vec(void* p, int64_t i, const float (&x)[V], bool bf16) {
    if (bf16) {
        Vec<uint16_t, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) o.e[j] = osr::f32_to_bf16_bits(x[j]);
        *reinterpret_cast<Vec<uint16_t, V>*>(static_cast<uint16_t*>(p) + i) = o;
    } else {
        Vec<float, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) o.e[j] = x[j];
        *reinterpret_cast<Vec<float, V>*>(static_cast<float*>(p) + i) = o;
    }
}

// e^x through the hardware's 2^x.  Rounded to one float, the product x log2(e) costs a
// relative 1.2 |x| 2^-24 of the result (log2(e) as a float is 0.2 of that); ACC keeps what the
// product and the constant lose as a second part (5 operations more; without the constant's
// the result is off by 20 units at |x| = 80).  For bf16 logits, known to 2^-9 of their
// value, the first form serves.
template <bool ACC>
__device__ __forceinline__ float exp_of(float x) {
    constexpr float kLog2e = 1.44269504088896341f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147181f;
    const float hi = x * kLog2e;
    const float e = __builtin_amdgcn_exp2f(hi);
    if constexpr (!ACC) return e;
    const float lo = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -hi));
    // past the range of 2^x the low part is not wanted (it is NaN at infinite x)
    return fabsf(hi) < 128.0f ? fmaf(e, lo * kLn2, e) : e;
}

// s = sigmoid(x) and r = 1 - s, each to a few units of 2^-24 of its own value (ACC as
// above): with e = e^-x, s = 1 / (1 + e) and r = e s (1 once e is so large that s is
// below half a unit of 1; the product would be inf 0 there).  x = -inf gives
// s = 0, r = 1 and x = +inf gives s = 1, r = 0, exactly; NaN stays NaN.
template <bool ACC>
__device__ __forceinline__ void sigmoid2(float x, float& s, float& r) {
    const float e = exp_of<ACC>(-x);
    s = __builtin_amdgcn_rcpf(1.0f + e);
    r = e > 33554432.0f ? 1.0f : e * s;
}
template <typename T>
constexpr bool kAccurate = sizeof(T) == 4;  // logits of type T

// The scan's input weight w(mu), from mu and 1 - mu.
template <int WT>
__device__ __forceinline__ float weight_of(float m, float om) {
    if constexpr (WT == 1) return om;
    if constexpr (WT == 2) return __builtin_amdgcn_sqrtf(om * (1.0f + m));
    return 1.0f;
}

// Some rows of a tensor as a buffer of their own: an access past the last of them, or
// by a lane without channels (kOut), reads zero and writes nothing; so does every access
// to one of no bytes, which stands for an absent tensor.  Offsets are in bytes, whole in the
// address register (the part of the bounds check that needs no care); a buffer has at
// most 2^30 of them, so kOut plus a row's offset lies outside and does not wrap.
constexpr uint32_t kOut = 0x80000000u;
// Streamed once, rows are loaded non-temporally (B8 T4096 D2048 bf16 forward 90 -> 83 us; inputs that
// the 256 MB cache still holds lose: B7 T1531 D1001 fp32 36 -> 40).  The backward's stores too
// (training step 322 -> 306 us); not the forward's, whose y the next kernel reads.
constexpr int kNt = 2;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* p, int64_t first, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(static_cast<char*>(const_cast<void*>(p)) + first, 0, bytes, 0x00020000);
}
template <typename T>
__device__ __forceinline__ T load_row(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    if constexpr (sizeof(T) == 2)
        return __builtin_bit_cast(T, static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, kNt)));
    else
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, kNt));
}
// NT: written past the caches.
template <bool BF16, bool NT>
__device__ __forceinline__ void store_row(__amdgpu_buffer_rsrc_t r, uint32_t off, float x) {
    if constexpr (BF16)
        __builtin_amdgcn_raw_buffer_store_b16(osr::f32_to_bf16_bits(x), r, off, 0, NT ? kNt : 0);
    else
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), r, off, 0, NT ? kNt : 0);
}

// The value, in a register whose origin the compiler does not see: offsets taken from
// it are formed where they are used and not held from the top of the kernel (16 to 32 registers).
__device__ __forceinline__ uint32_t here(uint32_t x) {
    asm("" : "+v"(x));
    return x;
}

// The same, anew each time it is reached: what is read or computed from the result is
// not kept from the last time.
template <typename T>
__device__ __forceinline__ T anew(T x) {
    asm volatile("" : "+v"(x));
    return x;
}

// f(constant) for a flag that is the same in every thread: one branch around a whole
// loop instead of one in each of its steps.
template <typename F>
__device__ __forceinline__ void with_flag(bool flag, F&& f) {
    if (flag)
        f(std::true_type());
    else
        f(std::false_type());
}

}  // namespace layer
