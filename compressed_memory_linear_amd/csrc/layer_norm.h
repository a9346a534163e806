// layer_norm.h -- what the norm kernels share: the layout of a row over the
// lanes of a workgroup, row sums, the gates.
//
// A row of D values is held by TPR threads, 8 K values each, in registers: it is
// read once, and every statistic is taken from the registers.  Where D is a
// multiple of 8 and the rows are 16-byte aligned a thread's 8 values are
// neighbours (16 bytes of bf16 to a load); elsewhere they are TPR apart, so
// that any D and any alignment of whole elements works, one element to a load.
#pragma once

#include "layer_device.h"
#include "layer_launch.h"

namespace layer {

constexpr int kE = 8;  // values per thread and piece

// Rows are loaded non-temporally, and the backward's gradients stored so (R32768 D2048 bf16:
// backward 212 -> 206 us).  In the forward so is x_out, which is read again only after the next block, and
// not z, which the next kernel reads (both plain 130 us, both non-temporal 125, so 115).  Each
// workgroup walks over its rows with the next one in flight: 3 workgroups of 256 threads per
// compute unit in the forward and 2 in the backward measured best (forward 2: 115 us, 3: 113, 4: 115;
// backward 1: 288, 2: 206, 3: 226, 4: 254).
template <int TPR_, int K_>
struct NormShape {
    static constexpr int TPR = TPR_;                       // threads per row
    static constexpr int K = K_;                           // pieces of 8 values per thread
    static constexpr int NT = TPR_ < 256 ? 256 : TPR_;     // threads per workgroup
    static constexpr int ROWS = NT / TPR_;                 // rows of a workgroup at a time
    static constexpr int WPR = TPR_ <= 64 ? 1 : TPR_ / 64; // waves per row
};

// Index of value e of piece k in its row.
template <typename S, bool VEC>
__device__ __forceinline__ int col_of(int lane, int k, int e) {
    return VEC ? (k * S::TPR + lane) * kE + e : (k * kE + e) * S::TPR + lane;
}

template <typename T>
struct Piece {
    T e[kE];
};

// The rows that a workgroup takes at once, as one buffer per tensor (of no bytes where
// the tensor is absent or the rows lie past the last): loads and stores need no branch.
struct Rows {
    int64_t first;  // element
    int count;      // elements
};
template <typename S>
__device__ __forceinline__ Rows rows_of(uint32_t it, int R, int D) {
    const int64_t left = R - static_cast<int64_t>(it) * S::ROWS;
    const int rows = left <= 0 ? 0 : left < S::ROWS ? static_cast<int>(left) : S::ROWS;
    return Rows{static_cast<int64_t>(it) * S::ROWS * D, rows * D};
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t norm_rsrc(const void* p, bool bf16, Rows r) {
    const int e = bf16 ? 2 : 4;
    return rows_rsrc(p, r.first * e, p ? r.count * e : 0);
}
// Byte offset of this thread's value e of piece k among those rows.
template <typename S, bool VEC>
__device__ __forceinline__ uint32_t off_of(int lane, int sub, int k, int e, int D, int size) {
    const int c = col_of<S, VEC>(lane, k, e);
    return c < D ? static_cast<uint32_t>(sub * D + c) * size : kOut;
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
template <typename S, bool VEC, typename T>
__device__ __forceinline__ void load_piece(__amdgpu_buffer_rsrc_t r, int lane, int sub, int k, int D, Piece<T>& o) {
    if constexpr (VEC) {
        const uint32_t at = off_of<S, true>(lane, sub, k, 0, D, sizeof(T));
        constexpr int N = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < kE / N; ++i) {
            const auto v = __builtin_bit_cast(
                Vec<T, N>, __builtin_amdgcn_raw_buffer_load_b128(r, at + i * 16, 0, kNt));
#pragma unroll
            for (int j = 0; j < N; ++j) o.e[i * N + j] = v.e[j];
        }
    } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const uint32_t at = off_of<S, false>(lane, sub, k, e, D, sizeof(T));
            if constexpr (sizeof(T) == 2)
                o.e[e] = __builtin_bit_cast(T, static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0)));
            else
                o.e[e] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
        }
    }
}
// Piece k of a weight of D values; ones where it is absent.
template <typename S, bool VEC>
__device__ __forceinline__ void load_weights(const float* p, int lane, int k, int D, float (&o)[kE]) {
    Piece<float> w;
    load_piece<S, VEC>(rows_rsrc(p, 0, p ? D * 4 : 0), lane, 0, k, D, w);
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = p ? w.e[e] : 1.0f;
}
// NT: written past the caches.
template <typename S, bool VEC, bool NT>
__device__ __forceinline__ void store_piece(__amdgpu_buffer_rsrc_t r, bool bf16, int lane, int sub, int k, int D,
                                            const float (&x)[kE]) {
    with_flag(bf16, [&](auto b) {
        constexpr bool BF16 = decltype(b)::value;
        constexpr int size = BF16 ? 2 : 4;
        if constexpr (VEC) {
            const uint32_t at = off_of<S, true>(lane, sub, k, 0, D, size);
            if constexpr (BF16) {
                u32x4_t w;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = osr::f32_to_bf16_bits(x[2 * j]) |
                           static_cast<uint32_t>(osr::f32_to_bf16_bits(x[2 * j + 1])) << 16;
                __builtin_amdgcn_raw_buffer_store_b128(w, r, at, 0, NT ? kNt : 0);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    __builtin_amdgcn_raw_buffer_store_b128(
                        u32x4_t{__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3])}, r, at + 16 * i, 0, NT ? kNt : 0);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kE; ++e) store_row<BF16, NT>(r, off_of<S, false>(lane, sub, k, e, D, size), x[e]);
        }
    });
}

// Sums of up to 2 values over the threads of a row, in all of them, in a fixed order.  Across
// waves they meet in LDS: `buf` is used in turns of two, so that one barrier
// separates a read from the write two sums later.
template <typename S>
struct RowSum {
    float (*buf)[S::NT / 64][2];  // [2][waves][2]
    int turn = 0;
    template <int N>
    __device__ __forceinline__ void operator()(float (&x)[N]) {
        static_assert(N <= 2, "the buffer's width");
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = osr::group_sum<(S::TPR < 64 ? S::TPR : 64)>(x[n]);
        if (S::WPR == 1) return;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) buf[turn][wave][n] = x[n];
        }
        __syncthreads();
        const int first = wave / S::WPR * S::WPR;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < S::WPR; ++w) s += buf[turn][first + w][n];
            x[n] = s;
        }
        turn ^= 1;
    }
};

// 1 / sqrt(x) for normal x > 0, to the last place or so: the hardware's estimate
// and one Newton step, which infinite x (squares past fp32) does not take.
__device__ __forceinline__ float rsqrt_acc(float x) {
    const float r = __builtin_amdgcn_rsqf(x);
    return r > 0.0f ? r * fmaf(-0.5f * x * r, r, 1.5f) : r;
}

// GeLU's parts for a gate g: cdf = Phi(g), and e = exp(-g^2 / 2), which its density takes too.
// With a = |g| and t = 1 / (1 + 0.35 a), Phi(-a) = e t q(t): q is the polynomial of degree 8
// nearest to exp(a^2 / 2) Phi(-a) / t in relative error (1.72e-7 for a up to 20, fitted for this by
// reweighted least squares; past 14.5 e is 0), so the lower tail keeps its relative accuracy; the
// argument of the exponential, rounded, costs up to 1.12 g^2 2^-24, and the evaluation in fp32 up to 16 units of
// 2^-24 (8 seen in all).  A third of the operations of erfcf.
__device__ __forceinline__ void gelu_parts(float g, float& cdf, float& e) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.35f, fabsf(g), 1.0f));
    e = __builtin_amdgcn_exp2f(g * g * -0.72134752f);
    float q = -2.508340625e-02f;
    q = fmaf(q, t, 1.262319635e-01f);
    q = fmaf(q, t, -2.233420272e-01f);
    q = fmaf(q, t, 1.271268000e-01f);
    q = fmaf(q, t, -4.416478743e-03f);
    q = fmaf(q, t, 9.897989587e-02f);
    q = fmaf(q, t, 1.211549029e-01f);
    q = fmaf(q, t, 1.397210148e-01f);
    q = fmaf(q, t, 1.396274145e-01f);
    const float lower = q * t * e;
    cdf = g < 0.0f ? lower : 1.0f - lower;
}

// Calls f with the NormShape for rows of D values: the fewest threads that hold
// the row with one piece each, up to a workgroup of 1024; past 8192 two pieces.  A power of two of
// them: widths just above one idle their threads (D2560 bf16 4.2 TB/s forward and 3.7 backward, D5120 3.6 and
// 3.3, where 2048 and 4096 reach 5.8 and 5.0 or more).
template <typename F>
void with_shape(int D, F&& f) {
    if (D <= 64) f(NormShape<8, 1>());
    else if (D <= 128) f(NormShape<16, 1>());
    else if (D <= 256) f(NormShape<32, 1>());
    else if (D <= 512) f(NormShape<64, 1>());
    else if (D <= 1024) f(NormShape<128, 1>());
    else if (D <= 2048) f(NormShape<256, 1>());
    else if (D <= 4096) f(NormShape<512, 1>());
    else if (D <= 8192) f(NormShape<1024, 1>());
    else f(NormShape<1024, 2>());
}

}  // namespace layer
