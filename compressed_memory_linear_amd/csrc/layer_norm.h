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

// Piece k of a row (zeros past its end); p is the row's first value.
template <typename S, bool VEC, typename T>
__device__ __forceinline__ void load_piece(const T* p, int lane, int k, int D, Piece<T>& o) {
    if (VEC) {
        const int c = col_of<S, true>(lane, k, 0);
        constexpr int N = 16 / sizeof(T);
        if (c < D) {
#pragma unroll
            for (int i = 0; i < kE / N; ++i) {
                const Vec<T, N> v = load_vec<T, N>(p, c + i * N);
#pragma unroll
                for (int j = 0; j < N; ++j) o.e[i * N + j] = v.e[j];
            }
        } else {
#pragma unroll
            for (int e = 0; e < kE; ++e) o.e[e] = T(0);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const int c = col_of<S, false>(lane, k, e);
            o.e[e] = c < D ? p[c] : T(0);
        }
    }
}
template <typename S, bool VEC>
__device__ __forceinline__ void load_weights(const float* p, int lane, int k, int D, float (&o)[kE]) {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int c = col_of<S, VEC>(lane, k, e);
        o[e] = c < D ? (p ? p[c] : 1.0f) : 0.0f;
    }
}
template <typename S, bool VEC>
__device__ __forceinline__ void store_piece(void* p, bool bf16, int64_t row, int lane, int k, int D,
                                            const float (&x)[kE]) {
    if (VEC) {
        const int c = col_of<S, true>(lane, k, 0);
        if (c >= D) return;
        if (bf16) {
            store_vec<kE>(p, row + c, x, true);
        } else {
            const float lo[4] = {x[0], x[1], x[2], x[3]}, hi[4] = {x[4], x[5], x[6], x[7]};
            store_vec<4>(p, row + c, lo, false);
            store_vec<4>(p, row + c + 4, hi, false);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const int c = col_of<S, false>(lane, k, e);
            const float v[1] = {x[e]};
            if (c < D) store_vec<1>(p, row + c, v, bf16);
        }
    }
}

// Sums of N values over the threads of a row, in all of them, in a fixed order.  Across
// waves they meet in LDS: `buf` is used in turns of two, so that one barrier
// separates a read from the write two sums later.
template <typename S, int N>
struct RowSum {
    float (*buf)[S::NT / 64][N];  // [2][waves][N]
    int turn = 0;
    __device__ __forceinline__ void operator()(float (&x)[N]) {
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

// Calls f with the NormShape for rows of D values: the fewest threads that hold
// the row with one piece each, up to a workgroup of 1024; past 8192 two pieces.
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
