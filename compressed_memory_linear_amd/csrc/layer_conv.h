// layer_conv.h -- what the kernels of the short causal convolution share.
//     p_t = bias + sum_j w[j] x_{t-W+1+j},   y_t = p_t sigmoid(p_t)  (or p_t);
//     dp = dy act'(p),  dx_s = sum_k w[W-1-k] dp_{s+k},  dw[j] = sum_t dp_t x_{t-W+1+j},  dbias = sum dp.
// A thread takes a run of tokens of V neighbouring channels: every row is read once per run, and those in front of
// it again.  A border between documents empties the registers of the rows before it, which is all that
// segments take.
#pragma once

#include "layer_device.h"
#include "layer_launch.h"

namespace layer {

constexpr int kConvRun = 16;       // tokens a thread of the forward walks over
constexpr int kConvBwdRun = 128;   // and of the backward, in groups of
constexpr int kConvGroup = 4;

// The filters of one thread's channels.
template <int V, int W>
struct Taps {
    float w[W][V], bias[V];
    __device__ __forceinline__ void load(const ConvParams& p, int c) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            bias[e] = p.bias ? p.bias[c + e] : 0.0f;
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = p.w[static_cast<int64_t>(c + e) * W + j];
        }
    }
};

__device__ __forceinline__ int conv_length(const ConvParams& p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}
// Whether token t begins a document (the first one goes on from the history).
__device__ __forceinline__ bool begins(const ConvParams& p, int b, int t) {
    if (!p.segments || t <= 0) return false;
    const int64_t i = static_cast<int64_t>(b) * p.T + t;
    return p.segments[i] != p.segments[i - 1];
}
// Row t > -W of a sequence, the history in front of it.
template <typename TIn, int V, int W>
__device__ __forceinline__ Vec<TIn, V> conv_row(const ConvParams& p, int b, int t, int c) {
    if (t >= 0) return load_vec<TIn, V>(static_cast<const TIn*>(p.x), (static_cast<int64_t>(b) * p.T + t) * p.x_row + c);
    if (!p.hist_in) return Vec<TIn, V>{};
    return load_vec<TIn, V>(static_cast<const TIn*>(p.hist_in),
                            (static_cast<int64_t>(b) * (W - 1) + t + W - 1) * p.D + c);
}
template <typename TIn, int V>
__device__ __forceinline__ void put_vec(void* to, int64_t i, const Vec<TIn, V>& v) {
    *reinterpret_cast<Vec<TIn, V>*>(static_cast<TIn*>(to) + i) = v;
}

// Call f with the taps, and with the inputs' type and the channels of a thread.
template <typename F>
void with_taps(int W, F&& f) {
    switch (W) {
        case 1: f(std::integral_constant<int, 1>()); break;
        case 2: f(std::integral_constant<int, 2>()); break;
        case 3: f(std::integral_constant<int, 3>()); break;
        case 4: f(std::integral_constant<int, 4>()); break;
        case 5: f(std::integral_constant<int, 5>()); break;
        case 6: f(std::integral_constant<int, 6>()); break;
        case 7: f(std::integral_constant<int, 7>()); break;
        default: f(std::integral_constant<int, 8>()); break;
    }
}
template <typename F>
void with_types(const ConvParams& p, F&& f) {
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 4> four;
    if (p.in_bf16)
        p.vec ? f(uint16_t(), four) : f(uint16_t(), one);
    else
        p.vec ? f(float(), four) : f(float(), one);
}

}  // namespace layer
