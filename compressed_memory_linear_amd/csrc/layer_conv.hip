// layer_conv.hip -- the short causal convolution in front of a recurrence:
// forward, backward and single step.
//     p_t = bias + sum_j w[j] x_{t-W+1+j},   y_t = p_t sigmoid(p_t)  (or p_t);
//     dp = dy act'(p),  dx_s = sum_k w[W-1-k] dp_{s+k},  dw[j] = sum_t dp_t x_{t-W+1+j},  dbias = sum dp.
// A thread walks over a run of tokens of V neighbouring channels with the W - 1 rows before
// the present one in registers: every row is read once per run, and those in front of it again.  A
// border between documents empties those registers, which is all that segments take.
#include "layer_device.h"
#include "layer_launch.h"

namespace layer {
namespace {

constexpr int kConvRun = 16;       // tokens a thread of the forward walks over
constexpr int kConvBwdRun = 128;   // and of the backward

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

template <typename TIn, int V, int W>
__global__ __launch_bounds__(256) void layer_conv_fwd_kernel(ConvParams p) {
    const int cols = p.D / V;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t run = id / cols;
    const int runs = (p.T + kConvRun - 1) / kConvRun;
    if (run >= static_cast<int64_t>(p.B) * runs) return;
    const int c = static_cast<int>(id % cols) * V;
    const int b = static_cast<int>(run / runs), t0 = static_cast<int>(run % runs) * kConvRun;
    const int len = conv_length(p, b), end = min(t0 + kConvRun, p.T);
    Taps<V, W> f;
    f.load(p, c);
    Vec<TIn, V> win[W];  // win[W - 1]: the present row
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (begins(p, b, t0 - (W - 1) + j))
#pragma unroll
            for (int i = 0; i < j; ++i) win[i] = Vec<TIn, V>{};
        win[j] = conv_row<TIn, V, W>(p, b, t0 - (W - 1) + j, c);
    }
    auto put_history = [&]() {  // the W - 1 rows before the present one
        if (!p.hist_out) return;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            put_vec<TIn, V>(p.hist_out, (static_cast<int64_t>(b) * (W - 1) + j) * p.D + c, win[j]);
    };
    if (len == 0 && t0 == 0) put_history();
    for (int t = t0; t < end; ++t) {
        float y[V] = {};
        if (t < len) {
            if (begins(p, b, t))
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j] = Vec<TIn, V>{};
            win[W - 1] = conv_row<TIn, V, W>(p, b, t, c);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float a = f.bias[e];
#pragma unroll
                for (int j = 0; j < W; ++j) a = fmaf(f.w[j][e], widen(win[j].e[e]), a);
                if (p.act) {
                    float s, r;
                    sigmoid2<true>(a, s, r);
                    a *= s;
                }
                y[e] = a;
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
            if (t == len - 1) put_history();
        }
        store_vec<V>(p.y, (static_cast<int64_t>(b) * p.T + t) * p.D + c, y, p.y_bf16);
    }
}

template <typename TIn, typename TDy, int V, int W>
__global__ __launch_bounds__(64) void layer_conv_bwd_kernel(ConvParams p) {
    const int c = (blockIdx.y * 64 + threadIdx.x) * V;
    if (c >= p.D) return;
    const int runs = (p.T + kConvBwdRun - 1) / kConvBwdRun;
    const int group = blockIdx.x;
    const int b = group / runs, t0 = group % runs * kConvBwdRun;
    const int len = conv_length(p, b), end = min(t0 + kConvBwdRun, p.T);
    Taps<V, W> f;
    f.load(p, c);
    float dw[W][V] = {}, db[V] = {};
    Vec<TIn, V> win[W];
    int age = W - 1;  // rows before the present one that belong to its document
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (begins(p, b, t0 - (W - 1) + j)) {
            age = 0;
#pragma unroll
            for (int i = 0; i < j; ++i) win[i] = Vec<TIn, V>{};
        } else {
            age = min(age + 1, W - 1);
        }
        win[j] = conv_row<TIn, V, W>(p, b, t0 - (W - 1) + j, c);
    }
    // gradients of the rows t - W + 1 .. t; a row is stored when the last token that reads it is done
    float acc[W][V] = {};
    auto store_row_of = [&](int t, const float (&g)[V]) {
        if (t >= t0) {
            if (t < end) store_vec<V>(p.dx, (static_cast<int64_t>(b) * p.T + t) * p.D + c, g, p.grad_bf16);
        } else if (t0 == 0 && p.dhist_in) {
            store_vec<V>(p.dhist_in, (static_cast<int64_t>(b) * (W - 1) + t + W - 1) * p.D + c, g, p.grad_bf16);
        }
    };
    // acc[j] belongs to row t - W + 1 + j of the present token t
    auto shift = [&](int t) {
        store_row_of(t - W + 1, acc[0]);
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[j][e] = j + 1 < W ? acc[j + 1][e] : 0.0f;
    };
    // behind the last token: the history's gradient reaches the last W - 1 rows of its document
    auto last = [&]() {
        if (!p.dhist_out) return;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (W - 2 - j > age) continue;
            const int64_t i = (static_cast<int64_t>(b) * (W - 1) + j) * p.D + c;
#pragma unroll
            for (int e = 0; e < V; ++e)
                acc[j][e] += p.grad_bf16 ? widen(static_cast<const uint16_t*>(p.dhist_out)[i + e])
                                         : static_cast<const float*>(p.dhist_out)[i + e];
        }
    };
    for (int t = t0; t < end + W - 1; ++t) {
        if (t == len) last();
        if (t < len) {
            if (begins(p, b, t)) {
                age = 0;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j] = Vec<TIn, V>{};
            } else {
                age = min(age + 1, W - 1);
            }
            win[W - 1] = conv_row<TIn, V, W>(p, b, t, c);
            const Vec<TDy, V> dy =
                load_vec<TDy, V>(static_cast<const TDy*>(p.dy), (static_cast<int64_t>(b) * p.T + t) * p.D + c);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float a = f.bias[e];
#pragma unroll
                for (int j = 0; j < W; ++j) a = fmaf(f.w[j][e], widen(win[j].e[e]), a);
                float d = widen(dy.e[e]);
                if (p.act) {
                    float s, r;
                    sigmoid2<true>(a, s, r);
                    d *= s * fmaf(a, r, 1.0f);
                }
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    acc[j][e] = W - 1 - j <= age ? fmaf(f.w[j][e], d, acc[j][e]) : acc[j][e];
                    if (t < end) dw[j][e] = fmaf(d, widen(win[j].e[e]), dw[j][e]);
                }
                if (t < end) db[e] += d;
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
        }
        shift(t);
    }
    if (!p.part) return;
    float* part = p.part + static_cast<int64_t>(group) * (W + 1) * p.D + c;
#pragma unroll
    for (int j = 0; j < W; ++j) store_vec<V>(part, static_cast<int64_t>(j) * p.D, dw[j], false);
    store_vec<V>(part, static_cast<int64_t>(W) * p.D, db, false);
}

// One token; hist_out may be hist_in (each channel is read, then written, by one thread).
template <typename TIn, int V, int W>
__global__ __launch_bounds__(64) void layer_conv_step_kernel(ConvParams p) {
    const int cols = p.D / V;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    if (id >= static_cast<int64_t>(p.B) * cols) return;
    const int b = static_cast<int>(id / cols), c = static_cast<int>(id % cols) * V;
    Vec<TIn, V> win[W];
#pragma unroll
    for (int j = 0; j < W; ++j) win[j] = conv_row<TIn, V, W>(p, b, j - (W - 1), c);
    Taps<V, W> f;
    f.load(p, c);
    float y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float a = f.bias[e];
#pragma unroll
        for (int j = 0; j < W; ++j) a = fmaf(f.w[j][e], widen(win[j].e[e]), a);
        if (p.act) {
            float s, r;
            sigmoid2<true>(a, s, r);
            a *= s;
        }
        y[e] = a;
    }
#pragma unroll
    for (int j = 1; j < W; ++j)
        put_vec<TIn, V>(p.hist_out, (static_cast<int64_t>(b) * (W - 1) + j - 1) * p.D + c, win[j]);
    store_vec<V>(p.y, static_cast<int64_t>(b) * p.D + c, y, p.y_bf16);
}

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

}  // namespace

int conv_groups(int B, int T) { return static_cast<int>(tiles_of(T, kConvBwdRun) * B); }

int launch_conv_fwd(const ConvParams& p, hipStream_t st) {
    with_types(p, [&](auto in, auto v) {
        with_taps(p.W, [&](auto w) {
            const int64_t n = tiles_of(p.T, kConvRun) * p.B * (p.D / v());
            hipLaunchKernelGGL((layer_conv_fwd_kernel<decltype(in), v(), w()>), dim3(tiles_of(n, 256)), dim3(256), 0, st,
                               p);
        });
    });
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

int launch_conv_bwd(const ConvParams& p, hipStream_t st) {
    const int groups = conv_groups(p.B, p.T);
    with_types(p, [&](auto in, auto v) {
        with_taps(p.W, [&](auto w) {
            const dim3 grid(groups, tiles_of(p.D / v(), 64));
            if (p.y_bf16)
                hipLaunchKernelGGL((layer_conv_bwd_kernel<decltype(in), uint16_t, v(), w()>), grid, dim3(64), 0, st, p);
            else
                hipLaunchKernelGGL((layer_conv_bwd_kernel<decltype(in), float, v(), w()>), grid, dim3(64), 0, st, p);
        });
    });
    if (p.part) launch_col_sums(ColSums{p.part, groups, p.W + 1, p.D, p.W, p.dw, p.dbias, nullptr}, st);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

int launch_conv_step(const ConvParams& p, hipStream_t st) {
    with_types(p, [&](auto in, auto v) {
        with_taps(p.W, [&](auto w) {
            const int64_t n = static_cast<int64_t>(p.B) * (p.D / v());
            hipLaunchKernelGGL((layer_conv_step_kernel<decltype(in), v(), w()>), dim3(tiles_of(n, 64)), dim3(64), 0, st,
                               p);
        });
    });
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace layer
