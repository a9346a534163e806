// layer_conv.hip -- the short causal convolution in front of a recurrence: forward and single step (layer_conv.h).
//
// Bound by HBM: B8 T4096 D2048 W4 bf16 moves 268 MB in 48 to 61 us, 4.4 to 5.6 TB/s, fp32 twice that in 107, 5.0 TB/s
// (bf16 a token at a time, its row asked for when it is needed, 68).  One token of one sequence: 3 us, and 9 for the host's call.
#include "layer_conv.h"

namespace layer {
namespace {

// One run of tokens of V channels to a thread: its rows are asked for together, without a branch, and lie in
// registers.  A wave's lanes are neighbouring channels of one run (ALONE), or of several where a row is short.
template <typename TIn, int V, int W, bool ALONE>
__global__ __launch_bounds__(256) void layer_conv_fwd_kernel(ConvParams p, int lanes) {
    constexpr int R = kConvRun;
    const int cols = p.D / V, runs = (p.T + R - 1) / R;
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int l = threadIdx.x & 63;
    int64_t run;
    int col;
    if (ALONE) {
        const int across = (cols + 63) / 64;
        run = wave / across;
        col = static_cast<int>(wave % across) * 64 + l;
    } else {
        run = wave * (64 / lanes) + l / lanes;
        col = l % lanes;
    }
    if (ALONE ? run >= static_cast<int64_t>(p.B) * runs : run >= static_cast<int64_t>(p.B) * runs || col >= cols) return;
    const bool in = col < cols;  // (past the row's end a lane takes part in the ballot alone)
    const int c = in ? col * V : 0;
    const int b = static_cast<int>(run / runs), t0 = static_cast<int>(run % runs) * R;
    const int len = conv_length(p, b);
    Vec<TIn, V> row[R + W - 1];  // of tokens t0 - W + 1 on
    const TIn* x = static_cast<const TIn*>(p.x) + static_cast<int64_t>(b) * p.T * p.x_row + c;
    const TIn* hist = p.hist_in ? static_cast<const TIn*>(p.hist_in) + static_cast<int64_t>(b) * (W - 1) * p.D + c : x;
#pragma unroll
    for (int j = 0; j < R + W - 1; ++j) {
        const int t = t0 - (W - 1) + j;
        // a row that is not there is read from one that is
        const TIn* from = t >= 0 ? x + static_cast<int64_t>(min(t, p.T - 1)) * p.x_row
                                 : hist + (p.hist_in ? static_cast<int64_t>(t + W - 1) * p.D : 0);
        row[j] = load_vec<TIn, V>(from, 0);
    }
    Taps<V, W> f;
    f.load(p, c);
    if (!p.hist_in && t0 < W - 1) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            if (t0 - (W - 1) + j < 0) row[j] = Vec<TIn, V>{};
    }
    // borders among the rows, bit j for row j
    uint32_t cuts = 0;
    if (p.segments) {
        if (ALONE) {
            const int t = t0 - (W - 1) + l;
            cuts = static_cast<uint32_t>(__ballot(l < R + W - 1 && t < len && begins(p, b, t)));
        } else {
            for (int j = 0; j < R + W - 1; ++j)
                if (t0 - (W - 1) + j < len && begins(p, b, t0 - (W - 1) + j)) cuts |= 1u << j;
        }
    }
    if (!in) return;
    const int64_t out = (static_cast<int64_t>(b) * p.T + t0) * p.D + c;
    auto put_history = [&](auto first) {
        if (!p.hist_out) return;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            put_vec<TIn, V>(p.hist_out, (static_cast<int64_t>(b) * (W - 1) + j) * p.D + c, row[first() + j]);
    };
    if (len == 0 && t0 == 0) put_history(std::integral_constant<int, 0>());
    const bool partly = cuts || t0 + R >= len;
    with_flag(partly, [&](auto part) {
        if (part()) {  // what a border in front of the run leaves of the rows there
            each<W - 1>([&](auto jc) {
                constexpr int j = jc();
                if (cuts >> j & 1) {
#pragma unroll
                    for (int i = 0; i < j; ++i) row[i] = Vec<TIn, V>{};
                }
            });
        }
        each<R>([&](auto ic) {
            constexpr int i = ic();
            const int t = t0 + i;
            float y[V] = {};
            if (!part() || t < len) {
                if (part() && (cuts >> (i + W - 1) & 1)) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) row[i + j] = Vec<TIn, V>{};
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float a = f.bias[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) a = fmaf(f.w[j][e], widen(row[i + j].e[e]), a);
                    y[e] = a;
                }
                if (p.act) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float s, r;
                        sigmoid2<kAccurate<TIn>>(y[e], s, r);
                        y[e] *= s;
                    }
                }
                if (part() && t == len - 1) put_history(std::integral_constant<int, i + 1>());
            }
            if (!part() || t < p.T) store_vec<V>(p.y, out + static_cast<int64_t>(i) * p.D, y, p.y_bf16);
        });
    });
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
            sigmoid2<kAccurate<TIn>>(a, s, r);
            a *= s;
        }
        y[e] = a;
    }
#pragma unroll
    for (int j = 1; j < W; ++j)
        put_vec<TIn, V>(p.hist_out, (static_cast<int64_t>(b) * (W - 1) + j - 1) * p.D + c, win[j]);
    store_vec<V>(p.y, static_cast<int64_t>(b) * p.D + c, y, p.y_bf16);
}

}  // namespace

int launch_conv_fwd(const ConvParams& p, hipStream_t st) {
    with_types(p, [&](auto in, auto v) {
        with_taps(p.W, [&](auto w) {
            const int cols = p.D / v();
            const int64_t runs = tiles_of(p.T, kConvRun) * p.B;
            int lanes = 1;
            while (lanes < cols && lanes < 64) lanes *= 2;
            if (cols >= 48) {
                const int64_t waves = runs * tiles_of(cols, 64);
                hipLaunchKernelGGL((layer_conv_fwd_kernel<decltype(in), v(), w(), true>), dim3(tiles_of(waves, 4)),
                                   dim3(256), 0, st, p, 64);
            } else {
                const int64_t waves = tiles_of(runs, 64 / lanes);
                hipLaunchKernelGGL((layer_conv_fwd_kernel<decltype(in), v(), w(), false>), dim3(tiles_of(waves, 4)),
                                   dim3(256), 0, st, p, lanes);
            }
        });
    });
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
