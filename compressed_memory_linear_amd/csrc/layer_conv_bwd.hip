// layer_conv_bwd.hip -- gradient of the short causal convolution (layer_conv.h).  The sum and its activation are
// taken again from x; nothing of the forward is kept.  The sums over tokens go to the workspace, one set to a run, and
// are added by a second kernel in a fixed order.
//
// B8 T4096 D2048 W4 bf16: 403 MB in 105 us, 3.8 TB/s, and 5 us for the second kernel (a token at a time: 235 in
// all); two to three waves to a vector unit (the next group's rows, the filters and their sums in registers) do not
// cover the loads.  fp32 604 MB in 182, 4.4 TB/s.  Runs of 64 tokens instead of 128 13 us slower, groups of 8 instead of 4
// 2 us.  The runs are that long whatever the size, so that a small call takes what one wave's run does: B1 T4096 D2048
// bf16 (256 waves) 57 us of 50 MB, B1 T2048 56; and rows of few channels leave lanes idle (B64 T4096 D64 86 us of 101 MB).
#include "layer_conv.h"

namespace layer {
namespace {

// A run of tokens of V channels to a thread, in groups whose rows are asked for a group ahead.
template <typename TIn, typename TDy, int V, int W>
__global__ __launch_bounds__(64) void layer_conv_bwd_kernel(ConvParams p) {
    constexpr int N = kConvGroup;
    const int l = threadIdx.x, col = blockIdx.y * 64 + l;
    const bool in = col * V < p.D;  // (past the row's end a lane takes part in the ballots alone)
    const int c = in ? col * V : 0;
    const int runs = (p.T + kConvBwdRun - 1) / kConvBwdRun;
    const int group = blockIdx.x;
    const int b = group / runs, t0 = group % runs * kConvBwdRun;
    const int len = conv_length(p, b), end = min(t0 + kConvBwdRun, p.T);
    const int64_t first = static_cast<int64_t>(b) * p.T;
    const TIn* x = static_cast<const TIn*>(p.x) + first * p.x_row + c;
    const TDy* dyp = static_cast<const TDy*>(p.dy) + first * p.D + c;
    struct Group {
        Vec<TIn, V> x[N];
        Vec<TDy, V> dy[N];
        bool cut;  // whether token l of the group begins a document
    } next;
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t at = min(t + i, p.T - 1);  // a row that is not there is read from one that is
            next.x[i] = load_vec<TIn, V>(x, at * p.x_row);
            next.dy[i] = load_vec<TDy, V>(dyp, at * p.D);
        }
        next.cut = l < N && t + l < len && begins(p, b, t + l);
    };
    fetch(t0);
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
        if (!in) return;
        if (t >= t0) {
            if (t < end) store_vec<V>(p.dx, (first + t) * p.D + c, g, p.grad_bf16);
        } else if (t0 == 0 && p.dhist_in) {
            store_vec<V>(p.dhist_in, (static_cast<int64_t>(b) * (W - 1) + t + W - 1) * p.D + c, g, p.grad_bf16);
        }
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
    for (int g0 = t0; g0 < end + W - 1; g0 += N) {
        const Group now = next;
        const uint64_t cuts = __ballot(now.cut);
        if (g0 + N < end + W - 1) fetch(g0 + N);
        // a group of tokens of this run alone, of one document back to their first taps
        const bool plain = g0 >= t0 + W - 1 && g0 + N <= min(end, len) && !cuts && age >= W - 1;
        with_flag(!plain, [&](auto partly) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int t = g0 + i;
                if (partly() && t == len) last();
                if (!partly() || t < len) {
                    if (partly()) {
                        if (cuts >> i & 1) {
                            age = 0;
#pragma unroll
                            for (int j = 0; j < W - 1; ++j) win[j] = Vec<TIn, V>{};
                        } else {
                            age = min(age + 1, W - 1);
                        }
                    }
                    win[W - 1] = now.x[i];
                    float a[V], d[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        a[e] = f.bias[e];
                        d[e] = widen(now.dy[i].e[e]);
#pragma unroll
                        for (int j = 0; j < W; ++j) a[e] = fmaf(f.w[j][e], widen(win[j].e[e]), a[e]);
                    }
                    if (p.act) {
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            float s, r;
                            sigmoid2<kAccurate<TIn>>(a[e], s, r);
                            d[e] *= s * fmaf(a[e], r, 1.0f);
                        }
                    }
                    const bool mine = !partly() || t < end;  // (the tokens behind the run are the next one's)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            if (!partly() || W - 1 - j <= age) acc[j][e] = fmaf(f.w[j][e], d[e], acc[j][e]);
                            if (mine) dw[j][e] = fmaf(d[e], widen(win[j].e[e]), dw[j][e]);
                        }
                        if (mine) db[e] += d[e];
                    }
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
                }
                if (!partly()) {
                    if (in) store_vec<V>(p.dx, (first + t - W + 1) * p.D + c, acc[0], p.grad_bf16);
                } else if (t < end + W - 1) {
                    store_row_of(t - W + 1, acc[0]);
                }
#pragma unroll
                for (int j = 0; j < W; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[j][e] = j + 1 < W ? acc[j + 1][e] : 0.0f;
            }
        });
    }
    if (!p.part || !in) return;
    float* part = p.part + static_cast<int64_t>(group) * (W + 1) * p.D + c;
#pragma unroll
    for (int j = 0; j < W; ++j) store_vec<V>(part, static_cast<int64_t>(j) * p.D, dw[j], false);
    store_vec<V>(part, static_cast<int64_t>(W) * p.D, db, false);
}

}  // namespace

int conv_groups(int B, int T) { return static_cast<int>(tiles_of(T, kConvBwdRun) * B); }

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

}  // namespace layer
