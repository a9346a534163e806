// layer_ln.hip -- the layer norm with the residual in front of it, forward and
// backward, in one pass over the rows:
//     x' = x + y,  m = mean(x'),  c = x' - m,  r = 1 / sqrt(mean(c^2) + eps),  n = c r,  z = n w + b;
//     t = dz w,  dx' = dx_out + r (t - mean(t) - n mean(t n)),  dw = sum dz n,  db = sum dz.
// Rows lie in registers as for the other norms (layer_norm.h): read once, the variance taken from
// the differences.  The backward takes the forward again from x and y, so that nothing of it is kept; its sums
// over rows stay with each thread's columns, go to the workspace and are added in a fixed order.
//
// Bound by HBM: R32768 D2048 bf16 with the residual, forward 537 MB in 86 us, 6.2 TB/s (part of it from the 256 MB cache),
// backward 671 MB in 119 us, 5.6 TB/s, and 5 us for the sums.  R2331 D1001 (odd rows, element by element, residual
// in fp32): 11 us for 29 MB, one to two rows to a workgroup and two sums over their waves; the sums 4 us.  Up to 8192 values
// as at 2048 (R8192 D8192: forward 6.0 TB/s in bf16 and 5.4 in fp32, backward 5.7 and 5.7).  Past those the backward
// with two pieces a thread and the next row in flight spills 97 to 211 of its 128 registers' values: R4096 D16384 366 us in
// bf16, 1.8 TB/s, and 810 in fp32, 1.7 (forward 6.2 and 5.7 TB/s); element by element 25 to 30 from 4097 on, R8192 D8191 308
// us in bf16, 2.2 TB/s, and 334 in fp32, 4.0.
#include "layer_norm.h"

namespace layer {
namespace {

template <typename S, bool VEC, typename TIn, typename TRes>
__global__ __launch_bounds__(S::NT) void layer_ln_fwd_kernel(LayerNormParams p) {
    __shared__ float red[2][S::NT / 64][2];
    RowSum<S> sum{red};
    const int lane = threadIdx.x % S::TPR, sub = threadIdx.x / S::TPR;
    const float inv = 1.0f / static_cast<float>(p.D);
    struct Raw {
        Piece<TIn> y;
        Piece<TRes> x;
    };
    auto fetch = [&](uint32_t it, Raw (&o)[S::K]) {
        const Rows rows = rows_of<S>(it, p.R, p.D);
        const auto yr = norm_rsrc(p.y, sizeof(TIn) == 2, rows), xr = norm_rsrc(p.x, sizeof(TRes) == 2, rows);
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            load_piece<S, VEC>(yr, lane, sub, k, p.D, o[k].y);
            load_piece<S, VEC>(xr, lane, sub, k, p.D, o[k].x);
        }
    };
    const uint32_t steps = (static_cast<uint32_t>(p.R) + S::ROWS - 1) / S::ROWS;
    Raw next[S::K];
    fetch(blockIdx.x, next);
    float w[S::K][kE], b[S::K][kE];
#pragma unroll
    for (int k = 0; k < S::K; ++k) {
        load_weights<S, VEC>(p.w, lane, k, p.D, w[k]);
        load_weights<S, VEC>(p.b, lane, k, p.D, b[k]);
#pragma unroll
        for (int e = 0; e < kE; ++e) b[k][e] = p.b ? b[k][e] : 0.0f;
    }
    for (uint32_t it = blockIdx.x; it < steps; it += gridDim.x) {
        // rows past the last are rows of zeros, in step with the barriers
        const Rows rows = rows_of<S>(it, p.R, p.D);
        float x[S::K][kE];
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                x[k][e] = widen(next[k].x.e[e]) + widen(next[k].y.e[e]);
                s[0] += x[k][e];
            }
        fetch(it + gridDim.x, next);  // in flight while this row is worked on
        const auto xr = norm_rsrc(p.x_out, p.res_bf16, rows);
#pragma unroll
        for (int k = 0; k < S::K; ++k) store_piece<S, VEC, true>(xr, p.res_bf16, lane, sub, k, p.D, x[k]);
        sum(s);
        const float m = s[0] * inv;
        s[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                x[k][e] = col_of<S, VEC>(lane, k, e) < p.D ? x[k][e] - m : 0.0f;
                s[0] = fmaf(x[k][e], x[k][e], s[0]);
            }
        sum(s);
        const float r = rsqrt_acc(fmaf(s[0], inv, p.eps));
        const auto zr = norm_rsrc(p.z, p.in_bf16, rows);
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
#pragma unroll
            for (int e = 0; e < kE; ++e) x[k][e] = fmaf(x[k][e] * r, w[k][e], b[k][e]);
            store_piece<S, VEC, false>(zr, p.in_bf16, lane, sub, k, p.D, x[k]);
        }
    }
}

template <typename S, bool VEC, typename TIn, typename TRes>
__global__ __launch_bounds__(S::NT) void layer_ln_bwd_kernel(LayerNormParams p) {
    __shared__ float red[2][S::NT / 64][2];
    __shared__ float cols[S::ROWS > 1 ? S::ROWS : 1][S::ROWS > 1 ? S::TPR * kE : 1];
    RowSum<S> sum{red};
    const int lane = threadIdx.x % S::TPR, sub = threadIdx.x / S::TPR;
    const float inv = 1.0f / static_cast<float>(p.D);
    struct Raw {
        Piece<TIn> y, z;
        Piece<TRes> x, d;
    };
    auto fetch = [&](uint32_t it, Raw (&o)[S::K]) {
        const Rows rows = rows_of<S>(it, p.R, p.D);
        const auto yr = norm_rsrc(p.y, sizeof(TIn) == 2, rows), zr = norm_rsrc(p.dz, sizeof(TIn) == 2, rows);
        const auto xr = norm_rsrc(p.x, sizeof(TRes) == 2, rows), dr = norm_rsrc(p.dx_out, sizeof(TRes) == 2, rows);
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            load_piece<S, VEC>(yr, lane, sub, k, p.D, o[k].y);
            load_piece<S, VEC>(xr, lane, sub, k, p.D, o[k].x);
            load_piece<S, VEC>(zr, lane, sub, k, p.D, o[k].z);
            load_piece<S, VEC>(dr, lane, sub, k, p.D, o[k].d);
        }
    };
    const uint32_t steps = (static_cast<uint32_t>(p.R) + S::ROWS - 1) / S::ROWS;
    Raw next[S::K];
    fetch(blockIdx.x, next);
    float w[S::K][kE], gw[S::K][kE] = {}, gb[S::K][kE] = {};
#pragma unroll
    for (int k = 0; k < S::K; ++k) load_weights<S, VEC>(p.w, lane, k, p.D, w[k]);
    for (uint32_t it = blockIdx.x; it < steps; it += gridDim.x) {
        const Rows rows = rows_of<S>(it, p.R, p.D);
        float x[S::K][kE], g[S::K][kE], d[S::K][kE];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                x[k][e] = widen(next[k].x.e[e]) + widen(next[k].y.e[e]);
                g[k][e] = widen(next[k].z.e[e]);
                d[k][e] = widen(next[k].d.e[e]);
                s[0] += x[k][e];
                s[1] = fmaf(g[k][e], w[k][e], s[1]);
            }
        // the next row, in flight while this one is worked on; kept in this place
        __builtin_amdgcn_sched_barrier(0);
        fetch(it + gridDim.x, next);
        __builtin_amdgcn_sched_barrier(0);
        sum(s);
        const float m = s[0] * inv, mt = s[1] * inv;
        s[0] = s[1] = 0.0f;
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                x[k][e] = col_of<S, VEC>(lane, k, e) < p.D ? x[k][e] - m : 0.0f;
                s[0] = fmaf(x[k][e], x[k][e], s[0]);
                s[1] = fmaf(g[k][e] * w[k][e], x[k][e], s[1]);
            }
        sum(s);
        const float r = rsqrt_acc(fmaf(s[0], inv, p.eps));
        const float mn = s[1] * inv * r;  // mean(t n)
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const float n = x[k][e] * r;
                gw[k][e] = fmaf(g[k][e], n, gw[k][e]);
                gb[k][e] += g[k][e];
                d[k][e] = fmaf(r, fmaf(-n, mn, fmaf(g[k][e], w[k][e], -mt)), d[k][e]);
            }
        const auto xr = norm_rsrc(p.dx, p.res_bf16, rows), yr = norm_rsrc(p.dy, p.grad_bf16, rows);
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            store_piece<S, VEC, true>(xr, p.res_bf16, lane, sub, k, p.D, d[k]);
            if (p.dy) store_piece<S, VEC, true>(yr, p.grad_bf16, lane, sub, k, p.D, d[k]);
        }
    }
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
    if (p.dw) put_columns<S, VEC>(part, &cols[0][0], lane, sub, p.D, gw);
    if (p.db) put_columns<S, VEC>(part + p.D, &cols[0][0], lane, sub, p.D, gb);
}

template <typename F>
void with_kernel(const LayerNormParams& p, F&& f) {
    with_shape(p.D, [&](auto s) {
        auto types = [&](auto vec) {
            if (p.in_bf16)
                p.res_bf16 ? f(s, vec, uint16_t(), uint16_t()) : f(s, vec, uint16_t(), float());
            else
                p.res_bf16 ? f(s, vec, float(), uint16_t()) : f(s, vec, float(), float());
        };
        p.vec ? types(std::true_type()) : types(std::false_type());
    });
}

}  // namespace

int launch_layernorm_fwd(const LayerNormParams& p, hipStream_t st) {
    with_kernel(p, [&](auto s, auto vec, auto in, auto res) {
        using S = decltype(s);
        hipLaunchKernelGGL((layer_ln_fwd_kernel<S, vec(), decltype(in), decltype(res)>), dim3(p.groups), dim3(S::NT),
                           0, st, p);
    });
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

int launch_layernorm_bwd(const LayerNormParams& p, hipStream_t st) {
    with_kernel(p, [&](auto s, auto vec, auto in, auto res) {
        using S = decltype(s);
        hipLaunchKernelGGL((layer_ln_bwd_kernel<S, vec(), decltype(in), decltype(res)>), dim3(p.groups), dim3(S::NT),
                           0, st, p);
    });
    if (p.dw || p.db) launch_col_sums(ColSums{p.part, p.groups, 2, p.D, 0, nullptr, p.dw, p.db}, st);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace layer
