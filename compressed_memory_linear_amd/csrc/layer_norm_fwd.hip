// layer_norm_fwd.hip -- the norm after a block, its gate, the residual and the
// norm before the next block, in one pass over the rows:
//     u = y phi(gate),  n = u / rms(u) w_post,  x' = x + scale n,
//     z = x' / rms(x') w_pre,   rms(a) = sqrt(mean(a^2) + eps).
// x' leaves rounded to its own type; z is taken from x' before that rounding.
//
// Bound by HBM: R32768 D2048 bf16 with every operand moves 671 MB in 114 us, 5.9 TB/s; R8192 D8192 128 us, 5.3;
// R4096 D16384 124 us, 5.4.  Past 8192 values all but bf16 throughout spill 4 to 19 registers (fp32 R2048 D16384
// 173 us, 3.9 TB/s), and single elements 49 or 50.  A decoding step's R256 D4096 (7 us for 13 MB) is one row per
// workgroup: the latency of its loads and of two sums over eight waves, one after the other.
#include "layer_norm.h"

namespace layer {
namespace {

template <typename S, bool VEC, typename TIn, typename TRes>
__global__ __launch_bounds__(S::NT) void layer_norm_fwd_kernel(NormParams p) {
    __shared__ float red[2][S::NT / 64][2];
    RowSum<S> sum{red};
    const int lane = threadIdx.x % S::TPR;
    const int sub = threadIdx.x / S::TPR;
    const float inv = 1.0f / static_cast<float>(p.D);

    struct Raw {
        Piece<TIn> y, g;
        Piece<TRes> x;
    };
    auto fetch = [&](uint32_t it, Raw (&o)[S::K]) {
        const Rows rows = rows_of<S>(it, p.R, p.D);
        const auto yr = norm_rsrc(p.y, sizeof(TIn) == 2, rows), gr = norm_rsrc(p.gate, sizeof(TIn) == 2, rows);
        const auto xr = norm_rsrc(p.x, sizeof(TRes) == 2, rows);
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            load_piece<S, VEC>(yr, lane, sub, k, p.D, o[k].y);
            load_piece<S, VEC>(gr, lane, sub, k, p.D, o[k].g);
            load_piece<S, VEC>(xr, lane, sub, k, p.D, o[k].x);
        }
    };
    const uint32_t steps = (static_cast<uint32_t>(p.R) + S::ROWS - 1) / S::ROWS;
    Raw next[S::K];
    fetch(blockIdx.x, next);
    float wpost[S::K][kE], sc[S::K][kE], wpre[S::K][kE];
#pragma unroll
    for (int k = 0; k < S::K; ++k) {
        load_weights<S, VEC>(p.w_post, lane, k, p.D, wpost[k]);
        load_weights<S, VEC>(p.scale, lane, k, p.D, sc[k]);
        load_weights<S, VEC>(p.w_pre, lane, k, p.D, wpre[k]);
    }
    for (uint32_t it = blockIdx.x; it < steps; it += gridDim.x) {
        // rows past the last are rows of zeros, in step with the barriers
        const Rows rows = rows_of<S>(it, p.R, p.D);
        float u[S::K][kE], xo[S::K][kE];
        float ss[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            const Raw raw = next[k];
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                u[k][e] = widen(raw.y.e[e]);
                xo[k][e] = widen(raw.x.e[e]);
            }
            if (p.gate_kind == 1) {
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    const float g = widen(raw.g.e[e]);
                    float cdf, ex;
                    gelu_parts(g, cdf, ex);
                    u[k][e] *= g * cdf;
                }
            } else if (p.gate_kind == 2) {
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    const float g = widen(raw.g.e[e]);
                    float s, r;
                    sigmoid2<kAccurate<TIn>>(g, s, r);
                    u[k][e] *= g * s;
                }
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) ss[0] = fmaf(u[k][e], u[k][e], ss[0]);
        }
        fetch(it + gridDim.x, next);  // in flight while this row is worked on
        if (p.y) {
            float r1 = 1.0f;
            if (p.post) {
                sum(ss);
                r1 = rsqrt_acc(fmaf(ss[0], inv, p.eps));
            }
#pragma unroll
            for (int k = 0; k < S::K; ++k)
#pragma unroll
                for (int e = 0; e < kE; ++e) xo[k][e] = fmaf(u[k][e] * r1 * wpost[k][e], sc[k][e], xo[k][e]);
        }
        const auto out = norm_rsrc(p.x_out, p.res_bf16, rows);
#pragma unroll
        for (int k = 0; k < S::K; ++k) store_piece<S, VEC, true>(out, p.res_bf16, lane, sub, k, p.D, xo[k]);
        if (p.pre) {
            ss[0] = 0.0f;
#pragma unroll
            for (int k = 0; k < S::K; ++k)
#pragma unroll
                for (int e = 0; e < kE; ++e) ss[0] = fmaf(xo[k][e], xo[k][e], ss[0]);
            sum(ss);
            const float r2 = rsqrt_acc(fmaf(ss[0], inv, p.eps));
            const auto zr = norm_rsrc(p.z, p.in_bf16, rows);
#pragma unroll
            for (int k = 0; k < S::K; ++k) {
#pragma unroll
                for (int e = 0; e < kE; ++e) xo[k][e] *= r2 * wpre[k][e];
                store_piece<S, VEC, false>(zr, p.in_bf16, lane, sub, k, p.D, xo[k]);
            }
        }
    }
}

template <typename TIn, typename TRes>
void launch(const NormParams& p, hipStream_t st) {
    with_shape(p.D, [&](auto s) {
        using S = decltype(s);
        if (p.vec)
            hipLaunchKernelGGL((layer_norm_fwd_kernel<S, true, TIn, TRes>), dim3(p.groups), dim3(S::NT), 0, st, p);
        else
            hipLaunchKernelGGL((layer_norm_fwd_kernel<S, false, TIn, TRes>), dim3(p.groups), dim3(S::NT), 0, st, p);
    });
}

}  // namespace

int norm_groups(int R, int D, bool backward) {
    int rows = 1, nt = 256;
    auto take = [&](auto s) { rows = decltype(s)::ROWS, nt = decltype(s)::NT; };
    with_shape(D, take);
    const int steps = static_cast<int>((static_cast<int64_t>(R) + rows - 1) / rows);
    // workgroups per compute unit (256): see NormShape
    const int most = 256 * (nt == 256 ? (backward ? 2 : 3) : nt == 512 && !backward ? 2 : 1);
    return steps < most ? steps : most;
}

int launch_norm_fwd(const NormParams& p, hipStream_t st) {
    if (p.in_bf16)
        p.res_bf16 ? launch<uint16_t, uint16_t>(p, st) : launch<uint16_t, float>(p, st);
    else
        p.res_bf16 ? launch<float, uint16_t>(p, st) : launch<float, float>(p, st);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace layer
