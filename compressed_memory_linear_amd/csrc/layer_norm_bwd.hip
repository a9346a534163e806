// layer_norm_bwd.hip -- gradient of the norms around a block (layer_norm_fwd.hip).
//
// With n1 = u / rms(u), n = n1 w_post, xh = x' / rms(x') and the means over a row,
//     dx' = dx_out + (t - xh mean(t xh)) / rms(x'),  t = dz w_pre,   dw_pre = sum dz xh,
//     dx = dx',  dscale = sum dx' n,  dn = scale dx',                dw_post = sum dn n1,
//     du = (s - n1 mean(s n1)) / rms(u),  s = dn w_post,
//     dy = du phi(gate),  dgate = du y phi'(gate).
// The forward is taken again from y, gate and x, which have to be read anyway,
// so that nothing of it is kept and x' is not read back rounded.  The sums over
// rows are held by each thread for its columns while its workgroup walks over
// its rows; the workgroups' sums go to the workspace and are added in a fixed
// order by a second kernel (no atomics: reruns agree bit for bit).
//
// Bound by HBM: R32768 D2048 bf16 with every operand moves 1.07 GB in 204 us, 5.3 TB/s (the
// device's own copy of 1 GiB: 5.4); 75 vector operations per value keep the vector units 65 %
// busy.  Rows of 64 values (R65536, SiLU, post-norm alone: 15 us for 34 MB) are bound by latency: 49 operations
// per value are 5.4 us and the bytes 6.3, but a workgroup's rows are four steps of load, sums and store.
#include "layer_norm.h"

namespace layer {
namespace {

// A row's five inputs, as stored.
template <typename TIn, typename TRes>
struct Raw {
    Piece<TIn> y, g, z;
    Piece<TRes> x, d;
};
template <typename S, bool VEC, typename TIn, typename TRes>
__device__ __forceinline__ void fetch(const NormParams& p, uint32_t it, int lane, int sub, Raw<TIn, TRes> (&o)[S::K]) {
    const Rows rows = rows_of<S>(it, p.R, p.D);
    const auto yr = norm_rsrc(p.y, sizeof(TIn) == 2, rows), gr = norm_rsrc(p.gate, sizeof(TIn) == 2, rows);
    const auto zr = norm_rsrc(p.dz, sizeof(TIn) == 2, rows), xr = norm_rsrc(p.x, sizeof(TRes) == 2, rows);
    const auto dr = norm_rsrc(p.dx_out, sizeof(TRes) == 2, rows);
#pragma unroll
    for (int k = 0; k < S::K; ++k) {
        load_piece<S, VEC>(yr, lane, sub, k, p.D, o[k].y);
        load_piece<S, VEC>(gr, lane, sub, k, p.D, o[k].g);
        load_piece<S, VEC>(xr, lane, sub, k, p.D, o[k].x);
        load_piece<S, VEC>(zr, lane, sub, k, p.D, o[k].z);
        load_piece<S, VEC>(dr, lane, sub, k, p.D, o[k].d);
    }
}
// phi and phi' of a piece's gates.
template <typename TIn>
__device__ __forceinline__ void gates(int kind, const Piece<TIn>& raw, float (&phi)[kE], float (&dphi)[kE]) {
    if (kind == 1) {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const float g = widen(raw.e[e]);
            float cdf, ex;
            gelu_parts(g, cdf, ex);
            phi[e] = g * cdf;
            dphi[e] = fmaf(g * 0.39894228040143268f, ex, cdf);
        }
    } else if (kind == 2) {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const float g = widen(raw.e[e]);
            float s, r;
            sigmoid2<kAccurate<TIn>>(g, s, r);
            phi[e] = g * s;
            dphi[e] = s * fmaf(g, r, 1.0f);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) phi[e] = 1.0f, dphi[e] = 0.0f;
    }
}
// This workgroup's column sums g, into its row of the workspace.
template <typename S, bool VEC>
__device__ __forceinline__ void put_columns(float* to, float* cols, int lane, int sub, int D, const float (&g)[S::K][kE]) {
    if constexpr (S::ROWS == 1) {
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const int c = col_of<S, VEC>(lane, k, e);
                if (c < D) to[c] = g[k][e];
            }
    } else {
        constexpr int kCols = S::TPR * kE;  // the row slots' sums meet in LDS
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kE; ++e) cols[sub * kCols + col_of<S, VEC>(lane, 0, e)] = g[0][e];
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += S::NT) {
            float s = 0.0f;
            for (int i = 0; i < S::ROWS; ++i) s += cols[i * kCols + c];
            to[c] = s;
        }
    }
}

template <typename S, bool VEC, typename TIn, typename TRes>
__global__ __launch_bounds__(S::NT) void layer_norm_bwd_kernel(NormParams p) {
    __shared__ float red[2][S::NT / 64][2];
    // column sums of the workgroup's row slots (where it has several)
    __shared__ float cols[S::ROWS > 1 ? S::ROWS : 1][S::ROWS > 1 ? S::TPR * kE : 1];
    RowSum<S> sum{red};
    const int lane = threadIdx.x % S::TPR;
    const int sub = threadIdx.x / S::TPR;
    const float inv = 1.0f / static_cast<float>(p.D);

    const uint32_t steps = (static_cast<uint32_t>(p.R) + S::ROWS - 1) / S::ROWS;
    Raw<TIn, TRes> next[S::K];
    fetch<S, VEC>(p, blockIdx.x, lane, sub, next);
    float wpost[S::K][kE], sc[S::K][kE], wpre[S::K][kE];
    float gpost[S::K][kE], gsc[S::K][kE], gpre[S::K][kE];
#pragma unroll
    for (int k = 0; k < S::K; ++k) {
        load_weights<S, VEC>(p.w_post, lane, k, p.D, wpost[k]);
        load_weights<S, VEC>(p.scale, lane, k, p.D, sc[k]);
        load_weights<S, VEC>(p.w_pre, lane, k, p.D, wpre[k]);
#pragma unroll
        for (int e = 0; e < kE; ++e) gpost[k][e] = gsc[k][e] = gpre[k][e] = 0.0f;
    }
    for (uint32_t it = blockIdx.x; it < steps; it += gridDim.x) {
        // rows past the last are rows of zeros, in step with the barriers
        const Rows rows = rows_of<S>(it, p.R, p.D);
        float yv[S::K][kE], phi[S::K][kE], dphi[S::K][kE], xo[S::K][kE], d[S::K][kE], t[S::K][kE];
        float ss[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            const Raw<TIn, TRes> raw = next[k];
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                yv[k][e] = widen(raw.y.e[e]);
                xo[k][e] = widen(raw.x.e[e]);
                d[k][e] = widen(raw.d.e[e]);
                t[k][e] = widen(raw.z.e[e]);
            }
            gates(p.gate_kind, raw.g, phi[k], dphi[k]);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const float u = yv[k][e] * phi[k][e];
                ss[0] = fmaf(u, u, ss[0]);
            }
        }
        // the next row, in flight while this one is worked on; kept in this place (the compiler moves it behind
        // part of what follows, which costs 10 of 205 us)
        __builtin_amdgcn_sched_barrier(0);
        fetch<S, VEC>(p, it + gridDim.x, lane, sub, next);
        __builtin_amdgcn_sched_barrier(0);
        float r1 = 1.0f;
        if (p.y) {
            if (p.post) {
                sum(ss);
                r1 = rsqrt_acc(fmaf(ss[0], inv, p.eps));
            }
#pragma unroll
            for (int k = 0; k < S::K; ++k)
#pragma unroll
                for (int e = 0; e < kE; ++e)
                    xo[k][e] = fmaf(yv[k][e] * phi[k][e] * r1 * wpost[k][e], sc[k][e], xo[k][e]);
        }
        if (p.pre) {
            ss[0] = ss[1] = 0.0f;
#pragma unroll
            for (int k = 0; k < S::K; ++k)
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    ss[0] = fmaf(xo[k][e], xo[k][e], ss[0]);
                    ss[1] = fmaf(t[k][e] * wpre[k][e], xo[k][e], ss[1]);
                }
            sum(ss);
            const float r2 = rsqrt_acc(fmaf(ss[0], inv, p.eps));
            const float m = ss[1] * inv * r2;  // mean(t xh)
#pragma unroll
            for (int k = 0; k < S::K; ++k)
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    const float xh = xo[k][e] * r2;
                    gpre[k][e] = fmaf(t[k][e], xh, gpre[k][e]);
                    d[k][e] = fmaf(r2, fmaf(-xh, m, t[k][e] * wpre[k][e]), d[k][e]);
                }
        }
        const auto dxr = norm_rsrc(p.dx, p.res_bf16, rows);
#pragma unroll
        for (int k = 0; k < S::K; ++k) store_piece<S, VEC, true>(dxr, p.res_bf16, lane, sub, k, p.D, d[k]);
        if (!p.y) continue;
        ss[0] = ss[1] = 0.0f;
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const float n1 = yv[k][e] * phi[k][e] * r1;
                gsc[k][e] = fmaf(d[k][e], n1 * wpost[k][e], gsc[k][e]);
                d[k][e] *= sc[k][e];
                gpost[k][e] = fmaf(d[k][e], n1, gpost[k][e]);
                d[k][e] *= wpost[k][e];
                ss[0] = fmaf(d[k][e], n1, ss[0]);
            }
        if (p.post) {
            sum(ss);
            const float m = ss[0] * inv;  // mean(s n1)
#pragma unroll
            for (int k = 0; k < S::K; ++k)
#pragma unroll
                for (int e = 0; e < kE; ++e) d[k][e] = r1 * fmaf(-(yv[k][e] * phi[k][e] * r1), m, d[k][e]);
        }
        const auto dyr = norm_rsrc(p.dy, p.grad_bf16, rows), dgr = norm_rsrc(p.dgate, p.grad_bf16, rows);
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            float o[kE];
#pragma unroll
            for (int e = 0; e < kE; ++e) o[e] = d[k][e] * phi[k][e];
            store_piece<S, VEC, true>(dyr, p.grad_bf16, lane, sub, k, p.D, o);
            if (p.dgate) {
#pragma unroll
                for (int e = 0; e < kE; ++e) o[e] = d[k][e] * yv[k][e] * dphi[k][e];
                store_piece<S, VEC, true>(dgr, p.grad_bf16, lane, sub, k, p.D, o);
            }
        }
    }
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 3 * p.D;
    if (p.dw_post) put_columns<S, VEC>(part, &cols[0][0], lane, sub, p.D, gpost);
    if (p.dscale) put_columns<S, VEC>(part + p.D, &cols[0][0], lane, sub, p.D, gsc);
    if (p.dw_pre) put_columns<S, VEC>(part + 2 * p.D, &cols[0][0], lane, sub, p.D, gpre);
}

// The same for wide rows, on 1024 threads of 128 registers each.  Much of what does not fit them lies
// in LDS, where every thread finds its own and no other's: the weights with one piece a thread,
// two of the three column sums with two (the weights are then read from the cache).  No row is
// loaded ahead, and the gates are taken twice.  Spilled all the same: nothing with one 16-byte piece a thread, 7 to 16
// registers with eight single elements, 22 to 37 and 80 to 98 with two pieces of either.
// R8192 D8192: bf16 252 us, 4.3 TB/s, fp32 467 us (the kernel above, spilling: 885 and 1946; this one
// with the next row in flight, spilling: 298 and 737; with the weights from the cache too, 430
// in bf16).  R4096 D16384 bf16: 479 us, 2.2 TB/s (2016; with every sum in registers 707); R5461 D12288 559 us,
// 1.9 TB/s.  Rows that do not fill the threads: R13107 D5120 bf16 321 us, 3.3 TB/s; element by element, R8192
// D8190 334 us, 3.2.  Bound by latency: one workgroup per compute unit, three sums over 16 waves per
// row, nothing else to run meanwhile.
template <typename S, bool VEC, typename TIn, typename TRes>
__global__ __launch_bounds__(S::NT) void layer_norm_bwd_wide_kernel(NormParams p) {
    constexpr bool kWeights = S::K == 1;  // in LDS
    __shared__ float red[2][S::NT / 64][2];
    __shared__ float4 mine[kWeights ? 3 : 2][2 * S::K][S::NT];  // the weights, or the sums of dscale and dw_post
    RowSum<S> sum{red};
    const int lane = threadIdx.x;
    const float inv = 1.0f / static_cast<float>(p.D);
    float gpost[S::K][kE] = {}, gsc[S::K][kE] = {}, gpre[S::K][kE] = {};  // with two pieces gpre alone
    auto get = [&](int n, int k, float (&o)[kE]) {
        const int t = anew(lane);
        const float4 a = mine[n][2 * k][t], b = mine[n][2 * k + 1][t];
        o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
    };
    auto put = [&](int n, int k, const float (&v)[kE]) {
        mine[n][2 * k][lane] = make_float4(v[0], v[1], v[2], v[3]);
        mine[n][2 * k + 1][lane] = make_float4(v[4], v[5], v[6], v[7]);
    };
    if (kWeights) {
        for (int n = 0; n < 3; ++n) {
            float v[kE];
            load_weights<S, VEC>(n == 0 ? p.w_post : n == 1 ? p.scale : p.w_pre, lane, 0, p.D, v);
            put(n, 0, v);
        }
    } else {
        const float zero[kE] = {};
#pragma unroll
        for (int k = 0; k < S::K; ++k) put(0, k, zero), put(1, k, zero);
    }
    auto weights = [&](int n, const float* from, int k, float (&o)[kE]) {
        if constexpr (kWeights) {
            get(n, 0, o);
        } else {
            load_weights<S, VEC>(from, anew(lane), k, p.D, o);
        }
    };
    for (uint32_t it = blockIdx.x; it < static_cast<uint32_t>(p.R); it += gridDim.x) {
        const Rows rows = rows_of<S>(it, p.R, p.D);
        Raw<TIn, TRes> raw[S::K];
        fetch<S, VEC>(p, it, lane, 0, raw);
        float u[S::K][kE], d[S::K][kE];
        float ss[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            float phi[kE], dphi[kE];
            gates(p.gate_kind, raw[k].g, phi, dphi);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                u[k][e] = widen(raw[k].y.e[e]) * phi[e];
                ss[0] = fmaf(u[k][e], u[k][e], ss[0]);
            }
        }
        float r1 = 1.0f;
        if (p.y && p.post) {
            sum(ss);
            r1 = rsqrt_acc(fmaf(ss[0], inv, p.eps));
        }
        if (p.pre) {
            float xs[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < S::K; ++k) {
                float wp[kE], sc[kE], wq[kE];
                weights(0, p.w_post, k, wp);
                weights(1, p.scale, k, sc);
                weights(2, p.w_pre, k, wq);
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    d[k][e] = fmaf(u[k][e] * r1 * wp[e], sc[e], widen(raw[k].x.e[e]));  // x'
                    xs[0] = fmaf(d[k][e], d[k][e], xs[0]);
                    xs[1] = fmaf(widen(raw[k].z.e[e]) * wq[e], d[k][e], xs[1]);
                }
            }
            sum(xs);
            const float r2 = rsqrt_acc(fmaf(xs[0], inv, p.eps));
            const float m = xs[1] * inv * r2;  // mean(t xh)
#pragma unroll
            for (int k = 0; k < S::K; ++k) {
                float wq[kE];
                weights(2, p.w_pre, k, wq);
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    const float xh = d[k][e] * r2, z = widen(raw[k].z.e[e]);
                    gpre[k][e] = fmaf(z, xh, gpre[k][e]);
                    d[k][e] = fmaf(r2, fmaf(-xh, m, z * wq[e]), widen(raw[k].d.e[e]));
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < S::K; ++k)
#pragma unroll
                for (int e = 0; e < kE; ++e) d[k][e] = widen(raw[k].d.e[e]);
        }
        const auto dxr = norm_rsrc(p.dx, p.res_bf16, rows);
#pragma unroll
        for (int k = 0; k < S::K; ++k) store_piece<S, VEC, true>(dxr, p.res_bf16, lane, 0, k, p.D, d[k]);
        if (!p.y) continue;
        ss[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            float wp[kE], sc[kE];
            weights(0, p.w_post, k, wp);
            weights(1, p.scale, k, sc);
            float as[kE], ap[kE];  // the sums of dscale and dw_post
            if constexpr (!kWeights) get(0, k, as), get(1, k, ap);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                u[k][e] *= r1;  // n1
                float &to_s = kWeights ? gsc[k][e] : as[e], &to_p = kWeights ? gpost[k][e] : ap[e];
                to_s = fmaf(d[k][e], u[k][e] * wp[e], to_s);
                d[k][e] *= sc[e];
                to_p = fmaf(d[k][e], u[k][e], to_p);
                d[k][e] *= wp[e];
                ss[0] = fmaf(d[k][e], u[k][e], ss[0]);
            }
            if constexpr (!kWeights) put(0, k, as), put(1, k, ap);
        }
        if (p.post) {
            sum(ss);
            const float m = ss[0] * inv;  // mean(s n1)
#pragma unroll
            for (int k = 0; k < S::K; ++k)
#pragma unroll
                for (int e = 0; e < kE; ++e) d[k][e] = r1 * fmaf(-u[k][e], m, d[k][e]);
        }
        const auto dyr = norm_rsrc(p.dy, p.grad_bf16, rows), dgr = norm_rsrc(p.dgate, p.grad_bf16, rows);
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            float phi[kE], dphi[kE], o[kE];
#pragma unroll
            for (int e = 0; e < kE; ++e) raw[k].g.e[e] = anew(raw[k].g.e[e]);
            gates(p.gate_kind, raw[k].g, phi, dphi);
#pragma unroll
            for (int e = 0; e < kE; ++e) o[e] = d[k][e] * phi[e];
            store_piece<S, VEC, true>(dyr, p.grad_bf16, lane, 0, k, p.D, o);
#pragma unroll
            for (int e = 0; e < kE; ++e) o[e] = d[k][e] * widen(raw[k].y.e[e]) * dphi[e];
            store_piece<S, VEC, true>(dgr, p.grad_bf16, lane, 0, k, p.D, o);
        }
    }
    if constexpr (!kWeights) {
#pragma unroll
        for (int k = 0; k < S::K; ++k) get(0, k, gsc[k]), get(1, k, gpost[k]);
    }
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 3 * p.D;
    if (p.dw_post) put_columns<S, VEC>(part, nullptr, lane, 0, p.D, gpost);
    if (p.dscale) put_columns<S, VEC>(part + p.D, nullptr, lane, 0, p.D, gsc);
    if (p.dw_pre) put_columns<S, VEC>(part + 2 * p.D, nullptr, lane, 0, p.D, gpre);
}

// out[c] = sum over the workgroups of part[g][which][c]: 32 columns and 32 rows of
// threads to a workgroup, each adding every 32nd row in order, 16 loads at a time, then a
// tree over the rows of threads.  (A row past the last reads zero.)
__global__ __launch_bounds__(1024) void layer_norm_cols_kernel(NormParams p) {
    __shared__ float s[32][32];
    const int which = blockIdx.y;
    float* out = which == 0 ? p.dw_post : which == 1 ? p.dscale : p.dw_pre;
    if (!out) return;
    const int l = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + l;
    const uint32_t row = 3 * p.D * 4;  // bytes
    const auto part = rows_rsrc(p.part, 0, p.groups * row);
    float a = 0.0f;
    for (int g0 = r; g0 < p.groups; g0 += 32 * 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = load_row<float>(part, c < p.D ? (g0 + 32 * i) * row + (which * p.D + c) * 4 : kOut);
#pragma unroll
        for (int i = 0; i < 16; ++i) a += v[i];
    }
    s[r][l] = a;
#pragma unroll
    for (int n = 16; n > 0; n /= 2) {
        __syncthreads();
        if (r < n) s[r][l] += s[r + n][l];
    }
    if (r == 0 && c < p.D) out[c] = s[0][l];
}

template <typename TIn, typename TRes>
void launch(const NormParams& p, hipStream_t st) {
    with_shape(p.D, [&](auto s) {
        using S = decltype(s);
        auto go = [&](auto vec) {
            if constexpr (S::NT < 1024)
                hipLaunchKernelGGL((layer_norm_bwd_kernel<S, vec(), TIn, TRes>), dim3(p.groups), dim3(S::NT), 0, st, p);
            else
                hipLaunchKernelGGL((layer_norm_bwd_wide_kernel<S, vec(), TIn, TRes>), dim3(p.groups), dim3(S::NT), 0,
                                   st, p);
        };
        p.vec ? go(std::true_type()) : go(std::false_type());
    });
}

}  // namespace

int launch_norm_bwd(const NormParams& p, hipStream_t st) {
    if (p.in_bf16)
        p.res_bf16 ? launch<uint16_t, uint16_t>(p, st) : launch<uint16_t, float>(p, st);
    else
        p.res_bf16 ? launch<float, uint16_t>(p, st) : launch<float, float>(p, st);
    if (p.dw_post || p.dscale || p.dw_pre)
        hipLaunchKernelGGL(layer_norm_cols_kernel, dim3((p.D + 31) / 32, 3), dim3(1024), 0, st, p);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace layer
