// layer_ssm.hip -- the selective state space scan, forward and single step (layer_ssm.h).
//
// Where the chains of 64 channels are too few to fill the device the time axis is split into segments: a first kernel
// takes every segment but the last from a state of zeros to its end, which gives the segment's map h -> exp(A S) h + H
// (S the sum of its steps); the second starts each segment from the maps before it, composed in order.
#include "layer_ssm.h"

namespace layer {
namespace {

constexpr int kTile = kSsmTile;
constexpr int kMaxSegs = 64;
#ifndef WANT
#define WANT 256
#endif

// The workspace: the segments' maps [chain][segment][state, sum of steps][64].
struct FwdSpace {
    float* maps;
    int segs;
    int64_t length;  // tokens per segment, whole tiles
    size_t bytes;
};
__host__ __device__ inline FwdSpace fwd_space(const SsmParams& p) {
    FwdSpace s;
    const int64_t blocks = (p.D / p.G + 63) / 64, chains = blocks * p.G * p.B, tiles = tiles_of(p.T, kTile);
    // workgroups of as many waves as a state has quads
    int64_t want = WANT / chains;
    want = want < 1 ? 1 : want > kMaxSegs ? kMaxSegs : want;
    if (want > tiles / 4) want = tiles / 4;
    if (want < 1) want = 1;
    const int64_t per = tiles_of(tiles, static_cast<int>(want));
    s.length = per * kTile;
    s.segs = static_cast<int>(tiles_of(tiles, static_cast<int>(per)));
    s.maps = static_cast<float*>(p.ws);
    s.bytes = s.segs > 1 ? static_cast<size_t>(chains) * s.segs * (ssm_padded(p.N) + 1) * 64 * sizeof(float) : 0;
    return s;
}

// Segment k of a chain's maps.
template <int NP>
__device__ __forceinline__ float* map_of(const FwdSpace& ws, int chain, int k) {
    return ws.maps + (static_cast<int64_t>(chain) * ws.segs + k) * (NP + 1) * 64;
}

// MAPS: the segments' maps alone.
template <typename TIn, int SN, int NW, bool MAPS, bool VEC>
__global__ __launch_bounds__(NW * 64) void layer_ssm_fwd_kernel(SsmParams p, FwdSpace ws) {
    constexpr int NP = SN * NW;            // states, with those that stand for none
    constexpr int NT = NW * 64;
    constexpr int K = kTile * 16 / NT;     // quads of a tile that a thread takes
    constexpr bool kAcc = kAccurate<TIn>;
    __shared__ float du[kTile][2][64];     // delta and u
    __shared__ float part[MAPS ? 1 : NW][MAPS ? 1 : kTile][64];  // a wave's part of y
    const int chains = p.B * p.G * ssm_blocks(p);
    const int chain = blockIdx.x % chains, seg = blockIdx.x / chains;
    const SsmPlace me = ssm_place(p, chain);
    const SsmQuad mine = ssm_quad(p, me, chain);
    const int wave = me.wave, l = me.l, c = me.c, n0 = wave * SN;
    float A[SN], h[SN], bias[4], skip[4];
    quad_weights(p.dt_bias, mine, bias);
    quad_weights(p.skip, mine, skip);
    const int64_t state = (static_cast<int64_t>(me.b) * p.D + c) * p.N + n0;
#pragma unroll
    for (int n = 0; n < SN; ++n) {
        const bool on = n0 + n < p.N;
        A[n] = on ? p.A[static_cast<int64_t>(c) * p.N + n0 + n] * kLog2e : 0.0f;
        h[n] = !MAPS && on && p.state_in ? p.state_in[state + n] : 0.0f;
    }
    if constexpr (!MAPS) {
        for (int k = 0; k < seg; ++k) {
            const float* m = map_of<NP>(ws, chain, k) + l;
            const float S = m[NP * 64];
#pragma unroll
            for (int n = 0; n < SN; ++n) {
                const float H = m[(n0 + n) * 64];
                // a segment with a document's border in it passes nothing on, whatever it is; a product of decays that
                // underflows is held above 0, so that an infinite state stays one as token by token
                const float P = fmaxf(__builtin_amdgcn_exp2f(A[n] * S), 1.40129846e-45f);
                h[n] = S == __builtin_inff() ? H : fmaf(P, h[n], H);
            }
        }
    }
    const int t_begin = static_cast<int>(seg * ws.length), t_end = static_cast<int>(min(t_begin + ws.length, static_cast<int64_t>(p.T)));
    struct Raw {
        Vec<TIn, 4> x[K], d[K], z[MAPS ? 1 : K];
        SsmRegs<TIn, SN, kTile, VEC> b, c;
    } next;
    auto fetch = [&](int t0) {
        const int valid = min(max(me.len - t0, 0), min(kTile, t_end - t0));
        const int64_t token = static_cast<int64_t>(me.b) * p.T + t0;
        const auto xr = ssm_rows<TIn>(p.x, token, valid, p.x_row, p.D);
        const auto dr = ssm_rows<TIn>(p.dt, token, valid, p.dt_row, p.D);
        const auto zr = ssm_rows<TIn>(p.z, token, MAPS ? 0 : valid, p.z_row, p.D);
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int row = mine.row + i * (NT / 16);
            next.x[i] = load_quad<TIn, VEC, true>(xr, quad_offset<TIn>(mine, row, p.x_row), mine.count);
            next.d[i] = load_quad<TIn, VEC, true>(dr, quad_offset<TIn>(mine, row, p.dt_row), mine.count);
            if constexpr (!MAPS) next.z[i] = load_quad<TIn, VEC, true>(zr, quad_offset<TIn>(mine, row, p.z_row), mine.count);
        }
        const TIn *Bg = static_cast<const TIn*>(p.Bm) + me.g * p.N, *Cg = static_cast<const TIn*>(p.Cm) + me.g * p.N;
        next.b.load(ssm_rows<TIn>(Bg, token, valid, p.b_row, p.N), l, n0, p.N, p.b_row);
        if constexpr (!MAPS) next.c.load(ssm_rows<TIn>(Cg, token, valid, p.c_row, p.N), l, n0, p.N, p.c_row);
    };
    fetch(t_begin);
    double steps[4] = {};  // the sums of this thread's tokens' steps
    bool dropped = false;
    for (int t0 = t_begin; t0 < t_end; t0 += kTile) {
        const int rows = min(kTile, t_end - t0), valid = min(max(me.len - t0, 0), rows);
        float x[K][4], z[MAPS ? 1 : K][4], B[kTile / 16][SN], C[kTile / 16][SN];
        next.b.get(B);
        if constexpr (!MAPS) next.c.get(C);
        float d[K][4];
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d[i][e] = widen(next.d[i].e[e]) + bias[e];
                x[i][e] = widen(next.x[i].e[e]);
                if constexpr (!MAPS) z[i][e] = widen(next.z[i].e[e]);
            }
        if (t0 + kTile < t_end) fetch(t0 + kTile);
        if (p.softplus) {
            float slope;
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) softplus_parts<kAcc>(d[i][e], d[i][e], slope);
        }
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int row = mine.row + i * (NT / 16);
            float4 dv, uv;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (row >= valid) d[i][e] = 0.0f;
                (&dv.x)[e] = d[i][e];
                (&uv.x)[e] = d[i][e] * x[i][e];
                if constexpr (MAPS) steps[e] += d[i][e];
            }
            *reinterpret_cast<float4*>(&du[row][0][(threadIdx.x & 15) * 4]) = dv;
            *reinterpret_cast<float4*>(&du[row][1][(threadIdx.x & 15) * 4]) = uv;
        }
        const uint64_t cuts = ssm_cuts(p, me.b, t0, valid, l);
        dropped = dropped || cuts != 0;
        __syncthreads();
        with_flag(cuts != 0, [&](auto with_cuts) {
            each<kTile>([&](auto tc) {
                constexpr int t = tc();
                if (with_cuts() && (cuts >> t & 1)) {
#pragma unroll
                    for (int n = 0; n < SN; ++n) h[n] = 0.0f;
                }
                if (!MAPS && t % kSsmSave == 0 && p.saved && t < rows && me.live) {
                    const int64_t tiles = tiles_of(p.T, kSsmSave);
                    float* to = p.saved + (me.b * tiles + (t0 + t) / kSsmSave) * p.N * p.D + c;
#pragma unroll
                    for (int n = 0; n < SN; ++n)
                        if (n0 + n < p.N) to[static_cast<int64_t>(n0 + n) * p.D] = h[n];
                }
                const float step = du[t][0][l], u = du[t][1][l];
                float y[SN];
#pragma unroll
                for (int n = 0; n < SN; ++n) {
                    h[n] = fmaf(__builtin_amdgcn_exp2f(step * A[n]), h[n], bcast<t % 16>(B[t / 16][n]) * u);
                    if constexpr (!MAPS) y[n] = bcast<t % 16>(C[t / 16][n]) * h[n];
                }
                if constexpr (!MAPS) {
#pragma unroll
                    for (int k = 1; k < SN; k *= 2)
#pragma unroll
                        for (int n = 0; n < SN; n += 2 * k) y[n] += y[n + k];
                    part[wave][t][l] = y[0];
                }
            });
        });
        __syncthreads();
        if constexpr (!MAPS) {
            const int size = p.y_bf16 ? 2 : 4;
            const auto yr = rows_rsrc(p.y, (static_cast<int64_t>(me.b) * p.T + t0) * p.D * size, rows * p.D * size);
            float y[K][4];
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const int row = mine.row + i * (NT / 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[i][e] = skip[e] * x[i][e];
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(&part[w][row][(threadIdx.x & 15) * 4]);
                    y[i][0] += v.x, y[i][1] += v.y, y[i][2] += v.z, y[i][3] += v.w;
                }
            }
            if (p.z) {
#pragma unroll
                for (int i = 0; i < K; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float s, r;
                        sigmoid2<kAcc>(z[i][e], s, r);
                        y[i][e] *= z[i][e] * s;
                    }
            }
            with_flag(p.y_bf16, [&](auto bf16) {
#pragma unroll
                for (int i = 0; i < K; ++i) {
                    const int row = mine.row + i * (NT / 16);
                    if (row >= valid) y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0.0f;
                    using T = std::conditional_t<bf16(), uint16_t, float>;
                    store_quad<VEC, bf16(), false>(yr, quad_offset<T>(mine, row, p.D), mine.count, y[i]);
                }
            });
        }
    }
    if constexpr (MAPS) {
        float* m = map_of<NP>(ws, chain, seg) + l;
#pragma unroll
        for (int n = 0; n < SN; ++n) m[(n0 + n) * 64] = h[n];
        // the sums of steps: 4 channels of NT / 16 threads each
        double* sums = reinterpret_cast<double*>(&du[0][0][0]);  // [NT / 16][64]; the last tile's steps are done with
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[mine.row * 64 + (threadIdx.x & 15) * 4 + e] = steps[e];
        __syncthreads();
        if (wave == 0) {
            double s = 0.0;
            for (int i = 0; i < NT / 16; ++i) s += sums[i * 64 + l];
            m[NP * 64] = dropped ? __builtin_inff() : static_cast<float>(s);
        }
    } else if (p.state_out && me.live && seg == ws.segs - 1) {
#pragma unroll
        for (int n = 0; n < SN; ++n)
            if (n0 + n < p.N) p.state_out[state + n] = h[n];
    }
}

// One token: L lanes to a channel, SN states each; state_out may be state_in (each value is read, then
// written, by one lane).
template <typename TIn, int L, int SN, bool VEC>
__global__ __launch_bounds__(256) void layer_ssm_step_kernel(SsmParams p) {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t i = id / L;  // b D + c
    const bool live = i < static_cast<int64_t>(p.B) * p.D;
    const int b = live ? static_cast<int>(i / p.D) : 0, c = live ? static_cast<int>(i % p.D) : 0;
    const int n0 = static_cast<int>(id % L) * SN, g = c / (p.D / p.G);
    const TIn* Bm = static_cast<const TIn*>(p.Bm) + static_cast<int64_t>(b) * p.b_row + g * p.N;
    const TIn* Cm = static_cast<const TIn*>(p.Cm) + static_cast<int64_t>(b) * p.c_row + g * p.N;
    const float x = widen(static_cast<const TIn*>(p.x)[static_cast<int64_t>(b) * p.x_row + c]);
    float d = widen(static_cast<const TIn*>(p.dt)[static_cast<int64_t>(b) * p.dt_row + c]) + (p.dt_bias ? p.dt_bias[c] : 0.0f);
    float slope;
    if (p.softplus) softplus_parts<kAccurate<TIn>>(d, d, slope);
    const float u = d * x;
    const int64_t s = (static_cast<int64_t>(b) * p.D + c) * p.N + n0, a = static_cast<int64_t>(c) * p.N + n0;
    float y[1] = {0.0f}, h[SN], A[SN];
    if (VEC && n0 < p.N) {
        const auto hv = load_vec<float, SN>(p.state_in, s), av = load_vec<float, SN>(p.A, a);
#pragma unroll
        for (int n = 0; n < SN; ++n) h[n] = hv.e[n], A[n] = av.e[n];
    } else {
#pragma unroll
        for (int n = 0; n < SN; ++n) {
            h[n] = n0 + n < p.N ? p.state_in[s + n] : 0.0f;
            A[n] = n0 + n < p.N ? p.A[a + n] : 0.0f;
        }
    }
#pragma unroll
    for (int n = 0; n < SN; ++n) {
        const bool on = n0 + n < p.N;
        h[n] = fmaf(__builtin_amdgcn_exp2f(d * (A[n] * kLog2e)), h[n], on ? u * widen(Bm[n0 + n]) : 0.0f);
        if (on) y[0] = fmaf(widen(Cm[n0 + n]), h[n], y[0]);
    }
    if (live) {
        if (VEC && n0 < p.N) {
            store_vec<SN>(p.state_out, s, h, false);
        } else {
#pragma unroll
            for (int n = 0; n < SN; ++n)
                if (n0 + n < p.N) p.state_out[s + n] = h[n];
        }
    }
    y[0] = osr::group_sum<L>(y[0]);
    if (!live || n0 != 0) return;
    if (p.skip) y[0] = fmaf(p.skip[c], x, y[0]);
    if (p.z) {
        const float z = widen(static_cast<const TIn*>(p.z)[static_cast<int64_t>(b) * p.z_row + c]);
        float sg, r;
        sigmoid2<kAccurate<TIn>>(z, sg, r);
        y[0] *= z * sg;
    }
    store_vec<1>(p.y, i, y, p.y_bf16);
}

template <typename TIn>
void launch_fwd(const SsmParams& p, hipStream_t st) {
    const FwdSpace ws = fwd_space(p);
    with_states(p.N, [&](auto sn, auto nw) {
        const unsigned chains = static_cast<unsigned>(p.B) * p.G * tiles_of(p.D / p.G, 64);
        auto go = [&](auto vec) {
            const dim3 block(nw() * 64);
            if (ws.segs > 1)
                hipLaunchKernelGGL((layer_ssm_fwd_kernel<TIn, sn(), nw(), true, vec()>), dim3(chains * (ws.segs - 1)), block,
                                   0, st, p, ws);
            hipLaunchKernelGGL((layer_ssm_fwd_kernel<TIn, sn(), nw(), false, vec()>), dim3(chains * ws.segs), block, 0, st, p,
                               ws);
        };
        ssm_vec(p) ? go(std::true_type()) : go(std::false_type());
    });
}

template <typename TIn>
void launch_step(const SsmParams& p, hipStream_t st) {
    const bool vec = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.state_in) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(p.state_out) % 16 == 0 && reinterpret_cast<uintptr_t>(p.A) % 16 == 0;
    auto go = [&](auto L) {
        const dim3 grid(static_cast<unsigned>(tiles_of(static_cast<int64_t>(p.B) * p.D * L(), 256)));
        if (vec)
            hipLaunchKernelGGL((layer_ssm_step_kernel<TIn, L(), 4, true>), grid, dim3(256), 0, st, p);
        else
            hipLaunchKernelGGL((layer_ssm_step_kernel<TIn, L(), 4, false>), grid, dim3(256), 0, st, p);
    };
    if (p.N <= 4) go(std::integral_constant<int, 1>());
    else if (p.N <= 8) go(std::integral_constant<int, 2>());
    else if (p.N <= 16) go(std::integral_constant<int, 4>());
    else if (p.N <= 32) go(std::integral_constant<int, 8>());
    else go(std::integral_constant<int, 16>());
}

}  // namespace

size_t ssm_workspace_bytes(const SsmParams& p) { return fwd_space(p).bytes; }

int launch_ssm_fwd(const SsmParams& p, hipStream_t st) {
    p.in_bf16 ? launch_fwd<uint16_t>(p, st) : launch_fwd<float>(p, st);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}
int launch_ssm_step(const SsmParams& p, hipStream_t st) {
    p.in_bf16 ? launch_step<uint16_t>(p, st) : launch_step<float>(p, st);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace layer
