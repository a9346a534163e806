// layer_ssm.hip -- the selective state space scan, forward and single step (layer_ssm.h).
#include "layer_ssm.h"

namespace layer {
namespace {

constexpr int kTile = 32;  // tokens per tile

template <typename TIn, int SN, int NW>
__global__ __launch_bounds__(NW * 64) void layer_ssm_fwd_kernel(SsmParams p) {
    constexpr int NP = SN * NW;     // states, with those that stand for none
    constexpr int R = kTile / NW;   // tokens of a tile whose inputs and outputs a wave takes
    __shared__ float2 du[kTile][64];
    __shared__ float bc[kTile][2 * NP];
    __shared__ float part[NW][kTile][64];
    const SsmPlace me = ssm_place(p, blockIdx.x);
    const int wave = me.wave, l = me.l, c = me.c, n0 = wave * SN, r0 = wave * R;
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, skip = p.skip ? p.skip[c] : 0.0f;
    float A[SN], h[SN];
    const int64_t state = (static_cast<int64_t>(me.b) * p.D + c) * p.N + n0;
#pragma unroll
    for (int n = 0; n < SN; ++n) {
        const bool on = n0 + n < p.N;
        A[n] = on ? p.A[static_cast<int64_t>(c) * p.N + n0 + n] * kLog2e : 0.0f;
        h[n] = on && p.state_in ? p.state_in[state + n] : 0.0f;
    }
    const uint32_t ex = me.live ? c * sizeof(TIn) : kOut;
    const uint32_t ey = me.live ? c * (p.y_bf16 ? 2u : 4u) : kOut, dy = p.D * (p.y_bf16 ? 2u : 4u);
    for (int t0 = 0; t0 < p.T; t0 += kTile) {
        const int rows = min(kTile, p.T - t0), valid = min(max(me.len - t0, 0), rows);
        const auto xr = ssm_rows<TIn>(p.x, me.b, p.T, t0, valid, p.x_row, p.D);
        const auto dr = ssm_rows<TIn>(p.dt, me.b, p.T, t0, valid, p.dt_row, p.D);
        const auto zr = ssm_rows<TIn>(p.z, me.b, p.T, t0, valid, p.z_row, p.D);
        TIn rx[R], rd[R], rz[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            rx[i] = load_row<TIn>(xr, ex + (r0 + i) * p.x_row * static_cast<uint32_t>(sizeof(TIn)));
            rd[i] = load_row<TIn>(dr, ex + (r0 + i) * p.dt_row * static_cast<uint32_t>(sizeof(TIn)));
            rz[i] = load_row<TIn>(zr, ex + (r0 + i) * p.z_row * static_cast<uint32_t>(sizeof(TIn)));
        }
        ssm_load_bc<TIn, NP, kTile, NW * 64>(p, me, t0, valid, bc);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float d = widen(rd[i]) + bias, slope;
            if (p.softplus) softplus_parts(d, d, slope);
            const bool on = r0 + i < valid;
            du[r0 + i][l] = make_float2(on ? d : 0.0f, on ? d * widen(rx[i]) : 0.0f);
        }
        const uint64_t cuts = ssm_cuts(p, me.b, t0, valid, l);
        __syncthreads();
        for (int t = 0; t < kTile; ++t) {
            if (cuts >> t & 1) {
#pragma unroll
                for (int n = 0; n < SN; ++n) h[n] = 0.0f;
            }
            if (p.saved && t % kSsmSave == 0 && t < rows && me.live) {
                const int64_t tiles = tiles_of(p.T, kSsmSave);
                float* to = p.saved + (me.b * tiles + (t0 + t) / kSsmSave) * p.N * p.D + c;
#pragma unroll
                for (int n = 0; n < SN; ++n)
                    if (n0 + n < p.N) to[static_cast<int64_t>(n0 + n) * p.D] = h[n];
            }
            const float2 v = du[t][l];
            float y = 0.0f;
#pragma unroll
            for (int n = 0; n < SN; ++n) {
                h[n] = fmaf(__builtin_amdgcn_exp2f(v.x * A[n]), h[n], v.y * bc[t][n0 + n]);
                y = fmaf(bc[t][NP + n0 + n], h[n], y);
            }
            part[wave][t][l] = y;
        }
        __syncthreads();
        const auto yr = rows_rsrc(p.y, (static_cast<int64_t>(me.b) * p.T + t0) * p.D * (p.y_bf16 ? 2 : 4), rows * p.D * (p.y_bf16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float y = skip * widen(rx[i]);
#pragma unroll
            for (int w = 0; w < NW; ++w) y += part[w][r0 + i][l];
            if (p.z) {
                const float z = widen(rz[i]);
                float s, r;
                sigmoid2<true>(z, s, r);
                y *= z * s;
            }
            if (r0 + i >= valid) y = 0.0f;
            if (p.y_bf16) store_row<true, false>(yr, ey + (r0 + i) * dy, y);
            else store_row<false, false>(yr, ey + (r0 + i) * dy, y);
        }
    }
    if (p.state_out && me.live) {
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
    if (p.softplus) softplus_parts(d, d, slope);
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
        sigmoid2<true>(z, sg, r);
        y[0] *= z * sg;
    }
    store_vec<1>(p.y, i, y, p.y_bf16);
}

template <typename TIn>
void launch_fwd(const SsmParams& p, hipStream_t st) {
    with_states(p.N, [&](auto sn, auto nw) {
        const unsigned chains = static_cast<unsigned>(p.B) * p.G * tiles_of(p.D / p.G, 64);
        hipLaunchKernelGGL((layer_ssm_fwd_kernel<TIn, sn(), nw()>), dim3(chains), dim3(nw() * 64), 0, st, p);
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

size_t ssm_workspace_bytes(const SsmParams&) { return 0; }

int launch_ssm_fwd(const SsmParams& p, hipStream_t st) {
    p.in_bf16 ? launch_fwd<uint16_t>(p, st) : launch_fwd<float>(p, st);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}
int launch_ssm_step(const SsmParams& p, hipStream_t st) {
    p.in_bf16 ? launch_step<uint16_t>(p, st) : launch_step<float>(p, st);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace layer
