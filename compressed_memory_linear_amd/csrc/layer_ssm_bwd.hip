// layer_ssm_bwd.hip -- gradient of the selective state space scan (layer_ssm.h).
//
// With g = dy phi(z), phi(z) = z sigmoid(z), a_t = exp(delta_t A) and l_t the gradient that reaches h_t,
//     l_t = C_t g_t + a_{t+1} l_{t+1}   (the last token's taking dstate_out in),
//     dC_t = sum_c g_t h_t,   dB_t = sum_c l_t u_t   over the channels of a group,
//     du_t = sum_n l_t B_t,   r_t = a_t l_t,   q_t = r_t h_{t-1},
//     ddelta_t = sum_n q_t A + du_t x_t,   dA = sum_t q_t delta_t,   dstate_in = r_0,
//     dx = du delta + skip g,   ddt = ddelta softplus'(dt + bias),   dz = dy (C h + skip x) phi'(z).
// A workgroup walks its chain backwards in tiles of kSsmSave tokens: it takes the states of the tile again from the one
// that the forward saved before it, keeps them with their decays in registers, and then runs backwards over them.
// The sums over channels go to the workspace, a block of 64 channels each, and are added by a second kernel in a
// fixed order (no atomics: reruns agree bit for bit); so are the sums over tokens.
#include "layer_ssm.h"

namespace layer {
namespace {

constexpr int kTile = kSsmSave;

template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t ssm_rows(const void* p, int64_t token, int rows, int row, int width) {
    const int bytes = p && rows > 0 ? ((rows - 1) * row + width) * static_cast<int>(sizeof(T)) : 0;
    return rows_rsrc(p, token * row * static_cast<int64_t>(sizeof(T)), bytes);
}

// B and C of a tile's tokens as floats [token][2][NP], zeros past N and at padding (so that
// whatever stands there reaches nothing).
template <typename TIn, int NP, int TILE, int NT>
__device__ __forceinline__ void ssm_load_bc(const SsmParams& p, const SsmPlace& me, int t0, int n, float (*bc)[2 * NP]) {
    const int64_t row = static_cast<int64_t>(me.b) * p.T + t0;
    const TIn* Bm = static_cast<const TIn*>(p.Bm) + row * p.b_row + me.g * p.N;
    const TIn* Cm = static_cast<const TIn*>(p.Cm) + row * p.c_row + me.g * p.N;
    for (int i = threadIdx.x; i < TILE * 2 * NP; i += NT) {
        const int t = i / (2 * NP), k = i % (2 * NP), s = k % NP;
        float v = 0.0f;
        if (t < n && s < p.N) v = widen(k < NP ? Bm[static_cast<int64_t>(t) * p.b_row + s] : Cm[static_cast<int64_t>(t) * p.c_row + s]);
        bc[t][k] = v;
    }
}

// The workspace: sums of B's and C's gradients [block][B T][G][2][N], then those over tokens
// [B][N + 2][D] (dA, dskip, ddt_bias).
struct BwdSpace {
    float *bc, *tok;
    size_t bytes;
};
__host__ __device__ inline BwdSpace bwd_space(const SsmParams& p) {
    BwdSpace s;
    const int64_t blocks = (p.D / p.G + 63) / 64;
    const int64_t nbc = blocks * p.B * p.T * p.G * 2 * p.N, ntok = static_cast<int64_t>(p.B) * (p.N + 2) * p.D;
    s.bc = static_cast<float*>(p.ws);
    s.tok = s.bc + nbc;
    s.bytes = static_cast<size_t>(nbc + ntok) * sizeof(float);
    return s;
}

template <typename TIn, typename TDy, int SN, int NW>
__global__ __launch_bounds__(NW * 64) void layer_ssm_bwd_kernel(SsmParams p) {
    constexpr int NP = SN * NW;
    constexpr int R = kTile / NW;
    constexpr bool kHold = SN == 4;  // the decays too
    __shared__ float4 in[kTile][64];  // delta, u, g
    __shared__ float bc[kTile][2 * NP];
    __shared__ float sums[kTile][2 * NP];  // dB and dC over the block
    __shared__ float2 part[NW][kTile][64];  // du and ddelta of a wave's states
    __shared__ float ypart[NW][kTile][64];
    const SsmPlace me = ssm_place(p, blockIdx.x);
    const int wave = me.wave, l = me.l, c = me.c, n0 = wave * SN, r0 = wave * R;
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, skip = p.skip ? p.skip[c] : 0.0f;
    float A[SN], lam[SN], dA[SN] = {}, dskip = 0.0f, dbias = 0.0f;
    const int64_t state = (static_cast<int64_t>(me.b) * p.D + c) * p.N + n0;
#pragma unroll
    for (int n = 0; n < SN; ++n) {
        const bool on = n0 + n < p.N;
        A[n] = on ? p.A[static_cast<int64_t>(c) * p.N + n0 + n] * kLog2e : 0.0f;
        lam[n] = on && me.live && p.dstate_out ? p.dstate_out[state + n] : 0.0f;
    }
    const int eg = p.grad_bf16 ? 2 : 4;
    const uint32_t ex = me.live ? c * sizeof(TIn) : kOut, edy = me.live ? c * sizeof(TDy) : kOut;
    const uint32_t ed = me.live ? c * eg : kOut, dd = p.D * eg;
    const int tiles = (p.T + kTile - 1) / kTile;
    const BwdSpace ws = bwd_space(p);
    const int blocks = ssm_blocks(p);
    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int t0 = tile * kTile;
        const int rows = min(kTile, p.T - t0), valid = min(max(me.len - t0, 0), rows);
        const int64_t token = static_cast<int64_t>(me.b) * p.T + t0;
        const auto xr = ssm_rows<TIn>(p.x, token, valid, p.x_row, p.D);
        const auto dr = ssm_rows<TIn>(p.dt, token, valid, p.dt_row, p.D);
        const auto zr = ssm_rows<TIn>(p.z, token, valid, p.z_row, p.D);
        const auto gr = ssm_rows<TDy>(p.dy, token, valid, p.D, p.D);
        float x[R], d[R], slope[R], z[R], dy[R], g[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            x[i] = widen(load_row<TIn>(xr, ex + (r0 + i) * p.x_row * static_cast<uint32_t>(sizeof(TIn))));
            d[i] = widen(load_row<TIn>(dr, ex + (r0 + i) * p.dt_row * static_cast<uint32_t>(sizeof(TIn)))) + bias;
            z[i] = widen(load_row<TIn>(zr, ex + (r0 + i) * p.z_row * static_cast<uint32_t>(sizeof(TIn))));
            dy[i] = widen(load_row<TDy>(gr, edy + (r0 + i) * p.D * static_cast<uint32_t>(sizeof(TDy))));
        }
        ssm_load_bc<TIn, NP, kTile, NW * 64>(p, me, t0, valid, bc);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            slope[i] = 1.0f;
            if (p.softplus) softplus_parts<kAccurate<TIn>>(d[i], d[i], slope[i]);
            if (r0 + i >= valid) d[i] = 0.0f;
            g[i] = dy[i];
            if (p.z) {
                float s, r;
                sigmoid2<kAccurate<TIn>>(z[i], s, r);
                g[i] *= z[i] * s;
            }
            in[r0 + i][l] = make_float4(d[i], d[i] * x[i], g[i], 0.0f);
        }
        const uint64_t cuts = ssm_cuts(p, me.b, t0, valid, l);
        float before[SN], h[kTile][SN], a[kHold ? kTile : 1][SN];
        const float* from = p.saved + (static_cast<int64_t>(me.b) * tiles + tile) * p.N * p.D + c;
#pragma unroll
        for (int n = 0; n < SN; ++n)
            before[n] = n0 + n < p.N && me.live && !(cuts & 1) ? from[static_cast<int64_t>(n0 + n) * p.D] : 0.0f;
        __syncthreads();
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
            const float4 v = in[t][l];
            const bool cut = cuts >> t & 1;
            float y = 0.0f;
#pragma unroll
            for (int n = 0; n < SN; ++n) {
                const float e = __builtin_amdgcn_exp2f(v.x * A[n]), hp = t ? h[t - 1][n] : before[n];
                h[t][n] = fmaf(e, cut ? 0.0f : hp, v.y * bc[t][n0 + n]);
                if constexpr (kHold) a[t][n] = e;
                y = fmaf(bc[t][NP + n0 + n], h[t][n], y);
            }
            if (p.z) ypart[wave][t][l] = y;
        }
#pragma unroll
        for (int t = kTile - 1; t >= 0; --t) {
            if (t >= valid) {
                if (l == 0) {
#pragma unroll
                    for (int n = 0; n < SN; ++n) sums[t][n0 + n] = sums[t][NP + n0 + n] = 0.0f;
                }
                continue;
            }
            const float4 v = in[t][l];
            const bool cut = cuts >> t & 1;
            float du = 0.0f, q = 0.0f;
#pragma unroll
            for (int n = 0; n < SN; ++n) {
                lam[n] = fmaf(bc[t][NP + n0 + n], v.z, lam[n]);
                const float sC = osr::group_sum<64>(v.z * h[t][n]);
                const float sB = osr::group_sum<64>(lam[n] * v.y);
                if (l == 0) sums[t][n0 + n] = sB, sums[t][NP + n0 + n] = sC;
                du = fmaf(lam[n], bc[t][n0 + n], du);
                float e;
                if constexpr (kHold) e = a[t][n];
                else e = __builtin_amdgcn_exp2f(v.x * A[n]);
                // a state that is dropped passes nothing back, whatever it was
                lam[n] = cut ? 0.0f : e * lam[n];
                const float k = cut ? 0.0f : lam[n] * (t ? h[t - 1][n] : before[n]);
                q = fmaf(k, A[n], q);
                dA[n] = fmaf(k, v.x, dA[n]);
            }
            part[wave][t][l] = make_float2(du, q * kLn2);
        }
        __syncthreads();
        {
            // the block's sums, by all threads
            const int64_t row = (static_cast<int64_t>(blockIdx.x % blocks) * p.B + me.b) * p.T + t0;
            float* to = ws.bc + (row * p.G + me.g) * 2 * p.N;
            for (int i = threadIdx.x; i < rows * 2 * p.N; i += NW * 64) {
                const int t = i / (2 * p.N), k = i % (2 * p.N);
                to[static_cast<int64_t>(t) * p.G * 2 * p.N + k] = sums[t][k < p.N ? k : NP + k - p.N];
            }
        }
        const int64_t first = (static_cast<int64_t>(me.b) * p.T + t0) * p.D * eg;
        const auto dxr = rows_rsrc(p.dx, first, rows * p.D * eg), ddr = rows_rsrc(p.ddt, first, rows * p.D * eg);
        const auto dzr = rows_rsrc(p.dz, first, p.dz ? rows * p.D * eg : 0);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = r0 + i;
            const bool on = t < valid;
            float du = 0.0f, q = 0.0f, y = skip * x[i];
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float2 v = part[w][t][l];
                du += v.x, q += v.y;
                if (p.z) y += ypart[w][t][l];
            }
            float dx = fmaf(du, d[i], skip * g[i]), ddt = fmaf(du, x[i], q) * slope[i], dz = 0.0f;
            if (p.z) {
                float s, r;
                sigmoid2<kAccurate<TIn>>(z[i], s, r);
                dz = dy[i] * y * (s * fmaf(z[i], r, 1.0f));
            }
            if (!on) dx = ddt = dz = 0.0f;
            if (on) {
                dskip = fmaf(g[i], x[i], dskip);
                dbias += ddt;
            }
            with_flag(p.grad_bf16, [&](auto bf16) {
                store_row<bf16(), true>(dxr, ed + t * dd, dx);
                store_row<bf16(), true>(ddr, ed + t * dd, ddt);
                store_row<bf16(), true>(dzr, ed + t * dd, dz);
            });
        }
        __syncthreads();
    }
    if (p.dstate_in && me.live) {
#pragma unroll
        for (int n = 0; n < SN; ++n)
            if (n0 + n < p.N) p.dstate_in[state + n] = lam[n];
    }
    // the sums over tokens
    float* tok = ws.tok + static_cast<int64_t>(me.b) * (p.N + 2) * p.D + c;
    if (me.live) {
#pragma unroll
        for (int n = 0; n < SN; ++n)
            if (n0 + n < p.N) tok[static_cast<int64_t>(n0 + n) * p.D] = dA[n];
    }
    part[wave][0][l] = make_float2(dskip, dbias);
    __syncthreads();
    if (wave == 0 && me.live) {
        float2 s = part[0][0][l];
#pragma unroll
        for (int w = 1; w < NW; ++w) s.x += part[w][0][l].x, s.y += part[w][0][l].y;
        tok[static_cast<int64_t>(p.N) * p.D] = s.x;
        tok[static_cast<int64_t>(p.N + 1) * p.D] = s.y;
    }
}

// dB and dC: the blocks' sums added in order.  One thread per value [B T][G][2][N].
__global__ __launch_bounds__(256) void layer_ssm_bc_kernel(SsmParams p) {
    const int64_t n = static_cast<int64_t>(p.B) * p.T * p.G * 2 * p.N;
    const int blocks = (p.D / p.G + 63) / 64;
    const float* bc = bwd_space(p).bc;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        float s = 0.0f;
        for (int k = 0; k < blocks; ++k) s += bc[k * n + i];
        const int64_t row = i / (2 * p.N);
        const int k = static_cast<int>(i % (2 * p.N));
        const float o[1] = {s};
        store_vec<1>(k < p.N ? p.dB : p.dC, row * p.N + k % p.N, o, p.grad_bf16);
    }
}

template <typename TIn, typename TDy>
void launch(const SsmParams& p, hipStream_t st) {
    with_states(p.N, [&](auto sn, auto nw) {
        const unsigned chains = static_cast<unsigned>(p.B) * p.G * tiles_of(p.D / p.G, 64);
        hipLaunchKernelGGL((layer_ssm_bwd_kernel<TIn, TDy, sn(), nw()>), dim3(chains), dim3(nw() * 64), 0, st, p);
    });
}

}  // namespace

size_t ssm_bwd_workspace_bytes(const SsmParams& p) { return bwd_space(p).bytes; }

int launch_ssm_bwd(const SsmParams& p, hipStream_t st) {
    if (p.in_bf16)
        p.y_bf16 ? launch<uint16_t, uint16_t>(p, st) : launch<uint16_t, float>(p, st);
    else
        p.y_bf16 ? launch<float, uint16_t>(p, st) : launch<float, float>(p, st);
    const int64_t n = static_cast<int64_t>(p.B) * p.T * p.G * 2 * p.N;
    hipLaunchKernelGGL(layer_ssm_bc_kernel, dim3(static_cast<unsigned>(tiles_of(n, 256) < 8192 ? tiles_of(n, 256) : 8192)),
                       dim3(256), 0, st, p);
    const float* tok = bwd_space(p).tok;
    launch_col_sums(ColSums{tok, p.B, p.N + 2, p.D, p.N, p.dA, p.dskip, p.ddt_bias}, st);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace layer
