// layer_ssm_bwd.hip -- the state space scan's gradient around its main kernel (layer_ssm_bwd.h): the segments' maps in
// front of it, the sums behind it.
#include "layer_ssm_bwd.h"

namespace layer {
namespace ssm_bwd {
namespace {

// The maps of the parts of all segments but the first: from a gradient of zeros behind each to the one in front of it.
template <typename TIn, typename TDy, int SN, int NW, bool VEC>
__global__ __launch_bounds__((NW + (NW < 4 ? 2 : 4)) * 64) void layer_ssm_bwd_maps_kernel(SsmParams p, BwdSpace ws) {
    constexpr int HT = (NW < 4 ? 2 : 4) * 64, K = kTile * 16 / HT, kStep = HT / 16, kIn = sizeof(TIn), NP = SN * NW;
    constexpr bool kAcc = kAccurate<TIn>;
    __shared__ float in[2][kTile][2][64];  // delta, g
    const int chains = p.B * p.G * ssm_blocks(p);
    const SsmPlace me = ssm_place(p, blockIdx.x % chains);
    const Segment s = segment_of(p, ws.per + blockIdx.x / chains, ws.part_length, me.len, chains);
    const int64_t token = static_cast<int64_t>(me.b) * p.T + s.t0(0);
    const std::integral_constant<int, 0> even;
    const std::integral_constant<int, 1> odd;
    if (me.wave >= NW) {
        const SsmQuad mine = ssm_quad(p, me, s.chain, threadIdx.x - NW * 64);
        float bias[4];
        quad_weights(p.dt_bias, mine, bias);
        SsmStream ds(p.dt, token, p.dt_row, p.D, kIn), zs(p.z, token, p.z_row, p.D, kIn), gs(p.dy, token, p.D, p.D, sizeof(TDy));
        const QuadOffsets<K> dO(mine, p.dt_row, kStep, kIn), zo(mine, p.z_row, kStep, kIn), go(mine, p.D, kStep, sizeof(TDy));
        struct Raw {
            Vec<TIn, 4> d[K], z[K];
            Vec<TDy, 4> dy[K];
        } raw[2];
        double steps[4] = {};
        auto fetch = [&](int i, auto b) {
            if (i >= s.tiles) return;
            const int valid = s.valid(i);
            const auto dr = ds.rows(valid), zr = zs.rows(valid), gr = gs.rows(valid);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                raw[b()].d[k] = load_quad<TIn, VEC, true>(dr, dO.at[k], mine.count);
                raw[b()].z[k] = load_quad<TIn, VEC, true>(zr, zo.at[k], mine.count);
                raw[b()].dy[k] = load_quad<TDy, VEC, true>(gr, go.at[k], mine.count);
            }
            ds.move(-kTile), zs.move(-kTile), gs.move(-kTile);
        };
        auto inputs = [&](int i, auto b) {
            if (i >= s.tiles) return;
            const Raw& next = raw[b()];
            const int valid = s.valid(i);
            float d[K][4], g[K][4];
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[k][e] = widen(next.d[k].e[e]) + bias[e], g[k][e] = widen(next.dy[k].e[e]);
            if (p.softplus) {
                float slope;
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) softplus_parts<kAcc>(d[k][e], d[k][e], slope);
            }
            if (p.z) {
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float z = widen(next.z[k].e[e]);
                        float sg, r;
                        sigmoid2<kAcc>(z, sg, r);
                        g[k][e] *= z * sg;
                    }
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int row = mine.row + k * kStep;
                float4 dv, gv;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (row >= valid) d[k][e] = 0.0f;
                    (&dv.x)[e] = d[k][e];
                    (&gv.x)[e] = g[k][e];
                    steps[e] += d[k][e];
                }
                *reinterpret_cast<float4*>(&in[b()][row][0][mine.at]) = dv;
                *reinterpret_cast<float4*>(&in[b()][row][1][mine.at]) = gv;
            }
        };
        fetch(0, even);
        fetch(1, odd);
        inputs(0, even);
        fetch(2, even);
        __syncthreads();
        for (int i = 0; i < s.tiles; i += 2) {
            inputs(i + 1, odd);
            fetch(i + 3, odd);
            __syncthreads();
            if (i + 1 >= s.tiles) break;
            inputs(i + 2, even);
            fetch(i + 4, even);
            __syncthreads();
        }
        double* sums = reinterpret_cast<double*>(&in[0][0][0][0]);  // [HT / 16][64]
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[mine.row * 64 + mine.at + e] = steps[e];
        __syncthreads();
        return;
    }
    const int l = me.l, n0 = me.wave * SN;
    float A[SN], r[SN] = {};
#pragma unroll
    for (int n = 0; n < SN; ++n)
        A[n] = n0 + n < p.N && me.live ? ssm_decay(p.A[static_cast<int64_t>(me.c) * p.N + n0 + n]) : 0.0f;
    SsmRegs<TIn, SN, VEC> nc[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) nc[k].place(l, n0, p.N, p.c_row);
    SsmStream cs(static_cast<const TIn*>(p.Cm) + me.g * p.N, token, p.c_row, p.N, kIn);
    auto fetch = [&](int i, auto b) {
        if (i >= s.tiles) return;
        nc[b()].load(cs.rows(s.valid(i)));
        cs.move(-kTile);
    };
    bool dropped = false;
    auto walk = [&](int i, auto b) {
        const int valid = s.valid(i);
        float C[SN];
        nc[b()].get(C);
        fetch(i + 2, b);
        if (valid <= 0) return;
        const uint64_t cuts = ssm_cuts(p, me.b, s.t0(i), valid, l);
        dropped = dropped || cuts != 0;
        with_flag(cuts != 0 || valid < kTile, [&](auto partly) {
            each<kTile>([&](auto tc) {
                constexpr int t = kTile - 1 - tc();
                if (partly() && t >= valid) return;
                const float d = in[b()][t][0][l], g = in[b()][t][1][l];
#pragma unroll
                for (int n = 0; n < SN; ++n) {
                    r[n] = __builtin_amdgcn_exp2f(d * A[n]) * (r[n] + bcast<t>(C[n]) * g);
                    if (partly() && (cuts >> t & 1)) r[n] = 0.0f;
                }
            });
        });
    };
    fetch(0, even);
    fetch(1, odd);
    __syncthreads();
    for (int i = 0; i < s.tiles; i += 2) {
        walk(i, even);
        __syncthreads();
        if (i + 1 >= s.tiles) break;
        walk(i + 1, odd);
        __syncthreads();
    }
    float* m = map_of<NP>(ws, s.chain, s.seg) + l;
#pragma unroll
    for (int n = 0; n < SN; ++n) m[(n0 + n) * 64] = r[n];
    __syncthreads();
    if (me.wave == 0) {
        const double* sums = reinterpret_cast<const double*>(&in[0][0][0][0]);
        double a = 0.0;
        for (int j = 0; j < HT / 16; ++j) a += sums[j * 64 + l];
        m[NP * 64] = ssm_steps(a, dropped);
    }
}

// dB and dC: the blocks' sums added in order.  One thread per value [B T][G][2][N].
__global__ __launch_bounds__(256) void layer_ssm_bc_kernel(SsmParams p, const float* bc) {
    const int64_t n = static_cast<int64_t>(p.B) * p.T * p.G * 2 * p.N;
    const int blocks = (p.D / p.G + 63) / 64;
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
void launch_maps(const SsmParams& p, const BwdSpace& ws, hipStream_t st) {
    with_states(p.N, [&](auto sn, auto nw) {
        const unsigned chains = static_cast<unsigned>(p.B) * p.G * tiles_of(p.D / p.G, 64);
        auto go = [&](auto vec) {
            hipLaunchKernelGGL((layer_ssm_bwd_maps_kernel<TIn, TDy, sn(), nw(), vec()>), dim3(chains * (ws.parts - ws.per)),
                               dim3((nw() + (nw() < 4 ? 2 : 4)) * 64), 0, st, p, ws);
        };
        ssm_vec(p) ? go(std::true_type()) : go(std::false_type());
    });
}

}  // namespace
}  // namespace ssm_bwd

size_t ssm_bwd_workspace_bytes(const SsmParams& p) { return ssm_bwd::bwd_space(p).bytes; }

int launch_ssm_bwd(const SsmParams& p, hipStream_t st) {
    using namespace ssm_bwd;
    const BwdSpace ws = bwd_space(p);
    if (ws.segs > 1) {
        if (p.in_bf16)
            p.y_bf16 ? launch_maps<uint16_t, uint16_t>(p, ws, st) : launch_maps<uint16_t, float>(p, ws, st);
        else
            p.y_bf16 ? launch_maps<float, uint16_t>(p, ws, st) : launch_maps<float, float>(p, ws, st);
    }
    p.in_bf16 ? launch_bf16(p, ws, st) : launch_f32(p, ws, st);
    const int64_t n = static_cast<int64_t>(p.B) * p.T * p.G * 2 * p.N;
    hipLaunchKernelGGL(layer_ssm_bc_kernel, dim3(static_cast<unsigned>(tiles_of(n, 256) < 8192 ? tiles_of(n, 256) : 8192)),
                       dim3(256), 0, st, p, ws.bc);
    launch_col_sums(ColSums{ws.tok, p.B * ws.segs, p.N + 2, p.D, p.N, p.dA, p.dskip, p.ddt_bias}, st);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace layer
