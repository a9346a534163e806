// layer_ssm.hip -- the selective state space scan, forward and single step (layer_ssm.h).
//
// Where the chains of 64 channels are too few to fill the device the time axis is split into segments: a first kernel
// takes every segment but the last from a state of zeros to its end, which gives the segment's map h -> exp(A S) h + H
// (S the sum of its steps); the second starts each segment from the maps before it, composed in order.
//
// Bound by the vector units: a state and token takes a product, an exponential (two slots), B's product, the state's step
// and 1.75 operations for y, 4 cycles each for 64 channels; another 36 to 40 instructions per token and 64 channels
// are softplus, gate, conversions and the sum over waves.  D2048 N16 bf16: B8 T4096 (one segment) 292 to 320 us, the
// units 92 % busy, 0.54 GB of 100 us; B1 T65536 (32 segments) 865 us, of which the maps are 40 %, the units
// busy throughout.  From a wave for all 16 states and B and C in LDS, a tile at a time (1099 and 17400 us): segments, B and C by lane
// broadcast, quads 433 and 1430; addresses kept, steps four tokens ahead 395; inputs and outputs by waves of their own 390 and
// 920; loads two tiles ahead 320 and 870.  Two states to a lane and twice the waves: 332 and 1071 with one
// and 8 segments, against 317 and 1049.  Tiles behind a sequence's end are computed as the others are, with steps of zero:
// B7 T1531 D1001 N13 fp32 takes 144 us at full lengths, 117 at half of them and 89 with no token at all.
#include "layer_ssm.h"

namespace layer {
namespace {

constexpr int kTile = kSsmTile;
static_assert(kTile == 16 && kTile == kSsmSave, "a tile's B and C lie across 16 lanes, and a state is saved before each");
// The workspace: the segments' maps [chain][segment][state, sum of steps][64], of which the last is none: there lies the
// state before the chain, since state_out may be where it was read and the segments start in any order.
struct FwdSpace {
    float* maps;
    int segs;
    int64_t length;  // tokens per segment, whole tiles
    size_t bytes;
};
inline FwdSpace fwd_space(const SsmParams& p) {
    FwdSpace s;
    const SsmSplit k = ssm_split(p, false);
    s.maps = static_cast<float*>(p.ws);
    s.segs = k.segs, s.length = k.length;
    s.bytes = s.segs > 1 ? static_cast<size_t>(k.chains) * s.segs * (ssm_padded(p.N) + 1) * 64 * sizeof(float) : 0;
    return s;
}

// Segment k of a chain's maps.
template <int NP>
__device__ __forceinline__ float* map_of(const FwdSpace& ws, int chain, int k) {
    return ws.maps + (static_cast<int64_t>(chain) * ws.segs + k) * (NP + 1) * 64;
}

// The first NW waves walk over the states of a tile while kHelpers<NW> more form the next tile's delta and u, and y of
// the tile before from the waves' parts of it; they meet once a tile.
// MAPS: the segments' maps alone.
template <int NW>
constexpr int kHelpers = NW < 4 ? 2 : 4;

template <typename TIn, int SN, int NW, bool MAPS, bool VEC>
__global__ __launch_bounds__((NW + kHelpers<NW>) * 64) void layer_ssm_fwd_kernel(SsmParams p, FwdSpace ws) {
    constexpr int NP = SN * NW;                     // states, with those that stand for none
    constexpr int HT = kHelpers<NW> * 64;           // threads that take inputs and outputs
    constexpr int K = kTile * 16 / HT;              // quads of a tile that each of them takes
    constexpr bool kAcc = kAccurate<TIn>;
    constexpr int kIn = sizeof(TIn);
    __shared__ float du[2][kTile][2][64];           // delta and u
    __shared__ float part[MAPS ? 1 : 2][MAPS ? 1 : NW][MAPS ? 1 : kTile][64];  // a wave's part of y
    const int chains = p.B * p.G * ssm_blocks(p);
    const int chain = blockIdx.x % chains, seg = blockIdx.x / chains;
    const SsmPlace me = ssm_place(p, chain);
    const int t_begin = static_cast<int>(seg * ws.length);
    const int t_end = static_cast<int>(min(t_begin + ws.length, static_cast<int64_t>(p.T)));
    const int tiles = (t_end - t_begin + kTile - 1) / kTile;
    const int64_t token = static_cast<int64_t>(me.b) * p.T + t_begin;
    // tokens of tile i of the segment, and those that are no padding
    auto rows_of = [&](int i) { return min(kTile, t_end - t_begin - i * kTile); };
    auto valid_of = [&](int i) { return min(me.len - t_begin - i * kTile, rows_of(i)); };

    if (me.wave >= NW) {
        const SsmQuad mine = ssm_quad(p, me, chain, threadIdx.x - NW * 64);
        float bias[4], skip[4];
        quad_weights(p.dt_bias, mine, bias);
        quad_weights(p.skip, mine, skip);
        const int ey = p.y_bf16 ? 2 : 4;
        SsmStream xs(p.x, token, p.x_row, p.D, kIn), ds(p.dt, token, p.dt_row, p.D, kIn), zs(p.z, token, p.z_row, p.D, kIn);
        SsmStream ys(p.y, token, p.D, p.D, ey);
        const QuadOffsets<K> xo(mine, p.x_row, HT / 16, kIn), dO(mine, p.dt_row, HT / 16, kIn), zo(mine, p.z_row, HT / 16, kIn);
        const QuadOffsets<K> yo(mine, p.D, HT / 16, ey);
        struct Raw {
            Vec<TIn, 4> x[K], z[MAPS ? 1 : K], d[K];
        } raw[2];  // inputs on their way, of a tile with an even and one with an odd number
        struct Kept {
            Vec<TIn, 4> x[K], z[K];
        } kept[2];  // what y takes of them
        double steps[4] = {};  // the sums of this thread's tokens' steps
        auto fetch = [&](int i, auto odd) {
            if (i >= tiles) return;
            Raw& next = raw[odd()];
            const int valid = valid_of(i);
            const auto xr = xs.rows(valid), dr = ds.rows(valid), zr = zs.rows(valid);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                next.x[k] = load_quad<TIn, VEC, true>(xr, xo.at[k], mine.count);
                next.d[k] = load_quad<TIn, VEC, true>(dr, dO.at[k], mine.count);
                if constexpr (!MAPS) next.z[k] = load_quad<TIn, VEC, true>(zr, zo.at[k], mine.count);
            }
            xs.move(kTile), ds.move(kTile), zs.move(kTile);
        };
        // delta and u of tile i
        auto inputs = [&](int i, auto odd) {
            if (i >= tiles) return;
            const Raw& next = raw[odd()];
            const int valid = valid_of(i);
            float d[K][4];
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[k][e] = widen(next.d[k].e[e]) + bias[e];
            if (p.softplus) {
                float slope;
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) softplus_parts<kAcc>(d[k][e], d[k][e], slope);
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int row = mine.row + k * (HT / 16);
                float4 dv, uv;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (row >= valid) d[k][e] = 0.0f;
                    (&dv.x)[e] = d[k][e];
                    (&uv.x)[e] = d[k][e] * widen(next.x[k].e[e]);
                    if constexpr (MAPS) steps[e] += d[k][e];
                }
                *reinterpret_cast<float4*>(&du[odd()][row][0][mine.at]) = dv;
                *reinterpret_cast<float4*>(&du[odd()][row][1][mine.at]) = uv;
                if constexpr (!MAPS) kept[odd()].x[k] = next.x[k], kept[odd()].z[k] = next.z[k];
            }
        };
        // y of tile i
        auto outputs = [&](int i, auto odd) {
            const Kept& before = kept[odd()];
            float y[K][4];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int row = mine.row + k * (HT / 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[k][e] = skip[e] * widen(before.x[k].e[e]);
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(&part[odd()][w][row][mine.at]);
                    y[k][0] += v.x, y[k][1] += v.y, y[k][2] += v.z, y[k][3] += v.w;
                }
            }
            if (p.z) {
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float z = widen(before.z[k].e[e]);
                        float s, r;
                        sigmoid2<kAcc>(z, s, r);
                        y[k][e] *= z * s;
                    }
            }
            const int valid = valid_of(i);
            const auto yr = ys.rows(rows_of(i));
            ys.move(kTile);
            with_flag(p.y_bf16, [&](auto bf16) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int row = mine.row + k * (HT / 16);
                    if (row >= valid) y[k][0] = y[k][1] = y[k][2] = y[k][3] = 0.0f;
                    store_quad<VEC, bf16(), false>(yr, yo.at[k], mine.count, y[k]);
                }
            });
        };
        const std::integral_constant<int, 0> even;
        const std::integral_constant<int, 1> odd;
        fetch(0, even);
        fetch(1, odd);
        inputs(0, even);
        fetch(2, even);
        __syncthreads();
        auto turn = [&](int i, auto other) {
            if constexpr (!MAPS) {
                if (i > 0) outputs(i - 1, other);
            }
            inputs(i + 1, other);
            fetch(i + 3, other);
            __syncthreads();
        };
        for (int i = 0; i < tiles; i += 2) {
            turn(i, odd);
            if (i + 1 < tiles) turn(i + 1, even);
        }
        if constexpr (MAPS) {
            // the sum of the steps, by channel; the last tile's are done with
            double* sums = reinterpret_cast<double*>(&du[0][0][0][0]);  // [HT / 16][64]
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[mine.row * 64 + mine.at + e] = steps[e];
            __syncthreads();
        } else {
            (tiles - 1) & 1 ? outputs(tiles - 1, odd) : outputs(tiles - 1, even);
        }
        return;
    }

    const int wave = me.wave, l = me.l, c = me.c, n0 = wave * SN;
    float A[SN], h[SN];
    const int64_t state = (static_cast<int64_t>(me.b) * p.D + c) * p.N + n0;
#pragma unroll
    for (int n = 0; n < SN; ++n) {
        const bool on = n0 + n < p.N;
        A[n] = on ? ssm_decay(p.A[static_cast<int64_t>(c) * p.N + n0 + n]) : 0.0f;
        h[n] = on && p.state_in && (MAPS ? seg == 0 : ws.segs == 1) ? p.state_in[state + n] : 0.0f;
    }
    if constexpr (MAPS) {
        if (seg == 0) {
            float* m = map_of<NP>(ws, chain, ws.segs - 1) + l;
#pragma unroll
            for (int n = 0; n < SN; ++n) m[(n0 + n) * 64] = h[n], h[n] = 0.0f;
        }
    } else {
        if (ws.segs > 1) {
            const float* m = map_of<NP>(ws, chain, ws.segs - 1) + l;
#pragma unroll
            for (int n = 0; n < SN; ++n) h[n] = m[(n0 + n) * 64];
        }
        for (int k = 0; k < seg; ++k) {
            const float* m = map_of<NP>(ws, chain, k) + l;
            const float S = m[NP * 64];
#pragma unroll
            for (int n = 0; n < SN; ++n) {
                const float H = m[(n0 + n) * 64];
                h[n] = ssm_across(A[n], S, h[n], H);
            }
        }
    }
    SsmRegs<TIn, SN, VEC> nb[2], nc[2];  // on their way, of tiles with even and with odd numbers
#pragma unroll
    for (int k = 0; k < 2; ++k) nb[k].place(l, n0, p.N, p.b_row), nc[k].place(l, n0, p.N, p.c_row);
    SsmStream bs(static_cast<const TIn*>(p.Bm) + me.g * p.N, token, p.b_row, p.N, kIn);
    SsmStream cs(static_cast<const TIn*>(p.Cm) + me.g * p.N, token, p.c_row, p.N, kIn);
    auto fetch = [&](int i, auto odd) {
        if (i >= tiles) return;
        const int valid = valid_of(i);
        nb[odd()].load(bs.rows(valid));
        if constexpr (!MAPS) nc[odd()].load(cs.rows(valid));
        bs.move(kTile), cs.move(kTile);
    };
    const std::integral_constant<int, 0> even;
    const std::integral_constant<int, 1> odd;
    fetch(0, even);
    fetch(1, odd);
    bool dropped = false;
    __syncthreads();
    auto turn = [&](int i, auto odd) {
        const int t0 = t_begin + i * kTile, valid = valid_of(i);
        float B[SN], C[SN];
        nb[odd()].get(B);
        if constexpr (!MAPS) nc[odd()].get(C);
        fetch(i + 2, odd);
        const uint64_t cuts = ssm_cuts(p, me.b, t0, valid, l);
        dropped = dropped || cuts != 0;
        if (!MAPS && p.saved && me.live) {
            const int64_t of = tiles_of(p.T, kSsmSave);
            float* to = p.saved + (me.b * of + t0 / kSsmSave) * p.N * p.D + c;
#pragma unroll
            for (int n = 0; n < SN; ++n)
                if (n0 + n < p.N) to[static_cast<int64_t>(n0 + n) * p.D] = cuts & 1 ? 0.0f : h[n];
        }
        with_flag(cuts != 0, [&](auto with_cuts) {
            const float(*from)[2][64] = du[odd()];
            float dn[2][4], un[2][4];  // steps and inputs of four tokens, and of the next four
#pragma unroll
            for (int j = 0; j < 4; ++j) dn[0][j] = from[j][0][l], un[0][j] = from[j][1][l];
            each<kTile>([&](auto tc) {
                constexpr int t = tc();
                if (with_cuts() && (cuts >> t & 1)) {
#pragma unroll
                    for (int n = 0; n < SN; ++n) h[n] = 0.0f;
                }
                if constexpr (t % 4 == 0 && t + 4 < kTile) {
                    constexpr int to = (t / 4 + 1) % 2;
#pragma unroll
                    for (int j = 0; j < 4; ++j) dn[to][j] = from[t + 4 + j][0][l], un[to][j] = from[t + 4 + j][1][l];
                }
                const float step = dn[t / 4 % 2][t % 4], u = un[t / 4 % 2][t % 4];
                float y[SN];
#pragma unroll
                for (int n = 0; n < SN; ++n) {
                    h[n] = fmaf(__builtin_amdgcn_exp2f(step * A[n]), h[n], bcast<t>(B[n]) * u);
                    if constexpr (!MAPS) y[n] = bcast<t>(C[n]) * h[n];
                }
                if constexpr (!MAPS) {
#pragma unroll
                    for (int k = 1; k < SN; k *= 2)
#pragma unroll
                        for (int n = 0; n < SN; n += 2 * k) y[n] += y[n + k];
                    part[odd()][wave][t][l] = y[0];
                }
            });
        });
        __syncthreads();
    };
    for (int i = 0; i < tiles; i += 2) {
        turn(i, even);
        if (i + 1 < tiles) turn(i + 1, odd);
    }
    if constexpr (MAPS) {
        float* m = map_of<NP>(ws, chain, seg) + l;
#pragma unroll
        for (int n = 0; n < SN; ++n) m[(n0 + n) * 64] = h[n];
        __syncthreads();
        if (wave == 0) {
            const double* sums = reinterpret_cast<const double*>(&du[0][0][0][0]);
            double s = 0.0;
            for (int j = 0; j < HT / 16; ++j) s += sums[j * 64 + l];
            m[NP * 64] = ssm_steps(s, dropped);
        }
    } else if (p.state_out && me.live && seg == ws.segs - 1) {
#pragma unroll
        for (int n = 0; n < SN; ++n)
            if (n0 + n < p.N) p.state_out[state + n] = h[n];
    }
}

// One token: L lanes to a channel, four states each, for NB sequences at a time; state_out may be state_in (each value
// is read, then written, by one lane).  Bound by HBM: B256 D4096 N16 moves 142 MB in 24 us (one sequence at a time and
// 64-bit divisions for its place: 43); four sequences from 16 on, one below, where workgroups are few.
template <typename TIn, int L, int NB, bool VEC>
__global__ __launch_bounds__(256) void layer_ssm_step_kernel(SsmParams p) {
    const int c = static_cast<int>(blockIdx.x) * (256 / L) + threadIdx.x / L, n0 = threadIdx.x % L * 4;
    if (c >= p.D) return;  // (with its whole group of L lanes)
    const int left = p.N - n0;  // states from n0 on: none in the last lanes of some widths
    const int g = c / (p.D / p.G);
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, skip = p.skip ? p.skip[c] : 0.0f;
    // four values at p, zeros past the last state
    auto quad = [&](const auto* from) {
        using T = std::remove_cv_t<std::remove_reference_t<decltype(*from)>>;
        Vec<T, 4> v = {};
        if (VEC) {
            if (left > 0) v = load_vec<T, 4>(from, 0);
        } else {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (n < left) v.e[n] = from[n];
        }
        return v;
    };
    const Vec<float, 4> A = quad(p.A + static_cast<int64_t>(c) * p.N + n0);
    for (int b0 = blockIdx.y * NB; b0 < p.B; b0 += gridDim.y * NB) {
        Vec<float, 4> h[NB];
        Vec<TIn, 4> B[NB], C[NB];
        TIn x[NB], dt[NB], z[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int64_t b = min(b0 + i, p.B - 1);  // a sequence past the last: another's values, not stored
            h[i] = quad(p.state_in + (b * p.D + c) * p.N + n0);
            B[i] = quad(static_cast<const TIn*>(p.Bm) + b * p.b_row + g * p.N + n0);
            C[i] = quad(static_cast<const TIn*>(p.Cm) + b * p.c_row + g * p.N + n0);
            x[i] = static_cast<const TIn*>(p.x)[b * p.x_row + c];
            dt[i] = static_cast<const TIn*>(p.dt)[b * p.dt_row + c];
            if (p.z) z[i] = static_cast<const TIn*>(p.z)[b * p.z_row + c];
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            float d = widen(dt[i]) + bias, slope;
            if (p.softplus) softplus_parts<kAccurate<TIn>>(d, d, slope);
            const float u = d * widen(x[i]);
            float y[1] = {0.0f}, o[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                o[n] = fmaf(__builtin_amdgcn_exp2f(d * ssm_decay(A.e[n])), h[i].e[n], u * widen(B[i].e[n]));
                if (n < left) y[0] = fmaf(widen(C[i].e[n]), o[n], y[0]);
            }
            y[0] = osr::group_sum<L>(y[0]);
            if (b0 + i >= p.B) continue;
            const int64_t at = static_cast<int64_t>(b0 + i) * p.D + c;
            float* to = p.state_out + at * p.N + n0;
            if (VEC) {
                if (left > 0) store_vec<4>(to, 0, o, false);
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    if (n < left) to[n] = o[n];
            }
            if (n0 != 0) continue;
            y[0] = fmaf(skip, widen(x[i]), y[0]);
            if (p.z) {
                const float zv = widen(z[i]);
                float s, r;
                sigmoid2<kAccurate<TIn>>(zv, s, r);
                y[0] *= zv * s;
            }
            store_vec<1>(p.y, at, y, p.y_bf16);
        }
    }
}

template <typename TIn>
void launch_fwd(const SsmParams& p, hipStream_t st) {
    const FwdSpace ws = fwd_space(p);
    with_states(p.N, [&](auto sn, auto nw) {
        const unsigned chains = static_cast<unsigned>(p.B) * p.G * tiles_of(p.D / p.G, 64);
        auto go = [&](auto vec) {
            const dim3 block((nw() + kHelpers<nw()>) * 64);
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
    bool vec = p.N % 4 == 0 && p.b_row % 4 == 0 && p.c_row % 4 == 0;
    for (const float* q : {p.state_in, static_cast<const float*>(p.state_out), p.A})
        vec = vec && reinterpret_cast<uintptr_t>(q) % 16 == 0;
    for (const void* q : {p.Bm, p.Cm}) vec = vec && reinterpret_cast<uintptr_t>(q) % (4 * sizeof(TIn)) == 0;
    auto go = [&](auto L, auto nb) {
        const int64_t rows = tiles_of(p.B, nb());
        const dim3 grid(static_cast<unsigned>(tiles_of(static_cast<int64_t>(p.D) * L(), 256)),
                        static_cast<unsigned>(rows < 32768 ? rows : 32768));
        if (vec)
            hipLaunchKernelGGL((layer_ssm_step_kernel<TIn, L(), nb(), true>), grid, dim3(256), 0, st, p);
        else
            hipLaunchKernelGGL((layer_ssm_step_kernel<TIn, L(), nb(), false>), grid, dim3(256), 0, st, p);
    };
    auto by_batch = [&](auto L) {
        p.B >= 16 ? go(L, std::integral_constant<int, 4>()) : go(L, std::integral_constant<int, 1>());
    };
    if (p.N <= 4) by_batch(std::integral_constant<int, 1>());
    else if (p.N <= 8) by_batch(std::integral_constant<int, 2>());
    else if (p.N <= 16) by_batch(std::integral_constant<int, 4>());
    else if (p.N <= 32) by_batch(std::integral_constant<int, 8>());
    else by_batch(std::integral_constant<int, 16>());
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
