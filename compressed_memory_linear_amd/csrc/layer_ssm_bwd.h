// layer_ssm_bwd.h -- gradient of the selective state space scan (layer_ssm.h).
//
// With g = dy phi(z), phi(z) = z sigmoid(z), a_t = exp(delta_t A) and l_t the gradient that reaches h_t,
//     l_t = C_t g_t + a_{t+1} l_{t+1}   (the last token's taking dstate_out in),
//     dC_t = sum_c g_t h_t,   dB_t = sum_c l_t u_t   over the channels of a group,
//     du_t = sum_n l_t B_t,   r_t = a_t l_t,   q_t = r_t h_{t-1},
//     ddelta_t = sum_n q_t A + du_t x_t,   dA = sum_t q_t delta_t,   dstate_in = r_0,
//     dx = du delta + skip g,   ddt = ddelta softplus'(dt + bias),   dz = dy (C h + skip x) phi'(z).
// A workgroup walks its chain backwards in tiles of kSsmSave tokens: it takes the states of the tile again from the one
// that the forward saved before it, keeps them with their decays in registers, and then runs backwards over them.
// Where the chains are few the time axis is split as in the forward: a segment maps the gradient that
// enters it from behind to the one that leaves it in front, r -> exp(A S) r + R, with the same S as the
// forward's.  The sums over channels go to the workspace, a block of 64 channels each, and are added by
// another kernel in a fixed order (no atomics: reruns agree bit for bit); so are the sums over tokens.
//
// Bound by the vector units, one wave that walks over states and one that takes inputs and outputs to each (256
// registers; 127 KB of LDS at 16 states): B4 T4096 D2048 N16 bf16, 4 segments, 560 to 640 us, the units 75 % busy.  Of about 22
// instructions per state and token six take the state again, nine are the gradients' and five the sums over
// channels, which permlane swaps of 8 cycles make 94 of 350 cycles per token and four states.  The maps in front 95 us, the
// kernels behind 14 and 8.  (The whole training step: 4825 us with one wave's sums over 64 lanes one by one, one
// segment and nothing ahead; 945 so.)  Past 16 states, where the
// threads that walk take inputs too, a tile's inputs on their way lie in registers across the walk, which spill: 32 to 76
// of them up to 32 states, 91 to 145 up to 64 (4 to 18 at 16).  64 states (B3 T777 D514 fp32): 239 us, with the decays held
// too 334, in one part of 16 tokens 400.
#pragma once

#include "layer_ssm.h"

namespace layer {

namespace ssm_bwd {
constexpr int kTile = kSsmSave;
static_assert(kTile == 16, "a tile's B and C lie across 16 lanes");

// The workspace: sums of B's and C's gradients [block][B T][G][2][N], those over tokens [B][segment][N + 2][D] (dA,
// dskip, ddt_bias), the maps [chain][part of a segment][state, sum of steps][64].  Those are formed by a kernel of small
// workgroups, for which the main kernel's segments are too few: a segment has several of them.
struct BwdSpace {
    float *bc, *tok, *maps;
    int segs, parts, per;  // segments of a chain, parts of all of them, parts of a segment
    int64_t length;        // tokens per segment, whole tiles
    int64_t part_length;
    size_t bytes;
};
inline BwdSpace bwd_space(const SsmParams& p) {
    BwdSpace s;
    const SsmSplit k = ssm_split(p, true);
    s.segs = k.segs, s.length = k.length;
    s.per = k.parts, s.part_length = k.length / k.parts;
    s.parts = static_cast<int>((p.T + s.part_length - 1) / s.part_length);
    const int64_t nbc = tiles_of(p.D / p.G, 64) * p.B * p.T * p.G * 2 * p.N;
    const int64_t ntok = static_cast<int64_t>(p.B) * s.segs * (p.N + 2) * p.D;
    const int64_t nmap = s.segs > 1 ? k.chains * s.parts * (ssm_padded(p.N) + 1) * 64 : 0;
    s.bc = static_cast<float*>(p.ws);
    s.tok = s.bc + nbc;
    s.maps = s.tok + ntok;
    s.bytes = static_cast<size_t>(nbc + ntok + nmap) * sizeof(float);
    return s;
}
template <int NP>
__device__ __forceinline__ float* map_of(const BwdSpace& ws, int chain, int k) {
    return ws.maps + (static_cast<int64_t>(chain) * ws.parts + k) * (NP + 1) * 64;
}

// Sixteen sums over the lanes at once, each step halving the registers: 35 operations where one by one they take 96.
// Every lane of quad k of row r is left with the sum of v[4 i + j], i = {2, 0, 3, 1}[k], j = {0, 2, 1, 3}[r].
__device__ __forceinline__ int sum16_index(int l) {
    const int k = l >> 2 & 3, r = l >> 4;
    return 4 * (k == 0 ? 2 : k == 1 ? 0 : k == 2 ? 3 : 1) + (r == 0 ? 0 : r == 1 ? 2 : r == 2 ? 1 : 3);
}
__device__ __forceinline__ float sum16(const float (&v)[16], int l) {
    float w[8], x[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]), false, false);
        w[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(w[2 * i]), __float_as_uint(w[2 * i + 1]), false, false);
        x[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    constexpr int kRor = 0x120;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] += osr::dpp_mov<kRor + 8>(x[i]);
    const float a = l & 8 ? x[1] : x[0], b = l & 8 ? x[3] : x[2];
    const float c = a + osr::dpp_mov<kRor + 4>(a), d = b + osr::dpp_mov<kRor + 12>(b);  // in every lane, then chosen
    float s = l & 4 ? c : d;
    s += osr::dpp_mov<osr::DPP_QUAD_1032>(s);
    return s + osr::dpp_mov<osr::DPP_QUAD_2301>(s);
}

// Up to four waves of states are joined by others that take the inputs and outputs, a tile ahead and one behind, as in
// the forward; eight, whose LDS holds one tile, take them themselves, in turns.
template <int NW>
struct Shape {
    static constexpr bool kApart = NW <= 4;
    static constexpr int kBuf = kApart ? 2 : 1;
    static constexpr int kHT = NW < 4 ? 128 : 256;  // threads that take inputs and outputs
    static constexpr int kNT = NW * 64 + (kApart ? kHT : 0);
    static constexpr int K = kTile * 16 / kHT;      // quads of a tile that each of them takes
};
template <int SN, int NW>
struct Shared {
    float in[Shape<NW>::kBuf][kTile][3][64];        // delta, u, g
    float part[Shape<NW>::kBuf][NW][kTile][2][64];  // du and ddelta of a wave's states
    float y[Shape<NW>::kBuf][NW][kTile][64];        // its part of C h
    float sums[Shape<NW>::kBuf][kTile][2 * SN * NW];  // dB and dC over the block
    // what the outputs take of the inputs (x, z, dy, softplus'), where the same threads walk over states in between
    float keep[Shape<NW>::kApart ? 1 : 4][Shape<NW>::kApart ? 1 : kTile][64];
};

// A segment of a chain, and its tiles from the last (0) to the first.
struct Segment {
    int chain, seg, t_begin, t_end, tiles, len, T;
    __device__ __forceinline__ int t0(int i) const { return t_begin + (tiles - 1 - i) * kTile; }
    __device__ __forceinline__ int rows(int i) const { return min(kTile, t_end - t0(i)); }
    __device__ __forceinline__ int valid(int i) const { return min(len - t0(i), rows(i)); }
};
__device__ __forceinline__ Segment segment_of(const SsmParams& p, int seg, int64_t length, int len, int chains) {
    Segment s;
    s.chain = blockIdx.x % chains, s.seg = seg;
    s.t_begin = static_cast<int>(seg * length);
    s.t_end = static_cast<int>(min(s.t_begin + length, static_cast<int64_t>(p.T)));
    s.tiles = (s.t_end - s.t_begin + kTile - 1) / kTile;
    s.len = len, s.T = p.T;
    return s;
}

// The threads that take the inputs of a tile and form its outputs.
template <typename TIn, typename TDy, int SN, int NW, bool VEC>
struct Taker {
    using Sh = Shape<NW>;
    static constexpr int K = Sh::K, kStep = Sh::kHT / 16, kIn = sizeof(TIn);
    static constexpr bool kAcc = kAccurate<TIn>;
    const SsmParams& p;
    const BwdSpace& ws;
    Shared<SN, NW>& sh;
    const Segment& s;
    const SsmPlace& me;
    SsmQuad mine;
    int id, eg, blocks;
    float bias[4], skip[4], dskip[4] = {}, dbias[4] = {};
    SsmStream xs, ds, zs, gs, dxs, dds, dzs;
    QuadOffsets<K> xo, dO, zo, go, oo;
    struct Raw {
        Vec<TIn, 4> x[K], d[K], z[K];
        Vec<TDy, 4> dy[K];
    } raw[Sh::kBuf];
    struct Kept {
        Vec<TIn, 4> x[K], z[K];
        Vec<TDy, 4> dy[K];
        float d[K][4], slope[K][4];
    } kept[Sh::kBuf];

    __device__ __forceinline__ Taker(const SsmParams& p_, const BwdSpace& ws_, Shared<SN, NW>& sh_, const Segment& s_,
                                     const SsmPlace& me_, int id_)
        : p(p_), ws(ws_), sh(sh_), s(s_), me(me_), mine(ssm_quad(p_, me_, s_.chain, id_)), id(id_),
          eg(p_.grad_bf16 ? 2 : 4), blocks(ssm_blocks(p_)),
          xs(p_.x, token(), p_.x_row, p_.D, kIn), ds(p_.dt, token(), p_.dt_row, p_.D, kIn),
          zs(p_.z, token(), p_.z_row, p_.D, kIn), gs(p_.dy, token(), p_.D, p_.D, sizeof(TDy)),
          dxs(p_.dx, token(), p_.D, p_.D, eg), dds(p_.ddt, token(), p_.D, p_.D, eg), dzs(p_.dz, token(), p_.D, p_.D, eg),
          xo(mine, p_.x_row, kStep, kIn), dO(mine, p_.dt_row, kStep, kIn), zo(mine, p_.z_row, kStep, kIn),
          go(mine, p_.D, kStep, sizeof(TDy)), oo(mine, p_.D, kStep, eg) {
        quad_weights(p.dt_bias, mine, bias);
        quad_weights(p.skip, mine, skip);
    }
    __device__ __forceinline__ int64_t token() const { return static_cast<int64_t>(me.b) * p.T + s.t0(0); }

    template <int B>
    __device__ __forceinline__ void fetch(int i) {
        if (i >= s.tiles) return;
        Raw& next = raw[B];
        const int valid = s.valid(i);
        const auto xr = xs.rows(valid), dr = ds.rows(valid), zr = zs.rows(valid), gr = gs.rows(valid);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            next.x[k] = load_quad<TIn, VEC, true>(xr, xo.at[k], mine.count);
            next.d[k] = load_quad<TIn, VEC, true>(dr, dO.at[k], mine.count);
            next.z[k] = load_quad<TIn, VEC, true>(zr, zo.at[k], mine.count);
            next.dy[k] = load_quad<TDy, VEC, true>(gr, go.at[k], mine.count);
        }
        xs.move(-kTile), ds.move(-kTile), zs.move(-kTile), gs.move(-kTile);
    }
    // delta, u and g of tile i
    template <int B>
    __device__ __forceinline__ void inputs(int i) {
        if (i >= s.tiles) return;
        const Raw& next = raw[B];
        const int valid = s.valid(i);
        float d[K][4], slope[K][4], g[K][4];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d[k][e] = widen(next.d[k].e[e]) + bias[e];
                slope[k][e] = 1.0f;
                g[k][e] = widen(next.dy[k].e[e]);
            }
        if (p.softplus) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) softplus_parts<kAcc>(d[k][e], d[k][e], slope[k][e]);
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
            float4 dv, uv, gv;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (row >= valid) d[k][e] = 0.0f;
                (&dv.x)[e] = d[k][e];
                (&uv.x)[e] = d[k][e] * widen(next.x[k].e[e]);
                (&gv.x)[e] = g[k][e];
            }
            *reinterpret_cast<float4*>(&sh.in[B][row][0][mine.at]) = dv;
            *reinterpret_cast<float4*>(&sh.in[B][row][1][mine.at]) = uv;
            *reinterpret_cast<float4*>(&sh.in[B][row][2][mine.at]) = gv;
            if constexpr (Sh::kApart) {
                Kept& keep = kept[B];
                keep.x[k] = next.x[k], keep.z[k] = next.z[k], keep.dy[k] = next.dy[k];
#pragma unroll
                for (int e = 0; e < 4; ++e) keep.d[k][e] = d[k][e], keep.slope[k][e] = slope[k][e];
            } else {
                float4 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    (&v[0].x)[e] = widen(next.x[k].e[e]), (&v[1].x)[e] = widen(next.z[k].e[e]);
                    (&v[2].x)[e] = widen(next.dy[k].e[e]), (&v[3].x)[e] = slope[k][e];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<float4*>(&sh.keep[j][row][mine.at]) = v[j];
            }
        }
    }
    // what inputs() kept for element e of quad k: x, z, dy, delta, softplus'
    struct Was {
        float x, z, dy, d, slope;
    };
    template <int B>
    __device__ __forceinline__ Was was(int k, int e) const {
        if constexpr (Sh::kApart) {
            const Kept& keep = kept[B];
            return Was{widen(keep.x[k].e[e]), widen(keep.z[k].e[e]), widen(keep.dy[k].e[e]), keep.d[k][e], keep.slope[k][e]};
        } else {
            const int row = mine.row + k * kStep, at = mine.at + e;
            return Was{sh.keep[0][row][at], sh.keep[1][row][at], sh.keep[2][row][at], sh.in[B][row][0][at], sh.keep[3][row][at]};
        }
    }
    // the gradients of tile i, and the block's sums of B's and C's
    template <int B>
    __device__ __forceinline__ void outputs(int i) {
        const int valid = s.valid(i), rows = s.rows(i);
        float dx[K][4], ddt[K][4], dz[K][4];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int row = mine.row + k * kStep;
            float du[4] = {}, q[4] = {}, y[4] = {};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float4 a = *reinterpret_cast<const float4*>(&sh.part[B][w][row][0][mine.at]);
                const float4 b = *reinterpret_cast<const float4*>(&sh.part[B][w][row][1][mine.at]);
                du[0] += a.x, du[1] += a.y, du[2] += a.z, du[3] += a.w;
                q[0] += b.x, q[1] += b.y, q[2] += b.z, q[3] += b.w;
            }
            if (p.z) {
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(&sh.y[B][w][row][mine.at]);
                    y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
                }
            }
            const bool on = row < valid;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Was in = was<B>(k, e);
                const float x = in.x, dy = in.dy;
                float g = dy;
                dz[k][e] = 0.0f;
                if (p.z) {
                    const float z = in.z;
                    float sg, r;
                    sigmoid2<kAcc>(z, sg, r);
                    g *= z * sg;
                    dz[k][e] = dy * fmaf(skip[e], x, y[e]) * (sg * fmaf(z, r, 1.0f));
                }
                dx[k][e] = fmaf(du[e], in.d, skip[e] * g);
                ddt[k][e] = fmaf(du[e], x, q[e] * kLn2) * in.slope;
                if (!on) dx[k][e] = ddt[k][e] = dz[k][e] = 0.0f;
                if (on) {
                    dskip[e] = fmaf(g, x, dskip[e]);
                    dbias[e] += ddt[k][e];
                }
            }
        }
        const auto dxr = dxs.rows(rows), ddr = dds.rows(rows), dzr = dzs.rows(rows);
        dxs.move(-kTile), dds.move(-kTile), dzs.move(-kTile);
        with_flag(p.grad_bf16, [&](auto bf16) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                store_quad<VEC, bf16(), true>(dxr, oo.at[k], mine.count, dx[k]);
                store_quad<VEC, bf16(), true>(ddr, oo.at[k], mine.count, ddt[k]);
                if (p.z) store_quad<VEC, bf16(), true>(dzr, oo.at[k], mine.count, dz[k]);
            }
        });
        constexpr int NP = SN * NW;
        const int64_t row = (static_cast<int64_t>(s.chain % blocks) * p.B + me.b) * p.T + s.t0(i);
        float* to = ws.bc + (row * p.G + me.g) * 2 * p.N;
        for (int j = id; j < rows * 2 * NP; j += Sh::kHT) {
            const int t = j / (2 * NP), k = j % (2 * NP), n = k % NP;
            if (n < p.N) to[static_cast<int64_t>(t) * p.G * 2 * p.N + (k < NP ? n : p.N + n)] = sh.sums[B][t][k];
        }
    }
};

// A wave's states.
template <typename TIn, int SN, int NW, bool VEC>
struct Walker {
    using Sh = Shape<NW>;
    static constexpr int NP = SN * NW;
    static constexpr bool kHold = SN == 4;   // the decays too
    static constexpr int kPart = 64 / SN;    // tokens whose states registers hold
    static constexpr int kPair = 8 / SN;     // tokens whose sums over the channels are taken together
    const SsmParams& p;
    Shared<SN, NW>& sh;
    const Segment& s;
    const SsmPlace& me;
    int wave, l, c, n0, sum_at;
    float A[SN], lam[SN], dA[SN] = {};
    SsmRegs<TIn, SN, VEC> nb[Sh::kBuf], nc[Sh::kBuf];
    float saved[Sh::kBuf][SN];
    SsmStream bs, cs;
    const float* from;  // the state before the tile that is fetched next
    int64_t state;

    __device__ __forceinline__ Walker(const SsmParams& p_, const BwdSpace& ws, Shared<SN, NW>& sh_, const Segment& s_,
                                      const SsmPlace& me_)
        : p(p_), sh(sh_), s(s_), me(me_), wave(me_.wave), l(me_.l), c(me_.c), n0(me_.wave * SN),
          bs(static_cast<const TIn*>(p_.Bm) + me_.g * p_.N, token(), p_.b_row, p_.N, sizeof(TIn)),
          cs(static_cast<const TIn*>(p_.Cm) + me_.g * p_.N, token(), p_.c_row, p_.N, sizeof(TIn)) {
        state = (static_cast<int64_t>(me.b) * p.D + c) * p.N + n0;
        // the value of sum16 that this lane is left with: of the pair's first or second token, of dB or dC, of a state
        const int v = sum16_index(l);
        sum_at = -(v / (2 * SN)) * 2 * NP + v / SN % 2 * NP + n0 + v % SN;
#pragma unroll
        for (int n = 0; n < SN; ++n) {
            // (lanes past the last channel hold zeros throughout, since the sums over channels take them in)
            const bool on = n0 + n < p.N && me.live;
            A[n] = on ? ssm_decay(p.A[static_cast<int64_t>(c) * p.N + n0 + n]) : 0.0f;
            lam[n] = on && p.dstate_out ? p.dstate_out[state + n] : 0.0f;
        }
        for (int k = ws.parts - 1; k >= (s.seg + 1) * ws.per; --k) {
            const float* m = map_of<NP>(ws, s.chain, k) + l;
            const float S = m[NP * 64];
#pragma unroll
            for (int n = 0; n < SN; ++n) {
                const float R = m[(n0 + n) * 64];
                lam[n] = ssm_across(A[n], S, lam[n], R);
            }
        }
#pragma unroll
        for (int k = 0; k < Sh::kBuf; ++k) nb[k].place(l, n0, p.N, p.b_row), nc[k].place(l, n0, p.N, p.c_row);
        const int64_t of = tiles_of(p.T, kTile);
        from = p.saved + (me.b * of + s.t0(0) / kTile) * p.N * p.D + c;
    }
    __device__ __forceinline__ int64_t token() const { return static_cast<int64_t>(me.b) * p.T + s.t0(0); }

    template <int B>
    __device__ __forceinline__ void fetch(int i) {
        if (i >= s.tiles) return;
        const int valid = s.valid(i);
        nb[B].load(bs.rows(valid));
        nc[B].load(cs.rows(valid));
        bs.move(-kTile), cs.move(-kTile);
#pragma unroll
        for (int n = 0; n < SN; ++n)
            saved[B][n] = n0 + n < p.N && me.live ? from[static_cast<int64_t>(n0 + n) * p.D] : 0.0f;
        from -= static_cast<int64_t>(p.N) * p.D;
    }

    // Tile i; then the loads of tile i + kBuf are asked for.
    template <int B>
    __device__ __forceinline__ void walk(int i) {
        const int valid = s.valid(i);
        float Bv[SN], Cv[SN], before[SN];
        nb[B].get(Bv);
        nc[B].get(Cv);
#pragma unroll
        for (int n = 0; n < SN; ++n) before[n] = saved[B][n];
        fetch<B>(i + Sh::kBuf);
        if (valid <= 0) {
            for (int j = l; j < kTile * 2 * SN; j += 64) sh.sums[B][j / (2 * SN)][j / SN % 2 * NP + n0 + j % SN] = 0.0f;
            return;
        }
        const uint64_t cuts = ssm_cuts(p, me.b, s.t0(i), valid, l);
        if (cuts & 1) {
#pragma unroll
            for (int n = 0; n < SN; ++n) before[n] = 0.0f;
        }
        with_flag(cuts != 0 || valid < kTile, [&](auto partly) {
            // a tile of more tokens than the registers hold goes in parts, from the last to the first, the state before
            // each being taken on the way to it
            constexpr int kParts = kTile / kPart;
            static_assert(kParts <= 2, "one state between the parts");
            auto decay = [&](float d, int n) { return __builtin_amdgcn_exp2f(d * A[n]); };
            float mid[SN];
            if constexpr (kParts == 2) {
#pragma unroll
                for (int n = 0; n < SN; ++n) mid[n] = before[n];
                each<kPart>([&](auto tc) {
                    constexpr int t = tc();
                    const float d = sh.in[B][t][0][l], u = sh.in[B][t][1][l];
                    const bool cut = partly() && (cuts >> t & 1);
#pragma unroll
                    for (int n = 0; n < SN; ++n) mid[n] = fmaf(decay(d, n), cut ? 0.0f : mid[n], bcast<t>(Bv[n]) * u);
                });
            }
            // (Eight states to a lane: tokens of the way back stay apart, and on the way forward where rows move element by
            // element, since what the compiler takes ahead it spills.  B4 T2048 D1024 N64 fp32 1083 us without, 928
            // so, 957 with both; B3 T777 D514, odd rows, 390, 383, 373.)
            each<kParts>([&](auto pc) {
                constexpr int first = (kParts - 1 - pc()) * kPart;
                const float(&start)[SN] = first ? mid : before;
                float h[kPart][SN], a[kHold ? kPart : 1][SN];
                each<kPart>([&](auto tc) {
                    constexpr int i = tc(), t = first + i;
                    const float d = sh.in[B][t][0][l], u = sh.in[B][t][1][l];
                    const bool cut = partly() && (cuts >> t & 1);
                    float y[SN];
#pragma unroll
                    for (int n = 0; n < SN; ++n) {
                        const float hp = i ? h[i ? i - 1 : 0][n] : start[n];
                        const float e = decay(d, n);
                        if constexpr (kHold) a[i][n] = e;
                        h[i][n] = fmaf(e, cut ? 0.0f : hp, bcast<t>(Bv[n]) * u);
                        y[n] = bcast<t>(Cv[n]) * h[i][n];
                    }
                    if (p.z) {
#pragma unroll
                        for (int k = 1; k < SN; k *= 2)
#pragma unroll
                            for (int n = 0; n < SN; n += 2 * k) y[n] += y[n + k];
                        sh.y[B][wave][t][l] = y[0];
                    }
                    if constexpr (!kHold && !VEC) __builtin_amdgcn_sched_barrier(0);
                });
                float v[16];
                each<kPart>([&](auto tc) {
                    constexpr int i = kPart - 1 - tc(), t = first + i, j = tc() % kPair;  // j: its place in the pair
                    if (partly() && t >= valid) {
#pragma unroll
                        for (int n = 0; n < 2 * SN; ++n) v[j * 2 * SN + n] = 0.0f;
                    } else {
                        const float d = sh.in[B][t][0][l], u = sh.in[B][t][1][l], g = sh.in[B][t][2][l];
                        const bool cut = partly() && (cuts >> t & 1);
                        float du[SN], q = 0.0f;
#pragma unroll
                        for (int n = 0; n < SN; ++n) {
                            lam[n] += bcast<t>(Cv[n]) * g;
                            v[j * 2 * SN + n] = lam[n] * u;
                            v[j * 2 * SN + SN + n] = g * h[i][n];
                            du[n] = bcast<t>(Bv[n]) * lam[n];
                            // a state that is dropped passes nothing back, whatever it was
                            lam[n] = cut ? 0.0f : (kHold ? a[kHold ? i : 0][n] : decay(d, n)) * lam[n];
                            const float k = cut ? 0.0f : lam[n] * (i ? h[i ? i - 1 : 0][n] : start[n]);
                            q = fmaf(k, A[n], q);
                            dA[n] = fmaf(k, d, dA[n]);
                        }
#pragma unroll
                        for (int k = 1; k < SN; k *= 2)
#pragma unroll
                            for (int n = 0; n < SN; n += 2 * k) du[n] += du[n + k];
                        sh.part[B][wave][t][0][l] = du[0];
                        sh.part[B][wave][t][1][l] = q;
                    }
                    if constexpr (j == kPair - 1) (&sh.sums[B][t + kPair - 1][0])[sum_at] = sum16(v, l);
                    if constexpr (!kHold) __builtin_amdgcn_sched_barrier(0);
                });
            });
        });
    }
    // The gradient of the state before the segment, and this lane's sums over its tokens.
    __device__ __forceinline__ void finish(float* tok) {
        if (!me.live) return;
#pragma unroll
        for (int n = 0; n < SN; ++n) {
            if (n0 + n >= p.N) continue;
            if (p.dstate_in && s.seg == 0) p.dstate_in[state + n] = lam[n];
            tok[static_cast<int64_t>(n0 + n) * p.D + c] = dA[n];
        }
    }
};

template <typename TIn, typename TDy, int SN, int NW, bool VEC>
__global__ __launch_bounds__(Shape<NW>::kNT) void layer_ssm_bwd_kernel(SsmParams p, BwdSpace ws) {
    using Sh = Shape<NW>;
    __shared__ Shared<SN, NW> sh;
    const int chains = p.B * p.G * ssm_blocks(p);
    const SsmPlace me = ssm_place(p, blockIdx.x % chains);
    const Segment s = segment_of(p, blockIdx.x / chains, ws.length, me.len, chains);
    float* tok = ws.tok + (static_cast<int64_t>(me.b) * ws.segs + s.seg) * (p.N + 2) * p.D;
    auto take_sums = [&](const Taker<TIn, TDy, SN, NW, VEC>& t) {
        // dskip and ddt_bias, of kHT / 16 threads each
        float(*all)[2][64] = reinterpret_cast<float(*)[2][64]>(&sh.in[0][0][0][0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) all[t.id >> 4][0][t.mine.at + e] = t.dskip[e], all[t.id >> 4][1][t.mine.at + e] = t.dbias[e];
    };
    auto put_sums = [&](int id, int chain) {
        if (id >= 128) return;
        const float(*all)[2][64] = reinterpret_cast<const float(*)[2][64]>(&sh.in[0][0][0][0]);
        const int which = id >> 6, k = chain % ssm_blocks(p) * 64 + (id & 63);
        float a = 0.0f;
        for (int j = 0; j < Sh::kHT / 16; ++j) a += all[j][which][id & 63];
        if (k < p.D / p.G) tok[static_cast<int64_t>(p.N + which) * p.D + me.g * (p.D / p.G) + k] = a;
    };
    if constexpr (Sh::kApart) {
        if (me.wave >= NW) {
            Taker<TIn, TDy, SN, NW, VEC> t(p, ws, sh, s, me, threadIdx.x - NW * 64);
            t.template fetch<0>(0);
            t.template fetch<1>(1);
            t.template inputs<0>(0);
            t.template fetch<0>(2);
            __syncthreads();
            for (int i = 0; i < s.tiles; i += 2) {
                if (i > 0) t.template outputs<1>(i - 1);
                t.template inputs<1>(i + 1);
                t.template fetch<1>(i + 3);
                __syncthreads();
                if (i + 1 >= s.tiles) break;
                t.template outputs<0>(i);
                t.template inputs<0>(i + 2);
                t.template fetch<0>(i + 4);
                __syncthreads();
            }
            (s.tiles - 1) & 1 ? t.template outputs<1>(s.tiles - 1) : t.template outputs<0>(s.tiles - 1);
            take_sums(t);
            __syncthreads();
            put_sums(t.id, s.chain);
        } else {
            Walker<TIn, SN, NW, VEC> w(p, ws, sh, s, me);
            w.template fetch<0>(0);
            w.template fetch<1>(1);
            __syncthreads();
            for (int i = 0; i < s.tiles; i += 2) {
                w.template walk<0>(i);
                __syncthreads();
                if (i + 1 >= s.tiles) break;
                w.template walk<1>(i + 1);
                __syncthreads();
            }
            w.finish(tok);
            __syncthreads();
        }
    } else {
        const bool takes = threadIdx.x < Sh::kHT;  // whole waves
        Taker<TIn, TDy, SN, NW, VEC> t(p, ws, sh, s, me, threadIdx.x & (Sh::kHT - 1));
        Walker<TIn, SN, NW, VEC> w(p, ws, sh, s, me);
        w.template fetch<0>(0);
        if (takes) t.template fetch<0>(0);
        for (int i = 0; i < s.tiles; ++i) {
            if (takes) {
                t.template inputs<0>(i);
                t.template fetch<0>(i + 1);
            }
            __syncthreads();
            w.template walk<0>(i);
            __syncthreads();
            if (takes) t.template outputs<0>(i);
        }
        w.finish(tok);
        __syncthreads();
        if (takes) take_sums(t);
        __syncthreads();
        if (takes) put_sums(t.id, s.chain);
    }
}

// Launches the kernel for inputs of type TIn (one translation unit each).
template <typename TIn>
void launch_kernel(const SsmParams& p, const BwdSpace& ws, hipStream_t st) {
    with_states(p.N, [&](auto sn, auto nw) {
        const unsigned chains = static_cast<unsigned>(p.B) * p.G * tiles_of(p.D / p.G, 64);
        auto go = [&](auto dy, auto vec) {
            hipLaunchKernelGGL((layer_ssm_bwd_kernel<TIn, decltype(dy), sn(), nw(), vec()>), dim3(chains * ws.segs),
                               dim3(Shape<nw()>::kNT), 0, st, p, ws);
        };
        const std::true_type yes;
        const std::false_type no;
        if (p.y_bf16)
            ssm_vec(p) ? go(uint16_t(), yes) : go(uint16_t(), no);
        else
            ssm_vec(p) ? go(float(), yes) : go(float(), no);
    });
}
void launch_bf16(const SsmParams& p, const BwdSpace& ws, hipStream_t st);
void launch_f32(const SsmParams& p, const BwdSpace& ws, hipStream_t st);

}  // namespace ssm_bwd
}  // namespace layer
