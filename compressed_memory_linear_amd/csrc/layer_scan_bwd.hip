// layer_scan_bwd.hip -- gradient of the element-wise gated recurrence.
//
// With l_t the gradient that reaches h_t (from y_t and from h_{t+1}),
//     l_t = dy_t + mu_{t+1} l_{t+1},   the last token's l taking dstate_out in,
//     dv_t = l_t w(mu_t) gamma_t,      dg_t = l_t w(mu_t) v_t gamma_t (1 - gamma_t),
//     df_t = l_t mu_t (1 - mu_t) (h_{t-1} + gamma_t v_t w'(mu_t)),   dstate_in = mu_0 l_0,
// where mu (1 - mu) w'(mu) is 0, -mu (1 - mu) or -mu^2 sqrt((1 - mu) / (1 + mu)):
// finite, and zero where a gate saturates.  A run of tokens maps the gradient
// r = mu_{t+1} l_{t+1} that enters it from behind to the one that leaves it in
// front, r -> A r + R, with the same A as the forward's map, so the tiles hand r on
// as the forward's do h (layer_chain.h), from the last to the first; each recomputes its h_{t-1}
// from the state the forward saved before it, and nothing else of the forward is kept.
//
// Bound by HBM and, with few chains, by the tiles' waits for one another (bf16, D2048): B8 T4096 with
// the writing intensity 940 MB in 187 to 209 us, 4.5 to 5.0 TB/s; B1 T65536 without 1.34 GB in 273
// to 284 us, 4.7 to 4.9 TB/s.  The vector units are 47 and 43 % busy.
// Runs of 16 tokens (126 registers with the intensity): 8 tokens 578 us for the latter's training
// step, 16 428, 24 408, but 334, 306 and 336 for the former's.  Weight 1 with the intensity holds both
// gates' factors over the second pass and spills 10 to 18 registers: 205 us at B8 T4096 where
// 1 - mu takes 193 and sqrt(1 - mu^2) 196.
#include "layer_chain.h"
#include "layer_device.h"
#include "layer_launch.h"

namespace layer {
namespace {

template <typename TIn, typename TDy, int WT, bool GAMMA>
__global__ __launch_bounds__(kScanWaves * 64, 4) void layer_scan_bwd_kernel(ScanParams p) {
    __shared__ Shared s;  // s.H: the runs' maps of r
    __shared__ float sH[kScanWaves][64];
    __shared__ uint32_t ticket;
    const int chains = p.B * ((p.D + 63) / 64);
    const int tiles = (p.T + kBwdTile - 1) / kBwdTile;
    const Place me = take_place(p.ws, p.D, chains, &ticket);
    const int tile = tiles - 1 - me.pos, b = me.b, wave = me.wave, l = me.l, c = me.c;
    const bool live = c < p.D;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int active = max(1, (len + kBwdTile - 1) / kBwdTile);  // tiles with tokens, the first in any case
    const int t0 = tile * kBwdTile;
    const int64_t first = (static_cast<int64_t>(b) * p.T + t0) * p.D;
    const int rows = min(kBwdTile, p.T - t0);
    const int r0 = wave * kBwdRun;
    // byte offsets of this lane's channel in the wave's first row, and from row to row
    const int eg = p.grad_bf16 ? 2 : 4;
    const uint32_t at = static_cast<uint32_t>(r0) * p.D + c;
    const uint32_t oin = live ? at * sizeof(TIn) : kOut, din = p.D * sizeof(TIn);
    const uint32_t ody = live ? at * sizeof(TDy) : kOut, ddy = p.D * sizeof(TDy);
    const uint32_t og = live ? at * eg : kOut, dog = p.D * eg;
    const auto dvr = rows_rsrc(p.dv, first * eg, rows * p.D * eg);
    const auto dfr = rows_rsrc(p.df, first * eg, rows * p.D * eg);
    const auto dgr = rows_rsrc(GAMMA ? p.dg : p.df, first * eg, rows * p.D * eg);
    if (tile >= active) {
        with_flag(p.grad_bf16, [&](auto bf16) {
#pragma unroll
            for (int i = 0; i < kBwdRun; ++i) {
                store_row<bf16(), true>(dvr, og + i * dog, 0.0f);
                store_row<bf16(), true>(dfr, og + i * dog, 0.0f);
                if (GAMMA) store_row<bf16(), true>(dgr, og + i * dog, 0.0f);
            }
        });
        return;
    }

    const int nin = rows * p.D * static_cast<int>(sizeof(TIn));
    const auto fr = rows_rsrc(p.f, first * sizeof(TIn), nin);
    const auto vr = rows_rsrc(p.v, first * sizeof(TIn), nin);
    const auto gr = rows_rsrc(GAMMA ? p.g : p.f, first * sizeof(TIn), nin);
    const auto yr = rows_rsrc(p.dy, first * sizeof(TDy), rows * p.D * static_cast<int>(sizeof(TDy)));
    TIn rf[kBwdRun], rv[kBwdRun], rg[GAMMA ? kBwdRun : 1];
    TDy ry[kBwdRun];
#pragma unroll
    for (int i = 0; i < kBwdRun; ++i) {
        rf[i] = load_row<TIn>(fr, oin + i * din);
        rv[i] = load_row<TIn>(vr, oin + i * din);
        if (GAMMA) rg[i] = load_row<TIn>(gr, oin + i * din);
        ry[i] = load_row<TDy>(yr, ody + i * ddy);
    }
    const int rank = active - 1 - tile;
    const int64_t sc = static_cast<int64_t>(b) * p.D + c;
    float h = 0.0f, behind = 0.0f;  // the state before the tile, the gradient from behind the chain
    if (live) {
        h = p.saved[(static_cast<int64_t>(b) * tiles + tile) * p.D + c];
        if (p.dstate_out && wave == 0 && rank < kScanWaves * kScanWaves) behind = p.dstate_out[sc];
    }

    // First pass: the run's maps of h and of r.
    float a[kBwdRun], om[kBwdRun], gam[GAMMA ? kBwdRun : 1], A = 1.0f, H = 0.0f, R = 0.0f;
    auto run_map = [&](int i) {
        const float x = widen(rv[i]) * weight_of<WT>(a[i], om[i]);
        A *= a[i];
        H = fmaf(a[i], H, GAMMA ? x * gam[GAMMA ? i : 0] : x);
    };
#pragma unroll
    for (int i = 0; i < kBwdRun; ++i) {
        sigmoid2<kAccurate<TIn>>(widen(rf[i]), a[i], om[i]);
        if (GAMMA) {
            float q;
            sigmoid2<kAccurate<TIn>>(widen(rg[i]), gam[i], q);
        }
        run_map(i);
    }
    // Padding passes the gradient on and keeps the state.  Set right afterwards, in the one tile
    // that has both, so that the others pay nothing.
    const bool padded = t0 + kBwdTile > len;
    if (padded) {
        A = 1.0f, H = 0.0f;
#pragma unroll
        for (int i = 0; i < kBwdRun; ++i) {
            if (t0 + r0 + i >= len) a[i] = 1.0f, rv[i] = TIn(0), ry[i] = TDy(0);
            run_map(i);
        }
    }
#pragma unroll
    for (int i = kBwdRun - 1; i >= 0; --i) R = a[i] * (R + widen(ry[i]));
    A = run_product(A, a);
    s.A[wave][l] = A, s.H[wave][l] = R, sH[wave][l] = H;
    const Chain links = chain_of(p.ws, chains, tiles);
    Carry from{s, links, me.chain, rank, wave, l};
    if (p.ws) from.begin();
    __syncthreads();
    const int waves = blockDim.x >> 6;
    if (wave == 0) {
        // the tile's map of r: the last run first
        A = 1.0f, R = 0.0f;
#pragma unroll
        for (int w = kScanWaves - 1; w >= 0; --w)
            if (w < waves) {
                R = fmaf(s.A[w][l], R, s.H[w][l]);
                A = times(A, s.A[w][l]);
            }
    }
    const bool last = tile == 0;
    if (p.ws) {
        from.finish(last, behind, A, R);
    } else {
        if (wave == 0) s.carry[l] = behind;
        __syncthreads();
    }
    float r = s.carry[l];
    if (p.dstate_in && last && wave == 0 && live) p.dstate_in[sc] = len > 0 ? fmaf(A, r, R) : r;
    for (int w = 0; w < wave; ++w) h = fmaf(s.A[w][l], h, sH[w][l]);
    for (int w = waves - 1; w > wave; --w) r = fmaf(s.A[w][l], r, s.H[w][l]);

    // Second pass, forwards: what l_t is multiplied with.  om becomes the factor of df, wg is that of
    // dv and gam that of dg.
    float wg[kBwdRun];
#pragma unroll
    for (int i = 0; i < kBwdRun; ++i) {
        const float m = a[i], o = om[i], w = weight_of<WT>(m, o);
        const float gx = GAMMA ? gam[GAMMA ? i : 0] * widen(rv[i]) : widen(rv[i]);
        wg[i] = GAMMA ? w * gam[GAMMA ? i : 0] : w;
        if constexpr (WT == 0) om[i] = m * o * h;
        if constexpr (WT == 1) om[i] = m * o * (h - gx);
        if constexpr (WT == 2) om[i] = m * fmaf(o, h, -m * w * __builtin_amdgcn_rcpf(1.0f + m) * gx);
        if constexpr (GAMMA) {
            float q, ng;
            sigmoid2<kAccurate<TIn>>(widen(rg[i]), q, ng);
            gam[i] = w * gx * ng;
        }
        h = fmaf(m, h, w * gx);
    }
    // Third pass, backwards: the gradients, in the factors' places.
#pragma unroll
    for (int i = kBwdRun - 1; i >= 0; --i) {
        const float lam = widen(ry[i]) + r;
        wg[i] *= lam;
        om[i] *= lam;
        if constexpr (GAMMA) gam[i] *= lam;
        r = a[i] * lam;
    }
    if (padded) {
#pragma unroll
        for (int i = 0; i < kBwdRun; ++i)
            if (t0 + r0 + i >= len) {
                wg[i] = om[i] = 0.0f;
                if constexpr (GAMMA) gam[i] = 0.0f;
            }
    }
    with_flag(p.grad_bf16, [&](auto bf16) {
        const uint32_t to = here(og);
#pragma unroll
        for (int i = 0; i < kBwdRun; ++i) {
            store_row<bf16(), true>(dvr, to + i * dog, wg[i]);
            store_row<bf16(), true>(dfr, to + i * dog, om[i]);
            if constexpr (GAMMA) store_row<bf16(), true>(dgr, to + i * dog, gam[i]);
        }
    });
}

template <typename TIn, typename TDy>
int pick(const ScanParams& p, hipStream_t st) {
    const unsigned groups = static_cast<unsigned>(tiles_of(p.D, 64) * p.B * tiles_of(p.T, kBwdTile));
    auto go = [&](auto wt, auto gamma) {
        hipLaunchKernelGGL((layer_scan_bwd_kernel<TIn, TDy, wt(), gamma()>), dim3(groups),
                           dim3(scan_threads(p.T, kBwdRun)), 0, st, p);
    };
    const std::integral_constant<int, 0> w0;
    const std::integral_constant<int, 1> w1;
    const std::integral_constant<int, 2> w2;
    const std::true_type yes;
    const std::false_type no;
    switch (p.weight) {
        case 0: p.g ? go(w0, yes) : go(w0, no); break;
        case 1: p.g ? go(w1, yes) : go(w1, no); break;
        default: p.g ? go(w2, yes) : go(w2, no); break;
    }
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace

int launch_scan_bwd(const ScanParams& p, hipStream_t st) {
    if (p.ws) clear_scan_workspace(p, kBwdTile, st);
    if (p.in_bf16) return p.y_bf16 ? pick<uint16_t, uint16_t>(p, st) : pick<uint16_t, float>(p, st);
    return p.y_bf16 ? pick<float, uint16_t>(p, st) : pick<float, float>(p, st);
}

}  // namespace layer
