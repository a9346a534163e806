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
#include "layer_chain.h"
#include "layer_device.h"
#include "layer_launch.h"

namespace layer {
namespace {

constexpr int kRun = 8;                  // tokens per wave of a tile
constexpr int kWaves = kBwdTile / kRun;  // waves per workgroup

template <typename TIn, typename TDy, int V, int WT, bool GAMMA>
__global__ __launch_bounds__(kWaves * 64, 4) void layer_scan_bwd_kernel(ScanParams p) {
    constexpr int CB = 64 * V;
    __shared__ Shared<kWaves, CB> s;
    __shared__ float sH[kWaves][CB];
    __shared__ uint32_t ticket;
    const int nblk = (p.D + CB - 1) / CB;
    const int chains = p.B * nblk;
    const int tiles = (p.T + kBwdTile - 1) / kBwdTile;
    uint32_t id = blockIdx.x;
    if (p.ws) {
        if (threadIdx.x == 0) ticket = atomicAdd(static_cast<uint32_t*>(p.ws), 1u);
        __syncthreads();
        id = __builtin_amdgcn_readfirstlane(ticket);
    }
    const int tile = tiles - 1 - static_cast<int>(id / chains), chain = static_cast<int>(id % chains);
    const int b = chain / nblk;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l = (threadIdx.x & 63) * V;
    const int c = chain % nblk * CB + l;
    const bool live = c < p.D;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int active = max(1, (len + kBwdTile - 1) / kBwdTile);
    const int t0 = tile * kBwdTile;
    const int64_t first = (static_cast<int64_t>(b) * p.T + t0) * p.D;
    const int rows = min(kBwdTile, p.T - t0);
    const int r0 = wave * kRun;
    const int eg = p.grad_bf16 ? 2 : 4;
    const uint32_t at = static_cast<uint32_t>(r0) * p.D + c;
    const uint32_t oin = live ? at * sizeof(TIn) : kOut, din = p.D * sizeof(TIn);
    const uint32_t ody = live ? at * sizeof(TDy) : kOut, ddy = p.D * sizeof(TDy);
    const uint32_t og = live ? at * eg : kOut, dog = p.D * eg;
    const auto dvr = rows_rsrc(p.dv, first * eg, rows * p.D * eg);
    const auto dfr = rows_rsrc(p.df, first * eg, rows * p.D * eg);
    const auto dgr = rows_rsrc(GAMMA ? p.dg : p.df, first * eg, rows * p.D * eg);
    if (tile >= active) {
        const float zero[V] = {};
        with_flag(p.grad_bf16, [&](auto bf16) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                store_rows<V, bf16()>(dvr, og + i * dog, zero);
                store_rows<V, bf16()>(dfr, og + i * dog, zero);
                if (GAMMA) store_rows<V, bf16()>(dgr, og + i * dog, zero);
            }
        });
        return;
    }

    const int nin = rows * p.D * static_cast<int>(sizeof(TIn));
    const auto fr = rows_rsrc(p.f, first * sizeof(TIn), nin);
    const auto vr = rows_rsrc(p.v, first * sizeof(TIn), nin);
    const auto gr = rows_rsrc(GAMMA ? p.g : p.f, first * sizeof(TIn), nin);
    const auto yr = rows_rsrc(p.dy, first * sizeof(TDy), rows * p.D * static_cast<int>(sizeof(TDy)));
    Vec<TIn, V> rf[kRun], rv[kRun], rg[GAMMA ? kRun : 1];
    Vec<TDy, V> ry[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        rf[i] = load_rows<TIn, V>(fr, oin + i * din);
        rv[i] = load_rows<TIn, V>(vr, oin + i * din);
        if (GAMMA) rg[i] = load_rows<TIn, V>(gr, oin + i * din);
        ry[i] = load_rows<TDy, V>(yr, ody + i * ddy);
    }
    float h[V] = {}, behind[V] = {};  // the state before the tile, the chain's first gradient
    const int rank = active - 1 - tile;
    const int64_t sc = static_cast<int64_t>(b) * p.D + c;
    if (live) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            h[j] = p.saved[(static_cast<int64_t>(b) * tiles + tile) * p.D + c + j];
            if (p.dstate_out && wave == 0 && rank < (p.ws ? p.group : 1)) behind[j] = p.dstate_out[sc + j];
        }
    }

    // First pass: the run's maps of h and of r.
    float a[kRun][V], om[kRun][V], gam[GAMMA ? kRun : 1][V], A[V], H[V], R[V];
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = 1.0f, H[j] = 0.0f, R[j] = 0.0f;
    auto run_map = [&](int i, int j) {
        const float x = widen(rv[i].e[j]) * weight_of<WT>(a[i][j], om[i][j]);
        A[j] *= a[i][j];
        H[j] = fmaf(a[i][j], H[j], GAMMA ? x * gam[GAMMA ? i : 0][j] : x);
    };
#pragma unroll
    for (int i = 0; i < kRun; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sigmoid2<kAccurate<TIn>>(widen(rf[i].e[j]), a[i][j], om[i][j]);
            if (GAMMA) {
                float q;
                sigmoid2<kAccurate<TIn>>(widen(rg[i].e[j]), gam[i][j], q);
            }
            run_map(i, j);
        }
    // Padding passes the gradient on and keeps the state.  Set right afterwards, in the one tile
    // that has both, so that the others pay nothing.
    const bool padded = t0 + kBwdTile > len;
    if (padded) {
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = 1.0f, H[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (t0 + r0 + i >= len) a[i][j] = 1.0f, rv[i].e[j] = TIn(0), ry[i].e[j] = TDy(0);
                run_map(i, j);
            }
    }
#pragma unroll
    for (int i = kRun - 1; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < V; ++j) R[j] = a[i][j] * (R[j] + widen(ry[i].e[j]));
#pragma unroll
    for (int j = 0; j < V; ++j) s.A[wave][l + j] = A[j], s.H[wave][l + j] = R[j], sH[wave][l + j] = H[j];
    __syncthreads();
    if (wave == 0) {
        // the tile's map of r: the last run first
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = 1.0f, R[j] = 0.0f;
#pragma unroll 2
        for (int w = kWaves - 1; w >= 0; --w)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                R[j] = fmaf(s.A[w][l + j], R[j], s.H[w][l + j]);
                A[j] *= s.A[w][l + j];
            }
    }
    const bool last = tile == 0;
    if (p.ws) {
        chain_carry<V>(s, chain_of(p.ws, chains, tiles, p.group, CB), chain, rank, last, behind, A, R);
    } else {
        if (wave == 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) s.carry[l + j] = behind[j];
        }
        __syncthreads();
    }
    float r[V];
#pragma unroll
    for (int j = 0; j < V; ++j) r[j] = s.carry[l + j];
    if (wave == 0 && live && last && p.dstate_in) {
#pragma unroll
        for (int j = 0; j < V; ++j) p.dstate_in[sc + j] = len > 0 ? fmaf(A[j], r[j], R[j]) : r[j];
    }
    for (int w = 0; w < wave; ++w)
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = fmaf(s.A[w][l + j], h[j], sH[w][l + j]);
    for (int w = kWaves - 1; w > wave; --w)
#pragma unroll
        for (int j = 0; j < V; ++j) r[j] = fmaf(s.A[w][l + j], r[j], s.H[w][l + j]);

    // Second pass, forwards: what l_t is multiplied with.  om becomes the factor of df, wg is that of
    // dv and gam that of dg.
    float wg[kRun][V];
#pragma unroll
    for (int i = 0; i < kRun; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float m = a[i][j], o = om[i][j], w = weight_of<WT>(m, o);
            const float gx = GAMMA ? gam[GAMMA ? i : 0][j] * widen(rv[i].e[j]) : widen(rv[i].e[j]);
            wg[i][j] = GAMMA ? w * gam[GAMMA ? i : 0][j] : w;
            if constexpr (WT == 0) om[i][j] = m * o * h[j];
            if constexpr (WT == 1) om[i][j] = m * o * (h[j] - gx);
            if constexpr (WT == 2) om[i][j] = m * fmaf(o, h[j], -m * w * __builtin_amdgcn_rcpf(1.0f + m) * gx);
            if constexpr (GAMMA) {
                float q, ng;
                sigmoid2<kAccurate<TIn>>(widen(rg[i].e[j]), q, ng);
                gam[i][j] = w * gx * ng;
            }
            h[j] = fmaf(m, h[j], w * gx);
        }
    // Third pass, backwards: the gradients, in the factors' places.
#pragma unroll
    for (int i = kRun - 1; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float lam = widen(ry[i].e[j]) + r[j];
            wg[i][j] *= lam;
            om[i][j] *= lam;
            if constexpr (GAMMA) gam[i][j] *= lam;
            r[j] = a[i][j] * lam;
        }
    if (padded) {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (t0 + r0 + i >= len) {
                    wg[i][j] = om[i][j] = 0.0f;
                    if constexpr (GAMMA) gam[i][j] = 0.0f;
                }
    }
    with_flag(p.grad_bf16, [&](auto bf16) {
        const uint32_t to = here(og);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            store_rows<V, bf16()>(dvr, to + i * dog, wg[i]);
            store_rows<V, bf16()>(dfr, to + i * dog, om[i]);
            if constexpr (GAMMA) store_rows<V, bf16()>(dgr, to + i * dog, gam[i]);
        }
    });
}

template <typename TIn, typename TDy, int V, int WT, bool GAMMA>
void launch(const ScanParams& p, hipStream_t st) {
    const unsigned nblk = static_cast<unsigned>((p.D + 64 * V - 1) / (64 * V));
    const unsigned tiles = static_cast<unsigned>(tiles_of(p.T, kBwdTile));
    hipLaunchKernelGGL((layer_scan_bwd_kernel<TIn, TDy, V, WT, GAMMA>), dim3(nblk * p.B * tiles), dim3(kWaves * 64), 0,
                       st, p);
}

template <typename TIn, typename TDy, int V>
void pick(const ScanParams& p, hipStream_t st) {
    const bool g = p.g != nullptr;
    switch (p.weight) {
        case 0: g ? launch<TIn, TDy, V, 0, true>(p, st) : launch<TIn, TDy, V, 0, false>(p, st); break;
        case 1: g ? launch<TIn, TDy, V, 1, true>(p, st) : launch<TIn, TDy, V, 1, false>(p, st); break;
        default: g ? launch<TIn, TDy, V, 2, true>(p, st) : launch<TIn, TDy, V, 2, false>(p, st); break;
    }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

int launch_scan_bwd(const ScanParams& p, hipStream_t st) {
    clear_scan_workspace(p, st);
    const size_t ein = 2 * (p.in_bf16 ? 2 : 4), ey = 2 * (p.y_bf16 ? 2 : 4), eg = 2 * (p.grad_bf16 ? 2 : 4);
    const bool two = p.D % 2 == 0 && aligned(p.v, ein) && aligned(p.f, ein) && aligned(p.g, ein) && aligned(p.dy, ey) &&
                     aligned(p.dv, eg) && aligned(p.df, eg) && aligned(p.dg, eg);
    if (p.in_bf16 && p.y_bf16)
        two ? pick<uint16_t, uint16_t, 2>(p, st) : pick<uint16_t, uint16_t, 1>(p, st);
    else if (p.in_bf16)
        two ? pick<uint16_t, float, 2>(p, st) : pick<uint16_t, float, 1>(p, st);
    else if (p.y_bf16)
        two ? pick<float, uint16_t, 2>(p, st) : pick<float, uint16_t, 1>(p, st);
    else
        two ? pick<float, float, 2>(p, st) : pick<float, float, 1>(p, st);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace layer
