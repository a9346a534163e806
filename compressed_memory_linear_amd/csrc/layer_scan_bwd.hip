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
    const uint32_t off = (live ? static_cast<uint32_t>(c) : kOut) + static_cast<uint32_t>(r0) * p.D;
    const auto dvr = rows_rsrc(p.dv, p.grad_bf16, first, rows, p.D);
    const auto dfr = rows_rsrc(p.df, p.grad_bf16, first, rows, p.D);
    const auto dgr = rows_rsrc(GAMMA ? p.dg : p.df, p.grad_bf16, first, rows, p.D);
    if (tile >= active) {
        const float zero[V] = {};
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            store_rows<V>(dvr, off + i * p.D, zero, p.grad_bf16);
            store_rows<V>(dfr, off + i * p.D, zero, p.grad_bf16);
            if (GAMMA) store_rows<V>(dgr, off + i * p.D, zero, p.grad_bf16);
        }
        return;
    }

    const auto fr = rows_rsrc(static_cast<const TIn*>(p.f) + first, rows, p.D);
    const auto vr = rows_rsrc(static_cast<const TIn*>(p.v) + first, rows, p.D);
    const auto gr = rows_rsrc(static_cast<const TIn*>(GAMMA ? p.g : p.f) + first, rows, p.D);
    const auto yr = rows_rsrc(static_cast<const TDy*>(p.dy) + first, rows, p.D);
    Vec<TIn, V> rf[kRun], rv[kRun], rg[GAMMA ? kRun : 1];
    Vec<TDy, V> ry[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        rf[i] = load_rows<TIn, V>(fr, off + i * p.D);
        rv[i] = load_rows<TIn, V>(vr, off + i * p.D);
        if (GAMMA) rg[i] = load_rows<TIn, V>(gr, off + i * p.D);
        ry[i] = load_rows<TDy, V>(yr, off + i * p.D);
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
#pragma unroll
    for (int i = 0; i < kRun; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool in = t0 + r0 + i < len;
            sigmoid2(widen(rf[i].e[j]), a[i][j], om[i][j]);
            float x = widen(rv[i].e[j]) * weight_of<WT>(a[i][j], om[i][j]);
            if (GAMMA) {
                float q;
                sigmoid2(widen(rg[i].e[j]), gam[i][j], q);
                x *= gam[i][j];
            }
            if (!in) a[i][j] = 1.0f, x = 0.0f;
            A[j] *= a[i][j];
            H[j] = fmaf(a[i][j], H[j], x);
        }
#pragma unroll
    for (int i = kRun - 1; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float dy = t0 + r0 + i < len ? widen(ry[i].e[j]) : 0.0f;
            R[j] = a[i][j] * (dy + R[j]);
        }
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
            const bool in = t0 + r0 + i < len;
            const float m = a[i][j], o = om[i][j], w = weight_of<WT>(m, o);
            const float gx = GAMMA ? gam[i][j] * widen(rv[i].e[j]) : widen(rv[i].e[j]);
            wg[i][j] = GAMMA ? w * gam[i][j] : w;
            float into = m * o * h[j];
            if (WT == 1) into = fmaf(-m * o, gx, into);
            if (WT == 2) into = fmaf(-m * m * w * __builtin_amdgcn_rcpf(1.0f + m), gx, into);
            om[i][j] = into;
            if (GAMMA) {
                float q, ng;
                sigmoid2(widen(rg[i].e[j]), q, ng);
                gam[i][j] = w * gx * ng;
            }
            h[j] = in ? fmaf(m, h[j], w * gx) : h[j];
        }
    // Third pass, backwards: the gradients.
#pragma unroll
    for (int i = kRun - 1; i >= 0; --i) {
        float dv[V], df[V], dg[V];
        const bool in = t0 + r0 + i < len;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float lam = (in ? widen(ry[i].e[j]) : 0.0f) + r[j];
            dv[j] = in ? lam * wg[i][j] : 0.0f;
            df[j] = in ? lam * om[i][j] : 0.0f;
            if (GAMMA) dg[j] = in ? lam * gam[i][j] : 0.0f;
            r[j] = a[i][j] * lam;
        }
        store_rows<V>(dvr, off + i * p.D, dv, p.grad_bf16);
        store_rows<V>(dfr, off + i * p.D, df, p.grad_bf16);
        if (GAMMA) store_rows<V>(dgr, off + i * p.D, dg, p.grad_bf16);
    }
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
