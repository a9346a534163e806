// layer_scan_bwd.hip -- gradient of the element-wise gated recurrence.
//
// With l_t the gradient that reaches h_t (from y_t and from h_{t+1}),
//     l_t = dy_t + mu_{t+1} l_{t+1},   the last token's l taking dstate_out in,
//     dv_t = l_t w(mu_t) gamma_t,      dg_t = l_t w(mu_t) v_t gamma_t (1 - gamma_t),
//     df_t = l_t mu_t (1 - mu_t) (h_{t-1} + gamma_t v_t w'(mu_t)),   dstate_in = mu_0 l_0,
// where mu (1 - mu) w'(mu) is 0, -mu (1 - mu) or -mu^2 sqrt((1 - mu) / (1 + mu)):
// finite, and zero where a gate saturates.  A run of tokens maps the gradient
// r = mu_{t+1} l_{t+1} that enters it from behind to the one that leaves it in
// front, r -> A r + R, with the same A as the forward's map: tiles are walked
// from the last to the first, each recomputing its h_{t-1} from the state the
// forward saved before it, so nothing of the forward but those states is kept.
#include "layer_device.h"
#include "layer_launch.h"

namespace layer {
namespace {

constexpr int kRun = 8;                   // tokens per wave of a tile
constexpr int kWaves = kScanTile / kRun;  // waves per workgroup

template <typename TIn, typename TDy, int V, int WT, bool GAMMA>
__global__ __launch_bounds__(kWaves * 64) void layer_scan_bwd_kernel(ScanParams p) {
    constexpr int CB = 64 * V;
    __shared__ float sA[kWaves][CB], sH[kWaves][CB], sR[kWaves][CB];
    const int nblk = (p.D + CB - 1) / CB;
    const int b = static_cast<int>(blockIdx.x / nblk);
    const int l = (threadIdx.x & 63) * V;
    const int c = static_cast<int>(blockIdx.x % nblk) * CB + l;
    const int wave = threadIdx.x >> 6;
    const bool live = c < p.D;
    const int cc = live ? c : 0;
    const int64_t base = static_cast<int64_t>(b) * p.T * p.D + cc;
    const TIn* vp = static_cast<const TIn*>(p.v) + base;
    const TIn* fp = static_cast<const TIn*>(p.f) + base;
    const TIn* gp = GAMMA ? static_cast<const TIn*>(p.g) + base : nullptr;
    const TDy* yp = static_cast<const TDy*>(p.dy) + base;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int tiles = (p.T + kScanTile - 1) / kScanTile;

    float r[V];  // the gradient entering from behind the tile
#pragma unroll
    for (int j = 0; j < V; ++j) r[j] = p.dstate_out ? p.dstate_out[static_cast<int64_t>(b) * p.D + cc + j] : 0.0f;

    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int t0 = tile * kScanTile + wave * kRun;
        Vec<TIn, V> rf[kRun], rv[kRun], rg[GAMMA ? kRun : 1];
        Vec<TDy, V> ry[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int64_t row = static_cast<int64_t>(min(t0 + i, p.T - 1)) * p.D;
            rf[i] = load_vec<TIn, V>(fp, row);
            rv[i] = load_vec<TIn, V>(vp, row);
            ry[i] = load_vec<TDy, V>(yp, row);
            if (GAMMA) rg[i] = load_vec<TIn, V>(gp, row);
        }
        float h[V];
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = p.saved[(static_cast<int64_t>(b) * tiles + tile) * p.D + cc + j];

        // a = mu, gx = gamma v, wg = w gamma: dv = l wg, dg = l wg v (1 - gamma); into: df = l into
        float a[kRun][V], wg[kRun][V], into[kRun][V], toG[kRun][V], dy[kRun][V], A[V], H[V], R[V];
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = 1.0f, H[j] = 0.0f, R[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const bool in = t0 + i < len;
                const float v = widen(rv[i].e[j]);
                float m, om, gam = 1.0f, ng = 0.0f;
                sigmoid2(widen(rf[i].e[j]), m, om);
                if (GAMMA) sigmoid2(widen(rg[i].e[j]), gam, ng);
                const float gx = gam * v;
                float w = 1.0f, pull = 0.0f;  // pull = mu (1 - mu) w'(mu)
                if (WT == 1) w = om, pull = -m * om;
                if (WT == 2) {
                    w = __builtin_amdgcn_sqrtf(om * (1.0f + m));
                    pull = -m * m * w * __builtin_amdgcn_rcpf(1.0f + m);
                }
                a[i][j] = in ? m : 1.0f;
                wg[i][j] = in ? w * gam : 0.0f;
                toG[i][j] = in ? w * gx * ng : 0.0f;
                dy[i][j] = in ? widen(ry[i].e[j]) : 0.0f;
                const float x = in ? w * gx : 0.0f;
                // into holds mu (1 - mu) w' gamma v until h_{t-1} is known
                into[i][j] = in ? pull * gx : 0.0f;
                A[j] *= a[i][j];
                H[j] = fmaf(a[i][j], H[j], x);
            }
#pragma unroll
        for (int i = kRun - 1; i >= 0; --i)
#pragma unroll
            for (int j = 0; j < V; ++j) R[j] = a[i][j] * (dy[i][j] + R[j]);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) sA[wave][l + j] = A[j], sH[wave][l + j] = H[j], sR[wave][l + j] = R[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) {
            for (int w = 0; w < wave; ++w) h[j] = fmaf(sA[w][l + j], h[j], sH[w][l + j]);
            float mine = 0.0f;
            for (int w = kWaves - 1; w >= 0; --w) {
                if (w == wave) mine = r[j];
                r[j] = fmaf(sA[w][l + j], r[j], sR[w][l + j]);
            }
            R[j] = mine;
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const bool in = t0 + i < len;
                float m, om;
                sigmoid2(widen(rf[i].e[j]), m, om);
                const float x = wg[i][j] * widen(rv[i].e[j]);
                if (in) into[i][j] = fmaf(m * om, h[j], into[i][j]);
                h[j] = fmaf(a[i][j], h[j], in ? x : 0.0f);
            }
#pragma unroll
        for (int i = kRun - 1; i >= 0; --i) {
            float dv[V], df[V], dg[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float lam = dy[i][j] + R[j];
                dv[j] = t0 + i < len ? lam * wg[i][j] : 0.0f;
                df[j] = t0 + i < len ? lam * into[i][j] : 0.0f;
                dg[j] = t0 + i < len ? lam * toG[i][j] : 0.0f;
                R[j] = a[i][j] * lam;
            }
            if (live && t0 + i < p.T) {
                const int64_t at = (static_cast<int64_t>(b) * p.T + t0 + i) * p.D + c;
                store_vec<V>(p.dv, at, dv, p.grad_bf16);
                store_vec<V>(p.df, at, df, p.grad_bf16);
                if (GAMMA) store_vec<V>(p.dg, at, dg, p.grad_bf16);
            }
        }
    }
    if (p.dstate_in && wave == 0 && live) {
#pragma unroll
        for (int j = 0; j < V; ++j) p.dstate_in[static_cast<int64_t>(b) * p.D + c + j] = r[j];
    }
}

template <typename TIn, typename TDy, int V, int WT, bool GAMMA>
void launch(const ScanParams& p, hipStream_t st) {
    const unsigned nblk = static_cast<unsigned>((p.D + 64 * V - 1) / (64 * V));
    hipLaunchKernelGGL((layer_scan_bwd_kernel<TIn, TDy, V, WT, GAMMA>), dim3(nblk * p.B), dim3(kWaves * 64), 0, st, p);
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
