// layer_scan.hip -- the element-wise gated recurrence, forward and single step.
//
// Per channel, with mu_t = sigmoid(f_t), gamma_t = sigmoid(g_t) (1 without g)
// and an input weight w(mu) = 1, 1 - mu or sqrt(1 - mu^2):
//     h_t = mu_t h_{t-1} + w(mu_t) gamma_t v_t,   y_t = h_t.
// A run of tokens is an affine map of the state before it, h -> A h + H with
// A the product of its mu and H its result from a zero state; two runs in a row
// compose to (A2 A1, A2 H1 + H2), which is what lets the time axis be split.
//
// A workgroup takes 64 V channels (a lane holds V neighbours, so a wave reads
// one contiguous piece of each token row) and kScanTile tokens at a time; each of its waves
// takes a run of kRun tokens of the tile, kept in registers as (mu, w gamma v).  The
// waves' (A, H) meet in LDS, every wave folds those before its own onto the
// tile's starting state and walks its run once more to form y.
#include "layer_device.h"
#include "layer_launch.h"

namespace layer {
namespace {

constexpr int kRun = 16;                   // tokens per wave of a tile
constexpr int kWaves = kScanTile / kRun;   // waves per workgroup

// (mu, w(mu) gamma v) of one element.
template <int WT, bool GAMMA>
__device__ __forceinline__ void coefficients(float f, float v, float g, float& a, float& b) {
    float r;
    sigmoid2(f, a, r);
    b = v;
    if (WT == 1) b *= r;
    if (WT == 2) b *= __builtin_amdgcn_sqrtf(r * (1.0f + a));
    if (GAMMA) {
        float s, q;
        sigmoid2(g, s, q);
        b *= s;
    }
}

template <typename TIn, int V, int WT, bool GAMMA>
__global__ __launch_bounds__(kWaves * 64) void layer_scan_fwd_kernel(ScanParams p) {
    constexpr int CB = 64 * V;  // channels per workgroup
    __shared__ float sA[kWaves][CB], sH[kWaves][CB];
    const int nblk = (p.D + CB - 1) / CB;
    const int b = static_cast<int>(blockIdx.x / nblk);
    const int c = static_cast<int>(blockIdx.x % nblk) * CB + (threadIdx.x & 63) * V;
    const int l = (threadIdx.x & 63) * V;
    const int wave = threadIdx.x >> 6;
    const bool live = c < p.D;  // V divides D: a lane's channels are all inside or all outside
    const int cc = live ? c : 0;
    const TIn* vp = static_cast<const TIn*>(p.v) + static_cast<int64_t>(b) * p.T * p.D + cc;
    const TIn* fp = static_cast<const TIn*>(p.f) + static_cast<int64_t>(b) * p.T * p.D + cc;
    const TIn* gp = GAMMA ? static_cast<const TIn*>(p.g) + static_cast<int64_t>(b) * p.T * p.D + cc : nullptr;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int tiles = (p.T + kScanTile - 1) / kScanTile;

    float carry[V];
#pragma unroll
    for (int j = 0; j < V; ++j) carry[j] = p.state_in ? p.state_in[static_cast<int64_t>(b) * p.D + cc + j] : 0.0f;

    for (int tile = 0; tile < tiles; ++tile) {
        const int t0 = tile * kScanTile + wave * kRun;
        Vec<TIn, V> rf[kRun], rv[kRun], rg[GAMMA ? kRun : 1];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int64_t row = static_cast<int64_t>(min(t0 + i, p.T - 1)) * p.D;
            rf[i] = load_vec<TIn, V>(fp, row);
            rv[i] = load_vec<TIn, V>(vp, row);
            if (GAMMA) rg[i] = load_vec<TIn, V>(gp, row);
        }
        float a[kRun][V], x[kRun][V], A[V], H[V];
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = 1.0f, H[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                coefficients<WT, GAMMA>(widen(rf[i].e[j]), widen(rv[i].e[j]), GAMMA ? widen(rg[i].e[j]) : 0.0f,
                                        a[i][j], x[i][j]);
                if (t0 + i >= len) a[i][j] = 1.0f, x[i][j] = 0.0f;
                A[j] *= a[i][j];
                H[j] = fmaf(a[i][j], H[j], x[i][j]);
            }
        __syncthreads();  // the tile before has been read
#pragma unroll
        for (int j = 0; j < V; ++j) sA[wave][l + j] = A[j], sH[wave][l + j] = H[j];
        __syncthreads();
        if (p.saved && wave == 0 && live) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                p.saved[(static_cast<int64_t>(b) * tiles + tile) * p.D + c + j] = carry[j];
        }
        float h[V];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (w == wave) h[j] = carry[j];
                carry[j] = fmaf(sA[w][l + j], carry[j], sH[w][l + j]);
            }
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                h[j] = fmaf(a[i][j], h[j], x[i][j]);
                o[j] = t0 + i < len ? h[j] : 0.0f;
            }
            if (live && t0 + i < p.T)
                store_vec<V>(p.y, (static_cast<int64_t>(b) * p.T + t0 + i) * p.D + c, o, p.y_bf16);
        }
    }
    if (p.state_out && wave == 0 && live) {
#pragma unroll
        for (int j = 0; j < V; ++j) p.state_out[static_cast<int64_t>(b) * p.D + c + j] = carry[j];
    }
}

// One token: state_out may be state_in (each channel is read, then written, by one thread).
template <typename TIn, int V, int WT, bool GAMMA>
__global__ __launch_bounds__(64) void layer_scan_step_kernel(ScanParams p) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x) * V;
    if (i >= static_cast<int64_t>(p.B) * p.D) return;
    const Vec<TIn, V> f = load_vec<TIn, V>(static_cast<const TIn*>(p.f), i);
    const Vec<TIn, V> v = load_vec<TIn, V>(static_cast<const TIn*>(p.v), i);
    Vec<TIn, V> g = {};
    if (GAMMA) g = load_vec<TIn, V>(static_cast<const TIn*>(p.g), i);
    Vec<float, V> s = {};
    if (p.state_in) s = load_vec<float, V>(p.state_in, i);
    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float a, x;
        coefficients<WT, GAMMA>(widen(f.e[j]), widen(v.e[j]), widen(g.e[j]), a, x);
        h[j] = fmaf(a, s.e[j], x);
    }
    store_vec<V>(p.state_out, i, h, false);
    store_vec<V>(p.y, i, h, p.y_bf16);
}

template <typename TIn, int V, int WT, bool GAMMA>
void launch(bool step, const ScanParams& p, hipStream_t st) {
    if (step) {
        const int64_t n = static_cast<int64_t>(p.B) * p.D / V;
        hipLaunchKernelGGL((layer_scan_step_kernel<TIn, V, WT, GAMMA>), dim3(static_cast<unsigned>((n + 63) / 64)),
                           dim3(64), 0, st, p);
        return;
    }
    const unsigned nblk = static_cast<unsigned>((p.D + 64 * V - 1) / (64 * V));
    hipLaunchKernelGGL((layer_scan_fwd_kernel<TIn, V, WT, GAMMA>), dim3(nblk * p.B), dim3(kWaves * 64), 0, st, p);
}

template <typename TIn, int V>
void pick(bool step, const ScanParams& p, hipStream_t st) {
    const bool g = p.g != nullptr;
    switch (p.weight) {
        case 0: g ? launch<TIn, V, 0, true>(step, p, st) : launch<TIn, V, 0, false>(step, p, st); break;
        case 1: g ? launch<TIn, V, 1, true>(step, p, st) : launch<TIn, V, 1, false>(step, p, st); break;
        default: g ? launch<TIn, V, 2, true>(step, p, st) : launch<TIn, V, 2, false>(step, p, st); break;
    }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int dispatch(bool step, const ScanParams& p, hipStream_t st) {
    const size_t ein = 2 * (p.in_bf16 ? 2 : 4), ey = 2 * (p.y_bf16 ? 2 : 4);
    const bool two = p.D % 2 == 0 && aligned(p.v, ein) && aligned(p.f, ein) && aligned(p.g, ein) && aligned(p.y, ey) &&
                     aligned(p.state_in, 8) && aligned(p.state_out, 8);
    if (p.in_bf16)
        two ? pick<uint16_t, 2>(step, p, st) : pick<uint16_t, 1>(step, p, st);
    else
        two ? pick<float, 2>(step, p, st) : pick<float, 1>(step, p, st);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace

int launch_scan_fwd(const ScanParams& p, hipStream_t st) { return dispatch(false, p, st); }
int launch_scan_step(const ScanParams& p, hipStream_t st) { return dispatch(true, p, st); }

}  // namespace layer
