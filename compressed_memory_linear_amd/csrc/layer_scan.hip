// layer_scan.hip -- the element-wise gated recurrence, forward and single step.
//
// Per channel, with mu_t = sigmoid(f_t), gamma_t = sigmoid(g_t) (1 without g)
// and an input weight w(mu) = 1, 1 - mu or sqrt(1 - mu^2):
//     h_t = mu_t h_{t-1} + w(mu_t) gamma_t v_t,   y_t = h_t.
// A run of tokens is an affine map of the state before it, h -> A h + H with
// A the product of its mu and H its result from a zero state; two runs in a row
// compose to (A2 A1, A2 H1 + H2), which is what lets the time axis be split.
//
// A workgroup takes one tile of kFwdTile tokens of 64 V channels (layer_chain.h): a lane
// holds V neighbouring channels, so a wave reads one contiguous piece of each
// token row, and each of its waves takes a run of kRun tokens, kept in registers as (mu, w gamma v).
// The waves' maps meet in LDS, the tile's starting state comes from its
// chain, every wave folds the runs before its own onto it and walks its run once more to form y.
// Every input is read once and every output written once.
#include "layer_chain.h"
#include "layer_device.h"
#include "layer_launch.h"

namespace layer {
namespace {

constexpr int kRun = 16;                   // tokens per wave of a tile
constexpr int kWaves = kFwdTile / kRun;   // waves per workgroup

// (mu, w(mu) gamma v) of one element.
template <int WT, bool GAMMA, bool ACC>
__device__ __forceinline__ void coefficients(float f, float v, float g, float& a, float& b) {
    float r;
    sigmoid2<ACC>(f, a, r);
    b = v * weight_of<WT>(a, r);
    if (GAMMA) {
        float s, q;
        sigmoid2<ACC>(g, s, q);
        b *= s;
    }
}

template <typename TIn, int V, int WT, bool GAMMA>
__global__ __launch_bounds__(kWaves * 64, 4) void layer_scan_fwd_kernel(ScanParams p) {
    constexpr int CB = 64 * V;  // channels per workgroup
    __shared__ Shared<kWaves, CB> s;
    __shared__ uint32_t ticket;
    const int nblk = (p.D + CB - 1) / CB;
    const int chains = p.B * nblk;
    const int tiles = (p.T + kFwdTile - 1) / kFwdTile;
    uint32_t id = blockIdx.x;
    if (p.ws) {
        if (threadIdx.x == 0) ticket = atomicAdd(static_cast<uint32_t*>(p.ws), 1u);
        __syncthreads();
        id = __builtin_amdgcn_readfirstlane(ticket);
    }
    const int tile = static_cast<int>(id / chains), chain = static_cast<int>(id % chains);
    const int b = chain / nblk;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l = (threadIdx.x & 63) * V;
    const int c = chain % nblk * CB + l;
    const bool live = c < p.D;  // V divides D: a lane's channels are all inside or all outside
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int active = max(1, (len + kFwdTile - 1) / kFwdTile);  // tiles with tokens, the first in any case
    const int t0 = tile * kFwdTile;
    const int64_t first = (static_cast<int64_t>(b) * p.T + t0) * p.D;
    const int rows = min(kFwdTile, p.T - t0);
    const int r0 = wave * kRun;  // this wave's rows of the tile
    // byte offsets of this lane's channels in the wave's first row, and from row to row
    const int ey = p.y_bf16 ? 2 : 4;
    const uint32_t oin = live ? (static_cast<uint32_t>(r0) * p.D + c) * sizeof(TIn) : kOut, din = p.D * sizeof(TIn);
    const uint32_t oy = live ? (static_cast<uint32_t>(r0) * p.D + c) * ey : kOut, dyo = p.D * ey;
    const auto yr = rows_rsrc(p.y, first * ey, rows * p.D * ey);
    if (tile >= active) {
        const float zero[V] = {};
        with_flag(p.y_bf16, [&](auto bf16) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) store_rows<V, bf16()>(yr, oy + i * dyo, zero);
        });
        return;
    }

    const auto fr = rows_rsrc(p.f, first * sizeof(TIn), rows * p.D * sizeof(TIn));
    const auto vr = rows_rsrc(p.v, first * sizeof(TIn), rows * p.D * sizeof(TIn));
    const auto gr = rows_rsrc(GAMMA ? p.g : p.f, first * sizeof(TIn), rows * p.D * sizeof(TIn));
    Vec<TIn, V> rf[kRun], rv[kRun], rg[GAMMA ? kRun : 1];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        rf[i] = load_rows<TIn, V>(fr, oin + i * din);
        rv[i] = load_rows<TIn, V>(vr, oin + i * din);
        if (GAMMA) rg[i] = load_rows<TIn, V>(gr, oin + i * din);
    }
    float before[V] = {};  // the chain's first state
    const int64_t sc = static_cast<int64_t>(b) * p.D + c;
    if (p.state_in && live && wave == 0 && tile < (p.ws ? p.group : 1)) {
#pragma unroll
        for (int j = 0; j < V; ++j) before[j] = p.state_in[sc + j];
    }

    float a[kRun][V], x[kRun][V], A[V], H[V];
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = 1.0f, H[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < kRun; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            coefficients<WT, GAMMA, kAccurate<TIn>>(widen(rf[i].e[j]), widen(rv[i].e[j]),
                                                    GAMMA ? widen(rg[i].e[j]) : 0.0f, a[i][j], x[i][j]);
            A[j] *= a[i][j];
            H[j] = fmaf(a[i][j], H[j], x[i][j]);
        }
    // Padding keeps the state.  Set right afterwards, in the one tile that has both, so that the
    // others pay nothing.
    const bool padded = t0 + kFwdTile > len;
    if (padded) {
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = 1.0f, H[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (t0 + r0 + i >= len) a[i][j] = 1.0f, x[i][j] = 0.0f;
                A[j] *= a[i][j];
                H[j] = fmaf(a[i][j], H[j], x[i][j]);
            }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s.A[wave][l + j] = A[j], s.H[wave][l + j] = H[j];
    __syncthreads();
    const bool last = tile == active - 1;
    if (wave == 0) {
        // the tile's map
#pragma unroll 2
        for (int w = 1; w < kWaves; ++w)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                H[j] = fmaf(s.A[w][l + j], H[j], s.H[w][l + j]);
                A[j] *= s.A[w][l + j];
            }
    }
    if (p.ws) {
        chain_carry<V>(s, chain_of(p.ws, chains, tiles, p.group, CB), chain, tile, last, before, A, H);
    } else {
        if (wave == 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) s.carry[l + j] = before[j];
        }
        __syncthreads();
    }
    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = s.carry[l + j];
    if (wave == 0 && live) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (p.state_out && last) p.state_out[sc + j] = len > 0 ? fmaf(A[j], h[j], H[j]) : h[j];
        }
    }
    for (int w = 0; w < wave; ++w)
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = fmaf(s.A[w][l + j], h[j], s.H[w][l + j]);
    if (p.saved && live && r0 % kBwdTile == 0 && r0 < rows) {
        const int64_t saves = (p.T + kBwdTile - 1) / kBwdTile;
#pragma unroll
        for (int j = 0; j < V; ++j) p.saved[(b * saves + (t0 + r0) / kBwdTile) * p.D + c + j] = h[j];
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) x[i][j] = h[j] = fmaf(a[i][j], h[j], x[i][j]);
    if (padded) {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (t0 + r0 + i >= len) x[i][j] = 0.0f;
    }
    with_flag(p.y_bf16, [&](auto bf16) {
        const uint32_t to = here(oy);
#pragma unroll
        for (int i = 0; i < kRun; ++i) store_rows<V, bf16()>(yr, to + i * dyo, x[i]);
    });
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
        coefficients<WT, GAMMA, kAccurate<TIn>>(widen(f.e[j]), widen(v.e[j]), widen(g.e[j]), a, x);
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
    const unsigned tiles = static_cast<unsigned>(tiles_of(p.T, kFwdTile));
    hipLaunchKernelGGL((layer_scan_fwd_kernel<TIn, V, WT, GAMMA>), dim3(nblk * p.B * tiles), dim3(kWaves * 64), 0, st,
                       p);
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

// Marks every hand-off of the workspace empty and sets the ticket to 0.
__global__ __launch_bounds__(256) void layer_scan_clear_kernel(uint64_t* ws, int64_t words) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < words; i += gridDim.x * 256)
        ws[i] = i < kTicketBytes / 8 ? 0 : ~UINT64_C(0);
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

int scan_group(int B, int T, int D) {
    (void)B, (void)T, (void)D;
    return 16;
}

size_t scan_workspace_bytes(int B, int T, int D) {
    const size_t tiles = tiles_of(T, kFwdTile < kBwdTile ? kFwdTile : kBwdTile);
    if (tiles == 1) return 0;
    const size_t groups = tiles_of(tiles, scan_group(B, T, D)), width = tiles_of(D, 128) * 128;
    return kTicketBytes + (tiles + groups) * width * B * sizeof(uint64_t);
}

void clear_scan_workspace(const ScanParams& p, hipStream_t st) {
    if (!p.ws) return;
    const int64_t words = static_cast<int64_t>(scan_workspace_bytes(p.B, p.T, p.D) / 8);
    const int64_t want = (words + 1023) / 1024;
    hipLaunchKernelGGL(layer_scan_clear_kernel, dim3(static_cast<unsigned>(want < 1024 ? want : 1024)), dim3(256), 0,
                       st, static_cast<uint64_t*>(p.ws), words);
}

int launch_scan_fwd(const ScanParams& p, hipStream_t st) {
    clear_scan_workspace(p, st);
    return dispatch(false, p, st);
}
int launch_scan_step(const ScanParams& p, hipStream_t st) { return dispatch(true, p, st); }

}  // namespace layer
