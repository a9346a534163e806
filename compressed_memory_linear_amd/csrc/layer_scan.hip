// layer_scan.hip -- the element-wise gated recurrence, forward and single step.
//
// Per channel, with mu_t = sigmoid(f_t), gamma_t = sigmoid(g_t) (1 without g)
// and an input weight w(mu) = 1, 1 - mu or sqrt(1 - mu^2):
//     h_t = mu_t h_{t-1} + w(mu_t) gamma_t v_t,   y_t = h_t.
// A run of tokens is an affine map of the state before it, h -> A h + H with
// A the product of its mu and H its result from a zero state; two runs in a row
// compose to (A2 A1, A2 H1 + H2), which is what lets the time axis be split.
//
// A workgroup takes one tile (layer_chain.h): each of its waves a run of kFwdRun
// tokens of 64 channels, kept in registers as (mu, w gamma v).
// The waves' maps meet in LDS, the tile's starting state comes from its
// chain, every wave folds the runs before its own onto it and walks its run once
// more to form y.  Every input is read once and every output written once.
//
// Bound by HBM (bf16, D2048): B8 T4096 403 MB in 79 us, 5.1 TB/s; B1 T65536 with the writing
// intensity 1.07 GB in 209 us, 5.1 TB/s (the device's own copy of 1 GiB: 5.4); 18 vector
// operations per element (24 with the intensity), two of the slow kind per gate, keep the vector units
// 43 % busy.  The kernel that clears the hand-off words costs 3 to 5 us more.
#include "layer_chain.h"
#include "layer_device.h"
#include "layer_launch.h"

namespace layer {
namespace {

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

template <typename TIn, int WT, bool GAMMA>
__global__ __launch_bounds__(kScanWaves * 64, 4) void layer_scan_fwd_kernel(ScanParams p) {
    __shared__ Shared s;
    __shared__ uint32_t ticket;
    const int chains = p.B * ((p.D + 63) / 64);
    const int tiles = (p.T + kFwdTile - 1) / kFwdTile;
    const Place me = take_place(p.ws, p.D, chains, &ticket);
    const int tile = me.pos, b = me.b, wave = me.wave, l = me.l, c = me.c;
    const bool live = c < p.D;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int active = max(1, (len + kFwdTile - 1) / kFwdTile);  // tiles with tokens, the first in any case
    const int t0 = tile * kFwdTile;
    const int64_t first = (static_cast<int64_t>(b) * p.T + t0) * p.D;
    const int rows = min(kFwdTile, p.T - t0);
    const int r0 = wave * kFwdRun;  // this wave's rows of the tile
    // byte offsets of this lane's channel in the wave's first row, and from row to row
    const int ey = p.y_bf16 ? 2 : 4;
    const uint32_t at = static_cast<uint32_t>(r0) * p.D + c;
    const uint32_t oin = live ? at * sizeof(TIn) : kOut, din = p.D * sizeof(TIn);
    const uint32_t oy = live ? at * ey : kOut, dyo = p.D * ey;
    const auto yr = rows_rsrc(p.y, first * ey, rows * p.D * ey);
    if (tile >= active) {
        with_flag(p.y_bf16, [&](auto bf16) {
#pragma unroll
            for (int i = 0; i < kFwdRun; ++i) store_row<bf16(), false>(yr, oy + i * dyo, 0.0f);
        });
        return;
    }

    const int nin = rows * p.D * static_cast<int>(sizeof(TIn));
    const auto fr = rows_rsrc(p.f, first * sizeof(TIn), nin);
    const auto vr = rows_rsrc(p.v, first * sizeof(TIn), nin);
    const auto gr = rows_rsrc(GAMMA ? p.g : p.f, first * sizeof(TIn), nin);
    TIn rf[kFwdRun], rv[kFwdRun], rg[GAMMA ? kFwdRun : 1];
#pragma unroll
    for (int i = 0; i < kFwdRun; ++i) {
        rf[i] = load_row<TIn>(fr, oin + i * din);
        rv[i] = load_row<TIn>(vr, oin + i * din);
        if (GAMMA) rg[i] = load_row<TIn>(gr, oin + i * din);
    }
    const int64_t sc = static_cast<int64_t>(b) * p.D + c;
    float before = 0.0f;  // the state before the chain
    if (p.state_in && live && wave == 0 && tile < kScanWaves * kScanWaves) before = p.state_in[sc];

    float a[kFwdRun], x[kFwdRun], A = 1.0f, H = 0.0f;
#pragma unroll
    for (int i = 0; i < kFwdRun; ++i) {
        coefficients<WT, GAMMA, kAccurate<TIn>>(widen(rf[i]), widen(rv[i]), GAMMA ? widen(rg[i]) : 0.0f, a[i], x[i]);
        A *= a[i];
        H = fmaf(a[i], H, x[i]);
    }
    // Padding keeps the state.  Set right afterwards, in the one tile that has both, so that the
    // others pay nothing.
    const bool padded = t0 + kFwdTile > len;
    if (padded) {
        A = 1.0f, H = 0.0f;
#pragma unroll
        for (int i = 0; i < kFwdRun; ++i) {
            if (t0 + r0 + i >= len) a[i] = 1.0f, x[i] = 0.0f;
            A *= a[i];
            H = fmaf(a[i], H, x[i]);
        }
    }
    A = run_product(A, a);
    s.A[wave][l] = A, s.H[wave][l] = H;
    const Chain links = chain_of(p.ws, chains, tiles);
    Carry from{s, links, me.chain, tile, wave, l};
    if (p.ws) from.begin();
    __syncthreads();
    const bool last = tile == active - 1;
    const int waves = blockDim.x >> 6;
    if (wave == 0) {
        // the tile's map
#pragma unroll
        for (int w = 1; w < kScanWaves; ++w)
            if (w < waves) {
                H = fmaf(s.A[w][l], H, s.H[w][l]);
                A = times(A, s.A[w][l]);
            }
    }
    if (p.ws) {
        from.finish(last, before, A, H);
    } else {
        if (wave == 0) s.carry[l] = before;
        __syncthreads();
    }
    float h = s.carry[l];
    if (p.state_out && last && wave == 0 && live) p.state_out[sc] = len > 0 ? fmaf(A, h, H) : h;
    for (int w = 0; w < wave; ++w) h = fmaf(s.A[w][l], h, s.H[w][l]);
    if (p.saved && live && (t0 + r0) % kBwdTile == 0 && r0 < rows) {
        const int64_t saves = (p.T + kBwdTile - 1) / kBwdTile;
        p.saved[(b * saves + (t0 + r0) / kBwdTile) * p.D + c] = h;
    }
#pragma unroll
    for (int i = 0; i < kFwdRun; ++i) x[i] = h = fmaf(a[i], h, x[i]);
    if (padded) {
#pragma unroll
        for (int i = 0; i < kFwdRun; ++i)
            if (t0 + r0 + i >= len) x[i] = 0.0f;
    }
    with_flag(p.y_bf16, [&](auto bf16) {
        const uint32_t to = here(oy);
#pragma unroll
        for (int i = 0; i < kFwdRun; ++i) store_row<bf16(), false>(yr, to + i * dyo, x[i]);
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
    const Vec<float, V> s = load_vec<float, V>(p.state_in, i);
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

template <typename TIn, int WT, bool GAMMA>
void launch(bool step, const ScanParams& p, hipStream_t st) {
    if (!step) {
        const unsigned chains = static_cast<unsigned>(tiles_of(p.D, 64)) * p.B;
        hipLaunchKernelGGL((layer_scan_fwd_kernel<TIn, WT, GAMMA>), dim3(chains * tiles_of(p.T, kFwdTile)),
                           dim3(scan_threads(p.T, kFwdRun)), 0, st, p);
        return;
    }
    // four neighbours a thread where every buffer is aligned for it
    const int64_t n = static_cast<int64_t>(p.B) * p.D;
    bool four = n % 4 == 0;
    for (const void* q : {p.v, p.f, p.g}) four = four && reinterpret_cast<uintptr_t>(q) % (4 * sizeof(TIn)) == 0;
    four = four && reinterpret_cast<uintptr_t>(p.y) % (p.y_bf16 ? 8 : 16) == 0;
    for (const float* q : {p.state_in, static_cast<const float*>(p.state_out)})
        four = four && reinterpret_cast<uintptr_t>(q) % 16 == 0;
    if (four)
        hipLaunchKernelGGL((layer_scan_step_kernel<TIn, 4, WT, GAMMA>), dim3(tiles_of(n, 256)), dim3(64), 0, st, p);
    else
        hipLaunchKernelGGL((layer_scan_step_kernel<TIn, 1, WT, GAMMA>), dim3(tiles_of(n, 64)), dim3(64), 0, st, p);
}

template <typename TIn>
int pick(bool step, const ScanParams& p, hipStream_t st) {
    const bool g = p.g != nullptr;
    switch (p.weight) {
        case 0: g ? launch<TIn, 0, true>(step, p, st) : launch<TIn, 0, false>(step, p, st); break;
        case 1: g ? launch<TIn, 1, true>(step, p, st) : launch<TIn, 1, false>(step, p, st); break;
        default: g ? launch<TIn, 2, true>(step, p, st) : launch<TIn, 2, false>(step, p, st); break;
    }
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

// Marks every hand-off of the workspace empty and sets the ticket to 0.  words is even:
// the ticket's and multiples of 64 channels.
__global__ __launch_bounds__(256) void layer_scan_clear_kernel(uint64_t* ws, int64_t words) {
    typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 2; i < words; i += gridDim.x * 512ll) {
        const uint64_t e = i < kTicketBytes / 8 ? 0 : ~UINT64_C(0);
        *reinterpret_cast<u64x2*>(ws + i) = u64x2{e, e};
    }
}

// Hand-off words of one direction: maps of the tiles and groups, states of the supergroups.
int64_t scan_words(int B, int T, int D, int tile) {
    const int64_t tiles = tiles_of(T, tile), groups = tiles_of(tiles, kScanWaves);
    return kTicketBytes / 8 + (tiles + groups + tiles_of(groups, kScanWaves)) * tiles_of(D, 64) * 64 * B;
}

}  // namespace

size_t scan_workspace_bytes(int B, int T, int D) {
    static_assert(kBwdTile <= kFwdTile, "the backward has the more tiles");
    return T <= kBwdTile ? 0 : scan_words(B, T, D, kBwdTile) * sizeof(uint64_t);
}

void clear_scan_workspace(const ScanParams& p, int tile, hipStream_t st) {
    const int64_t words = scan_words(p.B, p.T, p.D, tile), want = (words + 2047) / 2048;
    hipLaunchKernelGGL(layer_scan_clear_kernel, dim3(static_cast<unsigned>(want < 2048 ? want : 2048)), dim3(256), 0,
                       st, static_cast<uint64_t*>(p.ws), words);
}

int launch_scan_fwd(const ScanParams& p, hipStream_t st) {
    ScanParams q = p;
    if (p.T <= kFwdTile) q.ws = nullptr;  // one tile, nothing to hand on
    if (q.ws) clear_scan_workspace(q, kFwdTile, st);
    return p.in_bf16 ? pick<uint16_t>(false, q, st) : pick<float>(false, q, st);
}
int launch_scan_step(const ScanParams& p, hipStream_t st) {
    return p.in_bf16 ? pick<uint16_t>(true, p, st) : pick<float>(true, p, st);
}

}  // namespace layer
