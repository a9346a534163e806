// layer_ssm.h -- what the kernels of the selective state space scan share.
//
// Per channel, with delta = softplus(dt + bias) and u = delta x,
//     h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + u_t B_t[n],   y_t = sum_n C_t[n] h_t[n] + skip x_t.
// A lane holds SN of a channel's states, the NW waves of a workgroup take the N states of one block of 64
// channels between them, and the workgroup walks along the time axis in tiles: the waves share the work per token
// and channel (delta, u, the gate) through LDS and each sums its own states' part of y.
#pragma once

#include "layer_device.h"
#include "layer_launch.h"

namespace layer {

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// softplus(v) and its derivative.  With e = exp(-|v|) in [0, 1], softplus = max(v, 0) + log(1 + e) and
// log(1 + e) = 2 atanh(t), t = e / (2 + e) <= 1/3: an odd polynomial of degree 9, the nearest in relative
// error (4e-9, fitted for this by reweighted least squares), so that small steps keep their relative accuracy.
__device__ __forceinline__ void softplus_parts(float v, float& d, float& slope) {
    const float e = exp_of<true>(-fabsf(v));
    const float t = e * __builtin_amdgcn_rcpf(2.0f + e), q = t * t;
    float s = 0.281783342f;
    s = fmaf(s, q, 0.279606014f);
    s = fmaf(s, q, 0.400249094f);
    s = fmaf(s, q, 0.666663170f);
    s = fmaf(s, q, 2.0f);
    // NaN: e is NaN, and max(v, 0) is 0
    d = fmaf(t, s, fmaxf(v, 0.0f));
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    slope = v < 0.0f ? e * r : r;
}

// Channels of a workgroup: chain = (b G + g) blocks + block of 64 channels of the group.
struct SsmPlace {
    int b, g, c, wave, l;
    bool live;
    int len;
};
__device__ __forceinline__ int ssm_blocks(const SsmParams& p) { return (p.D / p.G + 63) / 64; }
__device__ __forceinline__ SsmPlace ssm_place(const SsmParams& p, int chain) {
    SsmPlace at;
    const int blocks = ssm_blocks(p), width = p.D / p.G;
    at.b = chain / blocks / p.G;
    at.g = chain / blocks % p.G;
    at.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    at.l = threadIdx.x & 63;
    const int k = chain % blocks * 64 + at.l;
    at.live = k < width;
    at.c = at.g * width + (at.live ? k : 0);
    at.len = p.lengths ? min(max(p.lengths[at.b], 0), p.T) : p.T;
    return at;
}

// Rows of a tensor [B,T,D] (row elements apart) from token t0 on, as a buffer.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t ssm_rows(const void* p, int b, int T_, int t0, int rows, int row, int D) {
    const int64_t first = (static_cast<int64_t>(b) * T_ + t0) * row;
    const int bytes = p && rows > 0 ? ((rows - 1) * row + D) * static_cast<int>(sizeof(T)) : 0;
    return rows_rsrc(p, first * static_cast<int64_t>(sizeof(T)), bytes);
}

// Which tokens of a tile of up to 64 begin a document (bit i: token t0 + i); the same in every lane.
__device__ __forceinline__ uint64_t ssm_cuts(const SsmParams& p, int b, int t0, int n, int l) {
    if (!p.segments) return 0;
    const int t = t0 + l;
    bool cut = false;
    if (l < n && t > 0) {
        const int32_t* s = p.segments + static_cast<int64_t>(b) * p.T + t;
        cut = s[0] != s[-1];
    }
    return __ballot(cut);
}

// B and C of a tile's tokens as floats [token][2][NP], zeros past N and at padding (so that
// whatever stands there reaches nothing).
template <typename TIn, int NP, int TILE, int NT>
__device__ __forceinline__ void ssm_load_bc(const SsmParams& p, const SsmPlace& me, int t0, int n, float (*bc)[2 * NP]) {
    const int64_t row = static_cast<int64_t>(me.b) * p.T + t0;
    const TIn* Bm = static_cast<const TIn*>(p.Bm) + row * p.b_row + me.g * p.N;
    const TIn* Cm = static_cast<const TIn*>(p.Cm) + row * p.c_row + me.g * p.N;
    for (int i = threadIdx.x; i < TILE * 2 * NP; i += NT) {
        const int t = i / (2 * NP), k = i % (2 * NP), s = k % NP;
        float v = 0.0f;
        if (t < n && s < p.N) v = widen(k < NP ? Bm[static_cast<int64_t>(t) * p.b_row + s] : Cm[static_cast<int64_t>(t) * p.c_row + s]);
        bc[t][k] = v;
    }
}

// Calls f with the states per lane and waves of a workgroup for N states.
template <typename F>
void with_states(int N, F&& f) {
    const std::integral_constant<int, 4> four;
    const std::integral_constant<int, 8> eight;
    if (N <= 4) f(four, std::integral_constant<int, 1>());
    else if (N <= 8) f(four, std::integral_constant<int, 2>());
    else if (N <= 16) f(four, four);
    else if (N <= 32) f(four, eight);
    else f(eight, eight);
}

}  // namespace layer
