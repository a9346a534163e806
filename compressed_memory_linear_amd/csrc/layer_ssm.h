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

constexpr int kSsmTile = 16;  // tokens per tile of the forward
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// softplus(v) and its derivative.  With e = exp(-|v|) in [0, 1], softplus = max(v, 0) + log(1 + e) and
// log(1 + e) = 2 atanh(t), t = e / (2 + e) <= 1/3: an odd polynomial of degree 9, the nearest in relative
// error (7.8e-9, fitted for this by reweighted least squares), so that small steps keep their relative accuracy.
template <bool ACC>
__device__ __forceinline__ void softplus_parts(float v, float& d, float& slope) {
    const float e = exp_of<ACC>(-fabsf(v));
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

// What the kernels hold of a decay: A log2(e), kept finite where A is (a step of zero keeps the state, whatever A).
__device__ __forceinline__ float ssm_decay(float a) {
    const float v = a * kLog2e;
    return fabsf(v) == __builtin_inff() ? __builtin_copysignf(3.40282347e38f, v) : v;
}

// A state (or a gradient) h across a segment of the time axis: exp(A sum) h + H, with the sum of the segment's steps and
// what it makes of zeros, H.  S is the sum times 2^-31, so that no sum of up to 2^30 finite steps is infinite.  A
// segment with a document's border in it (S = inf) passes nothing on, whatever it is.  The
// decay goes in two halves, each kept between the least and the largest float: an infinite h stays one where the
// product of decays underflows and a zero stays one where growth (A > 0) overflows, as token by token.
__device__ __forceinline__ float ssm_steps(double sum, bool dropped) {
    return dropped ? __builtin_inff() : static_cast<float>(sum * 0x1p-31);
}
__device__ __forceinline__ float ssm_across(float A, float S, float h, float H) {
    const float P = fminf(fmaxf(__builtin_amdgcn_exp2f(0x1p30f * (A * S)), 1.40129846e-45f), 3.40282347e38f);
    return S == __builtin_inff() ? H : fmaf(P * h, P, H);
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

// The rows of a tensor [B,T,D] (row elements apart) of one tile after the other, each as a buffer that ends with
// the last row in use (of no bytes where the tensor is absent); `width` elements of a row count.
struct SsmStream {
    uintptr_t at;
    uint32_t row_bytes, width_bytes;
    __device__ __forceinline__ SsmStream(const void* p, int64_t token, int row, int width, int size) {
        row_bytes = p ? row * size : 0;
        width_bytes = p ? width * size : 0;
        at = reinterpret_cast<uintptr_t>(p) + static_cast<uint64_t>(token) * row_bytes;
    }
    __device__ __forceinline__ void move(int rows) { at += static_cast<int64_t>(rows) * row_bytes; }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(int count) const {
        const uint32_t bytes = count > 0 ? (count - 1) * row_bytes + width_bytes : 0;
        return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at), 0, bytes, 0x00020000);
    }
};

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

// B and C are the same for every channel of a group.  A register holds one state's values of 16 tokens, the same in
// each row of 16 lanes, and the vector instruction that multiplies with one of them takes it from its lane by itself
// (row_newbcast): no load, no register and no instruction per value.  (As scalar loads, prefetched 4 tokens ahead
// from a packed copy, they kept a wave waiting for 60 % of its time.  The products are outer products of states and lanes,
// which the matrix cores' sixteen blocks of 4 x 4 x 1 form in fp32, but one of those instructions takes the
// vector unit 16 cycles beside other work, no less than the four that it stands for: B8 T4096 D2048 317 -> 373 us.)
template <int K>
__device__ __forceinline__ float bcast(float x) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x150 + K, 0xf, 0xf, true));
}

// Four neighbouring elements at byte offset off of a buffer: in one piece, or one by one, of which those from
// `count` on are outside.
template <typename T, bool VEC, bool NT>
__device__ __forceinline__ Vec<T, 4> load_quad(__amdgpu_buffer_rsrc_t r, uint32_t off, int count) {
    if constexpr (VEC && sizeof(T) == 2) {
        return __builtin_bit_cast(Vec<T, 4>, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, NT ? kNt : 0));
    } else if constexpr (VEC) {
        return __builtin_bit_cast(Vec<T, 4>, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, NT ? kNt : 0));
    } else {
        Vec<T, 4> v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v.e[e] = load_row<T, NT>(r, e < count ? off + e * static_cast<uint32_t>(sizeof(T)) : kOut);
        return v;
    }
}
template <bool VEC, bool BF16, bool NT>
__device__ __forceinline__ void store_quad(__amdgpu_buffer_rsrc_t r, uint32_t off, int count, const float (&x)[4]) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    if constexpr (VEC && BF16) {
        u32x2 w;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[j] = osr::f32_to_bf16_bits(x[2 * j]) | static_cast<uint32_t>(osr::f32_to_bf16_bits(x[2 * j + 1])) << 16;
        __builtin_amdgcn_raw_buffer_store_b64(w, r, off, 0, NT ? kNt : 0);
    } else if constexpr (VEC) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(x[j]);
        __builtin_amdgcn_raw_buffer_store_b128(w, r, off, 0, NT ? kNt : 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) store_row<BF16, NT>(r, e < count ? off + e * (BF16 ? 2u : 4u) : kOut, x[e]);
    }
}

// The channels whose inputs and outputs a thread takes: four neighbours, of every few tokens of each tile.  id: its
// number among the threads that do so.
struct SsmQuad {
    int row, c, count;  // the first of those tokens; channels c .. c + count - 1
    int at;             // c in its block of 64
};
__device__ __forceinline__ SsmQuad ssm_quad(const SsmParams& p, const SsmPlace& me, int chain, int id) {
    SsmQuad q;
    const int width = p.D / p.G, k = chain % ssm_blocks(p) * 64 + (id & 15) * 4;
    q.row = id >> 4;
    q.at = (id & 15) * 4;
    q.c = me.g * width + k;
    q.count = min(max(width - k, 0), 4);
    return q;
}
// Byte offsets of its quads in a tile's rows, every `step` tokens.
template <int K>
struct QuadOffsets {
    uint32_t at[K];
    __device__ __forceinline__ QuadOffsets(const SsmQuad& q, int stride, int step, int size) {
#pragma unroll
        for (int i = 0; i < K; ++i)
            at[i] = here(q.count > 0 ? static_cast<uint32_t>((q.row + i * step) * stride + q.c) * size : kOut);
    }
};
// A weight of four channels, zeros where it is absent.
__device__ __forceinline__ void quad_weights(const float* w, const SsmQuad& q, float (&o)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = w && e < q.count ? w[q.c + e] : 0.0f;
}

// B or C of a tile's 16 tokens, a register per state: lanes as tokens, the same in each row of 16.
template <typename T, int SN, bool VEC>
struct SsmRegs {
    static constexpr int Q = SN / 4;
    Vec<T, 4> raw[Q];
    uint32_t at[Q];
    int count;  // states from n0 on
    __device__ __forceinline__ void place(int l, int n0, int N, int row) {
        count = N - n0;
#pragma unroll
        for (int k = 0; k < Q; ++k)
            at[k] = here(4 * k < count ? static_cast<uint32_t>((l & 15) * row + n0 + 4 * k) * static_cast<uint32_t>(sizeof(T))
                                       : kOut);
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r) {
#pragma unroll
        for (int k = 0; k < Q; ++k) raw[k] = load_quad<T, VEC, false>(r, at[k], count - 4 * k);
    }
    __device__ __forceinline__ void get(float (&o)[SN]) const {
#pragma unroll
        for (int n = 0; n < SN; ++n) o[n] = widen(raw[n / 4].e[n % 4]);
    }
};

// Whether inputs and outputs can move in quads of elements: the quads lie within a group and every row of every
// tensor is aligned to one (B and C to a quad of states).
inline bool ssm_vec(const SsmParams& p) {
    if (p.D / p.G % 4 != 0 || p.N % 4 != 0) return false;
    for (int row : {p.x_row, p.dt_row, p.z_row, p.b_row, p.c_row})
        if (row % 4 != 0) return false;
    const uintptr_t in = p.in_bf16 ? 8 : 16, y = p.y_bf16 ? 8 : 16, g = p.grad_bf16 ? 8 : 16;
    for (const void* q : {p.x, p.dt, p.z, p.Bm, p.Cm})
        if (reinterpret_cast<uintptr_t>(q) % in != 0) return false;
    for (const void* q : {static_cast<const void*>(p.y), p.dy})
        if (reinterpret_cast<uintptr_t>(q) % y != 0) return false;
    for (const void* q : {p.dx, p.ddt, p.dz})
        if (reinterpret_cast<uintptr_t>(q) % g != 0) return false;
    return true;
}

__host__ __device__ inline int ssm_padded(int N) { return N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }

// The time axis in segments of whole tiles.  One of them where the chains nearly fill the device, since taking every
// segment twice costs more; else as many as fill it, and hide one another's waits.
// Forward, by the waves that walk over states for 1024 vector units (D2048 N16 bf16): B8 T4096 (1024 waves) 1 segment
// 321 us, 3 411; B1 T65536 (128 waves) 8 segments 1051, 24 876, 32 867; B7 T1531 D1001 N13 padded fp32 (448 waves) 2
// 149, 6 130, 9 122.  Past 32 states a wave holds twice as many: training step of B3 T777 D514 N64 with 7 segments
// forward 427 us, 10 471.  Backward, by workgroups, of which a compute unit's LDS holds one past 8 states: training step
// of B4 T4096 D2048 N16 (128 chains) 2 segments 1000 us, 4 970, 8 980; B3 T777 D514 N64 (30 chains) 4 749, 8 529, 12 597.
// Past 176 chains there is one: 256 of them (B8 T4096 D2048) take 1137 us, 288 (B9) two rounds of the device and 2235.
// The kernel of its maps has smaller workgroups and takes long segments in four parts (B4 T4096, 64 tiles a segment:
// 128 -> 95 us), short ones whole, since each segment reads the maps of all parts behind it (the training step of
// B3 T777, 7 tiles a segment: whole 393 us, in four parts 427).
struct SsmSplit {
    int64_t chains, length;
    int segs, parts;  // parts of a segment, each with a map of its own
};
inline SsmSplit ssm_split(const SsmParams& p, bool backward) {
    SsmSplit s;
    s.chains = tiles_of(p.D / p.G, 64) * p.G * p.B;
    const int64_t waves = s.chains * (p.N <= 4 ? 1 : p.N <= 8 ? 2 : p.N <= 16 ? 4 : 8), tiles = tiles_of(p.T, kSsmTile);
    int64_t want = waves > 704 ? 1 : (p.N <= 32 ? 4096 : 2048) / waves;
    if (backward) want = s.chains > 176 ? 1 : (p.N <= 16 ? 512 : 256) / s.chains;
    if (want > 64) want = 64;
    if (want > tiles / 4) want = tiles / 4;  // 64 tokens or more each
    if (want < 1) want = 1;
    int per = static_cast<int>(tiles_of(tiles, static_cast<int>(want)));
    s.parts = backward && want > 1 && per >= 16 ? 4 : 1;
    per = static_cast<int>(tiles_of(per, s.parts)) * s.parts;
    s.length = static_cast<int64_t>(per) * kSsmTile;
    s.segs = static_cast<int>(tiles_of(tiles, per));
    return s;
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
