// layer_chain.h -- the scan's tiles and the hand-off between their workgroups.
//
// The time axis is cut into tiles and the channels into
// blocks of 64 V; a workgroup takes one tile of one block of one sequence (a
// chain), reads it once, and needs from the rest of its chain only the state
// before the tile (forward; in the backward, which runs the tiles from the last to
// the first, the gradient from behind it).  A tile maps that state by
// h -> A h + H, and its (A, H) does not depend on the tiles before it, so it is
// published at once.  Tiles come in groups of `group`: a tile composes the maps of the
// tiles before it in its group, waits for the state before the group, and the
// group's last tile hands the state behind it on.  So a chain waits once per
// group instead of once per tile, and every sum has a fixed order.
//
// Which tile a workgroup takes follows a ticket that it draws when it starts
// (tiles of all chains in turn): whatever a workgroup waits for belongs to a lower
// ticket, so its owner has started, and the first unfinished ticket waits for
// nothing that is unfinished; every wait ends, whatever the order of dispatch.
//
// A hand-off is a pair of floats stored and loaded as one 64-bit word at agent
// scope.  The fill kernel in front marks all words empty; a word is read until it is
// not.  The word is its own flag: no ordering between words is needed.
#pragma once

#include <type_traits>

#include "layer_device.h"
#include "layer_launch.h"

namespace layer {

constexpr uint32_t kEmpty = 0xffffffffu;  // of the pair's first half
constexpr int kTicketBytes = 64;

// Words of a chain block: [chain][tile][64 V] maps, then [chain][group][64 V] states.
struct Chain {
    uint64_t *maps, *states;
    int tiles, groups, group, width;
    __device__ __forceinline__ uint64_t* map_at(int chain, int tile) const {
        return maps + (static_cast<int64_t>(chain) * tiles + tile) * width;
    }
    __device__ __forceinline__ uint64_t* state_at(int chain, int g) const {
        return states + (static_cast<int64_t>(chain) * groups + g) * width;
    }
};

__device__ __forceinline__ void put_pair(uint64_t* p, float a, float b) {
    // a NaN could look empty; any other NaN says the same
    const uint32_t x = a != a ? 0x7fc00000u : __float_as_uint(a);
    const uint64_t w = static_cast<uint64_t>(__float_as_uint(b)) << 32 | x;
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek_pair(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The pair at p once it is there.  The number of looks is bounded so that no fault elsewhere can
// turn into a hang; a wait that gives up leaves NaN behind.
__device__ __forceinline__ void get_pair(const uint64_t* p, uint64_t w, float& a, float& b) {
    for (int i = 0; static_cast<uint32_t>(w) == kEmpty && i < osr::XSPIN; ++i) {
        __builtin_amdgcn_s_sleep(1);
        w = peek_pair(p);
    }
    a = __uint_as_float(static_cast<uint32_t>(w));
    b = __uint_as_float(static_cast<uint32_t>(w >> 32));
}

// Rows of a tile as a buffer of their own: an access past the tile's last row, or
// by a lane without channels (kOut), reads zero and writes nothing.  Offsets are in
// bytes, whole in the address register (the part of the bounds check that needs no
// care); a tile has at most 2^29, so kOut plus a row's offset lies outside and does not wrap.
constexpr uint32_t kOut = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* p, int64_t first, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(static_cast<char*>(const_cast<void*>(p)) + first, 0, bytes, 0x00020000);
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_rows(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    constexpr int N = sizeof(T) * V;
    if constexpr (N == 2)
        return __builtin_bit_cast(Vec<T, V>, static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0)));
    else if constexpr (N == 4)
        return __builtin_bit_cast(Vec<T, V>, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
    else
        return __builtin_bit_cast(Vec<T, V>, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
}
template <int V, bool BF16>
__device__ __forceinline__ void store_rows(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&x)[V]) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    static_assert(V == 1 || V == 2, "one or two channels per lane");
    if constexpr (BF16 && V == 1)
        __builtin_amdgcn_raw_buffer_store_b16(osr::f32_to_bf16_bits(x[0]), r, off, 0, 0);
    else if constexpr (BF16)
        __builtin_amdgcn_raw_buffer_store_b32(
            osr::f32_to_bf16_bits(x[0]) | static_cast<uint32_t>(osr::f32_to_bf16_bits(x[1])) << 16, r, off, 0, 0);
    else if constexpr (V == 1)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[0]), r, off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(x[0]), __float_as_uint(x[1])}, r, off, 0, 0);
}

// The value, in a register whose origin the compiler does not see: offsets taken from
// it are formed where they are used and not held from the top of the kernel (16 to 32 registers).
__device__ __forceinline__ uint32_t here(uint32_t x) {
    asm("" : "+v"(x));
    return x;
}

// f(constant) for a flag that is the same in every thread: one branch around a whole
// loop instead of one in each of its steps.
template <typename F>
__device__ __forceinline__ void with_flag(bool flag, F&& f) {
    if (flag)
        f(std::true_type());
    else
        f(std::false_type());
}

// What the waves of a workgroup share: their runs' maps, the composed maps of the tiles
// before, the state before the tile.
template <int W, int CB>
struct Shared {
    float A[W][CB], H[W][CB];
    float PA[W][CB], PH[W][CB];
    float carry[CB];
};

// The state before this workgroup's tile, into s.carry (every wave calls this; barriers inside).
// Wave 0 holds the tile's own map (A, H) and the state before the chain, `first`.
// rank: the tile's place in its chain; last: no tile follows.
template <int V, int W, int CB>
__device__ __forceinline__ void chain_carry(Shared<W, CB>& s, const Chain& c, int chain, int rank, bool last,
                                            float (&first)[V], float (&A)[V], const float (&H)[V]) {
    const int wave = threadIdx.x >> 6, l = (threadIdx.x & 63) * V;
    const int g = rank / c.group, before = rank - g * c.group;
    const bool closes = before + 1 == c.group;
    if (wave == 0 && !last && !closes) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            // the map goes out after `first` has come in: the chain's last tile, which waits for
            // the map, may write its result where `first` was read
            asm volatile("" : "+v"(A[j]), "+v"(first[j]));
            put_pair(c.map_at(chain, rank) + l + j, A[j], H[j]);
        }
    }
    if (before > 0) {
        // wave w composes its share of the maps before
        const int per = (before + W - 1) / W;
        const int lo = min(wave * per, before), hi = min(lo + per, before);
        float PA[V], PH[V];
#pragma unroll
        for (int j = 0; j < V; ++j) PA[j] = 1.0f, PH[j] = 0.0f;
        constexpr int kBatch = 4;  // looked at together
        for (int k = lo; k < hi; k += kBatch) {
            uint64_t w[kBatch][V];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    w[i][j] = peek_pair(c.map_at(chain, g * c.group + min(k + i, hi - 1)) + l + j);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (k + i >= hi) break;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float a, h;
                    get_pair(c.map_at(chain, g * c.group + k + i) + l + j, w[i][j], a, h);
                    PH[j] = fmaf(a, PH[j], h);
                    PA[j] *= a;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) s.PA[wave][l + j] = PA[j], s.PH[wave][l + j] = PH[j];
        __syncthreads();
    }
    if (wave == 0) {
        float a[V], h[V], st[V];
        uint64_t w[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            a[j] = 1.0f, h[j] = 0.0f, st[j] = first[j];
            if (g > 0) w[j] = peek_pair(c.state_at(chain, g) + l + j);
        }
        if (before > 0) {
#pragma unroll 2
            for (int k = 0; k < W; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    h[j] = fmaf(s.PA[k][l + j], h[j], s.PH[k][l + j]);
                    a[j] *= s.PA[k][l + j];
                }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float tag;
            if (g > 0) get_pair(c.state_at(chain, g) + l + j, w[j], tag, st[j]);
            st[j] = fmaf(a[j], st[j], h[j]);
            if (!last && closes) put_pair(c.state_at(chain, g + 1) + l + j, 0.0f, fmaf(A[j], st[j], H[j]));
            s.carry[l + j] = st[j];
        }
    }
    __syncthreads();
}

// The chain block's layout in the workspace, for blocks of `width` channels.
__device__ inline Chain chain_of(void* ws, int chains, int tiles, int group, int width) {
    Chain c;
    c.tiles = tiles;
    c.group = group;
    c.groups = (c.tiles + group - 1) / group;
    c.width = width;
    c.maps = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + kTicketBytes);
    c.states = c.maps + static_cast<int64_t>(chains) * c.tiles * width;
    return c;
}

}  // namespace layer
