// layer_chain.h -- the scan's tiles and the hand-off between their workgroups.
//
// The time axis is cut into tiles and the channels into blocks of 64, one to a
// lane; a workgroup takes one tile of one block of one sequence (a
// chain), reads it once, and needs from the rest of its chain only the state
// before the tile (forward; in the backward, which runs the tiles from the last to
// the first, the gradient from behind it).  A tile maps that state by
// h -> A h + H, and its (A, H) does not depend on the tiles before it, so it is
// published at once.  Tiles come in groups of W = kScanWaves and groups in
// supergroups of W: a group's last tile composes the group's map and publishes that
// too, a supergroup's last tile hands the state behind it on.  A tile composes the
// maps of the tiles before it in its group and of the groups before it in its
// supergroup, and waits for the state before the supergroup.  So a chain waits for
// another's state once per W^2 tiles (16384 tokens in the forward), everything else is
// there as soon as the tiles before have been read, and every sum has a fixed order.
//
// Which tile a workgroup takes follows a ticket that it draws when it starts (one
// tile of every chain, then the next of every chain): whatever a workgroup waits for
// belongs to a lower ticket, so its owner has started, and the first unfinished ticket
// waits for nothing that is unfinished.  Every wait ends, whatever the order of dispatch.
//
// A hand-off is a pair of floats stored and loaded as one 64-bit word at agent
// scope.  A kernel in front marks all words empty; a word is read until it is
// not.  The word is its own flag: no ordering between words is needed.
//
// Long runs of narrow blocks measured best (B8 T4096 and, with the writing intensity, B1
// T65536 at D2048 bf16, forward): two channels a lane with 16 tokens a wave 85 and 219 us, one
// with 16 120 and 241, one with 24 94 and 206, one with 32 83 and 200; fewer tiles in
// flight per chain wait less for one another, and 32 tokens are what 128 registers hold.
#pragma once

#include "layer_device.h"
#include "layer_launch.h"

namespace layer {

constexpr uint32_t kEmpty = 0xffffffffu;  // of the pair's first half
constexpr int kTicketBytes = 64;

// The hand-off words of all chains: [chain][tile][64] maps, [chain][group][64]
// maps, [chain][supergroup][64] states (the first of each chain unused).
struct Chain {
    uint64_t *maps, *group_maps, *states;
    int tiles, groups, supers;
    __device__ __forceinline__ uint64_t* at(uint64_t* base, int chain, int count, int i) const {
        return base + (static_cast<int64_t>(chain) * count + i) * 64;
    }
};

// The product of two runs' A, each in [0, 1].  Where it underflows although neither is 0 it is the
// least positive number: an infinite state before it stays infinite, as token by token, and does
// not become 0 inf.  (Beside a finite state the two differ by 2^-149 of it.)  A NaN may
// be lost here; the run's H or R is NaN with it.  Three operations: the same with comparisons
// and a selection, in the chain's own latency, cost the training step of B1 T65536 D2048 444 -> 451 us.
constexpr float kLeast = 1.40129846e-45f;
__device__ __forceinline__ float times(float a, float b) {
    return fmaxf(a * b, fminf(fminf(a, b), kLeast));
}
// The same for a run's product A over its gates: told from a gate of 0 where it is 0 (a branch that
// only waves with such a product take).
template <int N>
__device__ __forceinline__ float run_product(float A, const float (&a)[N]) {
    if (__any(A == 0.0f)) {
        float least = a[0];
#pragma unroll
        for (int i = 1; i < N; ++i) least = fminf(least, a[i]);
        if (A == 0.0f && least > 0.0f) A = kLeast;
    }
    return A;
}

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

// What the waves of a workgroup share: their runs' maps, those of the tiles and of
// the groups before, the state before the tile.
struct Shared {
    float A[kScanWaves][64], H[kScanWaves][64];
    float PA[kScanWaves][64], PH[kScanWaves][64];
    float GA[kScanWaves][64], GH[kScanWaves][64];
    float carry[64];
};

// The state before this workgroup's tile, into s.carry.  Every count is the number
// of waves W: wave w fetches the map of the w-1st tile of the group and of the w-1st group of
// the supergroup, wave 0 the state before the supergroup, all asked for together (begin)
// while the waves' own maps meet in LDS.
// rank: the tile's place in its chain; last: no tile follows.
struct Carry {
    static constexpr int W = kScanWaves;
    Shared& s;
    const Chain& c;
    int chain, rank, wave, l;
    uint64_t wm, wg;  // wave 0: wm the state

    __device__ __forceinline__ int group() const { return rank / W; }
    __device__ __forceinline__ int super() const { return rank / (W * W); }
    __device__ __forceinline__ int tiles_before() const { return rank % W; }
    __device__ __forceinline__ int groups_before() const { return group() % W; }
    __device__ __forceinline__ uint64_t* map(int t) const { return c.at(c.maps, chain, c.tiles, t) + l; }
    __device__ __forceinline__ uint64_t* group_map(int g) const { return c.at(c.group_maps, chain, c.groups, g) + l; }
    __device__ __forceinline__ uint64_t* state(int k) const { return c.at(c.states, chain, c.supers, k) + l; }
    __device__ __forceinline__ uint64_t* my_map() const { return map(group() * W + wave - 1); }
    __device__ __forceinline__ uint64_t* my_group_map() const { return group_map(super() * W + wave - 1); }

    // Ask once; every wave, before the barrier that completes s.A and s.H.
    __device__ __forceinline__ void begin() {
        wm = wg = ~UINT64_C(0);
        if (wave == 0 ? super() > 0 : wave <= tiles_before()) wm = peek_pair(wave ? my_map() : state(super()));
        if (wave && wave <= groups_before()) wg = peek_pair(my_group_map());
    }
    // (a, h) = the first n maps that the waves fetched, composed in order
    __device__ __forceinline__ void compose(int n, const float (&A)[W][64], const float (&H)[W][64], float& a,
                                            float& h) const {
        a = 1.0f, h = 0.0f;
        for (int k = 1; k <= n; ++k) {
            h = fmaf(A[k][l], h, H[k][l]);
            a = times(a, A[k][l]);
        }
    }
    // After that barrier; wave 0 holds the tile's own map (A, H) and the state before the chain, `first`.
    __device__ __forceinline__ void finish(bool last, float first, float A, float H) {
        const bool closes = tiles_before() == W - 1, closes_super = closes && groups_before() == W - 1;
        float a, h;
        if (wave == 0) {
            if (!last && !closes) {
                // the map goes out after `first` has come in: the chain's last tile, which waits for
                // the map, may write its result where `first` was read
                asm volatile("" : "+v"(A), "+v"(first));
                put_pair(map(rank), A, H);
            }
        } else if (wave <= tiles_before()) {
            get_pair(my_map(), wm, s.PA[wave][l], s.PH[wave][l]);
        }
        if (closes && !closes_super && !last) {
            // the group's map goes out before anything outside the group is waited for
            __syncthreads();
            if (wave == 0) {
                compose(W - 1, s.PA, s.PH, a, h);
                a = times(a, A);
                asm volatile("" : "+v"(a), "+v"(first));
                put_pair(group_map(group()), a, fmaf(A, h, H));
            }
        }
        if (wave && wave <= groups_before()) get_pair(my_group_map(), wg, s.GA[wave][l], s.GH[wave][l]);
        __syncthreads();
        if (wave == 0) {
            float tag, st = first, ga, gh;
            compose(groups_before(), s.GA, s.GH, ga, gh);
            compose(tiles_before(), s.PA, s.PH, a, h);
            if (super() > 0) get_pair(state(super()), wm, tag, st);
            st = fmaf(a, fmaf(ga, st, gh), h);
            if (!last && closes_super) put_pair(state(super() + 1), 0.0f, fmaf(A, st, H));
            s.carry[l] = st;
        }
        __syncthreads();
    }
};

// The chains' layout in the workspace.
__device__ inline Chain chain_of(void* ws, int chains, int tiles) {
    Chain c;
    c.tiles = tiles;
    c.groups = (tiles + kScanWaves - 1) / kScanWaves;
    c.supers = (c.groups + kScanWaves - 1) / kScanWaves;
    c.maps = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + kTicketBytes);
    c.group_maps = c.maps + static_cast<int64_t>(chains) * c.tiles * 64;
    c.states = c.group_maps + static_cast<int64_t>(chains) * c.groups * 64;
    return c;
}

// What a workgroup works on: its ticket's tile and chain.
struct Place {
    int pos, chain, b, wave, l, c;  // pos: the tile's place in the order of tickets
};
__device__ __forceinline__ Place take_place(void* ws, int D, int chains, uint32_t* ticket) {
    uint32_t id = blockIdx.x;
    if (ws) {
        if (threadIdx.x == 0) *ticket = atomicAdd(static_cast<uint32_t*>(ws), 1u);
        __syncthreads();
        id = __builtin_amdgcn_readfirstlane(*ticket);
    }
    Place at;
    const int nblk = (D + 63) / 64;
    at.pos = static_cast<int>(id / chains);
    at.chain = static_cast<int>(id % chains);
    at.b = at.chain / nblk;
    at.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    at.l = threadIdx.x & 63;
    at.c = at.chain % nblk * 64 + at.l;
    return at;
}

}  // namespace layer
