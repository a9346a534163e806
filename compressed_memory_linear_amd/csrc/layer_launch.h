// layer_launch.h -- host-side launchers of the layer operators around the OSR
// recurrence: the element-wise gated recurrence (scan) and the norms of a
// block (internal to the library; the public interface is
// include/lattice_osr.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace layer {

// Tokens per tile (what a workgroup takes, each wave a run of them) of the scan's
// forward and backward.  A saving forward keeps the state before each of the backward's tiles.
constexpr int kScanWaves = 8;
constexpr int kFwdRun = 32, kFwdTile = kFwdRun * kScanWaves;
constexpr int kBwdRun = 16, kBwdTile = kBwdRun * kScanWaves;
static_assert(kFwdTile % kBwdTile == 0 && kBwdTile % kFwdRun == 0, "a saved state is one before a run");
inline int64_t tiles_of(int64_t T, int tile) { return (T + tile - 1) / tile; }
// Threads of a workgroup: a tile's waves, or those that have tokens where T is one tile at most (B64 T20
// D4096 bf16, forward: 8 waves 51 us, 1 wave 13).
inline unsigned scan_threads(int T, int run) {
    return 64 * static_cast<unsigned>(T < run * kScanWaves ? tiles_of(T, run) : kScanWaves);
}

// Parameters of the scan's kernels; layouts as in include/lattice_osr.h.
struct ScanParams {
    const void *v, *f, *g;    // [B,T,D]: input, forget-gate logits, writing-intensity logits (or null)
    const int32_t* lengths;   // [B] or null
    const float* state_in;    // [B,D] or null (zeros)
    float* state_out;         // [B,D] or null
    void* y;                  // [B,T,D] (forward)
    float* saved;             // [B, ceil(T / kBwdTile), D]: the state before each of those tiles, or null
    const void* dy;           // [B,T,D] (backward)
    const float* dstate_out;  // [B,D] or null
    void *dv, *df, *dg;       // [B,T,D] (backward; dg null where g is)
    float* dstate_in;         // [B,D] or null
    int B, T, D;
    int in_bf16;
    int y_bf16;     // y and dy
    int grad_bf16;  // dv, df, dg
    int weight;     // 0: 1, 1: 1 - mu, 2: sqrt(1 - mu^2)
    // Hand-offs between the workgroups of a chain (scan_workspace_bytes), or
    // null where T is one tile: a ticket counter, then the pairs (layer_chain.h).
    void* ws;
};

// Bytes of ScanParams::ws for B sequences of T tokens and D channels.
size_t scan_workspace_bytes(int B, int T, int D);
void clear_scan_workspace(const ScanParams& p, int tile, hipStream_t st);
// Return 0 or -5 (launch error).
int launch_scan_fwd(const ScanParams& p, hipStream_t st);
int launch_scan_bwd(const ScanParams& p, hipStream_t st);
int launch_scan_step(const ScanParams& p, hipStream_t st);

// Parameters of the norms around a block; rows of D values.
struct NormParams {
    const void *y, *gate, *x;              // [R,D] (gate, x may be null; y null: x alone)
    const float *w_post, *scale, *w_pre;   // [D] or null (ones)
    void *x_out, *z;                       // [R,D] (forward), each may be null
    const void *dx_out, *dz;               // [R,D] (backward), each may be null (zeros)
    void *dy, *dgate, *dx;                 // [R,D] (backward), each may be null
    float *dw_post, *dscale, *dw_pre;      // [D] (backward), each may be null
    float* part;                           // [groups][3][D]: one workgroup's sums over its rows
    int R, D;
    int in_bf16;    // y, gate, z, dz
    int res_bf16;   // x, x_out, dx_out, dx
    int grad_bf16;  // dy, dgate
    int gate_kind;  // 0: none, 1: GeLU, 2: SiLU
    int post, pre;  // whether the norm after / before the block is applied
    float eps;
    int vec;        // 1: D a multiple of 8 and every row buffer 16-byte aligned
    int groups;     // workgroups of the launch (the rows are dealt to them in turn)
};
constexpr int kNormMaxD = 16384;
// Workgroups of a launch over R rows of D values.
int norm_groups(int R, int D, bool backward);
int launch_norm_fwd(const NormParams& p, hipStream_t st);
int launch_norm_bwd(const NormParams& p, hipStream_t st);

}  // namespace layer
