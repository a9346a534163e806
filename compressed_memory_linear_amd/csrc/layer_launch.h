// layer_launch.h -- host-side launchers of the layer operators around the OSR
// recurrence: the element-wise gated recurrence (scan), the norms of a block,
// the short convolution, the selective state space scan and the layer norm
// (internal to the library; the public interface is include/lattice_osr.h).
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
__host__ __device__ inline int64_t tiles_of(int64_t T, int tile) { return (T + tile - 1) / tile; }
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

// Parameters of the short causal convolution.
constexpr int kConvMaxW = 8;
struct ConvParams {
    const void* x;                   // [B,T,D], rows x_row apart
    const float *w, *bias;           // [D,W]; [D] or null
    const int32_t *lengths, *segments;
    const void* hist_in;             // [B,W-1,D] or null
    void *hist_out, *y;              // hist_out may be null
    const void *dy, *dhist_out;      // backward; dhist_out may be null
    void *dx, *dhist_in;             // dhist_in may be null
    float *dw, *dbias;               // each may be null
    float* part;                     // [groups][W + 1][D]: one group of tokens' sums
    int B, T, D, W, x_row, act;
    int in_bf16, y_bf16, grad_bf16;
    int vec;                         // 1: D and x_row multiples of 8 and every buffer 16-byte aligned
};
// Groups of tokens that the backward's column sums come in.
int conv_groups(int B, int T);
int launch_conv_fwd(const ConvParams& p, hipStream_t st);
int launch_conv_bwd(const ConvParams& p, hipStream_t st);
int launch_conv_step(const ConvParams& p, hipStream_t st);

// Parameters of the selective state space scan.
constexpr int kSsmMaxN = 64;
constexpr int kSsmSave = 16;  // tokens between saved states, and per tile of the backward
struct SsmParams {
    const void *x, *dt, *Bm, *Cm, *z;  // z may be null
    const float *A, *skip, *dt_bias;   // skip, dt_bias may be null
    const int32_t *lengths, *segments;
    const float* state_in;             // [B,D,N] or null
    float* state_out;                  // or null
    void* y;
    float* saved;                      // [B, ceil(T / kSsmSave), N, D] or null
    const void* dy;                    // backward
    const float* dstate_out;
    void *dx, *ddt, *dz, *dB, *dC;
    float *dA, *dskip, *ddt_bias, *dstate_in;
    void* ws;
    int B, T, D, N, G;
    int x_row, dt_row, z_row, b_row, c_row;
    int in_bf16, y_bf16, grad_bf16, softplus;
};
size_t ssm_workspace_bytes(const SsmParams& p);
size_t ssm_bwd_workspace_bytes(const SsmParams& p);
int launch_ssm_fwd(const SsmParams& p, hipStream_t st);
int launch_ssm_bwd(const SsmParams& p, hipStream_t st);
int launch_ssm_step(const SsmParams& p, hipStream_t st);

// Parameters of the layer norm; rows of D values.
struct LayerNormParams {
    const void *x, *y;                 // y may be null
    const float *w, *b;                // or null
    void *x_out, *z;                   // x_out may be null
    const void *dx_out, *dz;           // dx_out may be null
    void *dx, *dy;                     // one of them may be null
    float *dw, *db;                    // each may be null
    float* part;                       // [groups][2][D]
    int R, D, in_bf16, res_bf16, grad_bf16;
    float eps;
    int vec, groups;
};
int launch_layernorm_fwd(const LayerNormParams& p, hipStream_t st);
int launch_layernorm_bwd(const LayerNormParams& p, hipStream_t st);

// Column sums: part is [groups][rows][D]; row r of the sum goes to mat[c * M + r] for r < M, row M to e0[c] and
// row M + 1 to e1[c] (each destination may be null).  Added in a fixed order.
struct ColSums {
    const float* part;
    int groups, rows, D, M;
    float *mat, *e0, *e1;
};
void launch_col_sums(const ColSums& p, hipStream_t st);

}  // namespace layer
