// layer_mixer_abi.hip -- the C ABI of the selective state space layer
// (include/lattice_osr.h: lattice_osr_conv_*, lattice_osr_ssm_*,
// lattice_osr_layernorm_*): host-side argument checks, buffer sizes and
// dispatch.  Every check runs before any HIP call; no C++ exception crosses
// the ABI.
#include <math.h>
#include <stdint.h>

#include "../../include/lattice_osr.h"
#include "layer_check.h"
#include "layer_launch.h"

namespace {

using layer::Buf;
using layer::check_buffers;
using layer::dtype_ok;
using layer::elem;

constexpr int kMaxRow = 1 << 22;  // elements from row to row: a tile's 16 rows of floats stay under 2^30 bytes

bool row_ok(int row, int64_t width) { return row == 0 || (row >= width && row <= kMaxRow); }
int row_of(int row, int width) { return row ? row : width; }
// Bytes from the first to the last element of `rows` rows.
size_t extent(int64_t rows, int64_t row, int64_t width, size_t e) {
    return static_cast<size_t>((rows - 1) * row + width) * e;
}

// The sizes that both recurrent operators share.
int check_sizes(int B, int T, int D) {
    if (B <= 0 || T <= 0 || D <= 0) return LATTICE_OSR_ERR_SHAPE;
    if (T > (1 << 30) || D > (1 << 20)) return LATTICE_OSR_ERR_SHAPE;
    if (static_cast<int64_t>(B) * T > (INT64_C(1) << 40) / D) return LATTICE_OSR_ERR_SHAPE;
    return LATTICE_OSR_OK;
}

// ---------------------------------------------------------------- conv ----
int check_conv(const lattice_osr_conv_desc* d) {
    if (!d) return LATTICE_OSR_ERR_NULL;
    const int rc = check_sizes(d->B, d->T, d->D);
    if (rc != LATTICE_OSR_OK) return rc;
    if (d->W < 1 || d->W > layer::kConvMaxW) return LATTICE_OSR_ERR_UNSUPPORTED;
    if (d->act != LATTICE_OSR_CONV_NONE && d->act != LATTICE_OSR_CONV_SILU) return LATTICE_OSR_ERR_UNSUPPORTED;
    if (!dtype_ok(d->in_dtype) || !dtype_ok(d->y_dtype) || !dtype_ok(d->grad_dtype)) return LATTICE_OSR_ERR_UNSUPPORTED;
    if (!row_ok(d->x_row, d->D)) return LATTICE_OSR_ERR_SHAPE;
    // a launch has fewer than 2^32 threads: the forward's at most two for each channel and 16 tokens
    if ((static_cast<int64_t>(d->T) + 15) / 16 * d->B * d->D >= INT64_C(1) << 31) return LATTICE_OSR_ERR_SHAPE;
    return LATTICE_OSR_OK;
}

// The backward's launch has 64 threads to a run, whatever D is.
int check_conv_bwd(const lattice_osr_conv_desc* d) {
    const int rc = check_conv(d);
    if (rc != LATTICE_OSR_OK) return rc;
    return layer::conv_groups(d->B, d->T) < 1 << 26 ? LATTICE_OSR_OK : LATTICE_OSR_ERR_SHAPE;
}

layer::ConvParams conv_params(const lattice_osr_conv_desc* d) {
    layer::ConvParams p = {};
    p.B = d->B, p.T = d->T, p.D = d->D, p.W = d->W, p.act = d->act;
    p.x_row = row_of(d->x_row, d->D);
    p.in_bf16 = d->in_dtype == LATTICE_OSR_BF16;
    p.y_bf16 = d->y_dtype == LATTICE_OSR_BF16;
    p.grad_bf16 = d->grad_dtype == LATTICE_OSR_BF16;
    return p;
}

size_t conv_part_bytes(const lattice_osr_conv_desc* d) {
    return static_cast<size_t>(layer::conv_groups(d->B, d->T)) * (d->W + 1) * d->D * sizeof(float);
}

bool conv_vec(const layer::ConvParams& p, const Buf* b, int n) {
    if (p.D % 8 != 0 || p.x_row % 8 != 0) return false;
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(b[i].p) % 16 != 0) return false;
    return true;
}

// ----------------------------------------------------------------- ssm ----
int64_t ssm_chains(const lattice_osr_ssm_desc* d) {
    return static_cast<int64_t>(d->B) * d->G * ((d->D / d->G + 63) / 64);
}

int check_ssm(const lattice_osr_ssm_desc* d) {
    if (!d) return LATTICE_OSR_ERR_NULL;
    const int rc = check_sizes(d->B, d->T, d->D);
    if (rc != LATTICE_OSR_OK) return rc;
    if (d->N < 1 || d->N > layer::kSsmMaxN) return LATTICE_OSR_ERR_UNSUPPORTED;
    if (d->G < 1 || d->D % d->G != 0) return LATTICE_OSR_ERR_SHAPE;
    if (!dtype_ok(d->in_dtype) || !dtype_ok(d->y_dtype) || !dtype_ok(d->grad_dtype)) return LATTICE_OSR_ERR_UNSUPPORTED;
    if (d->softplus != 0 && d->softplus != 1) return LATTICE_OSR_ERR_UNSUPPORTED;
    const int64_t gn = static_cast<int64_t>(d->G) * d->N;
    if (gn > kMaxRow || !row_ok(d->x_row, d->D) || !row_ok(d->dt_row, d->D) || !row_ok(d->z_row, d->D) ||
        !row_ok(d->b_row, gn) || !row_ok(d->c_row, gn))
        return LATTICE_OSR_ERR_SHAPE;
    if (ssm_chains(d) >= 1 << 22) return LATTICE_OSR_ERR_SHAPE;
    return LATTICE_OSR_OK;
}

layer::SsmParams ssm_params(const lattice_osr_ssm_desc* d) {
    layer::SsmParams p = {};
    p.B = d->B, p.T = d->T, p.D = d->D, p.N = d->N, p.G = d->G;
    p.x_row = row_of(d->x_row, d->D), p.dt_row = row_of(d->dt_row, d->D), p.z_row = row_of(d->z_row, d->D);
    p.b_row = row_of(d->b_row, d->G * d->N), p.c_row = row_of(d->c_row, d->G * d->N);
    p.in_bf16 = d->in_dtype == LATTICE_OSR_BF16;
    p.y_bf16 = d->y_dtype == LATTICE_OSR_BF16;
    p.grad_bf16 = d->grad_dtype == LATTICE_OSR_BF16;
    p.softplus = d->softplus;
    return p;
}

size_t ssm_saved_bytes(const lattice_osr_ssm_desc* d) {
    const size_t tiles = (static_cast<size_t>(d->T) + layer::kSsmSave - 1) / layer::kSsmSave;
    return static_cast<size_t>(d->B) * tiles * d->N * d->D * sizeof(float);
}

// ---------------------------------------------------------- layer norm ----
int check_ln(const lattice_osr_layernorm_desc* d) {
    if (!d) return LATTICE_OSR_ERR_NULL;
    if (d->R <= 0 || d->D <= 0) return LATTICE_OSR_ERR_SHAPE;
    if (d->D > layer::kNormMaxD) return LATTICE_OSR_ERR_UNSUPPORTED;
    if (!dtype_ok(d->in_dtype) || !dtype_ok(d->res_dtype) || !dtype_ok(d->grad_dtype))
        return LATTICE_OSR_ERR_UNSUPPORTED;
    if (!(d->eps >= 1.17549435e-38f) || !isfinite(d->eps)) return LATTICE_OSR_ERR_UNSUPPORTED;
    return LATTICE_OSR_OK;
}

layer::LayerNormParams ln_params(const lattice_osr_layernorm_desc* d, bool backward) {
    layer::LayerNormParams p = {};
    p.R = d->R, p.D = d->D;
    p.in_bf16 = d->in_dtype == LATTICE_OSR_BF16;
    p.res_bf16 = d->res_dtype == LATTICE_OSR_BF16;
    p.grad_bf16 = d->grad_dtype == LATTICE_OSR_BF16;
    p.eps = d->eps;
    p.groups = layer::norm_groups(d->R, d->D, backward);
    return p;
}

bool ln_vec(const lattice_osr_layernorm_desc* d, const Buf* b, int n) {
    if (d->D % 8 != 0) return false;
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(b[i].p) % 16 != 0) return false;
    return true;
}

}  // namespace

extern "C" {

size_t lattice_osr_conv_bwd_workspace_bytes(const lattice_osr_conv_desc* desc) {
    return check_conv_bwd(desc) != LATTICE_OSR_OK ? static_cast<size_t>(-1) : conv_part_bytes(desc);
}

int lattice_osr_conv_fwd(const lattice_osr_conv_desc* desc, const void* x, const float* w, const float* bias,
                         const int32_t* lengths, const int32_t* segments, const void* hist_in, void* hist_out,
                         void* y, void* hip_stream) {
    int rc = check_conv(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    if (!x || !w || !y) return LATTICE_OSR_ERR_NULL;
    if (desc->W == 1) hist_in = nullptr, hist_out = nullptr;
    layer::ConvParams p = conv_params(desc);
    const int64_t rows = static_cast<int64_t>(p.B) * p.T;
    const size_t ei = elem(desc->in_dtype), ey = elem(desc->y_dtype);
    const size_t nh = static_cast<size_t>(p.B) * (p.W - 1) * p.D * ei, nd = static_cast<size_t>(p.D) * 4;
    const Buf bufs[] = {{x, extent(rows, p.x_row, p.D, ei), ei, false},
                        {hist_in, nh, ei, false},
                        {hist_out, nh, ei, true},
                        {y, static_cast<size_t>(rows) * p.D * ey, ey, true},
                        {w, nd * p.W, 4, false},
                        {bias, nd, 4, false},
                        {lengths, p.B * sizeof(int32_t), 4, false},
                        {segments, rows * sizeof(int32_t), 4, false}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    p.vec = conv_vec(p, bufs, 6);
    p.x = x, p.w = w, p.bias = bias, p.lengths = lengths, p.segments = segments;
    p.hist_in = hist_in, p.hist_out = hist_out, p.y = y;
    return layer::launch_conv_fwd(p, static_cast<hipStream_t>(hip_stream));
}

int lattice_osr_conv_bwd(const lattice_osr_conv_desc* desc, const void* x, const float* w, const float* bias,
                         const int32_t* lengths, const int32_t* segments, const void* hist_in, const void* dy,
                         const void* dhist_out, void* dx, float* dw, float* dbias, void* dhist_in, void* workspace,
                         size_t workspace_bytes, void* hip_stream) {
    int rc = check_conv_bwd(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    if (!x || !w || !dy || !dx) return LATTICE_OSR_ERR_NULL;
    const bool sums = dw || dbias;
    const size_t need = sums ? conv_part_bytes(desc) : 0;
    if (sums && !workspace) return LATTICE_OSR_ERR_NULL;
    if (sums && workspace_bytes < need) return LATTICE_OSR_ERR_WORKSPACE;
    if (desc->W == 1) hist_in = dhist_out = nullptr, dhist_in = nullptr;
    layer::ConvParams p = conv_params(desc);
    const int64_t rows = static_cast<int64_t>(p.B) * p.T;
    const size_t ei = elem(desc->in_dtype), ey = elem(desc->y_dtype), eg = elem(desc->grad_dtype);
    const size_t n = static_cast<size_t>(rows) * p.D, nh = static_cast<size_t>(p.B) * (p.W - 1) * p.D;
    const size_t nd = static_cast<size_t>(p.D) * 4;
    const Buf bufs[] = {{x, extent(rows, p.x_row, p.D, ei), ei, false},
                        {hist_in, nh * ei, ei, false},
                        {dy, n * ey, ey, false},
                        {dhist_out, nh * eg, eg, false},
                        {dx, n * eg, eg, true},
                        {dhist_in, nh * eg, eg, true},
                        {w, nd * p.W, 4, false},
                        {bias, nd, 4, false},
                        {sums ? workspace : nullptr, need, 16, true},
                        {dw, nd * p.W, 4, true},
                        {dbias, nd, 4, true},
                        {lengths, p.B * sizeof(int32_t), 4, false},
                        {segments, rows * sizeof(int32_t), 4, false}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    p.vec = conv_vec(p, bufs, 8);
    p.x = x, p.w = w, p.bias = bias, p.lengths = lengths, p.segments = segments, p.hist_in = hist_in;
    p.dy = dy, p.dhist_out = dhist_out, p.dx = dx, p.dhist_in = dhist_in, p.dw = dw, p.dbias = dbias;
    p.part = sums ? static_cast<float*>(workspace) : nullptr;
    return layer::launch_conv_bwd(p, static_cast<hipStream_t>(hip_stream));
}

int lattice_osr_conv_step(const lattice_osr_conv_desc* desc, const void* x, const float* w, const float* bias,
                          const void* hist_in, void* hist_out, void* y, void* hip_stream) {
    int rc = check_conv(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    if (desc->T != 1 || desc->W < 2) return LATTICE_OSR_ERR_SHAPE;
    if (!x || !w || !hist_in || !hist_out || !y) return LATTICE_OSR_ERR_NULL;
    layer::ConvParams p = conv_params(desc);
    const size_t ei = elem(desc->in_dtype), ey = elem(desc->y_dtype);
    const size_t nh = static_cast<size_t>(p.B) * (p.W - 1) * p.D * ei, nd = static_cast<size_t>(p.D) * 4;
    const Buf bufs[] = {{x, extent(p.B, p.x_row, p.D, ei), ei, false},
                        {hist_in == hist_out ? nullptr : hist_in, nh, ei, false},
                        {hist_out, nh, ei, true},
                        {y, static_cast<size_t>(p.B) * p.D * ey, ey, true},
                        {w, nd * p.W, 4, false},
                        {bias, nd, 4, false}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    p.vec = conv_vec(p, bufs, 6);
    p.x = x, p.w = w, p.bias = bias, p.hist_in = hist_in, p.hist_out = hist_out, p.y = y;
    return layer::launch_conv_step(p, static_cast<hipStream_t>(hip_stream));
}

size_t lattice_osr_ssm_saved_bytes(const lattice_osr_ssm_desc* desc) {
    return check_ssm(desc) != LATTICE_OSR_OK ? static_cast<size_t>(-1) : ssm_saved_bytes(desc);
}
size_t lattice_osr_ssm_workspace_bytes(const lattice_osr_ssm_desc* desc) {
    return check_ssm(desc) != LATTICE_OSR_OK ? static_cast<size_t>(-1) : layer::ssm_workspace_bytes(ssm_params(desc));
}
size_t lattice_osr_ssm_bwd_workspace_bytes(const lattice_osr_ssm_desc* desc) {
    return check_ssm(desc) != LATTICE_OSR_OK ? static_cast<size_t>(-1) : layer::ssm_bwd_workspace_bytes(ssm_params(desc));
}

int lattice_osr_ssm_fwd(const lattice_osr_ssm_desc* desc, const void* x, const void* dt, const float* A,
                        const void* Bm, const void* Cm, const float* skip, const void* z, const float* dt_bias,
                        const int32_t* lengths, const int32_t* segments, const float* state_in, float* state_out,
                        void* y, void* saved, size_t saved_bytes, void* workspace, size_t workspace_bytes,
                        void* hip_stream) {
    int rc = check_ssm(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    if (!x || !dt || !A || !Bm || !Cm || !y) return LATTICE_OSR_ERR_NULL;
    if (saved && saved_bytes < ssm_saved_bytes(desc)) return LATTICE_OSR_ERR_WORKSPACE;
    layer::SsmParams p = ssm_params(desc);
    const size_t need = layer::ssm_workspace_bytes(p);
    if (need && !workspace) return LATTICE_OSR_ERR_NULL;
    if (workspace_bytes < need) return LATTICE_OSR_ERR_WORKSPACE;
    const int64_t rows = static_cast<int64_t>(p.B) * p.T;
    const size_t ei = elem(desc->in_dtype), ey = elem(desc->y_dtype), nd = static_cast<size_t>(p.D) * 4;
    const size_t ns = static_cast<size_t>(p.B) * p.D * p.N * 4;
    const int gn = p.G * p.N;
    const Buf bufs[] = {{x, extent(rows, p.x_row, p.D, ei), ei, false},
                        {dt, extent(rows, p.dt_row, p.D, ei), ei, false},
                        {z, extent(rows, p.z_row, p.D, ei), ei, false},
                        {Bm, extent(rows, p.b_row, gn, ei), ei, false},
                        {Cm, extent(rows, p.c_row, gn, ei), ei, false},
                        {A, nd * p.N, 4, false},
                        {skip, nd, 4, false},
                        {dt_bias, nd, 4, false},
                        {lengths, p.B * sizeof(int32_t), 4, false},
                        {segments, rows * sizeof(int32_t), 4, false},
                        {state_in == state_out ? nullptr : state_in, ns, 4, false},
                        {state_out, ns, 4, true},
                        {y, static_cast<size_t>(rows) * p.D * ey, ey, true},
                        {saved, ssm_saved_bytes(desc), 4, true},
                        {need ? workspace : nullptr, need, 16, true}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    p.x = x, p.dt = dt, p.A = A, p.Bm = Bm, p.Cm = Cm, p.skip = skip, p.z = z, p.dt_bias = dt_bias;
    p.lengths = lengths, p.segments = segments, p.state_in = state_in, p.state_out = state_out;
    p.y = y, p.saved = static_cast<float*>(saved), p.ws = need ? workspace : nullptr;
    return layer::launch_ssm_fwd(p, static_cast<hipStream_t>(hip_stream));
}

int lattice_osr_ssm_bwd(const lattice_osr_ssm_desc* desc, const void* x, const void* dt, const float* A,
                        const void* Bm, const void* Cm, const float* skip, const void* z, const float* dt_bias,
                        const int32_t* lengths, const int32_t* segments, const void* saved, size_t saved_bytes,
                        const void* dy, const float* dstate_out, void* dx, void* ddt, float* dA, void* dB, void* dC,
                        float* dskip, void* dz, float* ddt_bias, float* dstate_in, void* workspace,
                        size_t workspace_bytes, void* hip_stream) {
    int rc = check_ssm(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    if (!x || !dt || !A || !Bm || !Cm || !saved || !dy || !dx || !ddt || !dB || !dC || (z && !dz))
        return LATTICE_OSR_ERR_NULL;
    if ((!z && dz) || (!skip && dskip) || (!dt_bias && ddt_bias)) return LATTICE_OSR_ERR_UNSUPPORTED;
    if (saved_bytes < ssm_saved_bytes(desc)) return LATTICE_OSR_ERR_WORKSPACE;
    layer::SsmParams p = ssm_params(desc);
    const size_t need = layer::ssm_bwd_workspace_bytes(p);
    if (!workspace) return LATTICE_OSR_ERR_NULL;
    if (workspace_bytes < need) return LATTICE_OSR_ERR_WORKSPACE;
    const int64_t rows = static_cast<int64_t>(p.B) * p.T;
    const size_t ei = elem(desc->in_dtype), ey = elem(desc->y_dtype), eg = elem(desc->grad_dtype);
    const size_t nd = static_cast<size_t>(p.D) * 4, n = static_cast<size_t>(rows) * p.D;
    const size_t ns = static_cast<size_t>(p.B) * p.D * p.N * 4;
    const int gn = p.G * p.N;
    const size_t nbc = static_cast<size_t>(rows) * gn * eg;
    const Buf bufs[] = {{x, extent(rows, p.x_row, p.D, ei), ei, false},
                        {dt, extent(rows, p.dt_row, p.D, ei), ei, false},
                        {z, extent(rows, p.z_row, p.D, ei), ei, false},
                        {Bm, extent(rows, p.b_row, gn, ei), ei, false},
                        {Cm, extent(rows, p.c_row, gn, ei), ei, false},
                        {A, nd * p.N, 4, false},
                        {skip, nd, 4, false},
                        {dt_bias, nd, 4, false},
                        {lengths, p.B * sizeof(int32_t), 4, false},
                        {segments, rows * sizeof(int32_t), 4, false},
                        {saved, ssm_saved_bytes(desc), 4, false},
                        {dy, n * ey, ey, false},
                        {dstate_out, ns, 4, false},
                        {dx, n * eg, eg, true},
                        {ddt, n * eg, eg, true},
                        {dA, nd * p.N, 4, true},
                        {dB, nbc, eg, true},
                        {dC, nbc, eg, true},
                        {dskip, nd, 4, true},
                        {dz, n * eg, eg, true},
                        {ddt_bias, nd, 4, true},
                        {dstate_in, ns, 4, true},
                        {workspace, need, 16, true}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    p.x = x, p.dt = dt, p.A = A, p.Bm = Bm, p.Cm = Cm, p.skip = skip, p.z = z, p.dt_bias = dt_bias;
    p.lengths = lengths, p.segments = segments;
    p.saved = const_cast<float*>(static_cast<const float*>(saved));
    p.dy = dy, p.dstate_out = dstate_out, p.dx = dx, p.ddt = ddt, p.dz = dz, p.dB = dB, p.dC = dC;
    p.dA = dA, p.dskip = dskip, p.ddt_bias = ddt_bias, p.dstate_in = dstate_in, p.ws = workspace;
    return layer::launch_ssm_bwd(p, static_cast<hipStream_t>(hip_stream));
}

int lattice_osr_ssm_step(const lattice_osr_ssm_desc* desc, const void* x, const void* dt, const float* A,
                         const void* Bm, const void* Cm, const float* skip, const void* z, const float* dt_bias,
                         const float* state_in, float* state_out, void* y, void* hip_stream) {
    int rc = check_ssm(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    if (desc->T != 1) return LATTICE_OSR_ERR_SHAPE;
    if (!x || !dt || !A || !Bm || !Cm || !state_in || !state_out || !y) return LATTICE_OSR_ERR_NULL;
    layer::SsmParams p = ssm_params(desc);
    const size_t ei = elem(desc->in_dtype), ey = elem(desc->y_dtype), nd = static_cast<size_t>(p.D) * 4;
    const size_t ns = static_cast<size_t>(p.B) * p.D * p.N * 4;
    const int gn = p.G * p.N;
    const Buf bufs[] = {{x, extent(p.B, p.x_row, p.D, ei), ei, false},
                        {dt, extent(p.B, p.dt_row, p.D, ei), ei, false},
                        {z, extent(p.B, p.z_row, p.D, ei), ei, false},
                        {Bm, extent(p.B, p.b_row, gn, ei), ei, false},
                        {Cm, extent(p.B, p.c_row, gn, ei), ei, false},
                        {A, nd * p.N, 4, false},
                        {skip, nd, 4, false},
                        {dt_bias, nd, 4, false},
                        {state_in == state_out ? nullptr : state_in, ns, 4, false},
                        {state_out, ns, 4, true},
                        {y, static_cast<size_t>(p.B) * p.D * ey, ey, true}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    p.x = x, p.dt = dt, p.A = A, p.Bm = Bm, p.Cm = Cm, p.skip = skip, p.z = z, p.dt_bias = dt_bias;
    p.state_in = state_in, p.state_out = state_out, p.y = y;
    return layer::launch_ssm_step(p, static_cast<hipStream_t>(hip_stream));
}

size_t lattice_osr_layernorm_bwd_workspace_bytes(const lattice_osr_layernorm_desc* desc) {
    if (check_ln(desc) != LATTICE_OSR_OK) return static_cast<size_t>(-1);
    return static_cast<size_t>(layer::norm_groups(desc->R, desc->D, true)) * 2 * desc->D * sizeof(float);
}

int lattice_osr_layernorm_fwd(const lattice_osr_layernorm_desc* desc, const void* x, const void* y, const float* w,
                              const float* b, void* x_out, void* z, void* hip_stream) {
    int rc = check_ln(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    if (!x || !z) return LATTICE_OSR_ERR_NULL;
    if (!y && x_out) return LATTICE_OSR_ERR_UNSUPPORTED;
    const size_t n = static_cast<size_t>(desc->R) * desc->D, nd = static_cast<size_t>(desc->D) * 4;
    const size_t ei = elem(desc->in_dtype), er = elem(desc->res_dtype);
    const Buf bufs[] = {{x_out && x == x_out ? nullptr : x, n * er, er, false},
                        {y, n * ei, ei, false},
                        {w, nd, 4, false},
                        {b, nd, 4, false},
                        {x_out, n * er, er, true},
                        {z, n * ei, ei, true}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    layer::LayerNormParams p = ln_params(desc, false);
    p.vec = ln_vec(desc, bufs, 6);
    p.x = x, p.y = y, p.w = w, p.b = b, p.x_out = x_out, p.z = z;
    return layer::launch_layernorm_fwd(p, static_cast<hipStream_t>(hip_stream));
}

int lattice_osr_layernorm_bwd(const lattice_osr_layernorm_desc* desc, const void* x, const void* y, const float* w,
                              const void* dx_out, const void* dz, void* dx, void* dy, float* dw, float* db,
                              void* workspace, size_t workspace_bytes, void* hip_stream) {
    int rc = check_ln(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    if (!x || !dz || (!dx && !dy)) return LATTICE_OSR_ERR_NULL;
    if (!y && dy) return LATTICE_OSR_ERR_UNSUPPORTED;
    const bool sums = dw || db;
    const size_t need = sums ? lattice_osr_layernorm_bwd_workspace_bytes(desc) : 0;
    if (sums && !workspace) return LATTICE_OSR_ERR_NULL;
    if (sums && workspace_bytes < need) return LATTICE_OSR_ERR_WORKSPACE;
    const size_t n = static_cast<size_t>(desc->R) * desc->D, nd = static_cast<size_t>(desc->D) * 4;
    const size_t ei = elem(desc->in_dtype), er = elem(desc->res_dtype), eg = elem(desc->grad_dtype);
    const Buf bufs[] = {{x, n * er, er, false},
                        {y, n * ei, ei, false},
                        {w, nd, 4, false},
                        {dx && dx == dx_out ? nullptr : dx_out, n * er, er, false},
                        {dz, n * ei, ei, false},
                        {dx, n * er, er, true},
                        {dy, n * eg, eg, true},
                        {dw, nd, 4, true},
                        {db, nd, 4, true},
                        {sums ? workspace : nullptr, need, 4, true}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    layer::LayerNormParams p = ln_params(desc, true);
    p.vec = ln_vec(desc, bufs, 7);
    p.x = x, p.y = y, p.w = w, p.dx_out = dx_out, p.dz = dz, p.dx = dx, p.dy = dy, p.dw = dw, p.db = db;
    p.part = static_cast<float*>(workspace);
    return layer::launch_layernorm_bwd(p, static_cast<hipStream_t>(hip_stream));
}

}  // extern "C"
