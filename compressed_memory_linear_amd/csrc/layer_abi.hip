// layer_abi.hip -- the C ABI of the layer operators around the OSR recurrence
// (include/lattice_osr.h: lattice_osr_scan_*, lattice_osr_norm_*): host-side
// argument checks, buffer sizes and dispatch.  Every check runs before any HIP
// call; no C++ exception crosses the ABI.
#include <limits.h>
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

int check_scan(const lattice_osr_scan_desc* d) {
    if (!d) return LATTICE_OSR_ERR_NULL;
    if (d->B <= 0 || d->T <= 0 || d->D <= 0) return LATTICE_OSR_ERR_SHAPE;
    if (d->T > (1 << 30) || d->D > (1 << 20)) return LATTICE_OSR_ERR_SHAPE;
    if (static_cast<int64_t>(d->B) * d->T > (INT64_C(1) << 40) / d->D) return LATTICE_OSR_ERR_SHAPE;
    // A launch has fewer than 2^32 threads: at most 1024 for each tile of 64 channels.  (The product
    // is at most 65 x 129 / 2^13 times B T D, which the line before bounds.)
    const int64_t tiles = layer::tiles_of(d->T, layer::kBwdTile);
    if (layer::tiles_of(d->D, 64) * d->B * tiles >= INT64_C(1) << 22) return LATTICE_OSR_ERR_SHAPE;
    if (!dtype_ok(d->in_dtype) || !dtype_ok(d->y_dtype) || !dtype_ok(d->grad_dtype)) return LATTICE_OSR_ERR_UNSUPPORTED;
    if (d->input_weight < LATTICE_OSR_SCAN_ONE || d->input_weight > LATTICE_OSR_SCAN_NORM)
        return LATTICE_OSR_ERR_UNSUPPORTED;
    return LATTICE_OSR_OK;
}

size_t scan_saved_bytes(const lattice_osr_scan_desc* d) {
    return static_cast<size_t>(d->B) * layer::tiles_of(d->T, layer::kBwdTile) * d->D * sizeof(float);
}

layer::ScanParams scan_params(const lattice_osr_scan_desc* d) {
    layer::ScanParams p = {};
    p.B = d->B, p.T = d->T, p.D = d->D;
    p.in_bf16 = d->in_dtype == LATTICE_OSR_BF16;
    p.y_bf16 = d->y_dtype == LATTICE_OSR_BF16;
    p.grad_bf16 = d->grad_dtype == LATTICE_OSR_BF16;
    p.weight = d->input_weight;
    return p;
}

int check_norm(const lattice_osr_norm_desc* d) {
    if (!d) return LATTICE_OSR_ERR_NULL;
    if (d->R <= 0 || d->D <= 0) return LATTICE_OSR_ERR_SHAPE;
    if (d->D > layer::kNormMaxD) return LATTICE_OSR_ERR_UNSUPPORTED;
    if (!dtype_ok(d->in_dtype) || !dtype_ok(d->res_dtype) || !dtype_ok(d->grad_dtype))
        return LATTICE_OSR_ERR_UNSUPPORTED;
    if (d->gate_kind < LATTICE_OSR_GATE_NONE || d->gate_kind > LATTICE_OSR_GATE_SILU) return LATTICE_OSR_ERR_UNSUPPORTED;
    if ((d->post_norm != 0 && d->post_norm != 1) || (d->pre_norm != 0 && d->pre_norm != 1))
        return LATTICE_OSR_ERR_UNSUPPORTED;
    // below the smallest normal float the reciprocal root of a row of zeros is not finite
    if (!(d->eps >= 1.17549435e-38f) || !isfinite(d->eps)) return LATTICE_OSR_ERR_UNSUPPORTED;
    return LATTICE_OSR_OK;
}

// The operands both directions share: which of them a descriptor asks for.
int check_norm_operands(const lattice_osr_norm_desc* d, const void* y, const void* gate, const void* x,
                        const float* w_post, const float* scale, const float* w_pre) {
    if (!y && !x) return LATTICE_OSR_ERR_NULL;
    if ((d->gate_kind != LATTICE_OSR_GATE_NONE) != (gate != nullptr))
        return gate ? LATTICE_OSR_ERR_UNSUPPORTED : LATTICE_OSR_ERR_NULL;
    if (!y && (gate || d->post_norm || scale || !d->pre_norm)) return LATTICE_OSR_ERR_UNSUPPORTED;
    if ((w_post && !d->post_norm) || (w_pre && !d->pre_norm)) return LATTICE_OSR_ERR_UNSUPPORTED;
    return LATTICE_OSR_OK;
}

layer::NormParams norm_params(const lattice_osr_norm_desc* d, bool backward) {
    layer::NormParams p = {};
    p.R = d->R, p.D = d->D;
    p.in_bf16 = d->in_dtype == LATTICE_OSR_BF16;
    p.res_bf16 = d->res_dtype == LATTICE_OSR_BF16;
    p.grad_bf16 = d->grad_dtype == LATTICE_OSR_BF16;
    p.gate_kind = d->gate_kind;
    p.post = d->post_norm, p.pre = d->pre_norm;
    p.eps = d->eps;
    p.groups = layer::norm_groups(d->R, d->D, backward);
    return p;
}

// Whether the rows and weights can move in 16-byte pieces.
bool norm_vec(const lattice_osr_norm_desc* d, const Buf* b, int n) {
    if (d->D % 8 != 0) return false;
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(b[i].p) % 16 != 0) return false;
    return true;
}

}  // namespace

extern "C" {

size_t lattice_osr_scan_saved_bytes(const lattice_osr_scan_desc* desc) {
    return check_scan(desc) != LATTICE_OSR_OK ? static_cast<size_t>(-1) : scan_saved_bytes(desc);
}

size_t lattice_osr_scan_workspace_bytes(const lattice_osr_scan_desc* desc) {
    if (check_scan(desc) != LATTICE_OSR_OK) return static_cast<size_t>(-1);
    return layer::scan_workspace_bytes(desc->B, desc->T, desc->D);
}

int lattice_osr_scan_fwd(const lattice_osr_scan_desc* desc, const void* v, const void* mu_logit,
                         const void* gamma_logit, const int32_t* lengths, const float* state_in, float* state_out,
                         void* y, void* saved, size_t saved_bytes, void* workspace, size_t workspace_bytes,
                         void* hip_stream) {
    int rc = check_scan(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    if (!v || !mu_logit || !y) return LATTICE_OSR_ERR_NULL;
    if (saved && saved_bytes < scan_saved_bytes(desc)) return LATTICE_OSR_ERR_WORKSPACE;
    const size_t need = layer::scan_workspace_bytes(desc->B, desc->T, desc->D);
    if (need && !workspace) return LATTICE_OSR_ERR_NULL;
    if (workspace_bytes < need) return LATTICE_OSR_ERR_WORKSPACE;
    const size_t n = static_cast<size_t>(desc->B) * desc->T * desc->D, nb = static_cast<size_t>(desc->B) * desc->D;
    const size_t ei = elem(desc->in_dtype), ey = elem(desc->y_dtype);
    const Buf bufs[] = {{v, n * ei, ei, false},
                        {mu_logit, n * ei, ei, false},
                        {gamma_logit, n * ei, ei, false},
                        {lengths, desc->B * sizeof(int32_t), 4, false},
                        {state_in == state_out ? nullptr : state_in, nb * 4, 4, false},
                        {state_out, nb * 4, 4, true},
                        {y, n * ey, ey, true},
                        {saved, scan_saved_bytes(desc), 4, true},
                        {need ? workspace : nullptr, need, 16, true}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    layer::ScanParams p = scan_params(desc);
    p.v = v, p.f = mu_logit, p.g = gamma_logit, p.lengths = lengths;
    p.state_in = state_in, p.state_out = state_out, p.y = y, p.saved = static_cast<float*>(saved);
    p.ws = need ? workspace : nullptr;
    return layer::launch_scan_fwd(p, static_cast<hipStream_t>(hip_stream));
}

int lattice_osr_scan_bwd(const lattice_osr_scan_desc* desc, const void* v, const void* mu_logit,
                         const void* gamma_logit, const int32_t* lengths, const void* saved, size_t saved_bytes,
                         const void* dy, const float* dstate_out, void* dv, void* dmu_logit, void* dgamma_logit,
                         float* dstate_in, void* workspace, size_t workspace_bytes, void* hip_stream) {
    int rc = check_scan(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    if (!v || !mu_logit || !saved || !dy || !dv || !dmu_logit) return LATTICE_OSR_ERR_NULL;
    if (gamma_logit && !dgamma_logit) return LATTICE_OSR_ERR_NULL;
    if (!gamma_logit && dgamma_logit) return LATTICE_OSR_ERR_UNSUPPORTED;
    if (saved_bytes < scan_saved_bytes(desc)) return LATTICE_OSR_ERR_WORKSPACE;
    const size_t need = layer::scan_workspace_bytes(desc->B, desc->T, desc->D);
    if (need && !workspace) return LATTICE_OSR_ERR_NULL;
    if (workspace_bytes < need) return LATTICE_OSR_ERR_WORKSPACE;
    const size_t n = static_cast<size_t>(desc->B) * desc->T * desc->D, nb = static_cast<size_t>(desc->B) * desc->D;
    const size_t ei = elem(desc->in_dtype), ey = elem(desc->y_dtype), eg = elem(desc->grad_dtype);
    const Buf bufs[] = {{v, n * ei, ei, false},
                        {mu_logit, n * ei, ei, false},
                        {gamma_logit, n * ei, ei, false},
                        {lengths, desc->B * sizeof(int32_t), 4, false},
                        {saved, scan_saved_bytes(desc), 4, false},
                        {dy, n * ey, ey, false},
                        {dstate_out, nb * 4, 4, false},
                        {dv, n * eg, eg, true},
                        {dmu_logit, n * eg, eg, true},
                        {dgamma_logit, n * eg, eg, true},
                        {dstate_in, nb * 4, 4, true},
                        {need ? workspace : nullptr, need, 16, true}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    layer::ScanParams p = scan_params(desc);
    p.v = v, p.f = mu_logit, p.g = gamma_logit, p.lengths = lengths;
    p.saved = const_cast<float*>(static_cast<const float*>(saved));
    p.dy = dy, p.dstate_out = dstate_out;
    p.ws = need ? workspace : nullptr;
    p.dv = dv, p.df = dmu_logit, p.dg = dgamma_logit, p.dstate_in = dstate_in;
    return layer::launch_scan_bwd(p, static_cast<hipStream_t>(hip_stream));
}

int lattice_osr_scan_step(const lattice_osr_scan_desc* desc, const void* v, const void* mu_logit,
                          const void* gamma_logit, const float* state_in, float* state_out, void* y,
                          void* hip_stream) {
    int rc = check_scan(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    if (desc->T != 1) return LATTICE_OSR_ERR_SHAPE;
    if (!v || !mu_logit || !state_in || !state_out || !y) return LATTICE_OSR_ERR_NULL;
    const size_t n = static_cast<size_t>(desc->B) * desc->D;
    const size_t ei = elem(desc->in_dtype), ey = elem(desc->y_dtype);
    const Buf bufs[] = {{v, n * ei, ei, false},
                        {mu_logit, n * ei, ei, false},
                        {gamma_logit, n * ei, ei, false},
                        {state_in == state_out ? nullptr : state_in, n * 4, 4, false},
                        {state_out, n * 4, 4, true},
                        {y, n * ey, ey, true}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    layer::ScanParams p = scan_params(desc);
    p.v = v, p.f = mu_logit, p.g = gamma_logit;
    p.state_in = state_in, p.state_out = state_out, p.y = y;
    return layer::launch_scan_step(p, static_cast<hipStream_t>(hip_stream));
}

size_t lattice_osr_norm_bwd_workspace_bytes(const lattice_osr_norm_desc* desc) {
    if (check_norm(desc) != LATTICE_OSR_OK) return static_cast<size_t>(-1);
    return static_cast<size_t>(layer::norm_groups(desc->R, desc->D, true)) * 3 * desc->D * sizeof(float);
}

int lattice_osr_norm_fwd(const lattice_osr_norm_desc* desc, const void* y, const void* gate, const void* x,
                         const float* w_post, const float* scale, const float* w_pre, void* x_out, void* z,
                         void* hip_stream) {
    int rc = check_norm(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    rc = check_norm_operands(desc, y, gate, x, w_post, scale, w_pre);
    if (rc != LATTICE_OSR_OK) return rc;
    if ((desc->pre_norm && !z) || (!desc->pre_norm && !x_out)) return LATTICE_OSR_ERR_NULL;
    if ((!desc->pre_norm && z) || (!y && x_out)) return LATTICE_OSR_ERR_UNSUPPORTED;
    const size_t n = static_cast<size_t>(desc->R) * desc->D, nd = static_cast<size_t>(desc->D) * 4;
    const size_t ei = elem(desc->in_dtype), er = elem(desc->res_dtype);
    const Buf bufs[] = {{y, n * ei, ei, false},      {gate, n * ei, ei, false},
                        {x_out && x == x_out ? nullptr : x, n * er, er, false},
                        {x_out, n * er, er, true},   {z, n * ei, ei, true},
                        {w_post, nd, 4, false},      {scale, nd, 4, false},
                        {w_pre, nd, 4, false}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    layer::NormParams p = norm_params(desc, false);
    p.vec = norm_vec(desc, bufs, 8);
    p.y = y, p.gate = gate, p.x = x;
    p.w_post = w_post, p.scale = scale, p.w_pre = w_pre;
    p.x_out = x_out, p.z = z;
    return layer::launch_norm_fwd(p, static_cast<hipStream_t>(hip_stream));
}

int lattice_osr_norm_bwd(const lattice_osr_norm_desc* desc, const void* y, const void* gate, const void* x,
                         const float* w_post, const float* scale, const float* w_pre, const void* dx_out,
                         const void* dz, void* dy, void* dgate, void* dx, float* dw_post, float* dscale,
                         float* dw_pre, void* workspace, size_t workspace_bytes, void* hip_stream) {
    int rc = check_norm(desc);
    if (rc != LATTICE_OSR_OK) return rc;
    rc = check_norm_operands(desc, y, gate, x, w_post, scale, w_pre);
    if (rc != LATTICE_OSR_OK) return rc;
    if ((desc->pre_norm && !dz) || (!desc->pre_norm && !dx_out) || (y && !dy) || (gate && !dgate) || (!y && !dx))
        return LATTICE_OSR_ERR_NULL;
    if ((!desc->pre_norm && (dz || dw_pre)) || (!y && (dy || dscale)) || (!gate && dgate) || (!x && dx) ||
        (!desc->post_norm && dw_post))
        return LATTICE_OSR_ERR_UNSUPPORTED;
    const bool sums = dw_post || dscale || dw_pre;
    const size_t need = sums ? lattice_osr_norm_bwd_workspace_bytes(desc) : 0;
    if (sums && !workspace) return LATTICE_OSR_ERR_NULL;
    if (sums && workspace_bytes < need) return LATTICE_OSR_ERR_WORKSPACE;
    const size_t n = static_cast<size_t>(desc->R) * desc->D, nd = static_cast<size_t>(desc->D) * 4;
    const size_t ei = elem(desc->in_dtype), er = elem(desc->res_dtype), eg = elem(desc->grad_dtype);
    const Buf bufs[] = {{y, n * ei, ei, false},
                        {gate, n * ei, ei, false},
                        {x, n * er, er, false},
                        {dx && dx_out == dx ? nullptr : dx_out, n * er, er, false},
                        {dz, n * ei, ei, false},
                        {dy, n * eg, eg, true},
                        {dgate, n * eg, eg, true},
                        {dx, n * er, er, true},
                        {w_post, nd, 4, false},
                        {scale, nd, 4, false},
                        {w_pre, nd, 4, false},
                        {dw_post, nd, 4, true},
                        {dscale, nd, 4, true},
                        {dw_pre, nd, 4, true},
                        {sums ? workspace : nullptr, need, 4, true}};
    rc = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (rc != LATTICE_OSR_OK) return rc;
    layer::NormParams p = norm_params(desc, true);
    p.vec = norm_vec(desc, bufs, 11);
    p.y = y, p.gate = gate, p.x = x;
    p.w_post = w_post, p.scale = scale, p.w_pre = w_pre;
    p.dx_out = dx_out, p.dz = dz;
    p.dy = dy, p.dgate = dgate, p.dx = dx;
    p.dw_post = dw_post, p.dscale = dscale, p.dw_pre = dw_pre;
    p.part = static_cast<float*>(workspace);
    return layer::launch_norm_bwd(p, static_cast<hipStream_t>(hip_stream));
}

}  // extern "C"
