// gdn_layer_api.hip -- C entry points of the operators around the gated delta rule (gated scan,
// short convolution, RMS norm): argument checks and launches. Host code only; the kernels are in
// gdn_gscan.hip, gdn_conv.hip and gdn_rms.hip.
#include <math.h>
#include <string.h>

#include "../../include/gdn.h"
#include "gdn_kernels.h"
#include "gdn_layer.h"

using namespace gdn;

namespace {

constexpr int64_t kMaxTokens = INT32_MAX - 4096;  // token indices are 32-bit, elements 64-bit
constexpr int64_t kMaxChannels = 1 << 24;

bool zeros(const int32_t* r, int n) {
    for (int i = 0; i < n; ++i)
        if (r[i]) return false;
    return true;
}

// dtype in {bf16, fp32}, the second type equal to it or fp32
bool types_ok(int32_t dtype, int32_t other) {
    return (dtype == GDN_DTYPE_BF16 || dtype == GDN_DTYPE_FP32) && (other == dtype || other == GDN_DTYPE_FP32);
}

gdn_status check_sizes(int64_t B, int64_t T, int64_t D, const int32_t* cu, int32_t num_seqs, SeqView& seq) {
    if (B < 1 || T < 0 || D < 1) return GDN_ERR_INVALID_ARG;
    if (cu && (B != 1 || num_seqs < 1)) return GDN_ERR_INVALID_ARG;
    if (B > kMaxTokens || D > kMaxChannels || T > kMaxTokens / B) return GDN_ERR_UNSUPPORTED;
    seq.cu = cu;
    seq.T = (int32_t)T;
    seq.total = (int32_t)(B * T);
    seq.N = cu ? num_seqs : (int32_t)B;
    return GDN_OK;
}

gdn_status check_buf(const void* p, size_t need, size_t bytes) {
    if (!p || bytes < need) return GDN_ERR_WORKSPACE;
    return reinterpret_cast<uintptr_t>(p) % 256 ? GDN_ERR_WORKSPACE : GDN_OK;
}

gdn_status check_scan(const gdn_scan_desc* d, SeqView& seq) {
    if (!d || (d->flags & ~GDN_FLAG_ZERO_OUTSIDE) || !zeros(d->reserved, 4) || !types_ok(d->dtype, d->g_dtype)) return GDN_ERR_INVALID_ARG;
    return check_sizes(d->B, d->T, d->D, d->cu_seqlens, d->num_seqs, seq);
}

gdn_status check_conv(const gdn_conv_desc* d, SeqView& seq) {
    if (!d || (d->flags & ~GDN_FLAG_ZERO_OUTSIDE) || !zeros(d->reserved, 4) || !types_ok(d->dtype, d->w_dtype)) return GDN_ERR_INVALID_ARG;
    if (d->activation != GDN_ACT_NONE && d->activation != GDN_ACT_SILU) return GDN_ERR_INVALID_ARG;
    if (d->width < 2 || d->width > 4) return GDN_ERR_UNSUPPORTED;
    return check_sizes(d->B, d->T, d->D, d->cu_seqlens, d->num_seqs, seq);
}

gdn_status check_rms(const gdn_rmsnorm_desc* d) {
    if (!d || d->flags || !zeros(d->reserved, 4) || !types_ok(d->dtype, d->w_dtype)) return GDN_ERR_INVALID_ARG;
    if (d->rows < 0 || d->D < 1 || !(d->eps >= 0.f) || isinf(d->eps)) return GDN_ERR_INVALID_ARG;
    if (d->out_type != GDN_OUT_SAME && d->out_type != GDN_OUT_E4M3) return GDN_ERR_INVALID_ARG;
    if (d->scale_group != 0 && (d->scale_group != 128 || d->out_type != GDN_OUT_E4M3)) return GDN_ERR_INVALID_ARG;
    if (d->rows > kMaxTokens || d->D > kMaxChannels) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status launched(hipError_t e) {
    return e == hipSuccess ? GDN_OK : (e == hipErrorInvalidConfiguration ? GDN_ERR_UNSUPPORTED : GDN_ERR_HIP);
}

}  // namespace

extern "C" {

gdn_status gdn_gated_scan_fwd_workspace_size(const gdn_scan_desc* desc, size_t* bytes) {
    SeqView seq;
    if (!bytes) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_scan(desc, seq)) return s;
    *bytes = gscan_fwd_ws(seq, desc->D);
    return GDN_OK;
}

gdn_status gdn_gated_scan_bwd_workspace_size(const gdn_scan_desc* desc, size_t* bytes) {
    SeqView seq;
    if (!bytes) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_scan(desc, seq)) return s;
    *bytes = gscan_bwd_ws(seq, desc->D);
    return GDN_OK;
}

gdn_status gdn_gated_scan_states_size(const gdn_scan_desc* desc, size_t* bytes) {
    SeqView seq;
    if (!bytes) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_scan(desc, seq)) return s;
    *bytes = (size_t)((seq.total + (int64_t)kScanTile - 1) / kScanTile) * desc->D * 4;
    return GDN_OK;
}

gdn_status gdn_gated_scan_fwd(const gdn_scan_desc* desc, const void* x, const void* g, const float* initial_state,
                              void* h, float* final_state, void* states, void* workspace, size_t workspace_bytes,
                              void* stream) {
    GScanArgs a{};
    if (gdn_status s = check_scan(desc, a.seq)) return s;
    if (a.seq.total && (!x || !g || !h)) return GDN_ERR_INVALID_ARG;
    if (a.seq.total && (h == x || h == g)) return GDN_ERR_INVALID_ARG;
    const size_t need = gscan_fwd_ws(a.seq, desc->D);
    if (need)
        if (gdn_status s = check_buf(workspace, need, workspace_bytes)) return s;
    if (states && reinterpret_cast<uintptr_t>(states) % 256) return GDN_ERR_WORKSPACE;
    a.D = desc->D;
    a.x = x;
    a.g = g;
    a.s0 = initial_state;
    a.h = h;
    a.sT = final_state;
    a.states = static_cast<float*>(states);
    a.ws = static_cast<unsigned char*>(workspace);
    a.zero = desc->flags & GDN_FLAG_ZERO_OUTSIDE;
    ProfScope ps(kKGScanFwd, (hipStream_t)stream);
    return launched(launch_gscan_fwd(a, desc->dtype, desc->g_dtype, (hipStream_t)stream));
}

gdn_status gdn_gated_scan_bwd(const gdn_scan_desc* desc, const void* x, const void* g, const float* initial_state,
                              const void* d_h, const float* d_final_state, const void* states, void* dx, void* dg,
                              float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
    GScanArgs a{};
    if (gdn_status s = check_scan(desc, a.seq)) return s;
    if (a.seq.total && (!x || !g || !d_h || !dx || !dg)) return GDN_ERR_INVALID_ARG;
    if (a.seq.total && (dx == x || dx == g || dx == d_h || dg == x || dg == g || dg == d_h || dx == dg)) return GDN_ERR_INVALID_ARG;
    if (d_initial_state && (d_initial_state == initial_state || d_initial_state == d_final_state)) return GDN_ERR_INVALID_ARG;
    const size_t need = gscan_bwd_ws(a.seq, desc->D);
    if (need)
        if (gdn_status s = check_buf(workspace, need, workspace_bytes)) return s;
    if (states && reinterpret_cast<uintptr_t>(states) % 256) return GDN_ERR_WORKSPACE;
    a.D = desc->D;
    a.x = x;
    a.g = g;
    a.s0 = initial_state;
    a.d_h = d_h;
    a.d_sT = d_final_state;
    a.states = static_cast<float*>(const_cast<void*>(states));
    a.dx = dx;
    a.dg = dg;
    a.ds0 = d_initial_state;
    a.ws = static_cast<unsigned char*>(workspace);
    a.zero = desc->flags & GDN_FLAG_ZERO_OUTSIDE;
    ProfScope ps(kKGScanBwd, (hipStream_t)stream);
    return launched(launch_gscan_bwd(a, desc->dtype, desc->g_dtype, states != nullptr, (hipStream_t)stream));
}

gdn_status gdn_short_conv_bwd_workspace_size(const gdn_conv_desc* desc, size_t* bytes) {
    SeqView seq;
    if (!bytes) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_conv(desc, seq)) return s;
    *bytes = conv_bwd_ws(seq.total, desc->D, desc->width, desc->dtype);
    return GDN_OK;
}

gdn_status gdn_short_conv_fwd(const gdn_conv_desc* desc, const void* x, const void* weight, const void* bias,
                              const void* initial_state, void* y, void* final_state, void* stream) {
    ConvArgs a{};
    if (gdn_status s = check_conv(desc, a.seq)) return s;
    if (!weight || (a.seq.total && (!x || !y || x == y))) return GDN_ERR_INVALID_ARG;
    if (final_state && final_state == initial_state && (desc->cu_seqlens || desc->T > GDN_CONV_INPLACE_T))
        return GDN_ERR_INVALID_ARG;
    a.D = desc->D;
    a.W = desc->width;
    a.silu = desc->activation == GDN_ACT_SILU;
    a.x = x;
    a.w = weight;
    a.bias = bias;
    a.s0 = initial_state;
    a.sT = final_state;
    a.y = y;
    a.zero = desc->flags & GDN_FLAG_ZERO_OUTSIDE;
    ProfScope ps(kKConvFwd, (hipStream_t)stream);
    return launched(launch_conv_fwd(a, desc->dtype, desc->w_dtype, (hipStream_t)stream));
}

gdn_status gdn_short_conv_bwd(const gdn_conv_desc* desc, const void* x, const void* weight, const void* bias,
                              const void* initial_state, const void* d_y, const void* d_final_state, void* dx,
                              float* dweight, float* dbias, void* d_initial_state, void* workspace,
                              size_t workspace_bytes, void* stream) {
    ConvArgs a{};
    if (gdn_status s = check_conv(desc, a.seq)) return s;
    if (!weight || !dweight || (a.seq.total && (!x || !d_y || !dx || dx == x || dx == d_y))) return GDN_ERR_INVALID_ARG;
    if (d_initial_state && (d_initial_state == initial_state || d_initial_state == d_final_state)) return GDN_ERR_INVALID_ARG;
    const size_t need = conv_bwd_ws(a.seq.total, desc->D, desc->width, desc->dtype);
    if (need)
        if (gdn_status s = check_buf(workspace, need, workspace_bytes)) return s;
    a.D = desc->D;
    a.W = desc->width;
    a.silu = desc->activation == GDN_ACT_SILU;
    a.x = x;
    a.w = weight;
    a.bias = bias;
    a.s0 = initial_state;
    a.d_y = d_y;
    a.d_sT = d_final_state;
    a.dx = dx;
    a.dw = dweight;
    a.db = dbias;
    a.ds0 = d_initial_state;
    a.ws = static_cast<unsigned char*>(workspace);
    a.zero = desc->flags & GDN_FLAG_ZERO_OUTSIDE;
    ProfScope ps(kKConvBwd, (hipStream_t)stream);
    return launched(launch_conv_bwd(a, desc->dtype, desc->w_dtype, (hipStream_t)stream));
}

gdn_status gdn_rmsnorm_fwd(const gdn_rmsnorm_desc* desc, const void* x, const void* residual, const void* weight,
                           void* y, float* scale, void* residual_out, void* stream) {
    if (gdn_status s = check_rms(desc)) return s;
    if (!weight || (!residual) != (!residual_out)) return GDN_ERR_INVALID_ARG;
    if (desc->rows && (!x || !y || y == x || y == residual || y == residual_out)) return GDN_ERR_INVALID_ARG;
    if (desc->out_type == GDN_OUT_E4M3 ? (desc->rows && !scale) : scale != nullptr) return GDN_ERR_INVALID_ARG;
    RmsArgs a{};
    a.rows = desc->rows;
    a.D = desc->D;
    a.eps = desc->eps;
    a.group = desc->scale_group ? desc->scale_group : (int32_t)desc->D;
    a.x = x;
    a.res = residual;
    a.w = weight;
    a.y = y;
    a.scale = scale;
    a.res_out = residual_out;
    ProfScope ps(kKRmsFwd, (hipStream_t)stream);
    return launched(launch_rms_fwd(a, desc->dtype, desc->w_dtype, desc->out_type, (hipStream_t)stream));
}

gdn_status gdn_rmsnorm_bwd_workspace_size(const gdn_rmsnorm_desc* desc, size_t* bytes) {
    if (!bytes) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_rms(desc)) return s;
    *bytes = rms_bwd_ws(desc->rows, desc->D);
    return GDN_OK;
}

gdn_status gdn_rmsnorm_bwd(const gdn_rmsnorm_desc* desc, const void* r, const void* weight, const void* d_y,
                           const void* d_residual, void* dx, float* dweight, void* workspace,
                           size_t workspace_bytes, void* stream) {
    if (gdn_status s = check_rms(desc)) return s;
    if (!weight || (desc->rows && (!r || !d_y || !dx || dx == r || dx == d_y || dx == d_residual)))
        return GDN_ERR_INVALID_ARG;
    const size_t need = rms_bwd_ws(desc->rows, desc->D);
    if (need)
        if (gdn_status s = check_buf(workspace, need, workspace_bytes)) return s;
    RmsArgs a{};
    a.rows = desc->rows;
    a.D = desc->D;
    a.eps = desc->eps;
    a.x = r;
    a.w = weight;
    a.d_y = d_y;
    a.d_res = d_residual;
    a.dx = dx;
    a.dw = dweight;
    a.ws = static_cast<unsigned char*>(workspace);
    ProfScope ps(kKRmsBwd, (hipStream_t)stream);
    return launched(launch_rms_bwd(a, desc->dtype, desc->w_dtype, (hipStream_t)stream));
}

}  // extern "C"
