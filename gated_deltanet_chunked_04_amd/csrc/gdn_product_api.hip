// gdn_product_api.hip -- C entry points of the quantiser, the product of e4m3 matrices and the gated feed-forward
// block: argument checks and launches. Host code only; the kernels are in gdn_quant.hip, gdn_mm8.hip and gdn_ffn.hip.
#include <math.h>
#include <string.h>

#include <initializer_list>

#include "../../include/gdn.h"
#include "gdn_kernels.h"
#include "gdn_products.h"

using namespace gdn;

namespace {

constexpr int64_t kMaxRows = INT32_MAX - 4096;  // of a matrix, and values of a row
constexpr int64_t kMaxWidth = 1 << 24;          // of the feed-forward block

bool zeros(const int32_t* r, int n) {
    for (int i = 0; i < n; ++i)
        if (r[i]) return false;
    return true;
}

bool float_type(int32_t t) { return t == GDN_DTYPE_BF16 || t == GDN_DTYPE_FP32; }

bool is_one_of(const void* out, std::initializer_list<const void*> inputs) {
    for (const void* in : inputs)
        if (out == in) return true;
    return false;
}

gdn_status check_buf(const void* p, size_t need, size_t bytes) {
    if (!need) return GDN_OK;
    if (!p || bytes < need) return GDN_ERR_WORKSPACE;
    return reinterpret_cast<uintptr_t>(p) % 256 ? GDN_ERR_WORKSPACE : GDN_OK;
}

gdn_status check_quant(const gdn_quant_desc* d) {
    if (!d || d->flags || !zeros(d->reserved, 4) || !float_type(d->dtype)) return GDN_ERR_INVALID_ARG;
    if (d->rows < 0 || d->cols < 1) return GDN_ERR_INVALID_ARG;
    if (d->scales < GDN_SCALE_ROW || d->scales > GDN_SCALE_BLOCK) return GDN_ERR_INVALID_ARG;
    if ((d->transpose != 0 && d->transpose != 1) || (d->transpose && d->scales == GDN_SCALE_ROW)) return GDN_ERR_INVALID_ARG;
    if (d->rows > kMaxRows || d->cols > kMaxRows) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_matmul(const gdn_matmul_desc* d) {
    if (!d || (d->flags & ~GDN_FLAG_EXACT_SUMS) || !zeros(d->reserved, 5) || !float_type(d->out_dtype)) return GDN_ERR_INVALID_ARG;
    if (d->M < 0 || d->N < 1 || d->K < 0) return GDN_ERR_INVALID_ARG;
    if (d->scales < GDN_SCALE_ROW || d->scales > GDN_SCALE_BLOCK) return GDN_ERR_INVALID_ARG;
    if (d->M > kMaxRows || d->N > kMaxRows || d->K > kMaxRows) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// flags: which the call takes
gdn_status check_ffn(const gdn_ffn_desc* d, bool e4m3, int32_t flags = 0) {
    if (!d || (d->flags & ~flags) || !zeros(d->reserved, 4) || !float_type(d->dtype)) return GDN_ERR_INVALID_ARG;
    if (d->rows < 0 || d->K < 1 || d->F < 1) return GDN_ERR_INVALID_ARG;
    if (d->activation != GDN_ACT_SILU && d->activation != GDN_ACT_GELU_TANH) return GDN_ERR_INVALID_ARG;
    if (d->out_type != GDN_OUT_SAME && (!e4m3 || d->out_type != GDN_OUT_E4M3)) return GDN_ERR_INVALID_ARG;
    if (d->rows > kMaxRows || d->K > kMaxWidth || d->F > kMaxWidth) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status launched(hipError_t e) {
    return e == hipSuccess ? GDN_OK : (e == hipErrorInvalidConfiguration ? GDN_ERR_UNSUPPORTED : GDN_ERR_HIP);
}

}  // namespace

extern "C" {

gdn_status gdn_quant_e4m3(const gdn_quant_desc* desc, const void* x, void* q, float* scale, void* stream) {
    if (gdn_status s = check_quant(desc)) return s;
    if (desc->rows && (!x || !q || !scale || q == x || static_cast<const void*>(scale) == x || static_cast<void*>(scale) == q))
        return GDN_ERR_INVALID_ARG;
    const QuantArgs a{desc->rows, desc->cols, x, static_cast<uint8_t*>(q), scale};
    ProfScope ps(kKQuant, (hipStream_t)stream);
    return launched(launch_quant(a, desc->dtype, desc->scales, desc->transpose != 0, (hipStream_t)stream));
}

gdn_status gdn_matmul_e4m3_workspace_size(const gdn_matmul_desc* desc, size_t* bytes) {
    if (!bytes) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_matmul(desc)) return s;
    *bytes = mm8_ws(desc->M, desc->N, desc->K, desc->out_dtype, desc->scales, desc->flags != 0);
    return GDN_OK;
}

gdn_status gdn_matmul_e4m3(const gdn_matmul_desc* desc, const void* a, const float* a_scale, const void* b,
                           const float* b_scale, void* y, void* workspace, size_t workspace_bytes, void* stream) {
    if (gdn_status s = check_matmul(desc)) return s;
    if (desc->M && (!y || y == a || y == b || y == a_scale || y == b_scale)) return GDN_ERR_INVALID_ARG;
    if (desc->M && desc->K && (!a || !b || !a_scale || !b_scale)) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_buf(workspace, mm8_ws(desc->M, desc->N, desc->K, desc->out_dtype, desc->scales, desc->flags != 0), workspace_bytes)) return s;
    const Mm8Args m{desc->M, desc->N, desc->K, a, a_scale, b, b_scale, y, static_cast<unsigned char*>(workspace)};
    ProfScope ps(kKMatmul8, (hipStream_t)stream);
    return launched(launch_mm8(m, desc->out_dtype, desc->scales, desc->flags != 0, (hipStream_t)stream));
}

gdn_status gdn_gated_ffn_fwd_workspace_size(const gdn_ffn_desc* desc, size_t* bytes) {
    if (!bytes) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_ffn(desc, false)) return s;
    *bytes = ffn_fwd_ws(desc->rows, desc->K, desc->F, desc->dtype);
    return GDN_OK;
}

gdn_status gdn_gated_ffn_bwd_workspace_size(const gdn_ffn_desc* desc, size_t* bytes) {
    if (!bytes) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_ffn(desc, false, GDN_FLAG_GRAD_PAIRS)) return s;
    *bytes = ffn_bwd_ws(desc->rows, desc->K, desc->F, desc->dtype, desc->flags != 0);
    return GDN_OK;
}

gdn_status gdn_gated_ffn_fwd(const gdn_ffn_desc* desc, const void* x, const void* w_gate, const void* w_up, void* h,
                             float* pre, void* workspace, size_t workspace_bytes, void* stream) {
    if (gdn_status s = check_ffn(desc, false)) return s;
    if (!w_gate || !w_up || (desc->rows && (!x || !h || h == x || h == w_gate || h == w_up))) return GDN_ERR_INVALID_ARG;
    if (pre && (static_cast<void*>(pre) == h || is_one_of(pre, {x, w_gate, w_up}))) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_buf(workspace, ffn_fwd_ws(desc->rows, desc->K, desc->F, desc->dtype), workspace_bytes)) return s;
    FfnArgs a{};
    a.M = desc->rows;
    a.K = desc->K;
    a.F = desc->F;
    a.act = desc->activation;
    a.x = x;
    a.wg = w_gate;
    a.wu = w_up;
    a.h = h;
    a.pre = pre;
    a.ws = static_cast<unsigned char*>(workspace);
    ProfScope ps(kKFfnFwd, (hipStream_t)stream);
    return launched(launch_ffn_fwd(a, desc->dtype, (hipStream_t)stream));
}

gdn_status gdn_gated_ffn_bwd(const gdn_ffn_desc* desc, const void* x, const void* w_gate, const void* w_up,
                             const float* pre, const void* d_h, void* dx, void* dw_gate, void* dw_up, void* workspace,
                             size_t workspace_bytes, void* stream) {
    if (gdn_status s = check_ffn(desc, false, GDN_FLAG_GRAD_PAIRS)) return s;
    if (!w_gate || !w_up || (desc->rows && (!x || !d_h)) || (!dw_gate) != (!dw_up)) return GDN_ERR_INVALID_ARG;
    if (dw_gate && (dw_gate == dw_up || dw_gate == dx || dw_up == dx)) return GDN_ERR_INVALID_ARG;
    for (const void* out : {dx, dw_gate, dw_up})
        if (out && (out == x || out == w_gate || out == w_up || out == d_h || out == pre)) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_buf(workspace, ffn_bwd_ws(desc->rows, desc->K, desc->F, desc->dtype, desc->flags != 0), workspace_bytes)) return s;
    FfnArgs a{};
    a.M = desc->rows;
    a.K = desc->K;
    a.F = desc->F;
    a.act = desc->activation;
    a.pairs = desc->flags != 0;
    a.x = x;
    a.wg = w_gate;
    a.wu = w_up;
    a.pre = const_cast<float*>(pre);
    a.d_h = d_h;
    a.dx = dx;
    a.dwg = dw_gate;
    a.dwu = dw_up;
    a.ws = static_cast<unsigned char*>(workspace);
    ProfScope ps(kKFfnBwd, (hipStream_t)stream);
    return launched(launch_ffn_bwd(a, desc->dtype, (hipStream_t)stream));
}

gdn_status gdn_gated_ffn_e4m3_workspace_size(const gdn_ffn_desc* desc, size_t* bytes) {
    if (!bytes) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_ffn(desc, true, GDN_FLAG_EXACT_SUMS)) return s;
    *bytes = ffn8_ws(desc->rows, desc->K, desc->F, desc->dtype, desc->out_type == GDN_OUT_E4M3, desc->flags != 0);
    return GDN_OK;
}

gdn_status gdn_gated_ffn_e4m3(const gdn_ffn_desc* desc, const void* x, const float* x_scale, const void* w_gate,
                              const float* gate_scale, const void* w_up, const float* up_scale, void* h, float* scale,
                              void* workspace, size_t workspace_bytes, void* stream) {
    if (gdn_status s = check_ffn(desc, true, GDN_FLAG_EXACT_SUMS)) return s;
    if (!w_gate || !w_up || !gate_scale || !up_scale) return GDN_ERR_INVALID_ARG;
    const std::initializer_list<const void*> inputs = {x, x_scale, w_gate, gate_scale, w_up, up_scale};
    if (desc->rows && (!x || !x_scale || !h || is_one_of(h, inputs))) return GDN_ERR_INVALID_ARG;
    const bool quant = desc->out_type == GDN_OUT_E4M3;
    if (quant ? (desc->rows && (!scale || static_cast<void*>(scale) == h || is_one_of(scale, inputs))) : scale != nullptr) return GDN_ERR_INVALID_ARG;
    if (gdn_status s = check_buf(workspace, ffn8_ws(desc->rows, desc->K, desc->F, desc->dtype, quant, desc->flags != 0), workspace_bytes)) return s;
    FfnArgs a{};
    a.M = desc->rows;
    a.K = desc->K;
    a.F = desc->F;
    a.act = desc->activation;
    a.x = x;
    a.xs = x_scale;
    a.wg = w_gate;
    a.gs = gate_scale;
    a.wu = w_up;
    a.us = up_scale;
    a.h = h;
    a.hs = scale;
    a.ws = static_cast<unsigned char*>(workspace);
    ProfScope ps(kKFfn8, (hipStream_t)stream);
    return launched(launch_ffn8(a, desc->dtype, desc->flags != 0, (hipStream_t)stream));
}

}  // extern "C"
