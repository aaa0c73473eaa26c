// gdn_products.h -- quantisation to e4m3, the product of e4m3 matrices and the gated feed-forward block: argument
// structs and launchers. The C entry points are in gdn_product_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

struct QuantArgs {
    int64_t rows, cols;
    const void* x;
    uint8_t* q;
    float* scale;
};
// scales: 0 a row, 1 128 columns of a row, 2 128 x 128; turned: q is [cols, rows], and so are its scales' rows
hipError_t launch_quant(const QuantArgs& a, int dtype, int scales, bool turned, hipStream_t st);

struct Mm8Args {
    int64_t M, N, K;
    const void* a;
    const float* a_scale;
    const void* b;
    const float* b_scale;
    void* y;
    unsigned char* ws;
};
// exact: sums as in fp32 for an output in bf16 too (those of an output in fp32 always are)
size_t mm8_ws(int64_t M, int64_t N, int64_t K, int out_dtype, int scales, bool exact);
// scales as above, of b (a's are a row's where b's are, else of 128 columns)
hipError_t launch_mm8(const Mm8Args& a, int out_dtype, int scales, bool exact, hipStream_t st);

struct FfnArgs {
    int64_t M, K, F;
    int32_t act;
    bool pairs;  // gradients of gate and up as pairs of bf16 at any size
    const void* x;
    const void* wg;
    const void* wu;
    void* h;
    float* pre;
    const void* d_h;
    void* dx;
    void* dwg;
    void* dwu;
    // e4m3: scales of x, of the weights and of h (null: h is not quantised)
    const float* xs;
    const float* gs;
    const float* us;
    float* hs;
    unsigned char* ws;
};
size_t ffn_fwd_ws(int64_t M, int64_t K, int64_t F, int dtype);
size_t ffn_bwd_ws(int64_t M, int64_t K, int64_t F, int dtype, bool pairs);
size_t ffn8_ws(int64_t M, int64_t K, int64_t F, int dtype, bool quant, bool exact);
hipError_t launch_ffn_fwd(const FfnArgs& a, int dtype, hipStream_t st);
hipError_t launch_ffn_bwd(const FfnArgs& a, int dtype, hipStream_t st);
hipError_t launch_ffn8(const FfnArgs& a, int dtype, bool exact, hipStream_t st);

}  // namespace gdn
