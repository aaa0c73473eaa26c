// gdn_mm8.hip -- the product of two e4m3 matrices whose contraction is contiguous, with fp32 scales:
//   y[m, n] = sum over blocks kb of 128  a_scale[m, kb] b_scale[n, kb]  sum over k in kb of  a[m, k] b[n, k],
// b_scale[n, kb] being one value for 128 rows n (block), or a row's own (group); or one scale a row for the whole
// contraction in both (row). The scaled sums are kept in fp32: a step of the contraction is a block, its sum comes out
// of the matrix cores unscaled and is added with one fused product. Bounds and rates: at the tiles (gdn_mm.h).
#include "gdn_layer.h"
#include "gdn_mm.h"
#include "gdn_products.h"

namespace gdn {

namespace {

template <int KIND, int SC, typename T>
hipError_t mm8(const Mm8Args& a, hipStream_t st) {
    MmArgs p{};
    p.x[0] = static_cast<const uint8_t*>(a.a);
    p.w[0] = static_cast<const uint8_t*>(a.b);
    p.ldx = p.ldw = p.K = a.K;
    p.M = a.M;
    p.N = a.N;
    p.segs = p.outs = 1;
    p.xs = a.a_scale;
    p.ws[0] = a.b_scale;
    p.kb = (a.K + 127) / 128;
    p.out[0] = a.y;
    p.ldo = a.N;
    return mm_run<KIND, SC, false, false, false, kMmOut, T>(p, a.ws, st);
}
template <int KIND, typename T>
hipError_t mm8_s(const Mm8Args& a, int scales, hipStream_t st) {
    if (scales == 2) return mm8<KIND, kMmBlock, T>(a, st);
    return scales == 1 ? mm8<KIND, kMmGroup, T>(a, st) : mm8<KIND, kMmRow, T>(a, st);
}

}  // namespace

namespace {

MmScales scales_of(int scales) { return scales == 2 ? kMmBlock : (scales == 1 ? kMmGroup : kMmRow); }

}  // namespace

size_t mm8_ws(int64_t M, int64_t N, int64_t K, int out_dtype, int scales, bool exact) {
    return mm_plan(out_dtype == 1 || exact ? kMmF8x : kMmF8, scales_of(scales), M, N, K, 1, 1, false, false).bytes;
}

hipError_t launch_mm8(const Mm8Args& a, int out_dtype, int scales, bool exact, hipStream_t st) {
    if (a.M == 0) return hipSuccess;
    if (a.K == 0) scales = 2;  // zeros, whatever the rows' scales are: those of blocks are read with a block alone
    if (out_dtype == 1) return mm8_s<kMmF8x, float>(a, scales, st);
    return exact ? mm8_s<kMmF8x, bf16_t>(a, scales, st) : mm8_s<kMmF8, bf16_t>(a, scales, st);
}

}  // namespace gdn
