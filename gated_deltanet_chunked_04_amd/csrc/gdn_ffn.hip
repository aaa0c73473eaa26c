// gdn_ffn.hip -- the gated feed-forward block:  g = x Wg^T, u = x Wu^T, h = act(g) u,  and its gradients
//   dg = d_h u act'(g), du = d_h act(g),  dx = dg Wg + du Wu,  dWg = dg^T x, dWu = du^T x.
// Gate and up are computed side by side by the same waves, so h is made where both sums are and neither is written
// (`pre` keeps them in fp32 for the backward, which otherwise computes them again). 8,192 x 2,048 x 8,192 bf16: forward with pre
// 681 us (550 GFLOP, 0.8 GB written), dx 474, both weights' gradients 517: see the tiles (gdn_mm.h) for what bounds them.
#include "gdn_layer.h"
#include "gdn_mm.h"
#include "gdn_products.h"

namespace gdn {

namespace {

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

const uint8_t* u8(const void* p) { return static_cast<const uint8_t*>(p); }

MmArgs block_args(const FfnArgs& a, int64_t size) {
    MmArgs p{};
    p.x[0] = u8(a.x);
    p.w[0] = u8(a.wg);
    p.w[1] = u8(a.wu);
    p.ldx = p.ldw = a.K * size;
    p.M = a.M;
    p.N = a.F;
    p.K = a.K;
    p.segs = p.outs = 1;
    p.out[0] = a.h;
    p.ldo = a.F;
    p.pre = a.pre;
    p.act = a.act;
    return p;
}

// Gradients of gate and up from the forward's values, 8 at a time; bound by memory (14 bytes a value in bf16: 8,192 x 8,192
// 169 us, 5.6 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void k_ffn_act_bwd(MmArgs p) {
    const int64_t per = (p.N + 7) / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= per * p.M) return;
    const int64_t m = i / per, n = i % per * 8;
    float a[8], u[8];
    mm_load<float, 8>(p.pre + m * p.N + n, a, p.N - n);
    mm_load<float, 8>(p.pre + (p.M + m) * p.N + n, u, p.N - n);
    mm_gate<kMmFfnBwd, T, 8, false>(p, m, n, a, u);
}

// columns of the gradients of gate and up in the workspace: whole vectors, zeros behind F
int64_t grad_ld(int64_t F) { return (F + 7) / 8 * 8; }
// Whether bf16 gradients of gate and up are kept as two bf16 each, the rounded value and what that leaves (16 bits), side by side
// in a memory row. Rounded once, they make the error of dx and of the weights' gradients sqrt 2 times these results' own
// rounding; in small matrices, where few of them weigh most, up to 2.4 times (16 values; 1.3 to 1.8 with 256, 1.33 to 1.50 with
// 4,096, 1.40 to 1.43 with 65,536). As pairs they add nothing to it (1.00), for twice the matrix instructions and no second
// read of the weights or of x (mm_pair_row). Below 65,536 values in one of the matrices that is no time lost: 7 x 8,192 x 8,192
// all gradients 300 us, 8 rows, which are rounded once, 384; 32,768 x 8,192 with F = 7 648, with F = 9 870. Large ones pay it
// where the caller asks (8,192 x 2,048 x 8,192: all gradients 1,040 us, as pairs 2,690, for tiles of 64 rows too).
bool grad_pairs(int64_t M, int64_t K, int64_t F) {
    const int64_t few = 65536;
    return M * F < few || M * K < few || F * K < few;
}

// dx and both weights' gradients from the gradients of gate and up, d.
template <int KIND, typename T, bool PAIRS>
hipError_t bwd_products(const FfnArgs& a, void* const (&d)[2], int64_t ldd, void* part, hipStream_t st) {
    MmArgs p{};
    for (int i = 0; i < 2; ++i) p.x[i] = u8(d[i]);
    p.low = PAIRS ? ldd * (int64_t)sizeof(T) : 0;
    p.ldx = (PAIRS ? 2 : 1) * ldd * (int64_t)sizeof(T);
    p.ldw = a.K * (int64_t)sizeof(T);
    p.N = p.ldo = a.K;
    if (a.dx && a.M) {
        p.w[0] = u8(a.wg);
        p.w[1] = u8(a.wu);
        p.M = a.M;
        p.K = a.F;
        p.segs = 2;
        p.outs = 1;
        p.out[0] = a.dx;
        if (hipError_t e = mm_run<KIND, kMmPlain, false, true, false, kMmOut, T, PAIRS>(p, part, st)) return e;
    }
    if (a.dwg) {
        p.w[0] = u8(a.x);
        p.w[1] = nullptr;
        p.M = a.F;
        p.K = a.M;
        p.segs = 1;
        p.outs = 2;
        p.out[0] = a.dwg;
        p.out[1] = a.dwu;
        if (hipError_t e = mm_run<KIND, kMmPlain, true, true, false, kMmOut, T, PAIRS>(p, part, st)) return e;
    }
    return hipGetLastError();
}

template <int KIND, typename T>
hipError_t bwd(const FfnArgs& a, hipStream_t st) {
    const int64_t size = sizeof(T), ldd = grad_ld(a.F);
    const bool pairs = KIND == kMmBf16 && (a.pairs || grad_pairs(a.M, a.K, a.F));
    const size_t bytes = align256((size_t)((pairs ? 2 : 1) * a.M * ldd * size));
    void *const d[2] = {a.ws, a.ws + bytes}, *const part = a.ws + 2 * bytes;
    if (a.M) {
        MmArgs p = block_args(a, size);
        p.out[0] = d[0];
        p.out[1] = d[1];
        p.ldo = (pairs ? 2 : 1) * ldd;
        p.d_h = a.d_h;
        p.low = pairs ? ldd * size : 0;
        if (a.pre) {
            const int64_t blocks = ((a.F + 7) / 8 * a.M + 255) / 256;
            if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
            hipLaunchKernelGGL(k_ffn_act_bwd<T>, dim3((unsigned)blocks), dim3(256), 0, st, p);
        } else if (hipError_t e = mm_run<KIND, kMmPlain, false, false, true, kMmFfnBwd, T>(p, part, st)) {
            return e;
        }
    }
    if constexpr (KIND == kMmBf16)
        if (pairs) return bwd_products<KIND, T, true>(a, d, ldd, part, st);
    return bwd_products<KIND, T, false>(a, d, ldd, part, st);
}

template <int KIND, typename T, int EPI = kMmFfn>
hipError_t ffn8(const FfnArgs& a, void* h, void* part, hipStream_t st) {
    MmArgs p = block_args(a, 1);
    p.xs = a.xs;
    p.ws[0] = a.gs;
    p.ws[1] = a.us;
    p.kb = (a.K + 127) / 128;
    p.out[0] = h;
    p.scale = a.hs;
    return mm_run<KIND, kMmBlock, false, false, true, EPI, T>(p, part, st);
}

}  // namespace

size_t ffn_fwd_ws(int64_t M, int64_t K, int64_t F, int dtype) {
    return mm_plan(dtype == 1 ? kMmF32 : kMmBf16, kMmPlain, M, F, K, 1, 1, false, true).bytes;
}
size_t ffn_bwd_ws(int64_t M, int64_t K, int64_t F, int dtype, bool pairs) {
    const int kind = dtype == 1 ? kMmF32 : kMmBf16;
    pairs = kind == kMmBf16 && (pairs || grad_pairs(M, K, F));
    size_t part = mm_plan(kind, kMmPlain, M, F, K, 1, 1, false, true).bytes;
    for (size_t b : {mm_plan(kind, kMmPlain, M, K, F, 2, 1, true, false, pairs).bytes, mm_plan(kind, kMmPlain, F, K, M, 1, 2, true, false, pairs).bytes})
        if (b > part) part = b;
    return 2 * align256((size_t)((pairs ? 2 : 1) * M * grad_ld(F) * (dtype == 1 ? 4 : 2))) + part;
}
// Few rows, or a split contraction: the parts, and the block's fp32 output in front of its quantisation. Otherwise the
// workgroup that has a row's 128 columns quantises them.
size_t ffn8_ws(int64_t M, int64_t K, int64_t F, int dtype, bool quant, bool exact) {
    const MmPlan r = mm_plan(quant || exact || dtype == 1 ? kMmF8x : kMmF8, kMmBlock, M, F, K, 1, 1, false, true);
    return (quant && (r.few || r.splits) ? align256((size_t)(M * F * 4)) : 0) + r.bytes;
}

hipError_t launch_ffn_fwd(const FfnArgs& a, int dtype, hipStream_t st) {
    if (a.M == 0) return hipSuccess;
    if (dtype == 1) return mm_run<kMmF32, kMmPlain, false, false, true, kMmFfn, float>(block_args(a, 4), a.ws, st);
    return mm_run<kMmBf16, kMmPlain, false, false, true, kMmFfn, bf16_t>(block_args(a, 2), a.ws, st);
}
hipError_t launch_ffn_bwd(const FfnArgs& a, int dtype, hipStream_t st) {
    return dtype == 1 ? bwd<kMmF32, float>(a, st) : bwd<kMmBf16, bf16_t>(a, st);
}
hipError_t launch_ffn8(const FfnArgs& a, int dtype, bool exact, hipStream_t st) {
    if (a.M == 0) return hipSuccess;
    if (!a.hs && dtype == 1) return ffn8<kMmF8x, float>(a, a.h, a.ws, st);
    if (!a.hs) return exact ? ffn8<kMmF8x, bf16_t>(a, a.h, a.ws, st) : ffn8<kMmF8, bf16_t>(a, a.h, a.ws, st);
    const MmPlan r = mm_plan(kMmF8x, kMmBlock, a.M, a.F, a.K, 1, 1, false, true);
    if (!r.few && !r.splits) return ffn8<kMmF8x, float, kMmFfn8>(a, a.h, nullptr, st);
    if (hipError_t e = ffn8<kMmF8x, float>(a, a.ws, a.ws + align256((size_t)(a.M * a.F * 4)), st)) return e;
    const QuantArgs q{a.M, a.F, a.ws, static_cast<uint8_t*>(a.h), a.hs};
    return launch_quant(q, 1, 1, false, st);
}

}  // namespace gdn
