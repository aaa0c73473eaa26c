// gdn_layer.h -- the operators around the gated delta rule in a layer: the gated scan
// (gdn_gscan.hip), the short convolution (gdn_conv.hip) and the RMS norm with residual addition
// and 8-bit output (gdn_rms.hip): argument structs, launchers, and the view of packed sequences
// that the first two share. The C entry points are in gdn_layer_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_common.h"

namespace gdn {

// Sequences over the flattened token axis (B*T tokens). Packed: sequence n owns tokens
// [cu[n], cu[n+1]); otherwise sequence n is row n, tokens [nT, (n+1)T). Offsets read from the
// device are clamped into [0, total], so a bad array gives wrong values and no access out of range.
struct SeqView {
    const int32_t* cu;  // device, or null
    int32_t T;          // tokens per row (cu null)
    int32_t total;      // B * T
    int32_t N;
};
struct SeqPos {
    int32_t n, start, end;  // a token t belongs to the sequence iff start <= t < end
};

typedef const __attribute__((address_space(4))) int32_t seq_const_i32;
// Uniform reads of the offsets through the scalar cache (the kernels never write them).
__device__ __forceinline__ int32_t seq_off(const SeqView& s, int32_t n) {
    const int32_t v = ((seq_const_i32*)(uintptr_t)s.cu)[n];
    return v < 0 ? 0 : (v > s.total ? s.total : v);
}
__device__ __forceinline__ SeqPos seq_at(const SeqView& s, int32_t n) {
    if (!s.cu) return SeqPos{n, n * s.T, (n + 1) * s.T};
    return SeqPos{n, seq_off(s, n), seq_off(s, n + 1)};
}
// The sequence that holds token t (t wave-uniform, 0 <= t < total): the last n whose start is at
// or before t. Tokens before the first or behind the last sequence get a SeqPos that does not
// hold them.
__device__ __forceinline__ SeqPos seq_find(const SeqView& s, int32_t t) {
    if (!s.cu) return seq_at(s, t / s.T);
    int32_t lo = 0, hi = s.N - 1;
    while (lo < hi) {
        const int32_t mid = hi - ((hi - lo) >> 1);  // (no sum of the two: N may be near 2^31)
        if (seq_off(s, mid) <= t) lo = mid; else hi = mid - 1;
    }
    return seq_at(s, lo);
}
// Advance p to the sequence that holds t, t at or behind p's start: mostly the next one, else (behind sequences
// without tokens) by search.
__device__ __forceinline__ void seq_advance(const SeqView& s, SeqPos& p, int32_t t) {
    if (t < p.end || p.n + 1 >= s.N) return;
    p = seq_at(s, p.n + 1);
    if (t >= p.end) p = seq_find(s, t);
}
// The same backwards, t before p's end.
__device__ __forceinline__ void seq_retreat(const SeqView& s, SeqPos& p, int32_t t) {
    if (t >= p.start || p.n == 0) return;
    p = seq_at(s, p.n - 1);
    if (t < p.start || t >= p.end) p = seq_find(s, t);
}
// Calls f(n) (uniform) for every sequence without tokens, kEmptyRun sequences looked at together by each of `waves`
// waves. Whole waves call it.
constexpr int kEmptyRun = 8;
template <typename F>
__device__ __forceinline__ void for_each_empty(const SeqView& s, int wave, int waves, F f) {
    const int lane = threadIdx.x & 63;
    for (int64_t base = (int64_t)wave * kEmptyRun; base < s.N; base += (int64_t)waves * kEmptyRun) {
        const int64_t n = base + lane;
        bool empty = false;
        if (lane < kEmptyRun && n < s.N) {
            if (s.cu) {
                const int32_t a = s.cu[n], b = s.cu[n + 1];
                empty = min(max(a, 0), s.total) >= min(max(b, 0), s.total);
            } else {
                empty = s.T == 0;
            }
        }
        for (uint64_t m = __ballot(empty); m; m &= m - 1) f((int32_t)(base + __builtin_ctzll(m)));
    }
}
// Workgroups (per block of channels) of `waves` waves that look for sequences without tokens: one for every few
// sequences, 64 at most (one alone was the longest of the launch: 56 sequences of 10 tokens among 200 empty ones x 2048, scan
// 22.5 -> 15.3 us, convolution 33 -> 7.9; 2,048 of two tokens, each with an empty one, 129 -> 56 and 462 -> 27).
inline int empty_blocks(const SeqView& s, int waves) {
    const int64_t n = ((int64_t)s.N + kEmptyRun * waves - 1) / (kEmptyRun * waves);
    return (int)(n < 64 ? n : 64);
}

// A launch's threads are counted in 32 bits. Launchers return hipErrorInvalidConfiguration for more.
inline bool grid_fits(int64_t blocks, int threads) { return blocks <= (int64_t)UINT32_MAX / threads; }

// ---- gated scan ---------------------------------------------------------------------------
constexpr int kScanTile = 64;  // tokens between two entries of the kept states

struct GScanArgs {
    SeqView seq;
    int64_t D;
    const void* x;
    const void* g;
    const void* d_h;
    const float* s0;
    const float* d_sT;
    void* h;       // null: only the states are wanted
    float* sT;
    float* states;  // [ceil(total / 64), D]: the state entering every 64th token
    void* dx;
    void* dg;
    float* ds0;
    unsigned char* ws;
    bool zero;     // rows of no sequence get zeros
};
size_t gscan_fwd_ws(const SeqView& seq, int64_t D);
size_t gscan_bwd_ws(const SeqView& seq, int64_t D);
hipError_t launch_gscan_fwd(const GScanArgs& a, int dtype, int g_dtype, hipStream_t st);
hipError_t launch_gscan_bwd(const GScanArgs& a, int dtype, int g_dtype, bool have_states, hipStream_t st);

// ---- short convolution --------------------------------------------------------------------
struct ConvArgs {
    SeqView seq;
    int64_t D;
    int32_t W, silu;
    const void* x;
    const void* w;
    const void* bias;
    const void* s0;
    void* sT;
    void* y;
    const void* d_y;
    const void* d_sT;
    void* dx;
    float* dw;
    float* db;
    void* ds0;
    unsigned char* ws;
    bool zero;  // as above
};
size_t conv_bwd_ws(int64_t total, int64_t D, int W, int dtype);
hipError_t launch_conv_fwd(const ConvArgs& a, int dtype, int w_dtype, hipStream_t st);
hipError_t launch_conv_bwd(const ConvArgs& a, int dtype, int w_dtype, hipStream_t st);

// ---- RMS norm -----------------------------------------------------------------------------
struct RmsArgs {
    int64_t rows, D;
    float eps;
    int32_t group;  // columns per scale (D: one per row)
    const void* x;
    const void* res;
    const void* w;
    void* y;
    float* scale;
    void* res_out;
    const void* d_y;
    const void* d_res;
    void* dx;
    float* dw;
    unsigned char* ws;
};
size_t rms_bwd_ws(int64_t rows, int64_t D);
hipError_t launch_rms_fwd(const RmsArgs& a, int dtype, int w_dtype, int out, hipStream_t st);
hipError_t launch_rms_bwd(const RmsArgs& a, int dtype, int w_dtype, hipStream_t st);

}  // namespace gdn
