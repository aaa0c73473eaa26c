// gdn_gscan.hip -- the gated scan, the recurrence with a gate per channel instead of a matrix
// state per head: h_t = exp(g_t) h_{t-1} + x_t, and its gradient
//   mu_t = a_t (dh_t + mu_{t+1}),  dx_t = dh_t + mu_{t+1},  dg_t = mu_t h_{t-1},  dh_0 = mu_1,
// a = exp(g), mu behind the last token of a sequence = the gradient of its final state.
//
// The token axis is cut into tiles. A tile acts on the state that enters it as c -> A c + H, so
// three launches do it: the pair (A, H) of every tile, a scan over the pairs that leaves every
// tile's entering state, and the tiles again from their states. The gradient does the same from
// the other end, with the forward's entering states at hand to recompute h inside a tile in fp32.
#include "gdn_layer.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

// A c + H. A with its sign bit set marks a tile in which a sequence starts: nothing of c passes,
// whatever it holds. c = 0 passes nothing either, also where growing gates took A to infinity.
__device__ __forceinline__ float pass_on(float A, float H, float c) {
    return (__float_as_int(A) < 0 || c == 0.f) ? H : fmaf(A, c, H);
}

template <typename TX, typename TG, bool kRev>
__global__ __launch_bounds__(kThreads) void k_pairs(GScanArgs p, float2* pairs) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int32_t t0 = blockIdx.y * kScanTile;
    const int32_t t1 = min(t0 + kScanTile, p.seq.total);
    if (c >= p.D) return;
    const TX* x = static_cast<const TX*>(kRev ? p.d_h : p.x);
    const TG* g = static_cast<const TG*>(p.g);
    float A = 1.f, H = 0.f;
    if (!kRev) {
        SeqPos s = seq_find(p.seq, t0);
        for (int32_t t = t0; t < t1; ++t) {
            seq_advance(p.seq, s, t);
            if (t < s.start || t >= s.end) continue;
            const int64_t at = (int64_t)t * p.D + c;
            const float a = fast_exp(Elem<TG>::to_f(g[at]));
            if (t == s.start) {
                A = -1.f;
                H = p.s0 ? p.s0[(int64_t)s.n * p.D + c] : 0.f;
            }
            H = fmaf(a, H, Elem<TX>::to_f(x[at]));
            A *= a;
        }
    } else {
        for (int32_t t = t1 - 1; t >= t0; --t) {
            const SeqPos s = seq_find(p.seq, t);
            if (t < s.start || t >= s.end) continue;
            const int64_t at = (int64_t)t * p.D + c;
            const float a = fast_exp(Elem<TG>::to_f(g[at]));
            if (t + 1 == s.end) {
                A = -1.f;
                H = p.d_sT ? p.d_sT[(int64_t)s.n * p.D + c] : 0.f;
            }
            H = a * (Elem<TX>::to_f(x[at]) + H);
            A *= a;
        }
    }
    pairs[(int64_t)blockIdx.y * p.D + c] = make_float2(A, H);
}

template <bool kRev>
__global__ __launch_bounds__(kThreads) void k_carry(const float2* pairs, float* states, int tiles, int64_t D) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= D) return;
    float s = 0.f;
    for (int i = 0; i < tiles; ++i) {
        const int64_t at = (int64_t)(kRev ? tiles - 1 - i : i) * D + c;
        states[at] = s;
        const float2 q = pairs[at];
        s = pass_on(q.x, q.y, s);
    }
}

template <typename TX, typename TG>
__global__ __launch_bounds__(kThreads) void k_fwd(GScanArgs p) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int32_t t0 = blockIdx.y * kScanTile;
    const int32_t t1 = min(t0 + kScanTile, p.seq.total);
    if (c >= p.D) return;
    const TX* x = static_cast<const TX*>(p.x);
    const TG* g = static_cast<const TG*>(p.g);
    TX* out = static_cast<TX*>(p.h);
    float h = p.states[(int64_t)blockIdx.y * p.D + c];
    SeqPos s = seq_find(p.seq, t0);
    for (int32_t t = t0; t < t1; ++t) {
        seq_advance(p.seq, s, t);
        if (t < s.start || t >= s.end) continue;
        const int64_t at = (int64_t)t * p.D + c;
        if (t == s.start) h = p.s0 ? p.s0[(int64_t)s.n * p.D + c] : 0.f;
        h = fmaf(fast_exp(Elem<TG>::to_f(g[at])), h, Elem<TX>::to_f(x[at]));
        out[at] = Elem<TX>::from_f(h);
        if (t + 1 == s.end && p.sT) p.sT[(int64_t)s.n * p.D + c] = h;
    }
}

template <typename TX, typename TG>
__global__ __launch_bounds__(kThreads) void k_bwd(GScanArgs p, const float* rstates) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int32_t t0 = blockIdx.y * kScanTile;
    if (c >= p.D) return;
    const TX* x = static_cast<const TX*>(p.x);
    const TX* dh = static_cast<const TX*>(p.d_h);
    const TG* g = static_cast<const TG*>(p.g);
    TX* dx = static_cast<TX*>(p.dx);
    TG* dg = static_cast<TG*>(p.dg);
    float before[kScanTile];
    float h = p.states[(int64_t)blockIdx.y * p.D + c];
    SeqPos s = seq_find(p.seq, t0);
#pragma unroll
    for (int i = 0; i < kScanTile; ++i) {
        const int32_t t = t0 + i;
        if (t >= p.seq.total) continue;
        seq_advance(p.seq, s, t);
        if (t < s.start || t >= s.end) continue;
        const int64_t at = (int64_t)t * p.D + c;
        if (t == s.start) h = p.s0 ? p.s0[(int64_t)s.n * p.D + c] : 0.f;
        before[i] = h;
        h = fmaf(fast_exp(Elem<TG>::to_f(g[at])), h, Elem<TX>::to_f(x[at]));
    }
    float mu = rstates[(int64_t)blockIdx.y * p.D + c];
#pragma unroll
    for (int i = kScanTile - 1; i >= 0; --i) {
        const int32_t t = t0 + i;
        if (t >= p.seq.total) continue;
        s = seq_find(p.seq, t);
        if (t < s.start || t >= s.end) continue;
        const int64_t at = (int64_t)t * p.D + c;
        if (t + 1 == s.end) mu = p.d_sT ? p.d_sT[(int64_t)s.n * p.D + c] : 0.f;
        const float lam = Elem<TX>::to_f(dh[at]) + mu;
        mu = fast_exp(Elem<TG>::to_f(g[at])) * lam;
        dx[at] = Elem<TX>::from_f(lam);
        dg[at] = Elem<TG>::from_f(mu * before[i]);
        if (t == s.start && p.ds0) p.ds0[(int64_t)s.n * p.D + c] = mu;
    }
}

// Sequences without tokens: their state (or its gradient) passes through.
__global__ __launch_bounds__(kThreads) void k_empty(SeqView seq, int64_t D, const float* in, float* out) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    for (int32_t n = blockIdx.y; n < seq.N; n += gridDim.y) {
        const SeqPos s = seq_at(seq, n);
        if (s.start < s.end || c >= D) continue;
        out[(int64_t)n * D + c] = in ? in[(int64_t)n * D + c] : 0.f;
    }
}

hipError_t empties(const GScanArgs& a, const float* in, float* out, hipStream_t st) {
    if (!out || (!a.seq.cu && a.seq.T > 0)) return hipSuccess;
    const dim3 grid((unsigned)((a.D + kThreads - 1) / kThreads), (unsigned)(a.seq.N < 1024 ? a.seq.N : 1024));
    hipLaunchKernelGGL(k_empty, grid, dim3(kThreads), 0, st, a.seq, a.D, in, out);
    return hipGetLastError();
}

int tiles_of(int64_t total) { return (int)((total + kScanTile - 1) / kScanTile); }
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

template <typename TX, typename TG>
hipError_t fwd_states(const GScanArgs& a, float2* pairs, hipStream_t st) {
    const int tiles = tiles_of(a.seq.total);
    const dim3 grid((unsigned)((a.D + kThreads - 1) / kThreads), (unsigned)tiles);
    hipLaunchKernelGGL((k_pairs<TX, TG, false>), grid, dim3(kThreads), 0, st, a, pairs);
    hipLaunchKernelGGL((k_carry<false>), dim3(grid.x), dim3(kThreads), 0, st, pairs, a.states, tiles, a.D);
    return hipGetLastError();
}

template <typename TX, typename TG>
hipError_t fwd_t(GScanArgs a, hipStream_t st) {
    const int tiles = tiles_of(a.seq.total);
    if (tiles) {
        float2* pairs = reinterpret_cast<float2*>(a.ws);
        if (!a.states) a.states = reinterpret_cast<float*>(a.ws + align256((size_t)tiles * a.D * 8));
        if (hipError_t e = fwd_states<TX, TG>(a, pairs, st)) return e;
        const dim3 grid((unsigned)((a.D + kThreads - 1) / kThreads), (unsigned)tiles);
        hipLaunchKernelGGL((k_fwd<TX, TG>), grid, dim3(kThreads), 0, st, a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    return empties(a, a.s0, a.sT, st);
}

template <typename TX, typename TG>
hipError_t bwd_t(GScanArgs a, bool have, hipStream_t st) {
    const int tiles = tiles_of(a.seq.total);
    if (tiles) {
        float2* pairs = reinterpret_cast<float2*>(a.ws);
        float* rst = reinterpret_cast<float*>(a.ws + align256((size_t)tiles * a.D * 8));
        const dim3 grid((unsigned)((a.D + kThreads - 1) / kThreads), (unsigned)tiles);
        if (!have) {
            a.states = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(rst) + align256((size_t)tiles * a.D * 4));
            if (hipError_t e = fwd_states<TX, TG>(a, pairs, st)) return e;
        }
        hipLaunchKernelGGL((k_pairs<TX, TG, true>), grid, dim3(kThreads), 0, st, a, pairs);
        hipLaunchKernelGGL((k_carry<true>), dim3(grid.x), dim3(kThreads), 0, st, pairs, rst, tiles, a.D);
        hipLaunchKernelGGL((k_bwd<TX, TG>), grid, dim3(kThreads), 0, st, a, rst);
        if (hipError_t e = hipGetLastError()) return e;
    }
    return empties(a, a.d_sT, a.ds0, st);
}

}  // namespace

size_t gscan_fwd_ws(int64_t total, int64_t D) {
    const size_t n = (size_t)tiles_of(total) * D;
    return align256(n * 8) + align256(n * 4);
}
size_t gscan_bwd_ws(int64_t total, int64_t D) {
    const size_t n = (size_t)tiles_of(total) * D;
    return align256(n * 8) + 2 * align256(n * 4);
}

// dtype, g_dtype: gdn_dtype (0 bf16, 1 fp32); g in the type of x or fp32
hipError_t launch_gscan_fwd(const GScanArgs& a, int dtype, int g_dtype, hipStream_t st) {
    if (dtype == 1) return fwd_t<float, float>(a, st);
    return g_dtype == 1 ? fwd_t<bf16_t, float>(a, st) : fwd_t<bf16_t, bf16_t>(a, st);
}
hipError_t launch_gscan_bwd(const GScanArgs& a, int dtype, int g_dtype, bool have_states, hipStream_t st) {
    if (dtype == 1) return bwd_t<float, float>(a, have_states, st);
    return g_dtype == 1 ? bwd_t<bf16_t, float>(a, have_states, st) : bwd_t<bf16_t, bf16_t>(a, have_states, st);
}

}  // namespace gdn
