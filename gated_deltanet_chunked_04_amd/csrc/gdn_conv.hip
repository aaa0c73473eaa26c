// gdn_conv.hip -- the short causal convolution in front of the recurrences, one filter of W taps
// per channel: z_t = bias + sum_j w_j x_{t-W+1+j}, y = z or silu(z). The inputs before a sequence's
// first token are its entering state [W-1, D] (zeros without one); its last W-1 inputs leave as the
// final state. Gradient: dz = dy act'(z), z recomputed;
//   dx_s = sum_i w_{W-1-i} dz_{s+i},  dw_j = sum_t dz_t x_{t-W+1+j},  dbias = sum_t dz_t,
// positions before the first token giving the entering state's gradient.
#include "gdn_layer.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kSumTokens = 512;  // tokens per partial sum of dw and dbias

// Input at position t of sequence s: a token, or before its first one a row of the entering state.
template <typename T>
__device__ __forceinline__ float input_at(const ConvArgs& p, const SeqPos& s, int32_t t, int64_t c) {
    if (t >= s.start) return Elem<T>::to_f(static_cast<const T*>(p.x)[(int64_t)t * p.D + c]);
    if (!p.s0) return 0.f;
    const int64_t row = (int64_t)s.n * (p.W - 1) + (t - s.start + p.W - 1);
    return Elem<T>::to_f(static_cast<const T*>(p.s0)[row * p.D + c]);
}

template <typename T, typename TW>
__device__ __forceinline__ float pre_act(const ConvArgs& p, const SeqPos& s, int32_t t, int64_t c) {
    float z = p.bias ? Elem<TW>::to_f(static_cast<const TW*>(p.bias)[c]) : 0.f;
    for (int j = 0; j < p.W; ++j)
        z = fmaf(Elem<TW>::to_f(static_cast<const TW*>(p.w)[c * p.W + j]), input_at<T>(p, s, t - p.W + 1 + j, c), z);
    return z;
}

template <typename T, typename TW>
__device__ __forceinline__ float d_pre_act(const ConvArgs& p, const SeqPos& s, int32_t t, int64_t c) {
    const float dy = Elem<T>::to_f(static_cast<const T*>(p.d_y)[(int64_t)t * p.D + c]);
    if (!p.silu) return dy;
    const float z = pre_act<T, TW>(p, s, t, c);
    const float sg = 1.f / (1.f + fast_exp(-z));
    return dy * sg * (1.f + z * (1.f - sg));
}

template <typename T, typename TW>
__global__ __launch_bounds__(kThreads) void k_conv_fwd(ConvArgs p) {
    const int64_t c = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    const int32_t t = blockIdx.x;
    if (c >= p.D) return;
    const SeqPos s = seq_find(p.seq, t);
    if (t < s.start || t >= s.end) return;
    float z = pre_act<T, TW>(p, s, t, c);
    if (p.silu) z = z / (1.f + fast_exp(-z));
    static_cast<T*>(p.y)[(int64_t)t * p.D + c] = Elem<T>::from_f(z);
}

// Final states: a thread reads all W-1 rows of its channel before it writes them, so that the
// entering states may be overwritten in place.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_conv_final(ConvArgs p) {
    const int64_t c = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    if (c >= p.D) return;
    const SeqPos s = seq_at(p.seq, blockIdx.x);
    float v[3];
    const int32_t end = s.end > s.start ? s.end : s.start;
    for (int r = 0; r < p.W - 1; ++r) v[r] = input_at<T>(p, s, end - p.W + 1 + r, c);
    for (int r = 0; r < p.W - 1; ++r)
        static_cast<T*>(p.sT)[((int64_t)s.n * (p.W - 1) + r) * p.D + c] = Elem<T>::from_f(v[r]);
}

// dL/d(input at position t), t from W-1 before the sequence's first token to its last token.
template <typename T, typename TW>
__device__ __forceinline__ float d_input(const ConvArgs& p, const SeqPos& s, int32_t t, int64_t c) {
    float d = 0.f;
    for (int i = 0; i < p.W; ++i)
        if (t + i >= s.start && t + i < s.end)
            d = fmaf(Elem<TW>::to_f(static_cast<const TW*>(p.w)[c * p.W + p.W - 1 - i]),
                     d_pre_act<T, TW>(p, s, t + i, c), d);
    const int32_t end = s.end > s.start ? s.end : s.start;
    const int32_t r = t - (end - p.W + 1);
    if (p.d_sT && r >= 0)
        d += Elem<T>::to_f(static_cast<const T*>(p.d_sT)[((int64_t)s.n * (p.W - 1) + r) * p.D + c]);
    return d;
}

template <typename T, typename TW>
__global__ __launch_bounds__(kThreads) void k_conv_dx(ConvArgs p) {
    const int64_t c = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    const int32_t t = blockIdx.x;
    if (c >= p.D) return;
    const SeqPos s = seq_find(p.seq, t);
    if (t < s.start || t >= s.end) return;
    static_cast<T*>(p.dx)[(int64_t)t * p.D + c] = Elem<T>::from_f(d_input<T, TW>(p, s, t, c));
}

template <typename T, typename TW>
__global__ __launch_bounds__(kThreads) void k_conv_dstate(ConvArgs p) {
    const int64_t c = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    if (c >= p.D) return;
    const SeqPos s = seq_at(p.seq, blockIdx.x);
    for (int r = 0; r < p.W - 1; ++r)
        static_cast<T*>(p.ds0)[((int64_t)s.n * (p.W - 1) + r) * p.D + c] =
            Elem<T>::from_f(d_input<T, TW>(p, s, s.start - p.W + 1 + r, c));
}

// Partial sums over kSumTokens tokens, [parts, W + 1, D] (the taps, then the bias).
template <typename T, typename TW>
__global__ __launch_bounds__(kThreads) void k_conv_dw(ConvArgs p, float* part) {
    const int64_t c = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    if (c >= p.D) return;
    const int32_t t0 = blockIdx.x * kSumTokens, t1 = min(t0 + kSumTokens, p.seq.total);
    float acc[5] = {};
    SeqPos s = seq_find(p.seq, t0);
    for (int32_t t = t0; t < t1; ++t) {
        seq_advance(p.seq, s, t);
        if (t < s.start || t >= s.end) continue;
        const float dz = d_pre_act<T, TW>(p, s, t, c);
        for (int j = 0; j < p.W; ++j) acc[j] = fmaf(dz, input_at<T>(p, s, t - p.W + 1 + j, c), acc[j]);
        acc[4] += dz;
    }
    float* out = part + (int64_t)blockIdx.x * (p.W + 1) * p.D + c;
    for (int j = 0; j < p.W; ++j) out[j * p.D] = acc[j];
    out[p.W * p.D] = acc[4];
}

__global__ __launch_bounds__(kThreads) void k_conv_dw_sum(const float* part, int parts, int W, int64_t D, float* dw, float* db) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int j = blockIdx.y;
    if (c >= D) return;
    float s = 0.f;
    for (int i = 0; i < parts; ++i) s += part[((int64_t)i * (W + 1) + j) * D + c];
    if (j < W) dw[c * W + j] = s;
    else if (db) db[c] = s;
}

template <typename T, typename TW>
hipError_t fwd_t(const ConvArgs& a, hipStream_t st) {
    const unsigned cb = (unsigned)((a.D + kThreads - 1) / kThreads);
    if (a.seq.total)
        hipLaunchKernelGGL((k_conv_fwd<T, TW>), dim3((unsigned)a.seq.total, cb), dim3(kThreads), 0, st, a);
    if (a.sT) hipLaunchKernelGGL((k_conv_final<T>), dim3((unsigned)a.seq.N, cb), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

int parts_of(int64_t total) { return (int)((total + kSumTokens - 1) / kSumTokens); }

template <typename T, typename TW>
hipError_t bwd_t(const ConvArgs& a, hipStream_t st) {
    const unsigned cb = (unsigned)((a.D + kThreads - 1) / kThreads);
    const int parts = parts_of(a.seq.total);
    float* part = reinterpret_cast<float*>(a.ws);
    if (a.seq.total) {
        hipLaunchKernelGGL((k_conv_dx<T, TW>), dim3((unsigned)a.seq.total, cb), dim3(kThreads), 0, st, a);
        hipLaunchKernelGGL((k_conv_dw<T, TW>), dim3((unsigned)parts, cb), dim3(kThreads), 0, st, a, part);
    }
    if (a.ds0) hipLaunchKernelGGL((k_conv_dstate<T, TW>), dim3((unsigned)a.seq.N, cb), dim3(kThreads), 0, st, a);
    hipLaunchKernelGGL(k_conv_dw_sum, dim3(cb, (unsigned)a.W + 1), dim3(kThreads), 0, st, part, parts, a.W, a.D, a.dw, a.db);
    return hipGetLastError();
}

}  // namespace

size_t conv_bwd_ws(int64_t total, int64_t D, int W) { return (size_t)parts_of(total) * (W + 1) * D * 4; }

// dtype, w_dtype: gdn_dtype (0 bf16, 1 fp32); the filter in the type of x or fp32
hipError_t launch_conv_fwd(const ConvArgs& a, int dtype, int w_dtype, hipStream_t st) {
    if (dtype == 1) return fwd_t<float, float>(a, st);
    return w_dtype == 1 ? fwd_t<bf16_t, float>(a, st) : fwd_t<bf16_t, bf16_t>(a, st);
}
hipError_t launch_conv_bwd(const ConvArgs& a, int dtype, int w_dtype, hipStream_t st) {
    if (dtype == 1) return bwd_t<float, float>(a, st);
    return w_dtype == 1 ? bwd_t<bf16_t, float>(a, st) : bwd_t<bf16_t, bf16_t>(a, st);
}

}  // namespace gdn
