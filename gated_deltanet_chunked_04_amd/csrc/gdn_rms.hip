// gdn_rms.hip -- RMS norm over a row of D values, with the residual stream's addition in front and
// an output in the input's type or in 8 bits (e4m3) with scales behind:
//   r = x + residual (rounded to the input's type: the value the stream keeps is the value that is
//       normed, so the gradient sees what the forward saw),
//   y = r w / sqrt(mean(r^2) + eps),
//   8 bits: scale = max|y| / 448 over a row or over 128 columns (1 where all are zero),
//           q = e4m3(y / scale), from the fp32 y.
// Gradient, with rh = r / sqrt(mean(r^2) + eps) and u = w dy:
//   dr = (u - rh mean(u rh)) / sqrt(mean(r^2) + eps) + d_residual,  dw = sum over rows of dy rh.
#include "gdn_layer.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kSumRows = 64;  // rows per partial sum of dw
constexpr float kE4m3Max = 448.f;

// Sum over the workgroup, the same bits for every thread.
__device__ __forceinline__ float block_sum(float v, float* sh) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < kThreads / 64; ++i) s += sh[i];
    return s;
}
// Largest bit pattern over the workgroup (of absolute values: NaN above infinity above the rest).
__device__ __forceinline__ uint32_t block_umax(uint32_t v, uint32_t* sh) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    uint32_t s = 0;
    for (int i = 0; i < kThreads / 64; ++i) s = max(s, sh[i]);
    return s;
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// e4m3 (OCP) of v, to nearest even, clamped to +-448; NaN stays NaN.
__device__ __forceinline__ uint8_t to_e4m3(float v) {
    v = v > kE4m3Max ? kE4m3Max : (v < -kE4m3Max ? -kE4m3Max : v);
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xFF);
}

template <typename T, typename TW, bool kQuant>
__global__ __launch_bounds__(kThreads) void k_rms_fwd(RmsArgs p) {
    __shared__ float sh[kThreads / 64];
    __shared__ uint32_t shu[kThreads / 64];
    const int64_t base = (int64_t)blockIdx.x * p.D;
    const T* x = static_cast<const T*>(p.x) + base;
    const T* res = p.res ? static_cast<const T*>(p.res) + base : nullptr;
    const TW* w = static_cast<const TW*>(p.w);
    T* keep = p.res_out ? static_cast<T*>(p.res_out) + base : nullptr;
    auto value = [&](int64_t c) {
        float v = Elem<T>::to_f(x[c]);
        return v;
    };
    // the sum is formed once and kept: later reads come from the stream's new value
    const T* r = keep ? keep : x;
    float ss = 0.f;
    for (int64_t c = threadIdx.x; c < p.D; c += kThreads) {
        float v = value(c);
        if (res) {
            const T q = Elem<T>::from_f(v + Elem<T>::to_f(res[c]));
            keep[c] = q;
            v = Elem<T>::to_f(q);
        }
        ss = fmaf(v, v, ss);
    }
    const float rstd = 1.f / sqrtf(block_sum(ss, sh) / (float)p.D + p.eps);
    auto norm = [&](int64_t c) { return Elem<T>::to_f(r[c]) * rstd * Elem<TW>::to_f(w[c]); };
    if constexpr (!kQuant) {
        T* y = static_cast<T*>(p.y) + base;
        for (int64_t c = threadIdx.x; c < p.D; c += kThreads) y[c] = Elem<T>::from_f(norm(c));
    } else {
        uint8_t* y = static_cast<uint8_t*>(p.y) + base;
        const int64_t G = p.group, groups = (p.D + G - 1) / G;
        for (int64_t i = 0; i < groups; ++i) {
            const int64_t c1 = (i + 1) * G < p.D ? (i + 1) * G : p.D;
            uint32_t m = 0;
            for (int64_t c = i * G + threadIdx.x; c < c1; c += kThreads) m = max(m, abs_bits(norm(c)));
            const float amax = __uint_as_float(block_umax(m, shu));
            const float scale = amax == 0.f ? 1.f : amax / kE4m3Max;
            for (int64_t c = i * G + threadIdx.x; c < c1; c += kThreads) y[c] = to_e4m3(norm(c) / scale);
            if (threadIdx.x == 0) p.scale[(int64_t)blockIdx.x * groups + i] = scale;
        }
    }
}

template <typename T, typename TW>
__global__ __launch_bounds__(kThreads) void k_rms_dx(RmsArgs p, float* rstds) {
    __shared__ float sh[kThreads / 64];
    const int64_t base = (int64_t)blockIdx.x * p.D;
    const T* r = static_cast<const T*>(p.x) + base;
    const T* dy = static_cast<const T*>(p.d_y) + base;
    const T* dres = p.d_res ? static_cast<const T*>(p.d_res) + base : nullptr;
    const TW* w = static_cast<const TW*>(p.w);
    T* dx = static_cast<T*>(p.dx) + base;
    float ss = 0.f, dot = 0.f;
    for (int64_t c = threadIdx.x; c < p.D; c += kThreads) {
        const float v = Elem<T>::to_f(r[c]);
        ss = fmaf(v, v, ss);
        dot = fmaf(Elem<T>::to_f(dy[c]) * Elem<TW>::to_f(w[c]), v, dot);
    }
    const float rstd = 1.f / sqrtf(block_sum(ss, sh) / (float)p.D + p.eps);
    const float m = block_sum(dot, sh) * rstd / (float)p.D;
    for (int64_t c = threadIdx.x; c < p.D; c += kThreads) {
        const float rh = Elem<T>::to_f(r[c]) * rstd;
        float d = rstd * (Elem<T>::to_f(dy[c]) * Elem<TW>::to_f(w[c]) - rh * m);
        if (dres) d += Elem<T>::to_f(dres[c]);
        dx[c] = Elem<T>::from_f(d);
    }
    if (threadIdx.x == 0) rstds[blockIdx.x] = rstd;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_rms_dw(RmsArgs p, const float* rstds, float* part) {
    const int64_t c = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    if (c >= p.D) return;
    const int64_t r0 = (int64_t)blockIdx.x * kSumRows, r1 = r0 + kSumRows < p.rows ? r0 + kSumRows : p.rows;
    float s = 0.f;
    for (int64_t i = r0; i < r1; ++i)
        s = fmaf(Elem<T>::to_f(static_cast<const T*>(p.d_y)[i * p.D + c]),
                 Elem<T>::to_f(static_cast<const T*>(p.x)[i * p.D + c]) * rstds[i], s);
    part[(int64_t)blockIdx.x * p.D + c] = s;
}

__global__ __launch_bounds__(kThreads) void k_rms_dw_sum(const float* part, int64_t parts, int64_t D, float* dw) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= D) return;
    float s = 0.f;
    for (int64_t i = 0; i < parts; ++i) s += part[i * D + c];
    dw[c] = s;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
int64_t parts_of(int64_t rows) { return (rows + kSumRows - 1) / kSumRows; }

template <typename T, typename TW>
hipError_t fwd_t(const RmsArgs& a, int out, hipStream_t st) {
    if (a.rows == 0) return hipSuccess;
    if (out == 0) hipLaunchKernelGGL((k_rms_fwd<T, TW, false>), dim3((unsigned)a.rows), dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((k_rms_fwd<T, TW, true>), dim3((unsigned)a.rows), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

template <typename T, typename TW>
hipError_t bwd_t(const RmsArgs& a, hipStream_t st) {
    float* rstds = reinterpret_cast<float*>(a.ws);
    float* part = reinterpret_cast<float*>(a.ws + align256((size_t)a.rows * 4));
    const int64_t parts = parts_of(a.rows);
    const unsigned cb = (unsigned)((a.D + kThreads - 1) / kThreads);
    if (a.rows) {
        hipLaunchKernelGGL((k_rms_dx<T, TW>), dim3((unsigned)a.rows), dim3(kThreads), 0, st, a, rstds);
        if (a.dw) hipLaunchKernelGGL((k_rms_dw<T>), dim3((unsigned)parts, cb), dim3(kThreads), 0, st, a, rstds, part);
    }
    if (a.dw) hipLaunchKernelGGL(k_rms_dw_sum, dim3(cb), dim3(kThreads), 0, st, part, parts, a.D, a.dw);
    return hipGetLastError();
}

}  // namespace

size_t rms_bwd_ws(int64_t rows, int64_t D) { return align256((size_t)rows * 4) + (size_t)parts_of(rows) * D * 4; }

// dtype, w_dtype: gdn_dtype (0 bf16, 1 fp32); the weight in the type of x or fp32
hipError_t launch_rms_fwd(const RmsArgs& a, int dtype, int w_dtype, int out, hipStream_t st) {
    if (dtype == 1) return fwd_t<float, float>(a, out, st);
    return w_dtype == 1 ? fwd_t<bf16_t, float>(a, out, st) : fwd_t<bf16_t, bf16_t>(a, out, st);
}
hipError_t launch_rms_bwd(const RmsArgs& a, int dtype, int w_dtype, hipStream_t st) {
    if (dtype == 1) return bwd_t<float, float>(a, st);
    return w_dtype == 1 ? bwd_t<bf16_t, float>(a, st) : bwd_t<bf16_t, bf16_t>(a, st);
}

}  // namespace gdn
