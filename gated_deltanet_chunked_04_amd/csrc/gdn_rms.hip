// gdn_rms.hip -- RMS norm over a row of D values, with the residual stream's addition in front and
// an output in the input's type or in 8 bits (e4m3) with scales behind:
//   r = x + residual (rounded to the input's type: the value the stream keeps is the value that is
//       normed, so the gradient sees what the forward saw),
//   y = r w / sqrt(mean(r^2) + eps),
//   8 bits: scale = max|y| / 448 over a row or over 128 columns (at least 2^-126; 1 where all are zero),
//           q = e4m3(y / scale), from the fp32 y.
// Gradient, with rh = r / sqrt(mean(r^2) + eps) and u = w dy:
//   dr = (u - rh mean(u rh)) / sqrt(mean(r^2) + eps) + d_residual,  dw = sum over rows of dy rh.
//
// Bound by memory (about 6 operations per element forward and 10 backward against 7 or 8 bytes in
// bf16), so a row is read once and stays in registers between its sum and its output: a lane owns
// vectors of 8 neighbouring columns, a row belongs to 4 to 1,024 threads: up to 256 columns several rows share a
// wave, up to 512 a wave takes one and up to 1,024 two waves, above that a workgroup (shape_of). 16 lanes that sit
// side by side own 128 columns, so the maximum behind a scale of 128 columns is taken inside a row of 16 lanes.
// Rows too long for a workgroup's registers are read again.
#include "gdn_e4m3.h"
#include "gdn_layer.h"
#include "gdn_vec.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxWaves = 16;

// Sum (or largest) over the LANES threads of a row: 4, 16 or 32 lanes, a wave, or LANES / 64 waves through LDS. The
// same bits in every one. `slot`: which of the kernel's LDS words this call uses (two calls in a row use different
// ones, so one barrier per call is enough). All threads call it.
template <int LANES> constexpr int waves_of() { return LANES > 64 ? LANES / 64 : 1; }
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float (*sh)[kMaxWaves], int slot) {
    if constexpr (LANES == 4) {
        v += dpp_f<0xB1>(v);
        return v + dpp_f<0x4E>(v);
    }
    v = sum_ln(v);
    if constexpr (LANES == 16) return v;
    if constexpr (LANES == 32) return v + __shfl_xor(v, 16);
    v = sum_rows(v);
    if constexpr (LANES > 64) {
        const int first = (threadIdx.x / LANES) * waves_of<LANES>();
        if ((threadIdx.x & 63) == 0) sh[slot][threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < waves_of<LANES>(); ++i) v += sh[slot][first + i];
    }
    return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t row_umax(uint32_t v, float (*sh)[kMaxWaves], int slot) {
    if constexpr (LANES == 4) {
        v = max(v, dpp_u<0xB1>(v));
        return max(v, dpp_u<0x4E>(v));
    }
    v = umax_ln(v);
    if constexpr (LANES == 16) return v;
    v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    if constexpr (LANES == 32) return v;
    v = max(v, (uint32_t)__shfl_xor((int)v, 32));
    if constexpr (LANES > 64) {
        const int first = (threadIdx.x / LANES) * waves_of<LANES>();
        if ((threadIdx.x & 63) == 0) sh[slot][threadIdx.x >> 6] = __uint_as_float(v);
        __syncthreads();
        v = 0;
#pragma unroll
        for (int i = 0; i < waves_of<LANES>(); ++i) v = max(v, __float_as_uint(sh[slot][first + i]));
    }
    return v;
}

// A row's lane holds vectors at columns 8 (v LANES + lane), v < NV. Its first columns may belong to the
// lane before (Lane): they count for nothing in sums and maxima.
template <bool kOdd>
__device__ __forceinline__ float own(float x, int i, int skip) { return kOdd && i < skip ? 0.f : x; }

enum { kPlain = 0, kRowScale = 1, kGroupScale = 2 };

// A row per LANES threads, in workgroups of 256 or one row.
template <int LANES> constexpr int threads_of() { return LANES > kThreads ? LANES : kThreads; }
template <int LANES> constexpr int rows_of() { return threads_of<LANES>() / LANES; }

template <bool kOdd, typename T, typename TW, int LANES, int NV, int OUT>
__global__ __launch_bounds__(threads_of<LANES>()) void k_rms_fwd(RmsArgs p) {
    __shared__ float sh[2][kMaxWaves];
    const int lane = threadIdx.x % LANES;
    const int64_t row = (int64_t)blockIdx.x * rows_of<LANES>() + threadIdx.x / LANES;
    const bool active = rows_of<LANES>() == 1 || row < p.rows;  // (threads without a row take part in the sums)
    const int64_t base = active ? row * p.D : 0;
    Raw<T, 8> r[NV], s[NV];
    Raw<TW, 8> w[NV];
    int skip[NV];
    int64_t at[NV];
    bool live[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t c0 = 8 * ((int64_t)v * LANES + lane);
        const Lane ln(c0, p.D, 8);
        live[v] = active && c0 < p.D;
        at[v] = ln.at;
        skip[v] = ln.skip;
        r[v].clear();
        s[v].clear();
        w[v].clear();
        if (live[v]) {
            r[v] = load_raw<T, 8>(static_cast<const T*>(p.x) + base + at[v]);
            if (p.res) s[v] = load_raw<T, 8>(static_cast<const T*>(p.res) + base + at[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (live[v]) w[v] = load_raw<TW, 8>(static_cast<const TW*>(p.w) + at[v]);
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float a[8];
        if (p.res) {
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = r[v].get(i) + s[v].get(i);
            r[v].set(a);
            if (live[v]) store_own<kOdd, T, 8>(static_cast<T*>(p.res_out) + base + at[v], r[v], skip[v]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = own<kOdd>(r[v].get(i), i, skip[v]);
            ss = fmaf(x, x, ss);
        }
    }
    const float rstd = 1.f / sqrtf(row_sum<LANES>(ss, sh, 0) / (float)p.D + p.eps);
    if constexpr (OUT == kPlain) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = r[v].get(i) * rstd * w[v].get(i);
            if (live[v]) store_own<kOdd, T, 8>(static_cast<T*>(p.y) + base + at[v], y, skip[v]);
        }
    } else {
        float scale[NV];
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            uint32_t m = 0;
            if (live[v])
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, abs_bits(own<kOdd>(r[v].get(i) * rstd * w[v].get(i), i, skip[v])));
            if constexpr (OUT == kGroupScale) {
                scale[v] = scale_of(row_umax<(LANES < 16 ? LANES : 16)>(m, sh, 1));
                if (live[v] && lane % 16 == 0)
                    p.scale[row * ((p.D + 127) / 128) + (v * LANES + lane) / 16] = scale[v];
            } else {
                top = max(top, m);
            }
        }
        if constexpr (OUT == kRowScale) {
            const float sc = scale_of(row_umax<LANES>(top, sh, 1));
#pragma unroll
            for (int v = 0; v < NV; ++v) scale[v] = sc;
            if (active && lane == 0) p.scale[row] = sc;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const Divisor by(scale[v]);
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = r[v].get(i) * rstd * w[v].get(i);
            by.quotients(q);
            if (live[v])
                store_e4m3<kOdd>(static_cast<uint8_t*>(p.y) + base + at[v], pack_e4m3(q[0], q[1], q[2], q[3]),
                                 pack_e4m3(q[4], q[5], q[6], q[7]), skip[v]);
        }
    }
}

// Gradient: the workgroup's rows one after the other (256 / LANES at a time where a row has fewer threads), each lane
// adding its columns' dy rh in registers; at the end the workgroup's waves add theirs in LDS where they hold the same
// columns, and part[blockIdx.x] gets them.
template <bool kOdd, typename T, typename TW, int LANES, int NV>
__global__ __launch_bounds__(threads_of<LANES>()) void k_rms_bwd(RmsArgs p, float* part) {
    constexpr int kRows = rows_of<LANES>();
    static_assert(kRows == 1 || NV == 1, "rows that share a workgroup have one vector a lane");
    __shared__ float sh[4][kMaxWaves];
    __shared__ float shw[kRows > 1 ? kRows : 1][8][LANES];
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    int skip[NV];
    int64_t at[NV];
    bool live[NV];
    Raw<TW, 8> w[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t c0 = 8 * ((int64_t)v * LANES + lane);
        const Lane ln(c0, p.D, 8);
        live[v] = c0 < p.D;
        at[v] = live[v] ? ln.at : 0;
        skip[v] = ln.skip;
        w[v].clear();
        if (live[v]) w[v] = load_raw<TW, 8>(static_cast<const TW*>(p.w) + at[v]);
    }
    float dw[NV][8] = {};
    int slot = 0;
    // the next row is loaded while the present one is worked on, where both fit the registers of two waves a SIMD
    constexpr bool kAhead = NV < 4;
    Raw<T, 8> nr[NV], nd[NV], ns[NV];
    auto fetch = [&](int64_t first) {
        const int64_t row = first + sub, base = row * p.D;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            nr[v].clear();
            nd[v].clear();
            ns[v].clear();
            if (live[v] && (kRows == 1 || row < p.rows)) {
                nr[v] = load_raw<T, 8>(static_cast<const T*>(p.x) + base + at[v]);
                nd[v] = load_raw<T, 8>(static_cast<const T*>(p.d_y) + base + at[v]);
                if (p.d_res) ns[v] = load_raw<T, 8>(static_cast<const T*>(p.d_res) + base + at[v]);
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * kRows, begin = (int64_t)blockIdx.x * kRows;
    if (begin < p.rows) fetch(begin);
    for (int64_t first = begin; first < p.rows; first += step) {
        const int64_t row = first + sub, base = row * p.D;
        const bool active = kRows == 1 || row < p.rows;
        if (!kAhead && first != begin) fetch(first);
        Raw<T, 8> r[NV], d[NV], s[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            r[v] = nr[v];
            d[v] = nd[v];
            s[v] = ns[v];
        }
        if (kAhead && first + step < p.rows) fetch(first + step);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = own<kOdd>(r[v].get(i), i, skip[v]);
                ss = fmaf(x, x, ss);
                // (both factors masked: zero times an infinity would not count for nothing)
                dot = fmaf(own<kOdd>(d[v].get(i) * w[v].get(i), i, skip[v]), x, dot);
            }
        ss = row_sum<LANES>(ss, sh, slot);
        dot = row_sum<LANES>(dot, sh, slot + 1);
        slot ^= 2;
        const float rstd = active ? 1.f / sqrtf(ss / (float)p.D + p.eps) : 0.f;
        const float m = dot * rstd / (float)p.D;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float rh = r[v].get(i) * rstd;
                dw[v][i] = fmaf(d[v].get(i), rh, dw[v][i]);
                o[i] = rstd * (d[v].get(i) * w[v].get(i) - rh * m);
            }
            if (p.d_res)
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += s[v].get(i);
            if (live[v] && active) store_own<kOdd, T, 8>(static_cast<T*>(p.dx) + base + at[v], o, skip[v]);
        }
    }
    if (!p.dw) return;
    if constexpr (kRows > 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) shw[sub][i][lane] = dw[0][i];
        __syncthreads();
        if (sub > 0) return;
        for (int k = 1; k < kRows; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[0][i] += shw[k][i][lane];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (live[v]) store_own<kOdd, float, 8>(part + (int64_t)blockIdx.x * p.D + at[v], dw[v], skip[v]);
}

template <int COLS>
__global__ __launch_bounds__(kSumThreads) void k_rms_dw_sum(const float* part, int parts, int64_t D, float* dw) {
    __shared__ float sh[kSumThreads];
    const int64_t c0 = (int64_t)blockIdx.x * COLS;
    const float s = sum_parts<COLS>(part, parts, D, c0, sh);
    if (threadIdx.x < COLS && c0 + threadIdx.x < D) dw[c0 + threadIdx.x] = s;
}

// ---- rows of any length, element by element: fewer than 8 columns, or more than a workgroup's registers hold (4,000 x
// 32,776 bf16 454 us, x 32,768 190). A workgroup of 1,024 threads each, whatever the length, so 4,194,303 rows at most.
constexpr int kLoopThreads = 1024;
constexpr int kSlots = kLoopThreads / 64;

__device__ __forceinline__ float loop_sum(float v, float (*sh)[kMaxWaves]) {
    const float s = row_sum<kLoopThreads>(v, sh, 0);
    __syncthreads();
    return s;
}

template <typename T, typename TW, bool kQuant>
__global__ __launch_bounds__(kLoopThreads) void k_rms_fwd_loop(RmsArgs p) {
    __shared__ float sh[1][kMaxWaves];
    const int64_t base = (int64_t)blockIdx.x * p.D;
    const T* x = static_cast<const T*>(p.x) + base;
    const T* res = p.res ? static_cast<const T*>(p.res) + base : nullptr;
    const TW* w = static_cast<const TW*>(p.w);
    T* keep = p.res ? static_cast<T*>(p.res_out) + base : nullptr;
    float ss = 0.f;
    for (int64_t c = threadIdx.x; c < p.D; c += kLoopThreads) {
        float v = Elem<T>::to_f(x[c]);
        if (res) {
            const T q = Elem<T>::from_f(v + Elem<T>::to_f(res[c]));
            keep[c] = q;
            v = Elem<T>::to_f(q);
        }
        ss = fmaf(v, v, ss);
    }
    const float rstd = 1.f / sqrtf(loop_sum(ss, sh) / (float)p.D + p.eps);  // (a barrier: keep is complete)
    const T* r = res ? keep : x;
    auto norm = [&](int64_t c) { return Elem<T>::to_f(r[c]) * rstd * Elem<TW>::to_f(w[c]); };
    if constexpr (!kQuant) {
        T* y = static_cast<T*>(p.y) + base;
        for (int64_t c = threadIdx.x; c < p.D; c += kLoopThreads) y[c] = Elem<T>::from_f(norm(c));
    } else {
        uint8_t* y = static_cast<uint8_t*>(p.y) + base;
        const int64_t G = p.group, groups = (p.D + G - 1) / G;
        // a wave per group of 128 columns; a whole row by the workgroup
        const bool by_wave = G == 128;
        const int n = by_wave ? 64 : kLoopThreads, id = by_wave ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
        for (int64_t g = by_wave ? wave_id() : 0; g < groups; g += by_wave ? kSlots : 1) {
            const int64_t c1 = (g + 1) * G < p.D ? (g + 1) * G : p.D;
            uint32_t m = 0;
            for (int64_t c = g * G + id; c < c1; c += n) m = max(m, abs_bits(norm(c)));
            m = by_wave ? row_umax<64>(m, nullptr, 0) : row_umax<kLoopThreads>(m, sh, 0);
            const float scale = scale_of(m);
            const Divisor by(scale);
            for (int64_t c = g * G + id; c < c1; c += n) {
                float q[1] = {norm(c)};
                by.quotients(q);
                y[c] = (uint8_t)pack_e4m3(q[0], q[0], q[0], q[0]);
            }
            if (id == 0) p.scale[(int64_t)blockIdx.x * groups + g] = scale;
        }
    }
}

template <typename T, typename TW>
__global__ __launch_bounds__(kLoopThreads) void k_rms_dx_loop(RmsArgs p, float* rstds) {
    __shared__ float sh[1][kMaxWaves];
    const int64_t base = (int64_t)blockIdx.x * p.D;
    const T* r = static_cast<const T*>(p.x) + base;
    const T* dy = static_cast<const T*>(p.d_y) + base;
    const T* dres = p.d_res ? static_cast<const T*>(p.d_res) + base : nullptr;
    const TW* w = static_cast<const TW*>(p.w);
    T* dx = static_cast<T*>(p.dx) + base;
    float ss = 0.f, dot = 0.f;
    for (int64_t c = threadIdx.x; c < p.D; c += kLoopThreads) {
        const float v = Elem<T>::to_f(r[c]);
        ss = fmaf(v, v, ss);
        dot = fmaf(Elem<T>::to_f(dy[c]) * Elem<TW>::to_f(w[c]), v, dot);
    }
    const float rstd = 1.f / sqrtf(loop_sum(ss, sh) / (float)p.D + p.eps);
    const float m = loop_sum(dot, sh) * rstd / (float)p.D;
    for (int64_t c = threadIdx.x; c < p.D; c += kLoopThreads) {
        const float rh = Elem<T>::to_f(r[c]) * rstd;
        float d = rstd * (Elem<T>::to_f(dy[c]) * Elem<TW>::to_f(w[c]) - rh * m);
        if (dres) d += Elem<T>::to_f(dres[c]);
        dx[c] = Elem<T>::from_f(d);
    }
    if (threadIdx.x == 0) rstds[blockIdx.x] = rstd;
}

constexpr int kLoopSumRows = 64;  // rows per partial sum of dw behind k_rms_dx_loop
template <typename T>
__global__ __launch_bounds__(kThreads) void k_rms_dw_loop(RmsArgs p, const float* rstds, float* part) {
    const int64_t cblocks = (p.D + kThreads - 1) / kThreads, block = blockIdx.x / cblocks;
    const int64_t c = (blockIdx.x % cblocks) * kThreads + threadIdx.x;
    if (c >= p.D) return;
    const int64_t r0 = block * kLoopSumRows, r1 = r0 + kLoopSumRows < p.rows ? r0 + kLoopSumRows : p.rows;
    float s = 0.f;
    for (int64_t i = r0; i < r1; ++i)
        s = fmaf(Elem<T>::to_f(static_cast<const T*>(p.d_y)[i * p.D + c]),
                 Elem<T>::to_f(static_cast<const T*>(p.x)[i * p.D + c]) * rstds[i], s);
    part[block * p.D + c] = s;
}

// ---- launches -----------------------------------------------------------------------------

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Threads and vectors of a row: as many threads as it has vectors, in steps of 4 (32 columns), 16 (128), 32, 64, 128
// and 256, then up to four vectors a thread, of 256 threads to 8,192 columns and of 1,024 to 32,768; 0: by
// elements. (A wave for 2,048 columns, four vectors a lane, was slower: 32,768 rows of them to e4m3 took 85 us
// against 80, and 5,003 fp32 rows of 1,001 columns 19 against 15.5.)
struct Shape {
    int lanes, nv;
};
Shape shape_of(int64_t D) {
    if (D < 8 || D > 32768) return {0, 0};
    if (D <= 1024) return {D <= 32 ? 4 : (D <= 128 ? 16 : (D <= 256 ? 32 : (D <= 512 ? 64 : 128))), 1};
    const int lanes = D <= 8192 ? 256 : 1024;
    const int64_t n = (D + 8 * lanes - 1) / (8 * lanes);
    return {lanes, (int)(n <= 1 ? 1 : (n <= 2 ? 2 : 4))};
}
// The gradient's: its sums of dw double the registers a column takes, so 512 lanes and four vectors are the most. Those
// take all 256 registers, and 4 (fp32, rows that are not whole vectors) to 19 (bf16) of them spill, 80 bytes a lane at
// most: 8,000 x 16,384 bf16 201 us of a floor of 169, 4,000 x 16,384 fp32, which does not spill, 229.
Shape bwd_shape_of(int64_t D) {
    if (D > 16384) return {0, 0};
    return D > 8192 ? Shape{512, 4} : shape_of(D);
}

template <bool kOdd, typename T, typename TW, int OUT>
hipError_t fwd_o(const RmsArgs& a, hipStream_t st) {
    const Shape s = shape_of(a.D);
#define GDN_RMS_FWD(LANES, NV)                                                                              \
    if (s.lanes == LANES && s.nv == NV) {                                                                   \
        const int64_t groups = (a.rows + rows_of<LANES>() - 1) / rows_of<LANES>();                          \
        if (!grid_fits(groups, threads_of<LANES>())) return hipErrorInvalidConfiguration;                   \
        hipLaunchKernelGGL((k_rms_fwd<kOdd, T, TW, LANES, NV, OUT>), dim3((unsigned)groups),                \
                           dim3(threads_of<LANES>()), 0, st, a);                                            \
        return hipGetLastError();                                                                           \
    }
    GDN_RMS_FWD(4, 1)
    GDN_RMS_FWD(16, 1)
    GDN_RMS_FWD(32, 1)
    GDN_RMS_FWD(64, 1)
    GDN_RMS_FWD(128, 1)
    GDN_RMS_FWD(256, 1)
    GDN_RMS_FWD(256, 2)
    GDN_RMS_FWD(256, 4)
    GDN_RMS_FWD(1024, 2)
    GDN_RMS_FWD(1024, 4)
#undef GDN_RMS_FWD
    if (!grid_fits(a.rows, kLoopThreads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_rms_fwd_loop<T, TW, OUT != kPlain>), dim3((unsigned)a.rows), dim3(kLoopThreads), 0, st, a);
    return hipGetLastError();
}
template <typename T, typename TW>
hipError_t fwd_t(const RmsArgs& a, int out, hipStream_t st) {
    if (a.rows == 0) return hipSuccess;
    const bool odd = a.D % 8;
    if (out == 0) return odd ? fwd_o<true, T, TW, kPlain>(a, st) : fwd_o<false, T, TW, kPlain>(a, st);
    if (a.group == 128) return odd ? fwd_o<true, T, TW, kGroupScale>(a, st) : fwd_o<false, T, TW, kGroupScale>(a, st);
    return odd ? fwd_o<true, T, TW, kRowScale>(a, st) : fwd_o<false, T, TW, kRowScale>(a, st);
}

// Workgroups of the gradient, each with its own partial sums of dw: as many as the 256 compute units hold at a time
// (two each, one where a thread has four vectors), or fewer where there are fewer rows. 32,768 rows of 2,048: 256
// 124 us, 512 98, 1,024 106, 2,048 116; 8,000 rows of 8,192: 256 111, 512 117.
int64_t bwd_groups(int64_t rows, const Shape& s) {
    const int64_t per = s.lanes < kThreads ? kThreads / s.lanes : 1, most = s.nv == 4 ? 256 : 512;
    const int64_t n = (rows + per - 1) / per;
    return n < most ? n : most;
}
int64_t loop_parts(int64_t rows) { return (rows + kLoopSumRows - 1) / kLoopSumRows; }

template <bool kOdd, typename T, typename TW>
hipError_t bwd_o(const RmsArgs& a, hipStream_t st) {
    const Shape s = bwd_shape_of(a.D);
    int64_t parts = 0;
    float* part = reinterpret_cast<float*>(a.ws);
    if (a.rows && s.lanes) {
        parts = bwd_groups(a.rows, s);
        bool done = false;
#define GDN_RMS_BWD(LANES, NV)                                                                              \
        if (s.lanes == LANES && s.nv == NV) {                                                               \
            hipLaunchKernelGGL((k_rms_bwd<kOdd, T, TW, LANES, NV>), dim3((unsigned)parts),                  \
                               dim3(threads_of<LANES>()), 0, st, a, part);                                  \
            done = true;                                                                                    \
        }
        GDN_RMS_BWD(4, 1)
        GDN_RMS_BWD(16, 1)
        GDN_RMS_BWD(32, 1)
        GDN_RMS_BWD(64, 1)
        GDN_RMS_BWD(128, 1)
        GDN_RMS_BWD(256, 1)
        GDN_RMS_BWD(256, 2)
        GDN_RMS_BWD(256, 4)
        GDN_RMS_BWD(512, 4)
#undef GDN_RMS_BWD
        if (!done) return hipErrorInvalidValue;
    } else if (a.rows) {
        float* rstds = part;
        part = reinterpret_cast<float*>(a.ws + align256((size_t)a.rows * 4));
        parts = loop_parts(a.rows);
        if (!grid_fits(a.rows, kLoopThreads)) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((k_rms_dx_loop<T, TW>), dim3((unsigned)a.rows), dim3(kLoopThreads), 0, st, a, rstds);
        const unsigned cb = (unsigned)((a.D + kThreads - 1) / kThreads);
        if (a.dw) hipLaunchKernelGGL((k_rms_dw_loop<T>), dim3(cb * (unsigned)parts), dim3(kThreads), 0, st, a, rstds, part);
    }
    if (a.dw) {
        const int cols = sum_cols(a.D);
        const dim3 sums((unsigned)((a.D + cols - 1) / cols));
        if (cols == 64) hipLaunchKernelGGL(k_rms_dw_sum<64>, sums, dim3(kSumThreads), 0, st, part, (int)parts, a.D, a.dw);
        else hipLaunchKernelGGL(k_rms_dw_sum<16>, sums, dim3(kSumThreads), 0, st, part, (int)parts, a.D, a.dw);
    }
    return hipGetLastError();
}
template <typename T, typename TW>
hipError_t bwd_t(const RmsArgs& a, hipStream_t st) {
    return a.D % 8 ? bwd_o<true, T, TW>(a, st) : bwd_o<false, T, TW>(a, st);
}

}  // namespace

size_t rms_bwd_ws(int64_t rows, int64_t D) {
    const Shape s = bwd_shape_of(D);
    if (s.lanes) return (size_t)bwd_groups(rows, s) * D * 4;
    return align256((size_t)rows * 4) + (size_t)loop_parts(rows) * D * 4;
}

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
