// gdn_vec.h -- vectors of consecutive channels held by one lane, in storage form, for the streaming
// kernels of the layer operators. Rows of any length and buffers at any element-aligned address take
// the same code: a vector moves by one load or store at whatever alignment it has (the hardware takes
// any; 16-byte aligned ones are the fast case). Where a row does not end on a vector, its last lane's
// vector is moved back to end with the row (Lane::at), reads its neighbour's channels again and
// stores its own only (Lane::skip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_common.h"

namespace gdn {

template <typename T, int N>
struct Raw {
    static constexpr int kWords = (N * (int)sizeof(T) + 3) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void set(const float (&x)[N]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __float_as_uint(x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = pack_bf2(x[2 * i], 2 * i + 1 < N ? x[(2 * i + 1) % N] : 0.f);
        }
    }
};

// A lane's channels at .. at + N - 1 of a row of D >= N, of which it owns those from at + skip on.
struct Lane {
    int64_t at;
    int skip;
    __device__ __forceinline__ Lane(int64_t c0, int64_t D, int N) : at(c0 + N <= D ? c0 : D - N), skip((int)(c0 - at)) {}
};

template <typename T, int N>
__device__ __forceinline__ Raw<T, N> load_raw(const T* p) {
    Raw<T, N> r;
    if constexpr (N * sizeof(T) < 4) r.w[0] = p[0];
    else __builtin_memcpy(r.w, p, N * sizeof(T));
    return r;
}
// Results are stored non-temporally: they are not read again by the kernel, and the inputs that
// neighbouring waves share stay in the cache (the convolution's gradient of 32,768 x 6,144: 262 -> 249 us).
template <typename T, int N>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, N>& r) {
    if constexpr (N * sizeof(T) < 4) {
        p[0] = (T)r.w[0];
    } else {
        typedef uint32_t words __attribute__((ext_vector_type(Raw<T, N>::kWords), aligned(sizeof(T))));
        words v;
#pragma unroll
        for (int i = 0; i < Raw<T, N>::kWords; ++i) v[i] = r.w[i];
        __builtin_nontemporal_store(v, reinterpret_cast<words*>(p));
    }
}
// kOdd: rows that may not end on a vector (skip may be above zero).
template <bool kOdd, typename T, int N>
__device__ __forceinline__ void store_own(T* p, const Raw<T, N>& r, int skip) {
    if (!kOdd || skip == 0) return store_raw<T, N>(p, r);
#pragma unroll
    for (int i = 1; i < N; ++i)
        if (i >= skip) {
            if constexpr (sizeof(T) == 4) p[i] = __uint_as_float(r.w[i]);
            else p[i] = (T)(r.w[i / 2] >> (16 * (i & 1)));
        }
}
template <bool kOdd, typename T, int N>
__device__ __forceinline__ void store_own(T* p, const float (&x)[N], int skip) {
    Raw<T, N> r;
    r.set(x);
    store_own<kOdd, T, N>(p, r, skip);
}

// For tokens of no sequence, by the waves that meet them (no launch of its own; calls without such tokens take what
// they took within 1%).
template <bool kOdd, typename T, int N>
__device__ __forceinline__ void zero_own(T* p, int skip) {
    Raw<T, N> r;
    r.clear();
    store_own<kOdd, T, N>(p, r, skip);
}

// Sum over `parts` rows of partial sums [parts, n] for COLS columns from c0 on, by a workgroup of
// kSumThreads: COLS lanes side by side on the columns of a row, eight loads in flight per lane, then a tree
// over the rows in LDS (`sh`: kSumThreads words). The order of the additions depends on `parts` and COLS
// alone. Threads 0 .. COLS-1 get the sums of columns c0 + threadIdx.x. Many columns take 64 (whole cache lines),
// few 16, for more workgroups (171 parts of 30,720 columns: 64 6 us, 16 11; 512 of 2,048: 16 4.4 us).
constexpr int kSumThreads = 512;
inline int sum_cols(int64_t n) { return n >= 64 * 256 ? 64 : 16; }
template <int COLS>
__device__ __forceinline__ float sum_parts(const float* part, int parts, int64_t n, int64_t c0, float* sh) {
    constexpr int kRows = kSumThreads / COLS, kAhead = 8;
    const int col = threadIdx.x % COLS, row = threadIdx.x / COLS;
    float s[kAhead] = {};
    if (c0 + col < n) {
        const float* p = part + c0 + col;
        int i = row;
        for (; i + (kAhead - 1) * kRows < parts; i += kAhead * kRows)
#pragma unroll
            for (int u = 0; u < kAhead; ++u) s[u] += p[(int64_t)(i + kRows * u) * n];
        for (; i < parts; i += kRows) s[0] += p[(int64_t)i * n];
    }
    sh[threadIdx.x] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    __syncthreads();
    float t = 0.f;
    if (threadIdx.x < COLS)
#pragma unroll
        for (int r = 0; r < kRows; ++r) t += sh[r * COLS + threadIdx.x];
    return t;
}

}  // namespace gdn
