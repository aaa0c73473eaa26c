// gdn_quant.hip -- quantisation of a matrix to e4m3 with fp32 scales (gdn_e4m3.h): of a row, of 128 columns of a row,
// or of 128 x 128 values; the last two also turned, for products that contract over the rows.
// Bound by memory (2 or 4 bytes read and one written per value), so a value is read once and waits in its own type in the
// registers for its scale: 16 lanes own 128 columns of a row, a workgroup a tile of 128 x 128 or a row. 32,768 x 2,048
// bf16 by groups takes 32.4 us (6.2 TB/s). What a value costs in vector instructions shows all the same (without the
// clamp that quotients by a scale of their own never need, and with maxima of two bf16 bit patterns at a time, turned
// groups of 8,192 x 8,192 went from 49.0 us to 43.9, blocks from 45.2 to 38.2).
#include "gdn_layer.h"
#include "gdn_products.h"
#include "gdn_e4m3.h"
#include "gdn_vec.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

// Columns c .. c + 7 of a row of n, zeros behind it.
template <typename T>
__device__ __forceinline__ Raw<T, 8> load8(const T* p, int64_t c, int64_t n) {
    if (c + 8 <= n) return load_raw<T, 8>(p + c);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < n ? Elem<T>::to_f(p[c + i]) : 0.f;
    Raw<T, 8> r;
    r.set(v);
    return r;
}
__device__ __forceinline__ void store8(uint8_t* p, int64_t c, int64_t n, uint32_t lo, uint32_t hi) {
    if (c + 8 <= n) {
        store_e4m3<false>(p + c, lo, hi, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < n) p[c + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
}
// Absolute values and their maxima as bit patterns, bf16's two to a register.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
template <typename T> constexpr uint32_t kAbs = sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
template <typename T>
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) return max(a, b);
    else return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
template <typename T>
__device__ __forceinline__ uint32_t max_words(const Raw<T, 8>& v) {
    uint32_t m = v.w[0] & kAbs<T>;
#pragma unroll
    for (int i = 1; i < Raw<T, 8>::kWords; ++i) m = max_bits<T>(m, v.w[i] & kAbs<T>);
    return m;
}
// of the one or two values in a word, in fp32
template <typename T>
__device__ __forceinline__ uint32_t max_of(uint32_t m) {
    return sizeof(T) == 4 ? m : max(m << 16, m & 0xFFFF0000u);
}
template <typename T>
__device__ __forceinline__ uint32_t amax8(const Raw<T, 8>& v) { return max_of<T>(max_words<T>(v)); }
__device__ __forceinline__ void pack8(float (&v)[8], const Divisor& by, uint32_t& lo, uint32_t& hi) {
    by.quotients(v);
    lo = pack_e4m3_within(v[0], v[1], v[2], v[3]);
    hi = pack_e4m3_within(v[4], v[5], v[6], v[7]);
}

template <typename T>
__device__ __forceinline__ void pack8(const Raw<T, 8>& r, const Divisor& by, uint32_t& lo, uint32_t& hi) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.get(i);
    pack8(v, by, lo, hi);
}

// 128 columns of a row: 16 lanes, which take kGroups of them, a workgroup's width apart (32,768 x 2,048 bf16, before the above:
// one 35.4 us, two 33.0, four 33.6). WHOLE: rows are whole groups, so the matrix is one run of them (with rows and columns
// worked out 38.9).
constexpr int kGroups = 2;
template <typename T, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_quant_group(QuantArgs p) {
    const int64_t groups = (p.cols + 127) / 128, total = p.rows * groups;
    const int64_t begin = (int64_t)blockIdx.x * (kThreads / 16 * kGroups), first = begin + threadIdx.x / 16;
    const int l = 8 * (threadIdx.x & 15);
    Raw<T, 8> v[kGroups];
    int64_t at[kGroups], left[kGroups];  // of the lane's values, and columns from there to the row's end
    if constexpr (WHOLE) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) at[g] = min(first + g * (kThreads / 16), total - 1) * 128 + l, left[g] = 8;
    } else {
        const int64_t row0 = begin / groups;  // (of the workgroup; what lies behind it is counted in 32 bits)
        const uint32_t rest = (uint32_t)(begin - row0 * groups), per = (uint32_t)groups;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const uint32_t i = rest + (uint32_t)(min(first + g * (kThreads / 16), total - 1) - begin), r = i / per;
            const int64_t c = (int64_t)(i - r * per) * 128 + l;
            at[g] = (row0 + r) * p.cols + c;
            left[g] = p.cols - c;
        }
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) v[g] = load8(static_cast<const T*>(p.x) + at[g], 0, left[g]);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int64_t i = first + g * (kThreads / 16);
        const float scale = scale_of(umax_ln(amax8(v[g])));
        if (i >= total) return;
        const Divisor by(scale);
        uint32_t lo, hi;
        pack8(v[g], by, lo, hi);
        store8(p.q + at[g], 0, left[g], lo, hi);
        if (l == 0) p.scale[i] = scale;
    }
}

template <int THREADS>
__device__ __forceinline__ uint32_t block_umax(uint32_t m, uint32_t* sh) {
    m = umax_ln(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) m = max(m, sh[i]);
    return m;
}

// A row by a workgroup, in its registers up to 8 VECS columns a thread; a longer one (VECS 0) is read again for its values.
template <typename T, int THREADS, int VECS>
__global__ __launch_bounds__(THREADS) void k_quant_row(QuantArgs p) {
    __shared__ uint32_t sh[THREADS / 64];
    constexpr int kHeld = VECS ? VECS : 1;
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.cols;
    uint8_t* q = p.q + row * p.cols;
    Raw<T, 8> v[kHeld];
    uint32_t m = 0, lo, hi;
    if constexpr (VECS) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) v[i] = load8(x, 8 * ((int64_t)threadIdx.x + THREADS * i), p.cols);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) m = max(m, amax8(v[i]));
    } else {
        for (int64_t c = 8 * threadIdx.x; c < p.cols; c += 8 * THREADS) {
            v[0] = load8(x, c, p.cols);
            m = max(m, amax8(v[0]));
        }
    }
    const float scale = scale_of(block_umax<THREADS>(m, sh));
    const Divisor by(scale);
    if constexpr (VECS) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            pack8(v[i], by, lo, hi);
            store8(q, 8 * ((int64_t)threadIdx.x + THREADS * i), p.cols, lo, hi);
        }
    } else {
        for (int64_t c = 8 * threadIdx.x; c < p.cols; c += 8 * THREADS) {
            v[0] = load8(x, c, p.cols);
            pack8(v[0], by, lo, hi);
            store8(q, c, p.cols, lo, hi);
        }
    }
    if (threadIdx.x == 0) p.scale[row] = scale;
}
// The smallest workgroup whose registers hold a row.
template <typename T>
void quant_row(const QuantArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)a.rows);
    if (a.cols <= 2048) hipLaunchKernelGGL((k_quant_row<T, 256, 1>), grid, dim3(256), 0, st, a);
    else if (a.cols <= 4096) hipLaunchKernelGGL((k_quant_row<T, 256, 2>), grid, dim3(256), 0, st, a);
    else if (a.cols <= 8192) hipLaunchKernelGGL((k_quant_row<T, 256, 4>), grid, dim3(256), 0, st, a);
    else if (a.cols <= 32768) hipLaunchKernelGGL((k_quant_row<T, 1024, 4>), grid, dim3(1024), 0, st, a);
    else hipLaunchKernelGGL((k_quant_row<T, 1024, 0>), grid, dim3(1024), 0, st, a);
}

// 128 x 128 values: a thread holds 8 columns of 8 neighbouring rows. Turned: the 8 values of a column are 8 neighbours of
// the result's row and go through LDS as such, at a place that spreads the 16 lanes of a row over the banks; a row of the
// result leaves in pieces of 128 bytes. (Turned tiles have three barriers between loads and stores and a third more
// instructions: 8,192 x 8,192 bf16 43.9 us of 33.)
template <typename T, bool BLOCK, bool TURNED>
__global__ __launch_bounds__(kThreads) void k_quant_tile(QuantArgs p) {
    __shared__ uint32_t sh[4];
    __shared__ __align__(16) uint32_t top[BLOCK ? 1 : 16][128];
    __shared__ __align__(16) float scales[BLOCK ? 4 : 128];
    __shared__ u32x2 turn[TURNED ? 128 : 1][16];
    const uint32_t tiles = (uint32_t)((p.cols + 127) / 128);
    const int64_t br = blockIdx.x / tiles, bc = blockIdx.x % tiles;
    const int l = threadIdx.x & 15, g = threadIdx.x >> 4;
    const int64_t c = bc * 128 + 8 * l, r0 = br * 128 + 8 * g;
    Raw<T, 8> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (r0 + i < p.rows) {
            v[i] = load8(static_cast<const T*>(p.x) + (r0 + i) * p.cols, c, p.cols);
        } else {
            v[i].clear();
        }
    }
    float scale[8];
    if constexpr (BLOCK) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_bits<T>(m, max_words<T>(v[i]));
        const float s = scale_of(block_umax<kThreads>(max_of<T>(m), sh));
#pragma unroll
        for (int j = 0; j < 8; ++j) scale[j] = s;
        if (threadIdx.x == 0) p.scale[TURNED ? bc * ((p.rows + 127) / 128) + br : (int64_t)blockIdx.x] = s;
    } else {
        // the largest of each column over the tile's 128 rows
        Raw<T, 8> most8;
        most8.clear();
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < Raw<T, 8>::kWords; ++k) most8.w[k] = max_bits<T>(most8.w[k], v[i].w[k] & kAbs<T>);
        uint32_t m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = __float_as_uint(most8.get(j));
        *reinterpret_cast<u32x4*>(&top[g][8 * l]) = u32x4{m[0], m[1], m[2], m[3]};
        *reinterpret_cast<u32x4*>(&top[g][8 * l + 4]) = u32x4{m[4], m[5], m[6], m[7]};
        __syncthreads();
        if (threadIdx.x < 128) {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) most = max(most, top[i][threadIdx.x]);
            const float s = scale_of(most);
            scales[threadIdx.x] = s;
            const int64_t col = bc * 128 + threadIdx.x;
            if (col < p.cols) p.scale[col * ((p.rows + 127) / 128) + br] = s;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) scale[j] = scales[8 * l + j];
    }
    if constexpr (!TURNED) {
        const Divisor by(scale[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t lo, hi;
            pack8(v[i], by, lo, hi);
            if (r0 + i < p.rows) store8(p.q + (r0 + i) * p.cols, c, p.cols, lo, hi);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Divisor by(scale[j]);
            float column[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) column[i] = v[i].get(j);
            uint32_t lo, hi;
            pack8(column, by, lo, hi);
            turn[8 * l + j][g ^ l] = u32x2{lo, hi};
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = 16 * i + g;
            const int64_t col = bc * 128 + k;
            const u32x2 w = turn[k][l ^ (k >> 3)];
            if (col < p.cols) store8(p.q + col * p.rows, br * 128 + 8 * l, p.rows, w.x, w.y);
        }
    }
}

template <typename T>
hipError_t quant(const QuantArgs& a, int scales, bool turned, hipStream_t st) {
    const int64_t tiles = ((a.rows + 127) / 128) * ((a.cols + 127) / 128);
    int64_t blocks = tiles;
    if (scales == 0) blocks = a.rows;
    else if (scales == 1 && !turned) blocks = (a.rows * ((a.cols + 127) / 128) + kThreads / 16 * kGroups - 1) / (kThreads / 16 * kGroups);
    if (!grid_fits(blocks, scales == 0 && a.cols > 8192 ? 1024 : kThreads)) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), threads(kThreads);
    if (scales == 0) quant_row<T>(a, st);
    else if (scales == 1 && !turned && a.cols % 128 == 0) hipLaunchKernelGGL((k_quant_group<T, true>), grid, threads, 0, st, a);
    else if (scales == 1 && !turned) hipLaunchKernelGGL((k_quant_group<T, false>), grid, threads, 0, st, a);
    else if (scales == 1) hipLaunchKernelGGL((k_quant_tile<T, false, true>), grid, threads, 0, st, a);
    else if (turned) hipLaunchKernelGGL((k_quant_tile<T, true, true>), grid, threads, 0, st, a);
    else hipLaunchKernelGGL((k_quant_tile<T, true, false>), grid, threads, 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quant(const QuantArgs& a, int dtype, int scales, bool turned, hipStream_t st) {
    if (a.rows == 0) return hipSuccess;
    return dtype == 1 ? quant<float>(a, scales, turned, st) : quant<bf16_t>(a, scales, turned, st);
}

}  // namespace gdn
