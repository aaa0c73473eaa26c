// gdn_quant.hip -- quantisation of a matrix to e4m3 with fp32 scales (gdn_e4m3.h): of a row, of 128 columns of a row,
// or of 128 x 128 values; the last two also turned, for products that contract over the rows.
// Bound by memory (2 or 4 bytes read and one written per value, 3 operations), so a value is read once: 16 lanes own
// 128 columns of a row, a workgroup a tile of 128 x 128 or a row.
#include "gdn_layer.h"
#include "gdn_products.h"
#include "gdn_e4m3.h"
#include "gdn_vec.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

// Columns c .. c + 7 of a row of n, zeros behind it.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t c, int64_t n, float (&v)[8]) {
    if (c + 8 <= n) {
        const Raw<T, 8> r = load_raw<T, 8>(p + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = r.get(i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < n ? Elem<T>::to_f(p[c + i]) : 0.f;
    }
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
__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    return m;
}
__device__ __forceinline__ void pack8(const float (&v)[8], const Divisor& by, uint32_t& lo, uint32_t& hi) {
    lo = pack_e4m3(by.quotient(v[0]), by.quotient(v[1]), by.quotient(v[2]), by.quotient(v[3]));
    hi = pack_e4m3(by.quotient(v[4]), by.quotient(v[5]), by.quotient(v[6]), by.quotient(v[7]));
}

// 128 columns of a row: 16 lanes.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_quant_group(QuantArgs p) {
    const int64_t groups = (p.cols + 127) / 128, i = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 16;
    const bool live = i < p.rows * groups;
    const int64_t row = live ? i / groups : 0, c = (live ? i % groups : 0) * 128 + 8 * (threadIdx.x & 15);
    float v[8];
    load8(static_cast<const T*>(p.x) + row * p.cols, c, p.cols, v);
    const float scale = scale_of(umax_ln(amax8(v)));
    if (!live) return;
    const Divisor by(scale);
    uint32_t lo, hi;
    pack8(v, by, lo, hi);
    store8(p.q + row * p.cols, c, p.cols, lo, hi);
    if ((threadIdx.x & 15) == 0) p.scale[i] = scale;
}

__device__ __forceinline__ uint32_t block_umax(uint32_t m, uint32_t* sh) {
    m = umax_ln(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = m;
    __syncthreads();
    return max(max(sh[0], sh[1]), max(sh[2], sh[3]));
}

// A row by a workgroup; read again for its values.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_quant_row(QuantArgs p) {
    __shared__ uint32_t sh[4];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.cols;
    float v[8];
    uint32_t m = 0;
    for (int64_t c = 8 * threadIdx.x; c < p.cols; c += 8 * kThreads) {
        load8(x, c, p.cols, v);
        m = max(m, amax8(v));
    }
    const float scale = scale_of(block_umax(m, sh));
    const Divisor by(scale);
    for (int64_t c = 8 * threadIdx.x; c < p.cols; c += 8 * kThreads) {
        load8(x, c, p.cols, v);
        uint32_t lo, hi;
        pack8(v, by, lo, hi);
        store8(p.q + row * p.cols, c, p.cols, lo, hi);
    }
    if (threadIdx.x == 0) p.scale[row] = scale;
}

// 128 x 128 values: a thread holds 8 columns of 8 rows, 16 rows apart. Turned: the 8-bit values go through LDS, a row of
// the result (128 values of a column) in words of four.
template <typename T, bool BLOCK, bool TURNED>
__global__ __launch_bounds__(kThreads) void k_quant_tile(QuantArgs p) {
    __shared__ uint32_t sh[4];
    __shared__ uint32_t top[16][129];
    __shared__ __align__(16) uint8_t turn[TURNED ? 128 * 144 : 16];
    const int64_t tiles = (p.cols + 127) / 128, br = blockIdx.x / tiles, bc = blockIdx.x % tiles;
    const int64_t c = bc * 128 + 8 * (threadIdx.x & 15);
    const int r0 = threadIdx.x / 16;
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = br * 128 + r0 + 16 * i;
        if (r < p.rows) {
            load8(static_cast<const T*>(p.x) + r * p.cols, c, p.cols, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        }
    }
    float scale[8];
    if constexpr (BLOCK) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, amax8(v[i]));
        const float s = scale_of(block_umax(m, sh));
#pragma unroll
        for (int j = 0; j < 8; ++j) scale[j] = s;
        if (threadIdx.x == 0) p.scale[TURNED ? bc * ((p.rows + 127) / 128) + br : (int64_t)blockIdx.x] = s;
    } else {
        // the largest of each column over the tile's 128 rows
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i][j]));
            top[r0][8 * (threadIdx.x & 15) + j] = m;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) m = max(m, top[i][8 * (threadIdx.x & 15) + j]);
            scale[j] = scale_of(m);
        }
        if (r0 == 0)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < p.cols) p.scale[(c + j) * ((p.rows + 127) / 128) + br] = scale[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const Divisor by(scale[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i][j] = by.quotient(v[i][j]);
    }
    if constexpr (!TURNED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = br * 128 + r0 + 16 * i;
            if (r < p.rows)
                store8(p.q + r * p.cols, c, p.cols, pack_e4m3(v[i][0], v[i][1], v[i][2], v[i][3]), pack_e4m3(v[i][4], v[i][5], v[i][6], v[i][7]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t lo = pack_e4m3(v[0][j], v[1][j], v[2][j], v[3][j]), hi = pack_e4m3(v[4][j], v[5][j], v[6][j], v[7][j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) turn[(8 * (threadIdx.x & 15) + j) * 144 + r0 + 16 * i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 128 * 16; i += kThreads) {
            const int64_t col = bc * 128 + i / 16, r = br * 128 + 8 * (i % 16);
            if (col >= p.cols) break;
            const u32x2 w = *reinterpret_cast<const u32x2*>(turn + (i / 16) * 144 + 8 * (i % 16));
            store8(p.q + col * p.rows, r, p.rows, w.x, w.y);
        }
    }
}

template <typename T>
hipError_t quant(const QuantArgs& a, int scales, bool turned, hipStream_t st) {
    const int64_t tiles = ((a.rows + 127) / 128) * ((a.cols + 127) / 128);
    int64_t blocks = tiles;
    if (scales == 0) blocks = a.rows;
    else if (scales == 1 && !turned) blocks = (a.rows * ((a.cols + 127) / 128) + kThreads / 16 - 1) / (kThreads / 16);
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), threads(kThreads);
    if (scales == 0) hipLaunchKernelGGL(k_quant_row<T>, grid, threads, 0, st, a);
    else if (scales == 1 && !turned) hipLaunchKernelGGL(k_quant_group<T>, grid, threads, 0, st, a);
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
