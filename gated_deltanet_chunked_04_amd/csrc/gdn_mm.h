// gdn_mm.h -- matrix products on the matrix cores, shared by the e4m3 product (gdn_mm8.hip) and the gated
// feed-forward block (gdn_ffn.hip): operands, tiles in LDS, fragments, the loop over the contraction.
//
// Everything is  Y[m, n] = sum_k X[m, k] W[n, k]  with X on the lanes and W on the registers of a 16x16 accumulator
// tile (gdn_common.h: lane l holds rows 4 gq .. 4 gq + 3 of column ln; W's rows are the tile's rows and X's its
// columns), so a lane holds outputs of one m and, by the choice of which W rows make up a tile, runs of neighbouring n.
//
// A step of the contraction is 128 bytes of a row (64 bf16, 32 fp32, 128 e4m3 values: one scale of the e4m3 product),
// eight 16-byte chunks. Lane group gq takes chunks gq and gq + 4 of its row: which values of the contraction a matrix
// instruction sees in which slot does not matter as long as both operands agree.
//
// An operand lies in memory either by its rows (the contraction is contiguous) or turned (the contraction walks over
// memory rows: the gradients' products). Tiles keep that order in LDS; a turned bf16 tile is read by transposing reads.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_common.h"
#include "gdn_e4m3.h"
#include "gdn_vec.h"

namespace gdn {

// kMmF8 multiplies e4m3 by the 8-bit matrix instruction, kMmF8x widens e4m3 to bf16 (exact) first. The 8-bit
// instruction adds products in groups of eight that it aligns to the largest of them and cuts about 13 bits below it
// (measured: a product of 1 beside one of 448^2 in its group is lost; on quantised normal data its sums of 128 are off
// by 1.5e-5 in the 2-norm, the widened ones by 1e-8). That is a hundredth of a bf16 output's own rounding, so kMmF8 is
// for outputs in bf16, and kMmF8x for what is kept in 32 bits (fp32 outputs and the scales of an e4m3 output) and for bf16
// outputs of callers whose large products cancel, who ask for it (32,768 x 6,144 x 2,048 by blocks 430 us and 782).
enum MmKind { kMmBf16 = 0, kMmF32 = 1, kMmF8 = 2, kMmF8x = 3 };
template <int KIND> constexpr int mm_size() { return KIND == kMmBf16 ? 2 : (KIND == kMmF32 ? 4 : 1); }
constexpr int kMmStep = 128;  // bytes of a row per step

typedef int i32x8 __attribute__((ext_vector_type(8)));

// What a lane feeds for a step: its two chunks, in the form that the matrix instruction takes.
template <int KIND> struct MmFrag;
template <> struct MmFrag<kMmBf16> {
    bf16x8_t v[2];
    __device__ __forceinline__ void set(u32x4 a, u32x4 b) { v[0] = __builtin_bit_cast(bf16x8_t, a), v[1] = __builtin_bit_cast(bf16x8_t, b); }
};
template <> struct MmFrag<kMmF32> {
    f32x4 v[2];
    __device__ __forceinline__ void set(u32x4 a, u32x4 b) { v[0] = __builtin_bit_cast(f32x4, a), v[1] = __builtin_bit_cast(f32x4, b); }
};
template <> struct MmFrag<kMmF8> {
    i32x8 v;
    __device__ __forceinline__ void set(u32x4 a, u32x4 b) { v = i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w}; }
};
template <> struct MmFrag<kMmF8x> {
    bf16x8_t v[4];
    __device__ __forceinline__ void widen(int at, uint32_t lo, uint32_t hi) {
        const bf16x2_t p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false), q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
        const bf16x2_t r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false), s = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
        v[at] = bf16x8_t{p.x, p.y, q.x, q.y, r.x, r.y, s.x, s.y};
    }
    __device__ __forceinline__ void set(u32x4 a, u32x4 b) { widen(0, a.x, a.y), widen(1, a.z, a.w), widen(2, b.x, b.y), widen(3, b.z, b.w); }
};
// A step is mm_parts matrix instructions that add to one another.
template <int KIND> constexpr int mm_parts() { return KIND == kMmBf16 ? 2 : (KIND == kMmF32 ? 8 : (KIND == kMmF8 ? 1 : 4)); }
__device__ __forceinline__ f32x4 mm_part(int i, const MmFrag<kMmBf16>& w, const MmFrag<kMmBf16>& x, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mm_part(int i, const MmFrag<kMmF32>& w, const MmFrag<kMmF32>& x, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(w.v[i / 4][i % 4], x.v[i / 4][i % 4], c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mm_part(int, const MmFrag<kMmF8>& w, const MmFrag<kMmF8>& x, f32x4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mm_part(int i, const MmFrag<kMmF8x>& w, const MmFrag<kMmF8x>& x, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], c, 0, 0, 0);
}
template <int KIND>
__device__ __forceinline__ f32x4 mm_mma(const MmFrag<KIND>& w, const MmFrag<KIND>& x, f32x4 c) {
#pragma unroll
    for (int i = 0; i < mm_parts<KIND>(); ++i) c = mm_part(i, w, x, c);
    return c;
}

// ---- tiles in LDS ---------------------------------------------------------------------------
// By rows: [R][128 bytes], chunk c of row r at c ^ key(r), so that 8 lanes that read one chunk of 8 rows meet
// different banks. kFar: the tile's rows r come in fours that lie 2^kFar apart (the column order of W's tiles).
// Turned: [steps][R elements].
constexpr int kNear = 0;  // rows side by side
template <int kFar> __device__ __forceinline__ int mm_key(int r) {
    return kFar == kNear ? r & 7 : (r & 3) | ((((r >> 2) ^ (r >> kFar)) & 1) << 2);
}
template <int kFar> __device__ __forceinline__ int mm_at(int r, int c) { return r * kMmStep + ((c ^ mm_key<kFar>(r)) << 4); }

// Turned: chunk c of 16 bytes of memory row k; XOR over units of 32 bytes spreads the 16 rows that a transposing read
// meets (0-3, 8-11, 16-19, 24-27 of a half step) over the banks.
template <int R, int E> __device__ __forceinline__ int mm_turn_key(int k) {
    constexpr int kUnits = R * E / 32;
    return (((k & 3) | ((k >> 3) & 3) << 2) & (kUnits - 1)) << 1;
}
template <int R, int E> __device__ __forceinline__ int mm_turn_at(int k, int c) { return k * R * E + ((c ^ mm_turn_key<R, E>(k)) << 4); }

// The lane's two chunks of row r.
template <int kFar>
__device__ __forceinline__ void mm_read(u32x4 (&raw)[2], const uint8_t* tile, int r) {
    const int gq = threadIdx.x >> 4 & 3;
    raw[0] = *reinterpret_cast<const u32x4*>(tile + mm_at<kFar>(r, gq));
    raw[1] = *reinterpret_cast<const u32x4*>(tile + mm_at<kFar>(r, gq + 4));
}
template <int KIND, int kFar>
__device__ __forceinline__ void mm_read(MmFrag<KIND>& f, const uint8_t* tile, int r) {
    u32x4 raw[2];
    mm_read<kFar>(raw, tile, r);
    f.set(raw[0], raw[1]);
}
// The same for rows a whole number of 16 further on than the lane's row, whose two chunks lie at a and b: `by` bytes on.
__device__ __forceinline__ void mm_read_at(u32x4 (&raw)[2], uint32_t a, uint32_t b, int by) {
    typedef const __attribute__((address_space(3))) u32x4 lds_u32x4;
    raw[0] = *(lds_u32x4*)(uintptr_t)(a + by);
    raw[1] = *(lds_u32x4*)(uintptr_t)(b + by);
}
// A value that the compiler takes as new: offsets from it stay immediate offsets.
__device__ __forceinline__ uint32_t mm_fresh(uint32_t x) {
    asm volatile("" : "+v"(x));
    return x;
}
// The same from a turned tile of R rows, for 16 of them: r0 + far * g + i, lane ln = 4 g + i.
template <int KIND, int R>
__device__ __forceinline__ void mm_read_turned(MmFrag<KIND>& f, const uint8_t* tile, int r0, int far) {
    const int ln = threadIdx.x & 15, gq = threadIdx.x >> 4 & 3;
    if constexpr (KIND == kMmBf16) {
        const int col = r0 + far * (ln & 3);  // four neighbouring columns of memory row k
        u32x2 h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int k = (q >> 1) * 32 + gq * 8 + (q & 1) * 4 + (ln >> 2);
            h[q] = ds_read_tr16(reinterpret_cast<const bf16_t*>(tile + mm_turn_at<R, 2>(k, col >> 3) + (col & 7) * 2));
        }
        f.set(u32x4{h[0].x, h[0].y, h[1].x, h[1].y}, u32x4{h[2].x, h[2].y, h[3].x, h[3].y});
    } else {
        const int col = r0 + far * (ln >> 2) + (ln & 3);
        u32x4 h[2];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int k = (q >> 2) * 16 + gq * 4 + (q & 3);
            h[q >> 2][q & 3] = *reinterpret_cast<const uint32_t*>(tile + mm_turn_at<R, 4>(k, col >> 2) + (col & 3) * 4);
        }
        f.set(h[0], h[1]);
    }
}

// ---- memory to LDS --------------------------------------------------------------------------
// 16 bytes at p + off of a memory row of `limit` bytes, zeros behind it; at any address.
__device__ __forceinline__ u32x4 mm_chunk(const uint8_t* p, int64_t off, int64_t limit) {
    u32x4 v = {0, 0, 0, 0};
    if (off + 16 <= limit) {
        __builtin_memcpy(&v, p + off, 16);
    } else if (off < limit) {
        unsigned __int128 x = 0;
        if (limit >= 16) {  // the row's last 16 bytes, of which those in front of `off` go
            __builtin_memcpy(&x, p + limit - 16, 16);
            x >>= 8 * (int)(off + 16 - limit);
        } else {
#pragma unroll 1
            for (int i = (int)(limit - off) - 1; i >= 0; --i) x = x << 8 | p[off + i];
        }
        v = __builtin_bit_cast(u32x4, x);
    }
    return v;
}

// An operand's tile of R rows from row r0 on, in chunks: which memory row and byte a chunk has, and where it goes.
// Rows behind the operand's last one repeat it (they reach outputs that are not stored); steps behind the contraction
// are zeros.
// PAIRS: X's values are pairs, what rounding left of a value `low` bytes behind it in its memory row. The tile's rows are then
// 16 rows' values, the same rows' other halves, the next 16 rows' values, and so on: R / 2 rows, whose two halves meet one tile of W.
__device__ __forceinline__ int mm_pair_row(int r) { return (r >> 5) * 16 + (r & 15); }
__device__ __forceinline__ bool mm_pair_low(int r) { return r & 16; }
template <int E, int R, bool kTurned, int kFar, bool PAIRS = false>
struct MmTile {
    static constexpr int kChunks = R * 8;
    static constexpr int kWide = R * E / 16;  // chunks of a turned memory row
    static __device__ __forceinline__ int lds(int i) {
        return kTurned ? mm_turn_at<R, E>(i / kWide, i % kWide) : mm_at<kFar>(i >> 3, i & 7);
    }
    static __device__ __forceinline__ u32x4 load(const uint8_t* p, int64_t ld, int64_t r0, int64_t rows, int64_t k0, int64_t K, int i, int64_t low = 0) {
        const int at = kTurned ? i % kWide * (16 / E) : i >> 3;  // the tile's row
        if (PAIRS && mm_pair_low(at)) p += low;
        if constexpr (kTurned) {
            const int64_t k = k0 + i / kWide;
            return k < K ? mm_chunk(p + k * ld, (r0 + (PAIRS ? mm_pair_row(at) : at)) * E, rows * E) : u32x4{0, 0, 0, 0};
        } else {
            const int64_t r = r0 + (PAIRS ? mm_pair_row(at) : at);
            return mm_chunk(p + (r < rows ? r : rows - 1) * ld, k0 * E + 16 * (i & 7), K * E);
        }
    }
};

// ---- products -------------------------------------------------------------------------------
enum MmScales { kMmPlain = 0, kMmBlock = 1, kMmGroup = 2, kMmRow = 3 };

struct MmArgs {
    const uint8_t* x[2];  // per segment of the contraction (dx: d_gate, d_up), or per output (dw)
    const uint8_t* w[2];  // per segment, or gate and up side by side (the block's forward)
    int64_t low;          // 0, or the bytes from a value to what its rounding left (of d_gate and d_up), in the same memory row
    int64_t ldx, ldw;     // bytes between two memory rows
    int64_t M, N, K;      // rows of X, of W (of each where there are two side by side), contraction of a segment
    int32_t segs;         // segments of the contraction, 1 or 2
    int32_t outs;         // outputs, each with its x (dw)
    const float* xs;      // scales of e4m3 operands: [M, kb] (row: [M])
    const float* ws[2];   // block: [ceil(N/128), kb], group: [N, kb], row: [N]
    int64_t kb;           // scales of a row: ceil(K / 128)
    void* out[2];         // outputs [M, N] with ldo elements a row
    int64_t ldo;
    const void* d_h;      // [M, N]: the gradient that enters the block's backward
    float* pre;           // [2, M, N] gate and up in fp32, or null
    int32_t act;          // 1 silu, 2 gelu_tanh
    float* scale;         // of an e4m3 output [M, ceil(N/128)]
    float* part;          // where the contraction is split: sums of each part, [outs, splits, sides, M, N]
    int32_t splits;       // parts of the contraction (0: one, without part)
    int32_t share;        // steps of a part
};

// sigmoid and the slope of its argument: silu(a) = a sigmoid(a), gelu_tanh(a) = a sigmoid(2 c (a + 0.044715 a^3)).
struct Act {
    float f, df;  // activation and derivative
    __device__ __forceinline__ Act(float a, int act, bool grad) {
        constexpr float c = 1.5957691216057308f;  // 2 sqrt(2 / pi)
        const float a2 = a * a, p = act == 1 ? a : c * a * fmaf(0.044715f, a2, 1.f);
        const float s = __builtin_amdgcn_rcpf(1.f + fast_exp(-p));
        f = a * s;
        if (grad) {
            const float dp = act == 1 ? 1.f : c * fmaf(3.f * 0.044715f, a2, 1.f), t = s * (1.f - s);
            df = t == 0.f ? s : fmaf(a * t, dp, s);  // (where s is 0 or 1 the slope may have overflowed)
        } else {
            df = 0.f;
        }
    }
};

// N consecutive outputs at p, of which those in front of `n` exist.
template <typename T, int N>
__device__ __forceinline__ void mm_store(T* p, const float (&v)[N], int64_t n) {
    if (n >= N) {
        Raw<T, N> r;
        r.set(v);
        store_raw<T, N>(p, r);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = Elem<T>::from_f(v[i]);
    }
}
// 32 neighbouring fp32 columns of a row, of which lane group gq holds 8 gq .. 8 gq + 7: the groups trade halves, so that
// each of two stores writes 64 bytes in a row. p: the first of the 32. The four lanes of a row call it together.
__device__ __forceinline__ void mm_store32(float* p, const float (&v)[8]) {
    const int gq = threadIdx.x >> 4 & 3;
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[4 + i]), false, false);
        const auto y = __builtin_amdgcn_permlane32_swap(x[0], x[1], false, false);
        a[i] = __uint_as_float(y[0]);  // columns 4 gq + i
        b[i] = __uint_as_float(y[1]);  // columns 16 + 4 gq + i
    }
    mm_store<float, 4>(p + 4 * gq, a, 4);
    mm_store<float, 4>(p + 16 + 4 * gq, b, 4);
}
template <typename T, int N>
__device__ __forceinline__ void mm_load(const T* p, float (&v)[N], int64_t n) {
    if (n >= N) {
        const Raw<T, N> r = load_raw<T, N>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = r.get(i);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < n ? Elem<T>::to_f(p[i]) : 0.f;
    }
}

// What is done with a lane's sums. kMmOut: y = sums (with kMmRow, times the rows' scales). kMmFfn: h = act(gate) up, and
// gate and up themselves where `pre` is given. kMmFfnBwd: the gradients of gate and up from d_h. kMmPart: the sums of a
// part of the contraction, for k_mm_join. kMmFfn8: h in e4m3 with a scale for 128 columns (a tile's).
enum MmEpi { kMmOut = 0, kMmFfn = 1, kMmFfnBwd = 2, kMmPart = 3, kMmFfn8 = 4 };

// What rounding to T leaves of a value (nothing of those that are not finite, or become so).
template <typename T>
__device__ __forceinline__ float mm_left(float v) {
    const float d = v - Elem<T>::to_f(Elem<T>::from_f(v));
    return fabsf(d) < INFINITY ? d : 0.f;
}

// R columns of the block at (m, n). SHARED: by a wave whose four lane groups hold 32 neighbouring columns of a row.
template <int EPI, typename T, int R, bool SHARED>
__device__ __forceinline__ void mm_gate(const MmArgs& p, int64_t m, int64_t n, const float (&a)[R], const float (&u)[R]) {
    const int64_t left = p.N - n;
    if constexpr (EPI == kMmFfn) {
        float h[R];
#pragma unroll
        for (int i = 0; i < R; ++i) h[i] = Act(a[i], p.act, false).f * u[i];
        mm_store<T, R>(static_cast<T*>(p.out[0]) + m * p.ldo + n, h, left);
        if (p.pre) {
            if constexpr (R == 8) {
                const int64_t first = n - (8 * (threadIdx.x >> 4 & 3));
                if (SHARED && first + 32 <= p.N) {
                    mm_store32(p.pre + m * p.N + first, a);
                    mm_store32(p.pre + (p.M + m) * p.N + first, u);
                    return;
                }
            }
            mm_store<float, R>(p.pre + m * p.N + n, a, left);
            mm_store<float, R>(p.pre + (p.M + m) * p.N + n, u, left);
        }
    } else {
        float d[R], da[R], du[R];
        mm_load<T, R>(static_cast<const T*>(p.d_h) + m * p.N + n, d, left);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const Act f(a[i], p.act, true);
            da[i] = i < left ? d[i] * u[i] * f.df : 0.f;
            du[i] = i < left ? d[i] * f.f : 0.f;
        }
        // rounded to the inputs' type: they are operands of the products behind, which take whole vectors of their rows
        // and multiply what lies behind column N by zero
        T* const g = static_cast<T*>(p.out[0]) + m * p.ldo + n;
        T* const v = static_cast<T*>(p.out[1]) + m * p.ldo + n;
        mm_store<T, R>(g, da, R);
        mm_store<T, R>(v, du, R);
        if (p.low) {
#pragma unroll
            for (int i = 0; i < R; ++i) da[i] = mm_left<T>(da[i]), du[i] = mm_left<T>(du[i]);
            mm_store<T, R>(g + p.low / (int64_t)sizeof(T), da, R);
            mm_store<T, R>(v + p.low / (int64_t)sizeof(T), du, R);
        }
    }
}
// Columns that an epilogue writes: those of the gradients of gate and up to the end of their last vector.
template <int EPI> __host__ __device__ __forceinline__ int64_t mm_width(const MmArgs& p) { return EPI == kMmFfnBwd ? (p.N + 7) / 8 * 8 : p.N; }

// R columns of sums at (m, n): one side, or gate and up.
template <int EPI, typename T, int SC, bool DUAL, int R>
__device__ __forceinline__ void mm_finish(const MmArgs& p, void* out, int part, int64_t m, int64_t n, float (&v)[DUAL ? 2 : 1][R]) {
    if constexpr (EPI == kMmPart) {
#pragma unroll
        for (int i = 0; i < (DUAL ? 2 : 1); ++i)
            mm_store<float, R>(p.part + (((int64_t)part * (DUAL ? 2 : 1) + i) * p.M + m) * p.N + n, v[i], p.N - n);
    } else if constexpr (DUAL) {
        mm_gate<EPI, T, R, R == 8>(p, m, n, v[0], v[1]);
    } else {
        if (SC == kMmRow) {
            const float sx = p.xs[m];
#pragma unroll
            for (int i = 0; i < R; ++i) v[0][i] *= sx * p.ws[0][n + i < p.N ? n + i : p.N - 1];
        }
        mm_store<T, R>(static_cast<T*>(out) + m * p.ldo + n, v[0], p.N - n);
    }
}

// Adds the parts in their order; 4 columns a thread.
template <int SC, bool DUAL, int EPI, typename T>
__global__ __launch_bounds__(256) void k_mm_join(MmArgs p) {
    constexpr int kSides = DUAL ? 2 : 1;
    const int64_t per = (mm_width<EPI>(p) + 3) / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= per * p.M) return;
    const int64_t m = i / per, n = i % per * 4;
    const int z = blockIdx.y;
    float v[kSides][4] = {};
    if (n < p.N) {
        const float* from = p.part + ((int64_t)z * p.splits * kSides * p.M + m) * p.N + n;
        const int64_t side = p.M * p.N, left = p.N - n;
        constexpr int kAhead = 4;  // parts on their way together
        for (int s = 0; s < p.splits; s += kAhead) {
            float x[kAhead][kSides][4];
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
#pragma unroll
                for (int k = 0; k < kSides; ++k) mm_load<float, 4>(from + ((int64_t)min(s + a, p.splits - 1) * kSides + k) * side, x[a][k], left);
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
                if (s + a < p.splits)
#pragma unroll
                    for (int k = 0; k < kSides; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[k][j] += x[a][k][j];
        }
    }
    mm_finish<EPI, T, SC, DUAL, 4>(p, z ? p.out[1] : p.out[0], 0, m, n, v);
}

// Which of W's rows make up a wave's tile j of the register side: rows 4 g + i of the tile are rows
// mm_row(j) + far g + i of W. kPair: a lane's columns in tiles 2 q and 2 q + 1 are 8 neighbours (one 16-byte store of
// bf16, 64 bytes in a row by the four lane groups; gate and up: tiles 0, 1 and 2, 3); else 4 neighbours a tile (16
// bytes of fp32; turned tiles, whose transposing reads want neighbouring columns).
template <bool PAIR, bool DUAL> struct MmCols {
    static constexpr int kFar = PAIR ? 3 : kNear;  // for mm_key
    static constexpr int kStride = PAIR ? 8 : 4;
    static __device__ __forceinline__ constexpr int row(int j) { return PAIR ? (DUAL ? 0 : 32 * (j / 2)) + 4 * (j % 2) : 16 * j; }
    // the lane's first column of tile j
    static __device__ __forceinline__ int col(int j, int gq) { return row(j) + kStride * gq; }
};
// Which of the two X and W a segment of the contraction takes. Turned X (dw): the output's.
template <bool XT> __device__ __forceinline__ const uint8_t* mm_x(const MmArgs& p, int seg, int z) { return (XT ? z : seg) ? p.x[1] : p.x[0]; }
template <bool XT> __device__ __forceinline__ const uint8_t* mm_w(const MmArgs& p, int seg) { return !XT && seg ? p.w[1] : p.w[0]; }
template <typename T, bool WT, bool DUAL> constexpr bool mm_pair() { return DUAL || (sizeof(T) == 2 && !WT); }

// The sums of a wave's MT x NT tiles, scaled where the operands are e4m3. Shared by the kernels below.
template <int KIND, int SC, bool DUAL, int MT, int NT>
struct MmSums {
    static constexpr bool kScaled = SC == kMmBlock || SC == kMmGroup;
    f32x4 acc[MT][NT] = {};
    // A step's sums of X tile t and W tile j; sx: the scale of the lane's X row, sw of W's rows: one for all (block), or one
    // for each of the lane's columns (group).
    __device__ __forceinline__ void add(int t, int j, f32x4 c, float sx, const float (&sw)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(c[i], SC == kMmBlock ? sx * sw[0] : sx * sw[i], acc[t][j][i]);
    }
    // Hands the lane's outputs on: X's row m0 + 16 t + ln, the columns that MmCols names. PAIRS: tiles 2 t and 2 t + 1 are the
    // same rows'.
    template <int EPI, typename T, bool PAIR, bool PAIRS = false>
    __device__ __forceinline__ void finish(const MmArgs& p, void* out, int part, int64_t m0, int64_t n0) const {
        using C = MmCols<PAIR, DUAL>;
        constexpr int kRun = PAIR ? 8 : 4;
        const int ln = threadIdx.x & 15, gq = threadIdx.x >> 4 & 3;
        constexpr int kOf = PAIRS ? 2 : 1;
#pragma unroll
        for (int t = 0; t < MT / kOf; ++t) {
            const int64_t m = m0 + 16 * t + ln;
            if (m >= p.M) continue;
#pragma unroll
            for (int q = 0; q < NT; q += DUAL ? 4 : kRun / 4) {
                const int64_t n = n0 + C::col(q, gq);
                if (n >= mm_width<EPI>(p)) continue;
                float v[DUAL ? 2 : 1][kRun];
#pragma unroll
                for (int j = 0; j < (DUAL ? 4 : kRun / 4); ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& to = v[DUAL ? j / 2 : 0][(j % (kRun / 4)) * 4 + i];
                        to = acc[kOf * t][q + j][i];
                        if (PAIRS) to += acc[kOf * t + kOf - 1][q + j][i];
                    }
                mm_finish<EPI, T, SC, DUAL, kRun>(p, out, part, m, n, v);
            }
        }
    }
};

// h in e4m3: 128 columns of a row, which share a scale, are those of the four waves side by side. top: [rows of the tile][4]
// in LDS, row0 this wave's first row of it; all waves call it when they are done with the tiles.
template <class Sums, int MT>
__device__ __forceinline__ void mm_finish8(Sums& sums, const MmArgs& p, uint32_t* top, int row0, int wn, int64_t m0, int64_t n0) {
    const int ln = threadIdx.x & 15, gq = threadIdx.x >> 4 & 3;
    const int64_t n = n0 + 32 * wn + 8 * gq, left = p.N - n;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float h = Act(sums.acc[t][j][i], p.act, false).f * sums.acc[t][2 + j][i];
                sums.acc[t][j][i] = h;
                if (4 * j + i < left) m = max(m, abs_bits(h));
            }
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if (gq == 0) top[(row0 + 16 * t + ln) * 4 + wn] = m;
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t m = m0 + 16 * t + ln;
        if (m >= p.M || left <= 0) continue;
        const u32x4 a = *reinterpret_cast<const u32x4*>(top + (row0 + 16 * t + ln) * 4);
        const float scale = scale_of(max(max(a.x, a.y), max(a.z, a.w)));
        const Divisor by(scale);
        uint32_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float h[4] = {sums.acc[t][j][0], sums.acc[t][j][1], sums.acc[t][j][2], sums.acc[t][j][3]};
            by.quotients(h);
            w[j] = pack_e4m3_within(h[0], h[1], h[2], h[3]);
        }
        uint8_t* q = static_cast<uint8_t*>(p.out[0]) + m * p.N + n;
        if (left >= 8) {
            store_e4m3<false>(q, w[0], w[1], 0);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) q[i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
        }
        if (wn == 0 && gq == 0) p.scale[m * ((p.N + 127) / 128) + n0 / 128] = scale;
    }
}

// 128 x 64 WN outputs (two sides: half of each) by WM x WN waves of 128 / WM x 64, any sizes and addresses: chunks go
// through registers, the next step's on their way while one is multiplied; one tile of each operand in LDS. Eight waves,
// two on a SIMD, so that one's LDS reads pass behind the other's products (1,003 x 777 x 1,001 in e4m3, when the two were compared,
// 19.4 us, with four waves of 64 x 64 20.0; 16.3 now).
template <int KIND, int SC, bool XT, bool WT, bool DUAL, int EPI, typename T, int WM, int WN, bool PAIRS>
__global__ __launch_bounds__(64 * WM * WN) void k_mm_any(MmArgs p) {
    constexpr int E = mm_size<KIND>(), MT = 8 / WM, NT = 4;
    using C = MmCols<mm_pair<T, WT, DUAL>(), DUAL>;
    constexpr int kSteps = kMmStep / E;  // of the contraction per step
    constexpr int kRows = 64 * WN, kCols = DUAL ? kRows / 2 : kRows, kThreads = 64 * WM * WN;
    constexpr int kXC = 1024 / kThreads, kWC = kRows * 8 / kThreads;
    using Sums = MmSums<KIND, SC, DUAL, MT, NT>;
    using X = MmTile<E, 128, XT, kNear, PAIRS>;
    using W = MmTile<E, kCols, WT, C::kFar>;
    constexpr int kOf = PAIRS ? 2 : 1, BM = 128 / kOf;  // rows of X
    __shared__ __align__(16) uint8_t xt[128 * kMmStep], wt[kRows * kMmStep];
    const int wave = wave_id(), wm = wave % WM, wn = wave / WM;
    const int ln = threadIdx.x & 15, gq = threadIdx.x >> 4 & 3;
    const int64_t tm = (p.M + BM - 1) / BM, tn = (p.N + kCols - 1) / kCols;
    const int64_t m0 = (blockIdx.x % tm) * BM, n0 = (blockIdx.x / tm % tn) * kCols;
    const int rest = (int)(blockIdx.x / (tm * tn)), z = rest % p.outs, part = rest / p.outs;
    const int32_t per = (int32_t)((p.K + kSteps - 1) / kSteps);
    const int32_t begin = part * p.share, end = p.splits ? min(begin + p.share, per * p.segs) : per * p.segs;
    Sums sums;
    u32x4 cx[kXC], cw[kWC];
    auto load = [&](int32_t it) {
        const int seg = it >= per;
        const int64_t k0 = (int64_t)(it - seg * per) * kSteps;
#pragma unroll
        for (int i = 0; i < kXC; ++i) cx[i] = X::load(mm_x<XT>(p, seg, z), p.ldx, m0, p.M, k0, p.K, threadIdx.x + kThreads * i, p.low);
#pragma unroll
        for (int i = 0; i < kWC; ++i) {
            const int c = threadIdx.x + kThreads * i;
            if constexpr (DUAL) cw[i] = W::load(p.w[i / (kWC / 2)], p.ldw, n0, p.N, k0, p.K, c - kCols * 8 * (i / (kWC / 2)));
            else cw[i] = W::load(mm_w<XT>(p, seg), p.ldw, n0, p.N, k0, p.K, c);
        }
    };
    if (begin < end) load(begin);
    for (int32_t it = begin; it < end; ++it) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kXC; ++i) *reinterpret_cast<u32x4*>(xt + X::lds(threadIdx.x + kThreads * i)) = cx[i];
#pragma unroll
        for (int i = 0; i < kWC; ++i) {
            const int c = threadIdx.x + kThreads * i;
            if constexpr (DUAL) *reinterpret_cast<u32x4*>(wt + kCols * kMmStep * (i / (kWC / 2)) + W::lds(c - kCols * 8 * (i / (kWC / 2)))) = cw[i];
            else *reinterpret_cast<u32x4*>(wt + W::lds(c)) = cw[i];
        }
        __syncthreads();
        if (it + 1 < end) load(it + 1);
        MmFrag<KIND> fx, fw[NT];
        float sw[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if constexpr (WT) mm_read_turned<KIND, kRows>(fw[j], wt, wn * 64 + C::row(j), C::kStride);
            else mm_read<KIND, C::kFar>(fw[j], wt + (DUAL ? kCols * kMmStep * (j / 2) : 0), wn * (kCols / WN) + C::row(j) + C::kStride * (ln >> 2) + (ln & 3));
            if constexpr (Sums::kScaled)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (SC == kMmGroup) sw[j][i] = p.ws[0][min(n0 + wn * 64 + C::col(j, gq) + i, p.N - 1) * p.kb + it];
                    else sw[j][i] = p.ws[DUAL ? j / 2 : 0][n0 / 128 * p.kb + it];
                }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if constexpr (XT) mm_read_turned<KIND, 128>(fx, xt, wm * (16 * MT) + 16 * t, 4);
            else mm_read<KIND, kNear>(fx, xt, wm * (16 * MT) + 16 * t + ln);
            if constexpr (Sums::kScaled) {
                const float sx = p.xs[min(m0 + wm * (16 * MT) + 16 * t + ln, p.M - 1) * p.kb + it];
#pragma unroll
                for (int j = 0; j < NT; ++j) sums.add(t, j, mm_mma(fw[j], fx, f32x4{0.f, 0.f, 0.f, 0.f}), sx, sw[j]);
            } else {
#pragma unroll
                for (int j = 0; j < NT; ++j) sums.acc[t][j] = mm_mma(fw[j], fx, sums.acc[t][j]);
            }
        }
    }
    if constexpr (EPI == kMmFfn8) {
        __syncthreads();
        mm_finish8<Sums, MT>(sums, p, reinterpret_cast<uint32_t*>(xt), wm * (16 * MT), wn, m0 + wm * (16 * MT), n0);
    } else {
        sums.template finish<EPI, T, mm_pair<T, WT, DUAL>(), PAIRS>(p, z ? p.out[1] : p.out[0], z * p.splits + part, m0 + wm * (16 * MT / kOf), n0 + wn * (kCols / WN));
    }
}

// ---- the same, memory to LDS without registers ----------------------------------------------
// 16 bytes of each lane from base + off to LDS at lds + 16 lane. In assembly: the compiler takes the builtin for
// a write that every later LDS read has to wait for. Counted by vmcnt like a load; no register is written. M0, which holds the
// LDS address, is an operand, so that the compiler writes it and knows what it holds (as an instruction of the statement's own it
// went unseen; the compiler takes no clobber of it). It needs a wait state before the load that uses it.
__device__ __forceinline__ uint64_t mm_uniform(uint64_t a) {
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a) | (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32;
}
__device__ __forceinline__ uint64_t mm_uniform(const void* p) { return mm_uniform((uint64_t)(uintptr_t)p); }
__device__ __forceinline__ void mm_dma16(uint32_t lds, uint64_t base, uint32_t off) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(off), "s"(mm_uniform(base)) : "memory");
}
// All of this wave's loads to LDS have landed and its LDS reads are done; then the workgroup meets.
__device__ __forceinline__ void mm_meet() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
__device__ __forceinline__ uint32_t mm_lds(const void* p) { return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p; }

// Which tile a workgroup takes. Workgroups go round robin over the 8 XCDs, each with an L2 of its own: an XCD gets a
// run of tiles, in columns of 8 X tiles, so that the 32 tiles it works on at a time share 8 X and 4 W tiles.
struct MmPlace {
    int32_t m, n, rest;
    __device__ __forceinline__ MmPlace(int32_t id, int32_t total, int32_t tm, int32_t tn) {
        const int32_t xcd = id % 8, per = total / 8, more = total % 8;
        int32_t l = xcd * per + min(xcd, more) + id / 8;
        rest = l / (tm * tn);
        l -= rest * tm * tn;
        const int32_t group = l / (8 * tn), high = min(8, tm - 8 * group);
        l -= group * 8 * tn;
        m = 8 * group + l % high;
        n = l / high;
    }
};

// BM x 256 outputs (two sides: BM x 128 of each) by eight waves of BM/2 x 64; two steps' tiles in LDS, the next one on
// its way while one is multiplied. Memory rows and addresses are multiples of 16 bytes, 256 rows within 2^31 bytes.
// Bound by power and issue: 8,192 x 8,192 x 8,192 bf16 takes 813 us (1,352 TFLOP/s) at 1.83 GHz, 2,740 cycles a step whose
// matrix instructions need 2,048; without loads from memory 2,420 cycles, at a lower clock. e4m3 by blocks, 32,768 x 6,144 x
// 2,048: 430 us (1.9 PFLOP/s), with a scaled sum for each 128 products on the vector ALUs. BM is 128 where widened operands
// or fp32 leave no registers for 256, and where that fills the card better (mm_plan).
template <int KIND, int SC, bool XT, bool WT, bool DUAL, int EPI, typename T, int BM, bool PAIRS>
__global__ __launch_bounds__(512) void k_mm(MmArgs p) {
    constexpr int E = mm_size<KIND>(), MT = BM / 32, NT = 4, BN = 256;
    using C = MmCols<mm_pair<T, WT, DUAL>(), DUAL>;
    constexpr int kSteps = kMmStep / E;
    constexpr int kCols = DUAL ? 128 : 256;
    constexpr int kXB = BM * kMmStep, kWB = BN * kMmStep;
    constexpr int kXC = BM * 8 / 512, kWC = 4;  // chunks of a thread
    using Sums = MmSums<KIND, SC, DUAL, MT, NT>;
    using X = MmTile<E, BM, XT, kNear>;
    using W = MmTile<E, kCols, WT, C::kFar>;
    constexpr int kStage = kXB + kWB;
    constexpr int kSRows = Sums::kScaled ? BM + (SC == kMmGroup ? 256 : 2) : 0;  // rows of scales: X's, and W's or two of its blocks
    __shared__ __align__(128) uint8_t sh[2 * (kStage + kSRows * 16)];
    const int wave = wave_id(), lane = threadIdx.x & 63, wm = wave & 1, wn = wave >> 1;
    const int ln = lane & 15, gq = lane >> 4;
    constexpr int kOf = PAIRS ? 2 : 1, kXRows = BM / kOf;  // rows of X
    const int32_t tm = (int32_t)((p.M + kXRows - 1) / kXRows), tn = (int32_t)((p.N + kCols - 1) / kCols);
    const MmPlace at(blockIdx.x, gridDim.x, tm, tn);
    const int64_t m0 = (int64_t)at.m * kXRows, n0 = (int64_t)at.n * kCols;
    const int z = at.rest % p.outs, part = at.rest / p.outs;
    const int32_t per = (int32_t)((p.K + kSteps - 1) / kSteps);
    const int32_t begin = part * p.share, end = p.splits ? min(begin + p.share, per * p.segs) : per * p.segs;

    // Chunks behind an operand's last row or column repeat its last one (which starts in it, so it lies at or behind the
    // tile's start; a memory row is whole chunks).
    // A thread's chunk i of a tile is chunk threadIdx.x + 512 i as LDS has them; which of memory's that is, is the XOR undone.
    uint32_t xo[kXC], wo[kWC];
    int xk[kXC], wk[kWC];  // its place along the contraction: bytes of a row, or rows
#pragma unroll
    for (int i = 0; i < kXC; ++i) {
        const int c = threadIdx.x + 512 * i;
        if constexpr (XT) {
            const int k = c / X::kWide, r = ((c % X::kWide) ^ mm_turn_key<BM, E>(k)) * (16 / E);
            const int64_t col = (m0 + (PAIRS ? mm_pair_row(r) : r)) * E;
            xk[i] = k;
            xo[i] = (uint32_t)(k * p.ldx) + (uint32_t)(min(col, (p.M * E - 1) / 16 * 16) - m0 * E);
            if (PAIRS && mm_pair_low(r)) xo[i] += (uint32_t)p.low;
        } else {
            const int r = c >> 3, b = ((c & 7) ^ mm_key<kNear>(r)) * 16, row = PAIRS ? mm_pair_row(r) : r;
            xk[i] = b;
            xo[i] = (uint32_t)((m0 + row < p.M ? row : p.M - 1 - m0) * p.ldx) + b;
            if (PAIRS && mm_pair_low(r)) xo[i] += (uint32_t)p.low;
        }
    }
#pragma unroll
    for (int i = 0; i < kWC; ++i) {
        const int c = threadIdx.x + 512 * (DUAL ? i % 2 : i);
        if constexpr (WT) {
            const int k = c / W::kWide, b = ((c % W::kWide) ^ mm_turn_key<kCols, E>(k)) * 16;
            const int64_t col = n0 * E + b;
            wk[i] = k;
            wo[i] = (uint32_t)(k * p.ldw) + (uint32_t)(min(col, (p.N * E - 1) / 16 * 16) - n0 * E);
        } else {
            const int r = c >> 3, b = ((c & 7) ^ mm_key<C::kFar>(r)) * 16;
            wk[i] = b;
            wo[i] = (uint32_t)((n0 + r < p.N ? r : p.N - 1 - n0) * p.ldw) + b;
        }
    }
    // Scales pass through registers, those of four steps at a time: a thread has one row's, which lie side by side.
    const float* srow = nullptr;
    if constexpr (Sums::kScaled) {
        const int r = threadIdx.x - BM;
        if (r < 0) srow = p.xs + min(m0 + (int)threadIdx.x, p.M - 1) * p.kb;
        else if (SC == kMmGroup && r < 256) srow = p.ws[0] + min(n0 + r, p.N - 1) * p.kb;
        else if (SC == kMmBlock && r < 2) srow = (DUAL && r ? p.ws[1] : p.ws[0]) + (DUAL ? n0 / 128 : min(n0 / 128 + r, (p.N - 1) / 128)) * p.kb;
    }
    f32x4* const sring = reinterpret_cast<f32x4*>(sh + 2 * kStage);
    f32x4 snext = {};
    auto fetch_scales = [&](int32_t k) {  // of steps k .. k + 3
        if (srow) {
            if (k + 4 <= p.kb) __builtin_memcpy(&snext, srow + k, 16);
            else
#pragma unroll
                for (int i = 0; i < 4; ++i) snext[i] = srow[min((int64_t)k + i, p.kb - 1)];
        }
    };
    auto keep_scales = [&](int32_t k) {
        if (srow) sring[(k >> 2 & 1) * kSRows + threadIdx.x] = snext;
    };
    const uint32_t lds0 = mm_lds(sh) + wave * 1024;

    // Where the next step's tiles come from (scalars, whatever the compiler makes of the loop).
    const int64_t xstep = XT ? kSteps * p.ldx : kMmStep, wstep = WT ? kSteps * p.ldw : kMmStep;
    const int32_t whole = (int32_t)(p.K / kSteps), rest = (int32_t)(p.K % kSteps);
    const int64_t xat = XT ? m0 * E : m0 * p.ldx, wat = WT ? n0 * E : n0 * p.ldw;
    constexpr bool kSegs = WT && !XT;  // there may be two segments (dx)
    int32_t seg = kSegs ? begin >= per : 0, kt = begin - seg * per;
    uint64_t xs = mm_uniform(mm_x<XT>(p, seg, z) + xat + kt * xstep);
    uint64_t ws0 = mm_uniform((DUAL ? p.w[0] : mm_w<XT>(p, seg)) + wat + kt * wstep), ws1 = mm_uniform(p.w[1] + wat + kt * wstep);
    auto fetch = [&](int stage) {
        const uint32_t xl = lds0 + stage * kStage, wl = xl + kXB;
        if (__builtin_expect(kt < whole, 1)) {
#pragma unroll
            for (int i = 0; i < kXC; ++i) mm_dma16(xl + i * 8192, xs, xo[i]);
#pragma unroll
            for (int i = 0; i < kWC; ++i) mm_dma16(wl + i * 8192, DUAL && i >= 2 ? ws1 : ws0, wo[i]);
        } else {
            // the contraction's end: zeros behind it
            uint8_t* to = sh + stage * kStage + threadIdx.x * 16;
#pragma unroll
            for (int i = 0; i < kXC; ++i) {
                if (xk[i] < (XT ? rest : rest * E)) mm_dma16(xl + i * 8192, xs, xo[i]);
                else *reinterpret_cast<u32x4*>(to + i * 8192) = u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < kWC; ++i) {
                if (wk[i] < (WT ? rest : rest * E)) mm_dma16(wl + i * 8192, DUAL && i >= 2 ? ws1 : ws0, wo[i]);
                else *reinterpret_cast<u32x4*>(to + kXB + i * 8192) = u32x4{0, 0, 0, 0};
            }
        }
        xs += xstep;
        ws0 += wstep;
        if (DUAL) ws1 += wstep;
        ++kt;
        if (kSegs && kt == per && p.segs > 1) {
            kt = 0;
            ++seg;
            xs = mm_uniform(mm_x<XT>(p, seg, z) + xat);
            ws0 = mm_uniform(mm_w<XT>(p, seg) + wat);
        }
        kt = __builtin_amdgcn_readfirstlane(kt);
    };

    // The lane's chunks of its first X row; the rows of the next tiles lie whole numbers of 16 rows on, with the same keys.
    const uint32_t xl0 = mm_at<kNear>(wm * (BM / 2) + ln, gq), xl1 = mm_at<kNear>(wm * (BM / 2) + ln, gq + 4);
    Sums sums;
    if (begin < end) {  // (a part begins with a multiple of four steps)
        fetch(begin & 1);
        if constexpr (Sums::kScaled) {
            fetch_scales(begin);
            keep_scales(begin);
        }
    }
    for (int32_t it = begin; it < end; ++it) {
        mm_meet();
        if constexpr (Sums::kScaled) {
            // (what was loaded has arrived with the step's tiles)
            if ((it & 3) == 1 && it + 3 < end) keep_scales(it + 3);
            if ((it & 3) == 0 && it + 4 < end) fetch_scales(it + 4);
        }
        const uint8_t* xt = sh + (it & 1) * kStage;
        const uint8_t* wt = xt + kXB;
        const float* sc = reinterpret_cast<const float*>(sring + (it >> 2 & 1) * kSRows) + (it & 3);
        // X's chunks are read a tile ahead; e4m3 that is widened two tiles, and widened one ahead
        constexpr int kAhead = KIND == kMmF8x ? 2 : 1;
        MmFrag<KIND> fx[2], fw[NT];
        u32x4 raw[2][2], rw[NT][2];
        f32x4 c[2][NT];
        float sx[4] = {}, sw[NT][4];
        typedef const __attribute__((address_space(3))) float lds_float;
        const uint32_t xa = mm_fresh(mm_lds(xt) + xl0), xc = mm_fresh(mm_lds(xt) + xl1);
        const uint32_t sa = Sums::kScaled ? mm_fresh(mm_lds(sc) + 16 * (wm * (BM / 2) + ln)) : 0;
        auto read = [&](int t) {
            if constexpr (XT) mm_read_turned<KIND, BM>(fx[t & 1], xt, wm * (BM / 2) + 16 * t, 4);
            else mm_read_at(raw[t & 1], xa, xc, 16 * kMmStep * t);
            if constexpr (Sums::kScaled) sx[t & 3] = *(lds_float*)(uintptr_t)(sa + 256 * t);
        };
        auto ready = [&](int t) {
            if constexpr (!XT) fx[t & 1].set(raw[t & 1][0], raw[t & 1][1]);
        };
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if constexpr (WT) mm_read_turned<KIND, BN>(fw[j], wt, wn * 64 + C::row(j), C::kStride);
            else mm_read<C::kFar>(rw[j], wt + (DUAL ? 128 * kMmStep * (j / 2) : 0), wn * (kCols / 4) + C::row(j) + C::kStride * (ln >> 2) + (ln & 3));
        }
#pragma unroll
        for (int t = 0; t < kAhead; ++t) read(t);
        if constexpr (Sums::kScaled) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if constexpr (SC == kMmGroup) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) sw[j][i] = sc[4 * (BM + wn * 64 + C::col(j, gq) + i)];
                } else {
                    sw[j][0] = sc[4 * (BM + (DUAL ? j / 2 : wn / 2))];
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (it + 1 < end) fetch(~it & 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!WT)
#pragma unroll
            for (int j = 0; j < NT; ++j) fw[j].set(rw[j][0], rw[j][1]);
        ready(0);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if constexpr (KIND != kMmF8x) __builtin_amdgcn_sched_barrier(0);
            if (kAhead == 2 && t + 1 < MT) ready(t + 1);
            if (t + kAhead < MT) read(t + kAhead);
            // A tile's parts one after the other, or the four tiles' in turn (widened e4m3, 6,144 x 2,048 x 32,768 by groups
            // 1,031 us and 1,010; 16,384 x 16,384 x 2,048 by blocks 1,096 and 1,138).
            constexpr bool kTurn = KIND == kMmF8x && SC == kMmGroup;
            constexpr int kParts = mm_parts<KIND>();
#pragma unroll
            for (int k = 0; k < kParts * NT; ++k) {
                const int i = kTurn ? k / NT : k % kParts, j = kTurn ? k % NT : k / kParts;
                if constexpr (Sums::kScaled) c[t & 1][j] = mm_part(i, fw[j], fx[t & 1], i ? c[t & 1][j] : f32x4{0.f, 0.f, 0.f, 0.f});
                else sums.acc[t][j] = mm_part(i, fw[j], fx[t & 1], sums.acc[t][j]);
                // a tile's sums are added while the next one is multiplied
                if (Sums::kScaled && i == (kTurn ? 0 : kParts - 1) && t > 0) sums.add(t - 1, j, c[~t & 1][j], sx[(t - 1) & 3], sw[j]);
                // matrix instructions with vector ones between them (widened e4m3: three; by groups, 6,144 x 2,048 x 32,768, three
                // 969 us, four 1,010, five 990)
                if constexpr (Sums::kScaled) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    if (KIND == kMmF8x) __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
                    else if (t > 0) __builtin_amdgcn_sched_group_barrier(0x002, SC == kMmBlock ? 5 : 8, 0);
                }
            }
            if (kAhead == 1 && t + 1 < MT) ready(t + 1);
        }
        if constexpr (Sums::kScaled)
#pragma unroll
            for (int j = 0; j < NT; ++j) sums.add(MT - 1, j, c[(MT - 1) & 1][j], sx[(MT - 1) & 3], sw[j]);
    }
    if constexpr (EPI == kMmFfn8) {
        mm_meet();
        mm_finish8<Sums, MT>(sums, p, reinterpret_cast<uint32_t*>(sh), wm * (BM / 2), wn, m0 + wm * (BM / 2), n0);
    } else {
        sums.template finish<EPI, T, mm_pair<T, WT, DUAL>(), PAIRS>(p, z ? p.out[1] : p.out[0], z * p.splits + part, m0 + wm * (kXRows / 2), n0 + wn * (kCols / 4));
    }
}

// ---- few rows of X ---------------------------------------------------------------------------
// 16 W rows (of each side) by a workgroup whose waves share the contraction: W is read once, straight into the matrix
// instructions' registers, several steps of a wave at a time; X (at most 16 MT rows) comes from the caches. The waves' sums
// meet in LDS. WHOLE: memory rows are whole chunks. Bound by memory and by the latency of a few rounds of loads: gate and up of
// 1 x 2,048 x 5,632 bf16 13.0 us (46 MB, 3.6 TB/s), 16 x 6,144 x 2,048 e4m3 7.5.
template <int KIND, int SC, bool DUAL, int EPI, typename T, int MT, int WAVES, bool WHOLE>
__global__ __launch_bounds__(64 * WAVES) void k_mm_few(MmArgs p) {
    constexpr int E = mm_size<KIND>(), kSides = DUAL ? 2 : 1;
    // Steps at a time: what the registers of 4 waves a SIMD hold (gate and up of 2,048 x 8,192 in e4m3, 20 rows, two steps 10.7 us,
    // four, which leave room for 2 waves, 12.4; in fp32 at 5,648 x 5,952 124 and 118).
    constexpr int kAt = !WHOLE ? 1 : (WAVES == 16 ? (MT + kSides <= 3 ? 2 : 1) : (MT * kSides >= 8 ? 1 : (MT * kSides >= 4 ? 2 : 4)));
    constexpr int kSteps = kMmStep / E;
    constexpr bool kScaled = SC == kMmBlock || SC == kMmGroup;
    __shared__ f32x4 sh[WAVES][kSides * MT][64];
    const int wave = wave_id(), lane = threadIdx.x & 63, ln = lane & 15, gq = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int32_t per = (int32_t)((p.K + kSteps - 1) / kSteps);
    const uint8_t *wr[kSides], *xr[MT];
#pragma unroll
    for (int i = 0; i < kSides; ++i) wr[i] = p.w[i] + min(n0 + ln, p.N - 1) * p.ldw;
#pragma unroll
    for (int t = 0; t < MT; ++t) xr[t] = p.x[0] + min((int64_t)16 * t + ln, p.M - 1) * p.ldx;
    auto load = [&](const uint8_t* row, int64_t off) {
        if constexpr (WHOLE) return off < p.K * E ? *reinterpret_cast<const u32x4*>(row + off) : u32x4{0, 0, 0, 0};
        else return mm_chunk(row, off, p.K * E);
    };
    f32x4 acc[kSides][MT] = {};
    for (int32_t first = wave; first < per; first += WAVES * kAt) {
        u32x4 w[kAt][kSides][2], x[kAt][MT][2];
        float sx[kAt][MT], sw[kAt][kSides][4];
#pragma unroll
        for (int a = 0; a < kAt; ++a) {
            const int32_t kt = first + a * WAVES;
            if (kt >= per) break;
            const int64_t off = (int64_t)kt * kMmStep + 16 * gq;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < kSides; ++i) w[a][i][h] = load(wr[i], off + 64 * h);
#pragma unroll
                for (int t = 0; t < MT; ++t) x[a][t][h] = load(xr[t], off + 64 * h);
            }
            if constexpr (kScaled) {
#pragma unroll
                for (int t = 0; t < MT; ++t) sx[a][t] = p.xs[min((int64_t)16 * t + ln, p.M - 1) * p.kb + kt];
#pragma unroll
                for (int i = 0; i < kSides; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sw[a][i][j] = SC == kMmBlock ? p.ws[i][n0 / 128 * p.kb + kt] : p.ws[i][min(n0 + 4 * gq + j, p.N - 1) * p.kb + kt];
            }
        }
#pragma unroll
        for (int a = 0; a < kAt; ++a) {
            if (first + a * WAVES >= per) break;
            MmFrag<KIND> fw[kSides];
#pragma unroll
            for (int i = 0; i < kSides; ++i) fw[i].set(w[a][i][0], w[a][i][1]);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                MmFrag<KIND> fx;
                fx.set(x[a][t][0], x[a][t][1]);
#pragma unroll
                for (int i = 0; i < kSides; ++i) {
                    if constexpr (kScaled) {
                        const f32x4 c = mm_mma(fw[i], fx, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][t][j] = fmaf(c[j], sx[a][t] * sw[a][i][j], acc[i][t][j]);
                    } else {
                        acc[i][t] = mm_mma(fw[i], fx, acc[i][t]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kSides; ++i)
#pragma unroll
        for (int t = 0; t < MT; ++t) sh[wave][i * MT + t][lane] = acc[i][t];
    __syncthreads();
    if (wave >= MT) return;
    const int64_t m = 16 * wave + ln, n = n0 + 4 * gq;
    if (m >= p.M || n >= mm_width<EPI>(p)) return;
    float v[kSides][4] = {};
#pragma unroll
    for (int i = 0; i < kSides; ++i)
#pragma unroll
        for (int s = 0; s < WAVES; ++s) {
            const f32x4 c = sh[s][i * MT + wave][lane];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] += c[j];
        }
    mm_finish<EPI, T, SC, DUAL, 4>(p, p.out[0], 0, m, n, v);
}

// ---- which kernel ----------------------------------------------------------------------------
inline int64_t mm_blocks(int64_t M, int64_t N, bool dual, int BM) { return ((M + BM - 1) / BM) * ((N + (dual ? 127 : 255)) / (dual ? 128 : 256)); }
inline int64_t mm_any_blocks(int64_t M, int64_t N, bool dual, int BM) { return ((M + BM - 1) / BM) * ((N + (dual ? 63 : 127)) / (dual ? 64 : 128)); }

// Whether k_mm takes the operands.
inline bool mm_fits(const MmArgs& p) {
    uint64_t bits = (uint64_t)(p.ldx | p.ldw);
    for (int i = 0; i < 2; ++i) bits |= (uint64_t)(uintptr_t)p.x[i] | (uint64_t)(uintptr_t)p.w[i];
    return bits % 16 == 0 && p.ldx < (1 << 23) && p.ldw < (1 << 23);
}

// X rows of k_mm_few: 32, or 64 over short rows. Its workgroups read all of X each, so tiles pass it by as X grows (gate and up of
// 2,048 x 8,192 in e4m3, 40 rows: 14.9 us and 17.0; 5,648 x 5,952: 28.0 and 25.8, in fp32 194 and 152).
inline bool mm_is_few(int64_t M, int64_t row_bytes) { return M <= (row_bytes <= 3 * 1024 ? 64 : 32); }

// What a product of these sizes runs as: by sizes and types alone, so that the workspace can be told beforehand (k_mm and
// k_mm_any split alike, whichever the addresses ask for).
struct MmPlan {
    bool few;
    int bm;
    int splits, share;
    size_t bytes;  // of the parts
};
inline MmPlan mm_plan(int kind, int sc, int64_t M, int64_t N, int64_t K, int segs, int outs, bool turned, bool dual, bool pairs = false) {
    MmPlan r{};
    const int E = kind == kMmBf16 ? 2 : (kind == kMmF32 ? 4 : 1), steps = kMmStep / E;
    r.few = !turned && segs == 1 && outs == 1 && mm_is_few(M, K * E);
    if (r.few) return r;
    const int64_t total = (K + steps - 1) / steps * segs;
    // Memory rows that are no whole chunks go to k_mm_any (128 x 128, two workgroups a compute unit); others to k_mm with 256
    // rows of X a tile or 128. The contraction is taken whole or in parts. Whatever is quickest by this count of microseconds:
    // rounds of the workgroups that run at a time, what a step of a tile measured, and for parts another launch and what they
    // write and read at 4 TB/s.
    const bool odd = (turned ? N : K) * E % 16;
    const double step = odd ? (kind == kMmF32 ? 3.2 : (kind == kMmF8x ? 2.8 : 1.6)) : (kind == kMmF32 ? 4.0 : (kind == kMmF8x ? 2.0 : (kind == kMmF8 ? 1.2 : 1.0)));
    const int rows = pairs ? 64 : 128;  // of X in a tile of 128
    const int64_t tiles = (odd ? mm_any_blocks(M, N, dual, rows) : mm_blocks(M, N, dual, rows)) * outs, slots = odd ? 512 : 256;
    const double sums = 2e-6 * (double)M * (double)N * outs * (dual ? 2 : 1);
    double best = step * ((tiles + slots - 1) / slots) * total;
    r.bm = 128;
    const int64_t large = mm_blocks(M, N, dual, 256) * outs;
    const double large_us = (kind == kMmF8 ? 2.0 : 1.6) * ((large + 255) / 256) * total;
    if (!odd && !pairs && kind != kMmF8x && kind != kMmF32 && large_us <= best) {
        r.bm = 256;
        best = large_us;
    }
    const int unit = sc == kMmBlock || sc == kMmGroup ? 4 : 1;  // (scales come four steps at a time)
    for (int64_t parts = 2; parts <= 32 && parts < total && parts * tiles <= 2 * slots; ++parts) {
        const int64_t share = ((total + parts - 1) / parts + unit - 1) / unit * unit, got = (total + share - 1) / share;
        const double t = step * ((tiles * got + slots - 1) / slots) * share + 5 + sums * got;
        if (got > 1 && t < best) {
            best = t;
            r.bm = 128;
            r.share = (int)share;
            r.splits = (int)got;
        }
    }
    r.bytes = (size_t)outs * r.splits * (dual ? 2 : 1) * M * N * 4;
    return r;
}

template <int KIND, int SC, bool DUAL, int EPI, typename T, int MT, bool WHOLE>
hipError_t mm_few(const MmArgs& p, hipStream_t st) {
    const int64_t blocks = (mm_width<EPI>(p) + 15) / 16;
    const bool many = blocks <= 128 && p.K * mm_size<KIND>() >= 16 * kMmStep && MT * (DUAL ? 2 : 1) <= 4;
    if (blocks > UINT32_MAX / 1024) return hipErrorInvalidConfiguration;
    if constexpr (MT * (DUAL ? 2 : 1) <= 4)
        if (many) {
            hipLaunchKernelGGL((k_mm_few<KIND, SC, DUAL, EPI, T, MT, 16, WHOLE>), dim3((unsigned)blocks), dim3(1024), 0, st, p);
            return hipGetLastError();
        }
    hipLaunchKernelGGL((k_mm_few<KIND, SC, DUAL, EPI, T, MT, 8, WHOLE>), dim3((unsigned)blocks), dim3(512), 0, st, p);
    return hipGetLastError();
}
template <int KIND, int SC, bool DUAL, int EPI, typename T, int MT>
hipError_t mm_few(const MmArgs& p, hipStream_t st) {
    return mm_fits(p) ? mm_few<KIND, SC, DUAL, EPI, T, MT, true>(p, st) : mm_few<KIND, SC, DUAL, EPI, T, MT, false>(p, st);
}

template <int KIND, int SC, bool XT, bool WT, bool DUAL, int EPI, typename T, bool PAIRS>
hipError_t mm_tiles(const MmArgs& p, int bm, hipStream_t st) {
    const int64_t times = (int64_t)p.outs * (p.splits ? p.splits : 1);
    constexpr int kOf = PAIRS ? 2 : 1;
    if (mm_fits(p)) {
        const int64_t blocks = mm_blocks(p.M, p.N, DUAL, bm / kOf) * times;
        if (blocks > UINT32_MAX / 512 || blocks > INT32_MAX) return hipErrorInvalidConfiguration;
        if constexpr (KIND != kMmF8x && KIND != kMmF32 && EPI != kMmPart && !PAIRS)
            if (bm == 256) {
                hipLaunchKernelGGL((k_mm<KIND, SC, XT, WT, DUAL, EPI, T, 256, false>), dim3((unsigned)blocks), dim3(512), 0, st, p);
                return hipGetLastError();
            }
        hipLaunchKernelGGL((k_mm<KIND, SC, XT, WT, DUAL, EPI, T, 128, PAIRS>), dim3((unsigned)blocks), dim3(512), 0, st, p);
        return hipGetLastError();
    }
    constexpr int kWide = EPI == kMmFfn8 ? 4 : 2;  // (128 columns of h share a scale)
    const int64_t blocks = (kWide == 4 ? mm_blocks(p.M, p.N, DUAL, 128) : mm_any_blocks(p.M, p.N, DUAL, 128 / kOf)) * times;
    if (blocks > UINT32_MAX / 512) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_mm_any<KIND, SC, XT, WT, DUAL, EPI, T, 8 / kWide, kWide, PAIRS>), dim3((unsigned)blocks), dim3(512), 0, st, p);
    return hipGetLastError();
}

// `part`: the workspace that mm_plan asked for.
template <int KIND, int SC, bool XT, bool WT, bool DUAL, int EPI, typename T, bool PAIRS = false>
hipError_t mm_run(MmArgs p, void* part, hipStream_t st) {
    const MmPlan r = mm_plan(KIND, SC, p.M, p.N, p.K, p.segs, p.outs, XT || WT, DUAL, PAIRS);
    if constexpr (!XT && !WT && EPI != kMmFfn8)
        if (r.few) {
            if (p.M <= 16) return mm_few<KIND, SC, DUAL, EPI, T, 1>(p, st);
            if (p.M <= 32) return mm_few<KIND, SC, DUAL, EPI, T, 2>(p, st);
            return mm_few<KIND, SC, DUAL, EPI, T, 4>(p, st);
        }
    if constexpr (EPI != kMmFfn8)
        if (r.splits) {
            p.splits = r.splits;
            p.share = r.share;
            p.part = static_cast<float*>(part);
            if (hipError_t e = mm_tiles<KIND, SC, XT, WT, DUAL, kMmPart, T, PAIRS>(p, r.bm, st)) return e;
            const int64_t blocks = ((mm_width<EPI>(p) + 3) / 4 * p.M + 255) / 256;
            hipLaunchKernelGGL((k_mm_join<SC, DUAL, EPI, T>), dim3((unsigned)blocks, (unsigned)p.outs), dim3(256), 0, st, p);
            return hipGetLastError();
        }
    return mm_tiles<KIND, SC, XT, WT, DUAL, EPI, T, PAIRS>(p, r.bm, st);
}

}  // namespace gdn
