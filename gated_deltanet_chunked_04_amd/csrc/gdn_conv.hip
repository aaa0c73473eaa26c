// gdn_conv.hip -- the short causal convolution in front of the recurrences, one filter of W taps
// per channel: z_t = bias + sum_j w_j x_{t-W+1+j}, y = z or silu(z). The inputs before a sequence's
// first token are its entering state [W-1, D] (zeros without one); its last W-1 inputs leave as the
// final state. Gradient: dz = dy act'(z), z recomputed;
//   dx_s = sum_i w_{W-1-i} dz_{s+i},  dw_j = sum_t dz_t x_{t-W+1+j},  dbias = sum_t dz_t,
// positions before the first token giving the entering state's gradient.
//
// Bound by memory: 2W + 5 operations per element forward and 6W + 10 backward, against 4 and 6 bytes
// in bf16. So every input is read once: a wave walks a run of tokens down its block of channels (a
// lane holds a few neighbouring ones, so a wave reads whole cache lines of a token's row) with the
// last W-1 inputs, and in the gradient the last W-1 dz, in registers; only the W-1 tokens around the
// ends of a run are read by two waves, and what the gradient needs behind a run comes through LDS from
// the wave that starts there (240 -> 233 us). The next tokens' loads are issued before the present ones
// are used. Runs that lie inside one sequence take a path without any test per token.
#include <type_traits>

#include "gdn_layer.h"
#include "gdn_vec.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// The lane's filter, tap by tap, and its bias.
template <typename TW, int W, int VEC>
struct Filter {
    float w[W][VEC], b[VEC];
    __device__ __forceinline__ void load(const ConvArgs& p, int64_t c0) {
        const Raw<TW, VEC * W> r = load_raw<TW, VEC * W>(static_cast<const TW*>(p.w) + c0 * W);
        Raw<TW, VEC> rb;
        rb.clear();
        if (p.bias) rb = load_raw<TW, VEC>(static_cast<const TW*>(p.bias) + c0);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][v] = r.get(v * W + j);
            b[v] = rb.get(v);
        }
    }
};

// Row t of a [tokens, D] array, the lane's channels.
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> row(const void* a, int64_t t, const ConvArgs& p, int64_t c0) {
    return load_raw<T, VEC>(static_cast<const T*>(a) + t * p.D + c0);
}
// Row r of sequence n's state [W-1, D], zeros where there is none.
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> state_row(const void* a, int32_t n, int r, const ConvArgs& p, int64_t c0) {
    if (!a) {
        Raw<T, VEC> z;
        z.clear();
        return z;
    }
    return row<T, VEC>(a, (int64_t)n * (p.W - 1) + r, p, c0);
}

template <int W, int VEC>
__device__ __forceinline__ void shift_in(float (&win)[W - 1][VEC], const float (&x)[VEC]) {
#pragma unroll
    for (int r = 0; r + 1 < W - 1; ++r)
#pragma unroll
        for (int v = 0; v < VEC; ++v) win[r][v] = win[r + 1][v];
#pragma unroll
    for (int v = 0; v < VEC; ++v) win[W - 2][v] = x[v];
}

template <typename TW, int W, int VEC>
__device__ __forceinline__ void pre_act(const Filter<TW, W, VEC>& f, const float (&win)[W - 1][VEC], const float (&x)[VEC], float (&z)[VEC]) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        z[v] = f.b[v];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) z[v] = fmaf(f.w[j][v], win[j][v], z[v]);
        z[v] = fmaf(f.w[W - 1][v], x[v], z[v]);
    }
}
// 1 / (1 + exp(-z)); 0 where that is below fp32's normal range (z < -87.3: z sigmoid(z) is then off by up to 9e-37)
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + fast_exp(-z)); }

// Sequences without tokens: their state (or its gradient) passes through, by the workgroups behind
// the tokens': number `block` of `blocks`.
template <bool kOdd, typename T, int VEC>
__device__ void pass_empty(const ConvArgs& p, int block, int blocks, const void* in, void* out, int64_t c0, int skip, bool live) {
    for_each_empty(p.seq, block * kWaves + wave_id(), blocks * kWaves, [&](int32_t s) {
        if (!live) return;
        for (int r = 0; r < p.W - 1; ++r)
            store_own<kOdd, T, VEC>(static_cast<T*>(out) + ((int64_t)s * (p.W - 1) + r) * p.D + c0,
                                    state_row<T, VEC>(in, s, r, p, c0), skip);
    });
}

// U: tokens loaded ahead. `run`: tokens per wave.
template <bool kOdd, typename T, typename TW, int W, int VEC, int U>
__global__ __launch_bounds__(kThreads) void k_conv_fwd(ConvArgs p, int run, int token_blocks, int cblocks) {
    const int block = blockIdx.x / cblocks;  // of tokens
    const int64_t ch = ((int64_t)(blockIdx.x % cblocks) * kWave + (threadIdx.x & 63)) * VEC;
    const Lane ln(ch, p.D, VEC);
    const int64_t c0 = ln.at;
    if (block >= token_blocks)
        return pass_empty<kOdd, T, VEC>(p, block - token_blocks, gridDim.x / cblocks - token_blocks, p.s0, p.sT, c0, ln.skip, ch < p.D);
    if (ch >= p.D) return;
    const int64_t w0l = ((int64_t)block * kWaves + wave_id()) * run;
    if (w0l >= p.seq.total) return;
    const int32_t w0 = (int32_t)w0l;
    const int32_t w1 = w0l + run < p.seq.total ? w0 + run : p.seq.total;
    Raw<T, VEC> nx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) nx[u] = row<T, VEC>(p.x, min(w0 + u, w1 - 1), p, c0);
    Filter<TW, W, VEC> f;
    f.load(p, c0);
    SeqPos s = seq_find(p.seq, w0);
    float win[W - 1][VEC];
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        const int32_t at = w0 - (W - 1) + r;
        Raw<T, VEC> h;
        h.clear();
        if (w0 >= s.start && w0 < s.end)
            h = at >= s.start ? row<T, VEC>(p.x, at, p, c0) : state_row<T, VEC>(p.s0, s.n, at - s.start + W - 1, p, c0);
#pragma unroll
        for (int v = 0; v < VEC; ++v) win[r][v] = h.get(v);
    }
    T* y = static_cast<T*>(p.y);
    auto token = [&](int32_t t, const Raw<T, VEC>& raw) {
        float x[VEC], z[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) x[v] = raw.get(v);
        pre_act<TW, W, VEC>(f, win, x, z);
        if (p.silu)
#pragma unroll
            for (int v = 0; v < VEC; ++v) z[v] *= sigmoid(z[v]);
        store_own<kOdd, T, VEC>(y + (int64_t)t * p.D + c0, z, ln.skip);
        shift_in<W, VEC>(win, x);
    };
    const bool inside = w0 >= s.start && w1 < s.end;
    for (int32_t t0 = w0; t0 < w1; t0 += U) {
        Raw<T, VEC> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = nx[u];
        if (t0 + U < w1)
#pragma unroll
            for (int u = 0; u < U; ++u) nx[u] = row<T, VEC>(p.x, min(t0 + U + u, w1 - 1), p, c0);
        if (inside && t0 + U <= w1) {
#pragma unroll
            for (int u = 0; u < U; ++u) token(t0 + u, x[u]);
            continue;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t t = t0 + u;
            if (t >= w1) break;
            seq_advance(p.seq, s, t);
            if (t < s.start || t >= s.end) {
                if (p.zero) zero_own<kOdd, T, VEC>(y + (int64_t)t * p.D + c0, ln.skip);
                continue;
            }
            if (t == s.start && t > w0)
#pragma unroll
                for (int r = 0; r < W - 1; ++r) {
                    const Raw<T, VEC> h = state_row<T, VEC>(p.s0, s.n, r, p, c0);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) win[r][v] = h.get(v);
                }
            token(t, x[u]);
            // the window now holds the last W-1 inputs, exactly as they were read
            if (p.sT && t + 1 == s.end)
#pragma unroll
                for (int r = 0; r < W - 1; ++r)
                    store_own<kOdd, T, VEC>(static_cast<T*>(p.sT) + ((int64_t)s.n * (W - 1) + r) * p.D + c0, win[r], ln.skip);
        }
    }
}

// One workgroup: kWaves runs of `run` tokens (a multiple of 2 U) and 64 VEC channels; the partial sums of dw and dbias over
// its tokens go to part[block], [W + 1, D] (the taps, then the bias).
template <bool kOdd, typename T, typename TW, int W, int VEC, int U>
__global__ __launch_bounds__(kThreads) void k_conv_bwd(ConvArgs p, int run, int token_blocks, int cblocks, float* part) {
    __shared__ float sh[kWaves - 1][(W + 1) * VEC][kWave];
    const int lane = threadIdx.x & 63;
    const int wave = wave_id();
    const int block = blockIdx.x / cblocks;
    const int64_t ch = ((int64_t)(blockIdx.x % cblocks) * kWave + lane) * VEC;
    const bool live = ch < p.D;
    const Lane ln(ch, p.D, VEC);
    const int64_t c0 = ln.at;
    if (block >= token_blocks)
        return pass_empty<kOdd, T, VEC>(p, block - token_blocks, gridDim.x / cblocks - token_blocks, p.d_sT, p.ds0, c0, ln.skip, live);
    float dw[W][VEC] = {}, db[VEC] = {};
    struct Pair {
        Raw<T, VEC> x, d;
    };
    // The first W-1 tokens of each wave's run, for the wave before it, whose last results need them: read once.
    __shared__ Pair head[kWaves][W - 1][kWave];
    const int64_t w0l = ((int64_t)block * kWaves + wave) * run;
    const bool busy = live && w0l < p.seq.total;
    const int32_t w0 = w0l < p.seq.total ? (int32_t)w0l : 0;  // (uniform)
    const int32_t w1 = w0 + run < p.seq.total ? w0 + run : p.seq.total;
    const int32_t w2 = min(w1 + W - 1, p.seq.total);  // dx of the run's last tokens needs dz up to here
    auto fetch = [&](int32_t t, Pair (&q)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t at = min(t + u, w2 - 1);
            q[u].x = row<T, VEC>(p.x, at, p, c0);
            q[u].d = row<T, VEC>(p.d_y, at, p, c0);
        }
    };
    Pair qa[U];
    if (busy) {
        fetch(w0, qa);
#pragma unroll
        for (int r = 0; r < W - 1; ++r) head[wave][r][lane] = qa[r];
    }
    __syncthreads();
    if (busy) {
        Filter<TW, W, VEC> f;
        f.load(p, c0);
        SeqPos s = seq_find(p.seq, w0);
        float win[W - 1][VEC], dzw[W - 1][VEC];  // x and dz of the W-1 tokens before the present one
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            const int32_t at = w0 - (W - 1) + r;
            Raw<T, VEC> h;
            h.clear();
            if (w0 >= s.start && w0 < s.end)
                h = at >= s.start ? row<T, VEC>(p.x, at, p, c0) : state_row<T, VEC>(p.s0, s.n, at - s.start + W - 1, p, c0);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                win[r][v] = h.get(v);
                dzw[r][v] = 0.f;
            }
        }
        T* dx = static_cast<T*>(p.dx);
        // dz of a token, its part of the sums (own: the token is one of the run's), and the gradient of the
        // input W-1 positions back, which is whole now
        auto token = [&](const Pair& q, auto silu, bool own, float (&back)[VEC]) {
            float x[VEC], z[VEC], dz[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) x[v] = q.x.get(v);
            if constexpr (silu.value) {
                pre_act<TW, W, VEC>(f, win, x, z);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float sg = sigmoid(z[v]);
                    dz[v] = q.d.get(v) * (sg * (1.f + z[v] * (1.f - sg)));
                }
            } else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) dz[v] = q.d.get(v);
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                back[v] = f.w[0][v] * dz[v];
#pragma unroll
                for (int i = 0; i < W - 1; ++i) back[v] = fmaf(f.w[W - 1 - i][v], dzw[i][v], back[v]);
            }
            if (own) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) dw[j][v] = fmaf(dz[v], win[j][v], dw[j][v]);
                    dw[W - 1][v] = fmaf(dz[v], x[v], dw[W - 1][v]);
                    db[v] += dz[v];
                }
            }
            shift_in<W, VEC>(win, x);
            shift_in<W, VEC>(dzw, dz);
        };
        // Inside one sequence: blocks of U tokens, the next two in flight, in two buffers that take turns. The
        // first W-1 results belong to the wave before; W-1 tokens behind the run complete its last ones.
        auto inside = [&](auto silu) {
            static_assert(U >= W - 1, "the first block holds the tokens that the wave before needs");
            auto block = [&](const Pair (&q)[U], int32_t t, int from) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float back[VEC];
                    token(q[u], silu, true, back);
                    if (u >= from) store_own<kOdd, T, VEC>(dx + (int64_t)(t + u - (W - 1)) * p.D + c0, back, ln.skip);
                }
            };
            Pair qb[U], tail[W - 1];
            // (behind the run the loads stay on its last token, which the cache has)
            auto ahead = [&](int32_t t, Pair (&q)[U]) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int32_t at = min(t + u, w1 - 1);
                    q[u].x = row<T, VEC>(p.x, at, p, c0);
                    q[u].d = row<T, VEC>(p.d_y, at, p, c0);
                }
            };
            ahead(w0 + U, qb);
            block(qa, w0, W - 1);
            ahead(w0 + 2 * U, qa);
            int32_t t = w0 + U;
            for (; t + U < w1; t += 2 * U) {
                block(qb, t, 0);
                ahead(t + 2 * U, qb);
                block(qa, t + U, 0);
                ahead(t + 3 * U, qa);
            }
            // the tokens behind the run: the next wave's first, or from memory for the workgroup's last wave
#pragma unroll
            for (int r = 0; r < W - 1; ++r) {
                if (wave < kWaves - 1) {
                    tail[r] = head[wave + 1][r][lane];
                } else {
                    tail[r].x = row<T, VEC>(p.x, w1 + r, p, c0);
                    tail[r].d = row<T, VEC>(p.d_y, w1 + r, p, c0);
                }
            }
            block(qb, t, 0);
#pragma unroll
            for (int r = 0; r < W - 1; ++r) {
                float back[VEC];
                token(tail[r], silu, false, back);
                store_own<kOdd, T, VEC>(dx + (int64_t)(w1 + r - (W - 1)) * p.D + c0, back, ln.skip);
            }
        };
        // where the gradient of position t of sequence s goes: the token's owner stores it, positions before
        // the first token (rows of the entering state) go by the first token's owner
        auto put = [&](int32_t t, const float (&d)[VEC]) {
            if (t >= s.start) {
                if (t >= w0 && t < w1) store_own<kOdd, T, VEC>(dx + (int64_t)t * p.D + c0, d, ln.skip);
            } else if (p.ds0 && s.start >= w0 && s.start < w1) {
                store_own<kOdd, T, VEC>(static_cast<T*>(p.ds0) + ((int64_t)s.n * (W - 1) + t - s.start + W - 1) * p.D + c0, d, ln.skip);
            }
        };
        // Around the ends of sequences: token by token, U loads ahead.
        auto across = [&](auto silu) {
#pragma unroll 1
            for (int32_t t = w0; t < w2; ++t) {
                const Pair q = qa[0];
#pragma unroll
                for (int u = 0; u + 1 < U; ++u) qa[u] = qa[u + 1];
                const int32_t at = min(t + U, w2 - 1);
                qa[U - 1].x = row<T, VEC>(p.x, at, p, c0);
                qa[U - 1].d = row<T, VEC>(p.d_y, at, p, c0);
                // behind the run only the sequence that its last token is in matters
                if (t < w1) seq_advance(p.seq, s, t);
                if (t < s.start || t >= s.end) {
                    if (p.zero && t < w1) zero_own<kOdd, T, VEC>(dx + (int64_t)t * p.D + c0, ln.skip);
                    continue;
                }
                if (t == s.start && t > w0)
#pragma unroll
                    for (int r = 0; r < W - 1; ++r) {
                        const Raw<T, VEC> h = state_row<T, VEC>(p.s0, s.n, r, p, c0);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) {
                            win[r][v] = h.get(v);
                            dzw[r][v] = 0.f;
                        }
                    }
                float back[VEC];
                token(q, silu, t < w1, back);
                put(t - (W - 1), back);
                if (t + 1 == s.end) {
                    // the last W-1 positions: no tokens behind them, but the final state's gradient
#pragma unroll
                    for (int r = 0; r < W - 1; ++r) {
                        const Raw<T, VEC> g = state_row<T, VEC>(p.d_sT, s.n, r, p, c0);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) {
                            back[v] = g.get(v);
#pragma unroll
                            for (int i = 0; i + r < W - 1; ++i) back[v] = fmaf(f.w[W - 1 - i][v], dzw[r + i][v], back[v]);
                        }
                        put(s.end - (W - 1) + r, back);
                    }
                }
            }
        };
        const bool in_one = w0 - (W - 1) >= s.start && w2 < s.end;  // (then the run is whole)
        if (p.silu) {
            if (in_one) inside(std::true_type{});
            else across(std::true_type{});
        } else {
            if (in_one) inside(std::false_type{});
            else across(std::false_type{});
        }
    }
    if (wave > 0)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
#pragma unroll
            for (int j = 0; j < W; ++j) sh[wave - 1][j * VEC + v][lane] = dw[j][v];
            sh[wave - 1][W * VEC + v][lane] = db[v];
        }
    __syncthreads();
    if (wave > 0 || !live) return;
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][v] += sh[i][j * VEC + v][lane];
            db[v] += sh[i][W * VEC + v][lane];
        }
    float* out = part + (int64_t)block * (W + 1) * p.D + c0;
#pragma unroll
    for (int j = 0; j < W; ++j) store_own<kOdd, float, VEC>(out + j * p.D, dw[j], ln.skip);
    store_own<kOdd, float, VEC>(out + W * p.D, db, ln.skip);
}

template <int COLS>
__global__ __launch_bounds__(kSumThreads) void k_conv_dw_sum(const float* part, int parts, int W, int64_t D, float* dw, float* db) {
    __shared__ float sh[kSumThreads];
    const int64_t c0 = (int64_t)blockIdx.x * COLS, i = c0 + threadIdx.x;
    const float s = sum_parts<COLS>(part, parts, (W + 1) * D, c0, sh);
    if (threadIdx.x >= COLS || i >= (W + 1) * D) return;
    const int64_t j = i / D, c = i % D;
    if (j < W) dw[c * W + j] = s;
    else if (db) db[c] = s;
}

unsigned blocks_of(int64_t D, int vec) { return (unsigned)((D + (int64_t)kWave * vec - 1) / ((int64_t)kWave * vec)); }

// Channels per lane forward: 16 bytes of them; in rows of fewer than 64 such vectors 4 bytes, so that
// short rows still use a wave's lanes; one where a row has less than that.
template <typename T> int fwd_vec(int64_t D) {
    constexpr int wide = 16 / sizeof(T), slim = 4 / sizeof(T);
    return D >= 64 * wide ? wide : (D >= slim ? slim : 1);
}
// The gradient's: 4 (8 or 16 bytes), for its filter, its sums and two windows stay in registers beside
// the loads in flight.
template <typename T> int bwd_vec(int64_t D) {
    constexpr int wide = 4, slim = 4 / sizeof(T);
    return D >= 64 * wide ? wide : (D >= slim ? slim : 1);
}

// Tokens per wave: rows of at most 16 tokens go to one wave each (which makes their state's update in
// place safe: one wave reads it before it writes it). Longer axes take 16, or 8 where there are too few for 4,096
// waves of 16 (32K x 6144 bf16: 8 tokens 145 us, 16 139, 32 153, 64 164; 8192 x 2048: 15.0, 18.6).
int fwd_run(const SeqView& s, unsigned cblocks) {
    if (!s.cu && s.T <= 16) return s.T > 0 ? s.T : 1;
    return (int64_t)s.total * cblocks >= 4096 * 16 ? 16 : 8;
}

template <typename T, typename TW, int W, int VEC>
hipError_t fwd_v(const ConvArgs& a, hipStream_t st) {
    const unsigned cb = blocks_of(a.D, VEC);
    const int run = fwd_run(a.seq, cb);
    const int tb = (int)(((int64_t)a.seq.total + (int64_t)run * kWaves - 1) / ((int64_t)run * kWaves));
    const int extra = a.sT && (a.seq.cu || a.seq.T == 0) ? empty_blocks(a.seq, kWaves) : 0;
    if (tb + extra == 0) return hipSuccess;
    if (!grid_fits((int64_t)cb * (tb + extra), kThreads)) return hipErrorInvalidConfiguration;
    const dim3 grid(cb * (unsigned)(tb + extra));
    constexpr bool kMayOdd = VEC > 1;
    const bool odd = a.D % VEC;
    if (run < 8 && odd) hipLaunchKernelGGL((k_conv_fwd<kMayOdd, T, TW, W, VEC, 1>), grid, dim3(kThreads), 0, st, a, run, tb, (int)cb);
    else if (run < 8) hipLaunchKernelGGL((k_conv_fwd<false, T, TW, W, VEC, 1>), grid, dim3(kThreads), 0, st, a, run, tb, (int)cb);
    else if (odd) hipLaunchKernelGGL((k_conv_fwd<kMayOdd, T, TW, W, VEC, 8>), grid, dim3(kThreads), 0, st, a, run, tb, (int)cb);
    else hipLaunchKernelGGL((k_conv_fwd<false, T, TW, W, VEC, 8>), grid, dim3(kThreads), 0, st, a, run, tb, (int)cb);
    return hipGetLastError();
}
template <typename T, typename TW, int W>
hipError_t fwd_t(const ConvArgs& a, hipStream_t st) {
    constexpr int wide = 16 / sizeof(T), slim = 4 / sizeof(T);
    const int v = fwd_vec<T>(a.D);
    return v == wide ? fwd_v<T, TW, W, wide>(a, st) : (v == slim ? fwd_v<T, TW, W, slim>(a, st) : fwd_v<T, TW, W, 1>(a, st));
}

// Tokens per wave in the gradient: 24, or 16 or 8 where there are too few for 2,304 waves of 24, 2,048 of 16. Longer
// runs re-read less and leave fewer partial sums, shorter ones put more waves in flight and lose less where
// sequences end inside them (2 x 16384 x 6144 bf16, W = 4: 16 tokens 239 us, 24 233, 32 242, 40 232; 30,000 tokens in
// 50 sequences: 234, 232, 236, 240; 30,000 x 512: 8 tokens 34 us, 16 33, 24 31, 40 38; 2,048 x 6144: 8 tokens 26, 16 24,
// 24 28; 4,099 x 768 fp32, W = 3: 8 tokens 15.7 us, 16 19.9).
int bwd_run(int64_t total, unsigned cblocks) {
    const int64_t n = total * cblocks;
    return n >= 24 * 2304 ? 24 : (n >= 16 * 2048 ? 16 : 8);
}
int bwd_parts(int64_t total, int run) { return (int)((total + (int64_t)run * kWaves - 1) / ((int64_t)run * kWaves)); }

template <typename T, typename TW, int W, int VEC>
hipError_t bwd_v(const ConvArgs& a, hipStream_t st) {
    const unsigned cb = blocks_of(a.D, VEC);
    const int run = bwd_run(a.seq.total, cb);
    const int parts = bwd_parts(a.seq.total, run);
    const int extra = a.ds0 && (a.seq.cu || a.seq.T == 0) ? empty_blocks(a.seq, kWaves) : 0;
    float* part = reinterpret_cast<float*>(a.ws);
    if (!grid_fits((int64_t)cb * (parts + extra), kThreads)) return hipErrorInvalidConfiguration;
    const dim3 grid(cb * (unsigned)(parts + extra));
    if (parts + extra) {
        if (a.D % VEC) hipLaunchKernelGGL((k_conv_bwd<(VEC > 1), T, TW, W, VEC, 4>), grid, dim3(kThreads), 0, st, a, run, parts, (int)cb, part);
        else hipLaunchKernelGGL((k_conv_bwd<false, T, TW, W, VEC, 4>), grid, dim3(kThreads), 0, st, a, run, parts, (int)cb, part);
    }
    const int64_t n = (W + 1) * a.D;
    const int cols = sum_cols(n);
    const dim3 sums((unsigned)((n + cols - 1) / cols));
    if (cols == 64) hipLaunchKernelGGL(k_conv_dw_sum<64>, sums, dim3(kSumThreads), 0, st, part, parts, W, a.D, a.dw, a.db);
    else hipLaunchKernelGGL(k_conv_dw_sum<16>, sums, dim3(kSumThreads), 0, st, part, parts, W, a.D, a.dw, a.db);
    return hipGetLastError();
}
template <typename T, typename TW, int W>
hipError_t bwd_t(const ConvArgs& a, hipStream_t st) {
    constexpr int slim = 4 / sizeof(T);
    const int v = bwd_vec<T>(a.D);
    return v == 4 ? bwd_v<T, TW, W, 4>(a, st) : (v == slim ? bwd_v<T, TW, W, slim>(a, st) : bwd_v<T, TW, W, 1>(a, st));
}

template <typename T, typename TW>
hipError_t fwd_w(const ConvArgs& a, hipStream_t st) {
    return a.W == 2 ? fwd_t<T, TW, 2>(a, st) : (a.W == 3 ? fwd_t<T, TW, 3>(a, st) : fwd_t<T, TW, 4>(a, st));
}
template <typename T, typename TW>
hipError_t bwd_w(const ConvArgs& a, hipStream_t st) {
    return a.W == 2 ? bwd_t<T, TW, 2>(a, st) : (a.W == 3 ? bwd_t<T, TW, 3>(a, st) : bwd_t<T, TW, 4>(a, st));
}

}  // namespace

size_t conv_bwd_ws(int64_t total, int64_t D, int W, int dtype) {
    const unsigned cb = blocks_of(D, dtype == 1 ? bwd_vec<float>(D) : bwd_vec<bf16_t>(D));
    return (size_t)bwd_parts(total, bwd_run(total, cb)) * (W + 1) * D * 4;
}

// dtype, w_dtype: gdn_dtype (0 bf16, 1 fp32); the filter in the type of x or fp32
hipError_t launch_conv_fwd(const ConvArgs& a, int dtype, int w_dtype, hipStream_t st) {
    if (dtype == 1) return fwd_w<float, float>(a, st);
    return w_dtype == 1 ? fwd_w<bf16_t, float>(a, st) : fwd_w<bf16_t, bf16_t>(a, st);
}
hipError_t launch_conv_bwd(const ConvArgs& a, int dtype, int w_dtype, hipStream_t st) {
    if (dtype == 1) return bwd_w<float, float>(a, st);
    return w_dtype == 1 ? bwd_w<bf16_t, float>(a, st) : bwd_w<bf16_t, bf16_t>(a, st);
}

}  // namespace gdn
