// gdn_gscan.hip -- the gated scan, the recurrence with a gate per channel instead of a matrix
// state per head: h_t = exp(g_t) h_{t-1} + x_t, and its gradient
//   mu_t = a_t (dh_t + mu_{t+1}),  dx_t = dh_t + mu_{t+1},  dg_t = mu_t h_{t-1},  dh_0 = mu_1,
// a = exp(g), mu behind the last token of a sequence = the gradient of its final state.
//
// Bound by memory: 3 operations per element forward and 8 backward, against 8 and 14 bytes (bf16
// with fp32 gates). So every input is read once, in a single pass over the token axis:
//   * A workgroup of eight waves holds a tile of tokens by 64 VEC channels in registers, 8 or 16 tokens to a
//     wave. A run of tokens acts on the state that enters it as c -> A c + H; the waves' pairs (A, H) meet in
//     LDS and make the tile's pair.
//   * The tile publishes its pair, gathers the state that enters it from the tiles before it (enter_tile),
//     and each wave runs its tokens again from its own entering state, now with their outputs.
//   * Tiles are handed out in the order of the token axis by a counter, so a tile only ever waits for
//     tiles that are running or done, and those publish their pairs before they wait themselves.
//   * What is added to what is fixed by the tile's place, not by who was ready first, so results are
//     the same bits every time: the state entering a group of tiles comes from the group before it
//     as one published value, the tiles inside the group combine the pairs since then.
// Published words carry their own mark (all ones: not there yet), so no other ordering of memory is
// needed; a small launch clears them first. The gradient runs the same from the other end, and
// recomputes h inside its tile in fp32 from the state that the forward kept for every 64th token.
#include "gdn_layer.h"
#include "gdn_vec.h"

namespace gdn {

namespace {

constexpr int kWaves = 8;              // waves of a tile
constexpr int kThreads = kWaves * kWave;
constexpr int kMaxSpins = 1 << 20;     // (about a second) a wait gives up with NaN rather than hang

struct Chain {
    uint32_t* ticket;
    uint64_t* pairs;  // [tiles, D], in the order of the chain: A in the high word, H in the low one
    uint32_t* carry;  // [groups, D]: the state that enters the group
    int group;        // tiles between two published entering states
};

// A c + H. A with its sign bit set marks a run in which a sequence starts: nothing of c passes, whatever it
// holds. c = 0 passes nothing either, also where growing gates took A to infinity.
__device__ __forceinline__ float pass_on(float A, float H, float c) {
    return (__float_as_int(A) < 0 || c == 0.f) ? H : fmaf(A, c, H);
}
// (A, H) followed by (a, h).
__device__ __forceinline__ void then(float& A, float& H, float a, float h) {
    H = pass_on(a, h, H);
    A = __float_as_int(a) < 0 ? a : A * a;
}
// What several tiles do together to a state. The gates' product over them may leave fp32's range, though no tile's
// does, where growth follows decay or the state is small: its exponent is kept apart. In range it is the same bits as
// the plain product (64K x 64: 23.0 us, with the plain product 22.8; 32K x 2048 104 with either).
struct Span {
    float m = 1.f, H = 0.f;  // A = m 2^e
    int e = 0;
};
__device__ __forceinline__ void then(Span& s, float a, float h) {
    s.H = pass_on(a, h, s.H);
    if (__float_as_int(a) < 0) {
        s.m = -1.f;
    } else {
        s.m *= __builtin_amdgcn_frexp_mantf(a);  // (16 factors of 1/2 or more at most: no underflow)
        s.e += __builtin_amdgcn_frexp_expf(a);
    }
}
// m in [1, 2), or zero (whose exponent says nothing), or what passes nothing on.
__device__ __forceinline__ void settle(Span& s) {
    s.e = s.m == 0.f ? 0 : s.e + __builtin_amdgcn_frexp_expf(s.m) - 1;
    s.m = 2.f * __builtin_amdgcn_frexp_mantf(s.m);
}
// m times c 2^e, of a settled span: either is out of range only if A c is.
__device__ __forceinline__ float pass_on(const Span& s, float c) {
    const float h = fmaf(s.m, __builtin_amdgcn_ldexpf(c, s.e), s.H);
    return __float_as_int(s.m) < 0 || c == 0.f ? s.H : h;
}

// Bits that are never all ones.
__device__ __forceinline__ uint32_t mark(float x) { return x == x ? __float_as_uint(x) : 0x7FC00000u; }

template <typename W>
__device__ __forceinline__ W peek(const W* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W>
__device__ __forceinline__ void publish(W* p, W v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What the places from .. to - 1 of the chain do together to a state in channel c. Whole waves call it; `live`:
// this lane's channel exists. False if the wait was given up.
__device__ __forceinline__ bool gather(const Chain& ch, int64_t D, int64_t c, bool live, int from, int to, Span& s) {
    constexpr int kAhead = 4;
    for (int k = from; k < to; k += kAhead) {
        uint64_t v[kAhead];
        for (int spins = 0;;) {
            bool ok = true;
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (k + u < to) v[u] = live ? peek(ch.pairs + (int64_t)(k + u) * D + c) : 0;
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (k + u < to) ok = ok && v[u] != ~0ull;
            if (__all(ok)) break;
            if (++spins > kMaxSpins) return false;
            __builtin_amdgcn_s_sleep(1);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (k + u < to) then(s, __uint_as_float((uint32_t)(v[u] >> 32)), __uint_as_float((uint32_t)v[u]));
    }
    return true;
}
// The same places' pairs, all there by now, applied to the state one after the other.
__device__ __forceinline__ float in_turn(const Chain& ch, int64_t D, int64_t c, bool live, int from, int to, float s) {
#pragma unroll 4
    for (int k = from; k < to; ++k) {
        const uint64_t v = live ? peek(ch.pairs + (int64_t)k * D + c) : 0;
        s = pass_on(__uint_as_float((uint32_t)(v >> 32)), __uint_as_float((uint32_t)v), s);
    }
    return s;
}

// The state (or adjoint) that enters each of the tile's waves, for all channels of the block, into `cin`, from the
// waves' pairs in `agg`. Place `pos` of the chain; `first`: the place in which the sequence that enters it starts
// (pos: none enters). Publishes the tile's pair before it waits for anything. All threads call it: the places to
// look back over are split among kThreads / CH parts of the workgroup, so that each thread has few loads in flight
// beside its tokens. Ends with a barrier.
template <bool kRev, bool kChain, int CH>
__device__ __forceinline__ void enter_tile(const float2 (*agg)[CH], float2 (*mid)[CH], int (*mid_e)[CH], float (*cin)[CH], const Chain& ch,
                                           int64_t D, int64_t cbase, int pos, int tiles, int first) {
    constexpr int kParts = kThreads / CH;
    const int t = threadIdx.x % CH;
    const int part = __builtin_amdgcn_readfirstlane((int)threadIdx.x / CH);
    const int64_t c = cbase + t;
    const bool live = c < D;
    const float lost = __uint_as_float(0x7FC00000u);
    float s = 0.f, A = 1.f, H = 0.f;
    if constexpr (kChain) {
        if (part == 0) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float2 q = agg[kRev ? kWaves - 1 - w : w][t];
                then(A, H, q.x, q.y);
            }
            if (live && pos + 1 < tiles)
                publish(ch.pairs + (int64_t)pos * D + c, ((uint64_t)__float_as_uint(A) << 32) | mark(H));
        }
        if (first < pos) {
            const int group = pos / ch.group, begin = group * ch.group;
            const bool carried = first < begin;  // the state comes from the group before
            const int from = carried ? begin : first, each = (pos - from + kParts - 1) / kParts;
            const uint32_t* word = ch.carry + (int64_t)group * D + c;
            uint32_t v = 0;
            if (part == 0 && carried && live) v = peek(word);
            Span span;
            const int lo = min(from + part * each, pos), hi = min(lo + each, pos);
            if (!gather(ch, D, c, live, lo, hi, span)) {
                span.m = -1.f;
                span.H = lost;
            }
            settle(span);
            mid[part][t] = make_float2(span.m, span.H);
            mid_e[part][t] = span.e;
            __syncthreads();
            if (part == 0) {
                Span spans[kParts];  // (read before the wait: what is behind it is on every later group's way)
#pragma unroll
                for (int q = 0; q < kParts; ++q) spans[q] = Span{mid[q][t].x, mid[q][t].y, mid_e[q][t]};
                for (int spins = 0; !__all(v != ~0u);) {
                    if (++spins > kMaxSpins) {
                        v = __float_as_uint(lost);
                        break;
                    }
                    __builtin_amdgcn_s_sleep(1);
                    if (live) v = peek(word);
                }
                const float s0 = __uint_as_float(v);
                s = s0;
#pragma unroll
                for (int q = 0; q < kParts; ++q) s = pass_on(spans[q], s);
                // What the inputs leave behind a part's tiles from a zero state may pass the range where the true state
                // does not (they cancelled the state that entered, and growth followed).
                if (__any(fabsf(s0) < __builtin_inff() && !(fabsf(s) < __builtin_inff()))) s = in_turn(ch, D, c, live, from, pos, s0);
            }
        }
        if (part == 0 && live && (pos + 1) % ch.group == 0 && pos + 1 < tiles)
            publish(ch.carry + (int64_t)((pos + 1) / ch.group) * D + c, mark(pass_on(A, H, s)));
        asm volatile("" ::: "memory");  // the waves' pairs are read again rather than held through the wait
    }
    if (part == 0)
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float2 q = agg[kRev ? kWaves - 1 - w : w][t];
            cin[kRev ? kWaves - 1 - w : w][t] = s;
            s = pass_on(q.x, q.y, s);
        }
    __syncthreads();
}

template <int VEC>
__device__ __forceinline__ void load_f(const float* p, float (&x)[VEC]) {
    const Raw<float, VEC> r = load_raw<float, VEC>(p);
#pragma unroll
    for (int v = 0; v < VEC; ++v) x[v] = r.get(v);
}
template <int VEC>
__device__ __forceinline__ void state_of(const float* s, int32_t n, int64_t D, int64_t c, float (&x)[VEC]) {
    if (s) {
        load_f<VEC>(s + (int64_t)n * D + c, x);
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) x[v] = 0.f;
    }
}

// Sequences without tokens: their state (or its gradient) passes through, by the workgroups behind the tiles: number
// `block` of `blocks`.
template <bool kOdd, int VEC>
__device__ void pass_empty(const GScanArgs& p, int block, int blocks, const float* in, float* out, int64_t c, int skip, bool live) {
    for_each_empty(p.seq, block * kWaves + wave_id(), blocks * kWaves, [&](int32_t n) {
        if (!live) return;
        float x[VEC];
        state_of<VEC>(in, n, p.D, c, x);
        store_own<kOdd, float, VEC>(out + (int64_t)n * p.D + c, x, skip);
    });
}

// This workgroup's item: tile * cblocks + channel block, in the order in which workgroups got here.
__device__ __forceinline__ int take(const Chain& ch, bool chain, int* sh) {
    if (!chain) return blockIdx.x;
    if (threadIdx.x == 0) *sh = (int)__hip_atomic_fetch_add(ch.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*sh);
}

// A lane's first channel, counted from the block's (below zero where the vector is moved back, Lane). Lanes behind
// the row load a vector inside it too.
template <bool kOdd, int VEC>
__device__ __forceinline__ int first_channel(int64_t D, int64_t cbase, bool live, int lane, int skip) {
    if (live) return lane * VEC - skip;
    return kOdd && cbase + VEC > D ? (int)(D - VEC - cbase) : 0;
}

// `span`: tokens of a tile. A chain's tiles are full (kWaves kTokens); without a chain a tile is a whole row, or
// the only one.
template <bool kOdd, typename TX, typename TG, int VEC, int kTokens, bool kChain>
__global__ __launch_bounds__(kThreads) void k_gscan_fwd(GScanArgs p, int tiles, int span, int cblocks, Chain ch) {
    constexpr int kKeep = kScanTile / kTokens;  // waves between two kept states
    constexpr int CH = kWave * VEC;
    __shared__ __attribute__((aligned(16))) float2 agg[kWaves][CH];
    __shared__ __attribute__((aligned(16))) float cin[kWaves][CH];
    __shared__ __attribute__((aligned(16))) float2 mid[kChain ? kThreads / CH : 1][CH];
    __shared__ int mid_e[kChain ? kThreads / CH : 1][CH];
    __shared__ int sh_id, sh_first;
    const int id = take(ch, kChain, &sh_id);
    const int tile = id / cblocks, lane = threadIdx.x & 63, wave = wave_id();
    const int64_t cbase = (int64_t)(id % cblocks) * CH;
    const bool live = cbase + lane * VEC < p.D;
    const Lane ln(cbase + lane * VEC, p.D, VEC);
    const int skip = kOdd ? ln.skip : 0;
    const int lo = first_channel<kOdd, VEC>(p.D, cbase, live, lane, skip);
    const int64_t c = cbase + lo;
    if (tile >= tiles) return pass_empty<kOdd, VEC>(p, tile - tiles, gridDim.x / cblocks - tiles, p.s0, p.sT, c, skip, live);
    const int32_t t0 = tile * span, t1 = p.seq.total - t0 < span ? p.seq.total : t0 + span;
    const int32_t w0 = t1 - t0 < wave * kTokens ? t1 : t0 + wave * kTokens;
    const int32_t w1 = t1 - w0 < kTokens ? t1 : w0 + kTokens;
    Raw<TX, VEC> x[kTokens];
    Raw<TG, VEC> g[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int64_t at = (int64_t)min(w0 + i, p.seq.total - 1) * p.D + cbase;
        x[i] = load_raw<TX, VEC>(static_cast<const TX*>(p.x) + at + lo);
        g[i] = load_raw<TG, VEC>(static_cast<const TG*>(p.g) + at + lo);
    }
    const SeqPos s0 = seq_find(p.seq, min(w0, p.seq.total - 1));
    // all of the wave's tokens inside one sequence, none of them its first
    const bool inside = w0 > s0.start && w0 + kTokens <= s0.end;
    if (kChain && threadIdx.x == 0) sh_first = w0 >= s0.start && w0 < s0.end ? s0.start / span : tile;
    float A[VEC], H[VEC], last[VEC] = {};  // last: the entering state of the last sequence that starts here
    int32_t last_n = -1;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        A[v] = 1.f;
        H[v] = 0.f;
    }
    auto feed = [&](int i) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float a = fast_exp(g[i].get(v));
            H[v] = fmaf(a, H[v], x[i].get(v));
            A[v] *= a;
        }
    };
    if (inside) {
#pragma unroll
        for (int i = 0; i < kTokens; ++i) feed(i);
    } else {
        SeqPos s = s0;
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            const int32_t t = w0 + i;
            if (t >= w1) break;
            seq_advance(p.seq, s, t);
            if (t < s.start || t >= s.end) continue;
            if (t == s.start) {
                last_n = s.n;
                state_of<VEC>(p.s0, s.n, p.D, c, last);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    A[v] = -1.f;
                    H[v] = last[v];
                }
            }
            feed(i);
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v)
        if (!kOdd || (live && v >= skip)) agg[wave][lo + v] = make_float2(A[v], H[v]);
    __syncthreads();
    enter_tile<false, kChain, CH>(agg, mid, mid_e, cin, ch, p.D, cbase, tile, tiles, kChain ? __builtin_amdgcn_readfirstlane(sh_first) : tile);
    float h[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = cin[wave][kOdd ? max(lo + v, 0) : lo + v];
    if (!live || w0 >= w1) return;
    if (p.states && wave % kKeep == 0)
        store_own<kOdd, float, VEC>(p.states + (int64_t)(w0 / kScanTile) * p.D + c, h, skip);
    TX* out = static_cast<TX*>(p.h);
    auto step = [&](int i) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = fmaf(fast_exp(g[i].get(v)), h[v], x[i].get(v));
        if (out) store_own<kOdd, TX, VEC>(out + ((int64_t)(w0 + i) * p.D + cbase) + lo, h, skip);
    };
    if (inside) {
#pragma unroll
        for (int i = 0; i < kTokens; ++i) step(i);
        if (p.sT && w1 == s0.end) store_own<kOdd, float, VEC>(p.sT + (int64_t)s0.n * p.D + c, h, skip);
        return;
    }
    SeqPos s = s0;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int32_t t = w0 + i;
        if (t >= w1) break;
        seq_advance(p.seq, s, t);
        if (t < s.start || t >= s.end) {
            if (p.zero && out) zero_own<kOdd, TX, VEC>(out + ((int64_t)t * p.D + cbase) + lo, skip);
            continue;
        }
        if (t == s.start) {
            // final_state may be initial_state: the last sequence's end may lie in another workgroup, which may
            // have written it by now, so its start was kept; the others end in this wave, behind this read
            if (s.n == last_n) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) h[v] = last[v];
            } else {
                state_of<VEC>(p.s0, s.n, p.D, c, h);
            }
        }
        step(i);
        if (p.sT && t + 1 == s.end) store_own<kOdd, float, VEC>(p.sT + (int64_t)s.n * p.D + c, h, skip);
    }
}

template <bool kOdd, typename TX, typename TG, int VEC, int kTokens, bool kChain>
__global__ __launch_bounds__(kThreads) void k_gscan_bwd(GScanArgs p, int tiles, int span, int cblocks, Chain ch) {
    static_assert(kWaves * kTokens % kScanTile == 0, "a tile starts at a kept state");
    constexpr int CH = kWave * VEC;
    __shared__ __attribute__((aligned(16))) float2 agg[kWaves][CH];  // the forward's pairs, then the adjoint's
    __shared__ __attribute__((aligned(16))) float2 ragg[kWaves][CH];
    __shared__ __attribute__((aligned(16))) float cin[kWaves][CH];
    __shared__ __attribute__((aligned(16))) float rin[kWaves][CH];
    __shared__ __attribute__((aligned(16))) float2 mid[kChain ? kThreads / CH : 1][CH];
    __shared__ int mid_e[kChain ? kThreads / CH : 1][CH];
    __shared__ int sh_id, sh_first;
    const int id = take(ch, kChain, &sh_id);
    const int pos = id / cblocks, tile = tiles - 1 - pos, lane = threadIdx.x & 63, wave = wave_id();
    const int64_t cbase = (int64_t)(id % cblocks) * CH;
    const bool live = cbase + lane * VEC < p.D;
    const Lane ln(cbase + lane * VEC, p.D, VEC);
    const int skip = kOdd ? ln.skip : 0;
    const int lo = first_channel<kOdd, VEC>(p.D, cbase, live, lane, skip);
    const int64_t c = cbase + lo;
    if (pos >= tiles) return pass_empty<kOdd, VEC>(p, pos - tiles, gridDim.x / cblocks - tiles, p.d_sT, p.ds0, c, skip, live);
    const int32_t t0 = tile * span, t1 = p.seq.total - t0 < span ? p.seq.total : t0 + span;
    const int32_t w0 = t1 - t0 < wave * kTokens ? t1 : t0 + wave * kTokens;
    const int32_t w1 = t1 - w0 < kTokens ? t1 : w0 + kTokens;
    Raw<TX, VEC> x[kTokens], d[kTokens];
    Raw<TG, VEC> g[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int64_t at = (int64_t)min(w0 + i, p.seq.total - 1) * p.D + cbase;
        g[i] = load_raw<TG, VEC>(static_cast<const TG*>(p.g) + at + lo);
        x[i] = load_raw<TX, VEC>(static_cast<const TX*>(p.x) + at + lo);
        d[i] = load_raw<TX, VEC>(static_cast<const TX*>(p.d_h) + at + lo);
    }
    const SeqPos s0 = seq_find(p.seq, min(w0, p.seq.total - 1));
    // all of the wave's tokens inside one sequence, neither its first nor its last among them
    const bool inside = w0 > s0.start && w0 + kTokens < s0.end;
    if (kChain && threadIdx.x == kThreads - kWave) {
        // the chain comes from the sequence that goes on behind the tile
        const SeqPos e = seq_find(p.seq, t1 - 1);
        sh_first = t1 > e.start && t1 < e.end ? tiles - 1 - (e.end - 1) / span : pos;
    }
    float A[VEC], H[VEC], R[VEC], M[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        A[v] = R[v] = 1.f;
        H[v] = M[v] = 0.f;
    }
    if (inside) {
#pragma unroll
        for (int i = 0; i < kTokens; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float a = fast_exp(g[i].get(v));
                H[v] = fmaf(a, H[v], x[i].get(v));
                A[v] *= a;
            }
#pragma unroll
        for (int i = kTokens - 1; i >= 0; --i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) M[v] = fast_exp(g[i].get(v)) * (d[i].get(v) + M[v]);
#pragma unroll
        for (int v = 0; v < VEC; ++v) R[v] = A[v];
    } else {
        SeqPos s = s0;
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            const int32_t t = w0 + i;
            if (t >= w1) break;
            seq_advance(p.seq, s, t);
            if (t < s.start || t >= s.end) continue;
            if (t == s.start) {
                state_of<VEC>(p.s0, s.n, p.D, c, H);
#pragma unroll
                for (int v = 0; v < VEC; ++v) A[v] = -1.f;
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float a = fast_exp(g[i].get(v));
                H[v] = fmaf(a, H[v], x[i].get(v));
                A[v] *= a;
            }
        }
        SeqPos e = s;
        if (w0 < w1) e = seq_find(p.seq, w1 - 1);
#pragma unroll
        for (int i = kTokens - 1; i >= 0; --i) {
            const int32_t t = w0 + i;
            if (t >= w1) continue;
            seq_retreat(p.seq, e, t);
            if (t < e.start || t >= e.end) continue;
            if (t + 1 == e.end) {
                state_of<VEC>(p.d_sT, e.n, p.D, c, M);
#pragma unroll
                for (int v = 0; v < VEC; ++v) R[v] = -1.f;
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float a = fast_exp(g[i].get(v));
                M[v] = a * (d[i].get(v) + M[v]);
                R[v] *= a;
            }
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        if (!kOdd || (live && v >= skip)) {
            agg[wave][lo + v] = make_float2(A[v], H[v]);
            ragg[wave][lo + v] = make_float2(R[v], M[v]);
        }
    }
    __syncthreads();
    if (threadIdx.x >= kThreads - CH) {
        // the states that enter the waves, from the tile's kept one
        const int t = threadIdx.x - (kThreads - CH);
        // (none where nothing enters a tile from outside)
        float h = p.states && cbase + t < p.D ? p.states[(int64_t)(t0 / kScanTile) * p.D + cbase + t] : 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            cin[w][t] = h;
            h = pass_on(agg[w][t].x, agg[w][t].y, h);
        }
    }
    enter_tile<true, kChain, CH>(ragg, mid, mid_e, rin, ch, p.D, cbase, pos, tiles, kChain ? __builtin_amdgcn_readfirstlane(sh_first) : pos);
    if (!live || w0 >= w1) return;
    float h[VEC], mu[VEC], before[kTokens][VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        h[v] = cin[wave][kOdd ? max(lo + v, 0) : lo + v];
        mu[v] = rin[wave][kOdd ? max(lo + v, 0) : lo + v];
    }
    TX* dx = static_cast<TX*>(p.dx);
    TG* dg = static_cast<TG*>(p.dg);
    auto ahead = [&](int i) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            before[i][v] = h[v];
            h[v] = fmaf(fast_exp(g[i].get(v)), h[v], x[i].get(v));
        }
    };
    auto back = [&](int i) {
        float lam[VEC], dgv[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            lam[v] = d[i].get(v) + mu[v];
            mu[v] = fast_exp(g[i].get(v)) * lam[v];
            dgv[v] = mu[v] * before[i][v];
        }
        const int64_t at = (int64_t)(w0 + i) * p.D + cbase;
        store_own<kOdd, TX, VEC>(dx + at + lo, lam, skip);
        store_own<kOdd, TG, VEC>(dg + at + lo, dgv, skip);
    };
    if (inside) {
#pragma unroll
        for (int i = 0; i < kTokens; ++i) ahead(i);
#pragma unroll
        for (int i = kTokens - 1; i >= 0; --i) back(i);
        return;
    }
    SeqPos s = s0;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int32_t t = w0 + i;
        if (t >= w1) break;
        seq_advance(p.seq, s, t);
        if (t < s.start || t >= s.end) continue;
        if (t == s.start) state_of<VEC>(p.s0, s.n, p.D, c, h);
        ahead(i);
    }
    SeqPos e = seq_find(p.seq, w1 - 1);
#pragma unroll
    for (int i = kTokens - 1; i >= 0; --i) {
        const int32_t t = w0 + i;
        if (t >= w1) continue;
        seq_retreat(p.seq, e, t);
        if (t < e.start || t >= e.end) {
            const int64_t at = (int64_t)t * p.D + cbase;
            if (p.zero) {
                zero_own<kOdd, TX, VEC>(dx + at + lo, skip);
                zero_own<kOdd, TG, VEC>(dg + at + lo, skip);
            }
            continue;
        }
        if (t + 1 == e.end) state_of<VEC>(p.d_sT, e.n, p.D, c, mu);
        back(i);
        if (p.ds0 && t == e.start) store_own<kOdd, float, VEC>(p.ds0 + (int64_t)e.n * p.D + c, mu, skip);
    }
}

// Short sequences (decoding): a wave per sequence and block of channels walks the tokens; one launch, no workspace.
constexpr int kRowThreads = 256;
constexpr int kRowAhead = 8;  // tokens loaded ahead in a sequence of two such blocks or more (0.21 -> 0.11 us a token)
template <bool kOdd, typename TX, typename TG, int VEC>
__global__ __launch_bounds__(kRowThreads) void k_gscan_rows(GScanArgs p, int cblocks) {
    const int64_t item = (int64_t)blockIdx.x * (kRowThreads / kWave) + wave_id();
    const int64_t nl = item / cblocks;
    if (nl >= p.seq.N) return;
    const int64_t c0 = ((item % cblocks) * kWave + (threadIdx.x & 63)) * VEC;
    if (c0 >= p.D) return;
    const Lane ln(c0, p.D, VEC);
    const int64_t c = ln.at;
    const int skip = kOdd ? ln.skip : 0;
    const SeqPos s = seq_at(p.seq, (int32_t)nl);
    float h[VEC];
    state_of<VEC>(p.s0, s.n, p.D, c, h);
    const TX* x = static_cast<const TX*>(p.x) + c;
    const TG* g = static_cast<const TG*>(p.g) + c;
    TX* out = static_cast<TX*>(p.h);
    auto step = [&](int32_t t, const Raw<TX, VEC>& xt, const Raw<TG, VEC>& gt) {
        if (p.states && t % kScanTile == 0) store_own<kOdd, float, VEC>(p.states + (int64_t)(t / kScanTile) * p.D + c, h, skip);
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = fmaf(fast_exp(gt.get(v)), h[v], xt.get(v));
        if (out) store_own<kOdd, TX, VEC>(out + (int64_t)t * p.D + c, h, skip);
    };
    int32_t t = s.start;
    if (s.end - t >= 2 * kRowAhead) {
        Raw<TX, VEC> nx[kRowAhead];
        Raw<TG, VEC> ng[kRowAhead];
        auto fetch = [&](int32_t from) {
#pragma unroll
            for (int u = 0; u < kRowAhead; ++u) {
                const int64_t at = (int64_t)min(from + u, s.end - 1) * p.D;
                nx[u] = load_raw<TX, VEC>(x + at);
                ng[u] = load_raw<TG, VEC>(g + at);
            }
        };
        fetch(t);
        for (; s.end - t >= kRowAhead; t += kRowAhead) {
            Raw<TX, VEC> xt[kRowAhead];
            Raw<TG, VEC> gt[kRowAhead];
#pragma unroll
            for (int u = 0; u < kRowAhead; ++u) {
                xt[u] = nx[u];
                gt[u] = ng[u];
            }
            fetch(t + kRowAhead);
#pragma unroll
            for (int u = 0; u < kRowAhead; ++u) step(t + u, xt[u], gt[u]);
        }
    }
    Raw<TX, VEC> nx;
    Raw<TG, VEC> ng;
    if (t < s.end) {
        nx = load_raw<TX, VEC>(x + (int64_t)t * p.D);
        ng = load_raw<TG, VEC>(g + (int64_t)t * p.D);
    }
    for (; t < s.end; ++t) {
        const Raw<TX, VEC> xt = nx;
        const Raw<TG, VEC> gt = ng;
        if (t + 1 < s.end) {
            nx = load_raw<TX, VEC>(x + (int64_t)(t + 1) * p.D);
            ng = load_raw<TG, VEC>(g + (int64_t)(t + 1) * p.D);
        }
        step(t, xt, gt);
    }
    if (p.sT) store_own<kOdd, float, VEC>(p.sT + (int64_t)s.n * p.D + c, h, skip);
    if (p.zero && out) {  // in front of the first sequence and behind the last one
        for (int32_t t0 = 0; nl == 0 && t0 < s.start; ++t0) zero_own<kOdd, TX, VEC>(out + (int64_t)t0 * p.D + c, skip);
        for (int32_t t0 = s.end; nl == p.seq.N - 1 && t0 < p.seq.total; ++t0) zero_own<kOdd, TX, VEC>(out + (int64_t)t0 * p.D + c, skip);
    }
}

// A wave for every sequence: rows of up to 16 tokens, and packed batches that hold no more tokens than sequences
// (one each, as decoding has them) and at most 512 tokens. The lengths are on the device, so what bounds the loss is the longest
// walk that may be among them: a token costs 0.11 us there, and tiles take 13 to 20 us (x 2048 channels: 256
// sequences of a token 3.7 us by rows, 20 by tiles; 128 of one and one of 400 50 and 21; 1,024 of one and one of 2,048
// 285 and 33).
constexpr int kRowTokens = 512;
bool by_rows(const SeqView& s) { return s.cu ? s.total <= s.N && s.total <= kRowTokens : s.T <= 16; }

// Whether a tile of `span` tokens takes every row, or the whole of a packed batch: then no state passes from tile to
// tile (256 rows of 64 x 2048: 52 us, as a chain of full tiles 61; 16 rows of 24: 5.5 and 10).
bool one_tile(const SeqView& s, int span) { return (s.cu ? s.total : s.T) <= span; }

// Channels per lane and tokens per wave (with a chain). Forward 2 channels by 16 tokens: as many registers as 4 by 8,
// for tiles of half the channels and twice the tokens, which look back over half as many pairs and hand half as many
// states on (32K x 2048 fp32 gates 104 us, 4 by 8 111, 4 by 16 112, 2 by 32 111; 256K x 1024 376 and 429). The gradient
// 4 by 8, with more bytes a tile to each pair (2 by 16 was 4% slower). One channel in rows that would not fill a wave
// otherwise, 16 tokens (64K x 64: 8 tokens 35 us, 16 23, 32 17, but 2,000 x 64: 7.5, 8.6, 13).
constexpr int kFwdTokens = 16;
template <int VEC>
constexpr int bwd_tokens() { return VEC == 1 ? 16 : 8; }

// Clears a chain: the ticket to zero, every word behind it to "not there yet".
__global__ __launch_bounds__(256) void k_clear(u32x4* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const uint32_t v = i < 16 ? 0u : ~0u;
        p[i] = u32x4{v, v, v, v};
    }
}

int tiles_of(int64_t total, int tile) { return (int)((total + tile - 1) / tile); }
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Rows of fewer channels have one channel per lane.
constexpr int64_t kSlim = 128;

// A chain in the workspace: 256 bytes for the ticket, the pairs, the groups' states.
constexpr int kMinGroup = 8;
size_t chain_bytes(size_t tiles, int64_t D) {
    const size_t groups = (tiles + kMinGroup - 1) / kMinGroup;
    return 256 + align256(tiles * D * 8) + align256(groups * D * 4);
}
// A group hands its state on in about a microsecond, one group after the other, while a tile looks back over half
// a group's pairs. From `wide` channels on the memory takes longer than the chain, and small groups read less; with
// fewer, longer groups keep the chain short. us forward / backward in groups of 8, 16, 32 and 64 tiles:
//   64K x 4096   371 / 640   373 / 643   377 / 686   396 / 709
//   32K x 2048   106 / 173   106 / 176   108 / 179   114 / 199
//   64K x 1024   112 / 182   108 / 177   109 / 184   118 / 198
//   64K x  512    71 / 128    57 / 103    58 / 103    61 / 110
//   64K x  256    64 / 111    45 /  73    38 /  58    39 /  61
//   64K x   64    62 /  67    39 /  44    28 /  33    23 /  29
// Rows of fewer tiles have a shorter chain and care less (16 rows of 4096 x 256: 36 / 54, 35 / 54, 36 / 56, 36 / 57).
hipError_t make_chain(unsigned char* ws, size_t tiles, int64_t D, int64_t wide, Chain& ch, hipStream_t st) {
    const size_t bytes = chain_bytes(tiles, D);
    ch.group = D >= wide ? kMinGroup : (D >= 512 ? 16 : (D >= kSlim ? 32 : 64));
    ch.ticket = reinterpret_cast<uint32_t*>(ws);
    ch.pairs = reinterpret_cast<uint64_t*>(ws + 256);
    ch.carry = reinterpret_cast<uint32_t*>(ws + 256 + align256(tiles * D * 8));
    const int64_t n = (int64_t)(bytes / 16), blocks = (n + 1023) / 1024;
    hipLaunchKernelGGL(k_clear, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, reinterpret_cast<u32x4*>(ws), n);
    return hipGetLastError();
}

template <bool kOdd, typename TX, typename TG, int VEC, int TOK>
hipError_t fwd_tiles(const GScanArgs& a, int cb, hipStream_t st) {
    const int tiles = tiles_of(a.seq.total, kWaves * TOK);
    const int extra = a.sT && a.seq.cu ? empty_blocks(a.seq, kWaves) : 0;
    Chain ch{};
    if (!grid_fits((int64_t)(tiles + extra) * cb, kThreads)) return hipErrorInvalidConfiguration;
    if (hipError_t e = make_chain(a.ws, tiles, a.D, 4096, ch, st)) return e;
    hipLaunchKernelGGL((k_gscan_fwd<kOdd, TX, TG, VEC, TOK, true>), dim3((unsigned)(tiles + extra) * (unsigned)cb),
                       dim3(kThreads), 0, st, a, tiles, kWaves * TOK, cb, ch);
    return hipGetLastError();
}

// Without a chain, in one launch: rows that are a tile each, or a packed batch that is one.
template <bool kOdd, typename TX, typename TG, int VEC, int TOK>
hipError_t fwd_single(GScanArgs a, int cb, hipStream_t st) {
    const int tiles = a.seq.cu ? (a.seq.total > 0) : a.seq.N;
    const int extra = a.sT && a.seq.cu ? empty_blocks(a.seq, kWaves) : 0;
    if (tiles + extra == 0) return hipSuccess;
    if (!grid_fits((int64_t)(tiles + extra) * cb, kThreads)) return hipErrorInvalidConfiguration;
    a.states = nullptr;  // nothing enters a tile from outside: the gradient needs none
    hipLaunchKernelGGL((k_gscan_fwd<kOdd, TX, TG, VEC, TOK, false>), dim3((unsigned)(tiles + extra) * (unsigned)cb),
                       dim3(kThreads), 0, st, a, tiles, a.seq.cu ? kWaves * TOK : a.seq.T, cb, Chain{});
    return hipGetLastError();
}

template <bool kOdd, typename TX, typename TG, int VEC>
hipError_t fwd_v(const GScanArgs& a, hipStream_t st) {
    const int cb = (int)((a.D + kWave * VEC - 1) / (kWave * VEC));
    if (by_rows(a.seq)) {
        const int64_t items = (int64_t)a.seq.N * cb, per = kRowThreads / kWave;
        if (!grid_fits((items + per - 1) / per, kRowThreads)) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((k_gscan_rows<kOdd, TX, TG, VEC>), dim3((unsigned)((items + per - 1) / per)), dim3(kRowThreads), 0, st, a, cb);
        return hipGetLastError();
    }
    // Kept states lie 64 tokens apart, so rows that need them and have more take the chain.
    if (one_tile(a.seq, kScanTile)) return fwd_single<kOdd, TX, TG, VEC, 8>(a, cb, st);
    if (!a.states && one_tile(a.seq, 2 * kScanTile)) return fwd_single<kOdd, TX, TG, VEC, 16>(a, cb, st);
    return fwd_tiles<kOdd, TX, TG, VEC, kFwdTokens>(a, cb, st);
}

template <typename TX, typename TG>
hipError_t fwd_t(const GScanArgs& a, hipStream_t st) {
    if (a.D < kSlim) return fwd_v<false, TX, TG, 1>(a, st);
    return a.D % 2 ? fwd_v<true, TX, TG, 2>(a, st) : fwd_v<false, TX, TG, 2>(a, st);
}
template <bool kOdd, typename TX, typename TG, int VEC>
hipError_t bwd_v(GScanArgs a, bool have, hipStream_t st) {
    const int cb = (int)((a.D + kWave * VEC - 1) / (kWave * VEC));
    constexpr int kTok = bwd_tokens<VEC>();
    const bool single = one_tile(a.seq, kScanTile), rows = single && !a.seq.cu;  // (as forward)
    const int tiles = rows ? (a.seq.T > 0 ? a.seq.N : 0) : tiles_of(a.seq.total, single ? kScanTile : kWaves * kTok);
    const int extra = a.ds0 && (a.seq.cu || a.seq.T == 0) ? empty_blocks(a.seq, kWaves) : 0;
    if (tiles + extra == 0) return hipSuccess;
    if (!grid_fits((int64_t)(tiles + extra) * cb, kThreads)) return hipErrorInvalidConfiguration;
    if (single) {
        a.states = nullptr;  // nothing enters a tile from outside
    } else if (!have && tiles) {
        a.states = reinterpret_cast<float*>(a.ws + chain_bytes(tiles_of(a.seq.total, kScanTile), a.D));
        GScanArgs f = a;
        f.h = nullptr;
        f.sT = nullptr;
        if (hipError_t e = fwd_t<TX, TG>(f, st)) return e;
    }
    const dim3 grid((unsigned)(tiles + extra) * (unsigned)cb);
    if (single) {
        hipLaunchKernelGGL((k_gscan_bwd<kOdd, TX, TG, VEC, 8, false>), grid, dim3(kThreads), 0, st, a, tiles,
                           rows && a.seq.T ? a.seq.T : kScanTile, cb, Chain{});
        return hipGetLastError();
    }
    Chain ch{};
    if (hipError_t e = make_chain(a.ws, tiles, a.D, 2048, ch, st)) return e;
    hipLaunchKernelGGL((k_gscan_bwd<kOdd, TX, TG, VEC, kTok, true>), grid, dim3(kThreads), 0, st, a, tiles, kWaves * kTok, cb, ch);
    return hipGetLastError();
}

template <typename TX, typename TG>
hipError_t bwd_t(const GScanArgs& a, bool have, hipStream_t st) {
    if (a.D < kSlim) return bwd_v<false, TX, TG, 1>(a, have, st);
    return a.D % 4 ? bwd_v<true, TX, TG, 4>(a, have, st) : bwd_v<false, TX, TG, 4>(a, have, st);
}

}  // namespace

// (sized for 64-token tiles, whatever the types)
size_t gscan_fwd_ws(const SeqView& seq, int64_t D) {
    return by_rows(seq) || one_tile(seq, kScanTile) ? 0 : chain_bytes(tiles_of(seq.total, kScanTile), D);
}
size_t gscan_bwd_ws(const SeqView& seq, int64_t D) {
    if (one_tile(seq, kScanTile)) return 0;
    const size_t tiles = tiles_of(seq.total, kScanTile);
    return chain_bytes(tiles, D) + tiles * D * 4;
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
