// k_gate.hip -- the gated recurrence, its single step and its gradients.  Per
// batch row and channel, s_t = sigmoid(g_t), q_t = rate s_t:
//   a_t = exp(-q_t),  m_t = sqrt(1 - a_t^2) (or 1),  h_t = a_t h_{t-1} + m_t x_t
//   lam_t = dh_t + mu_{t+1},  mu_t = a_t lam_t,  dx_t = m_t lam_t,
//   dl_t = mu_t h_{t-1} - lam_t x_t a_t^2 / m_t   (the gradient of log a_t)
//   dg_t = -rate s_t (1 - s_t) dl_t,  drate = -sum s_t dl_t
// Everything is fp32 between the loads and the stores.  a_t next to 1 is 1 -
// e_t rounded, e_t = 1 - exp(-q_t) formed without cancellation and m_t^2 =
// e_t (2 - e_t); a smaller a_t is its exponential itself, since 1 - e_t would
// leave few of its digits (none from q_t = 17 on).  A rounded decay next to 1
// is off by the same amount at every token, 3e-5 of the state after 1000: so
// the state after a tile comes from the tile's sum of q_t (factor() below),
// and the rounded decays count within a tile alone.
//
// A workgroup takes a tile of tokens by 128 channels: 16 lanes hold a token's
// channels (eight each), and each such group a slice of S tokens.  A stretch
// of tokens maps the state p before it to f p + H, f = 2^-k; the slices' k and
// ends meet in LDS, one thread per channel folds them into the tile's, and
// every slice then runs again from the state it starts with.
//
// Tiles of one channel block (a chain) follow each other by looking back: a
// workgroup publishes its tile's (f, H) at once, waits until one of the kLook
// tiles before it holds an end state, applies the pairs since to it,
// and publishes its own end state.  The input is read once.  A pair travels
// in one 64-bit atomic word, so no fence is needed.  Workgroups take tiles in
// order from a counter and wait for earlier ones alone: of the tiles under
// way the first never waits, so every wait ends.
//
// Memory is the floor, and the arithmetic (two exponentials, a reciprocal and
// a root per element) is not hidden behind it whole.  Ten calls over one set of
// inputs in a graph, 2 x 8192 x 4096 bf16: 93 us (403 MB, 4.3 TB/s; a 1 GiB
// copy reaches 5.06): 85 without the waits, 81 without the gate's arithmetic,
// 75 without both; on changing inputs 103.  131072 x 1024: 239 us (814 MB,
// 3.4 TB/s): 176, 228 and 164, its eight chains wait for states; on changing
// inputs 235.  fp32 2 x 8192 x 4096: 190 us (805 MB, 4.2 TB/s).  Gradients of
// 2 x 8192 x 4096 bf16: 184 us (675 MB, 3.7 TB/s), on changing inputs 180.
// Persistent workgroups that load the next tile ahead took 118 and 305 us
// through registers, 114 and 275 through LDS, where these kernels took 96 and
// 235; tiles of 32 channels by 512 tokens 114 and 253.  Tiles in the order of
// the workgroups' indexes, without tickets, take 90 and 226 (239 with), but
// nothing says that workgroups start in that order, and the waits rest on it.
#include <algorithm>

#include "msr_quant.hpp"

#include "msr_lookback.hpp"

namespace {

using namespace msr;

struct GateArgs {
    const void *x, *g, *dh;         // dh: backward only
    const float *rate, *state_in;   // state_in: the state before token 0 (forward), the gradient of the last state (backward)
    void *y, *dg;                   // y: h (may be NULL), or dx
    float *state_out;               // the last state, or the gradient of state_in (may be NULL)
    float *carry;                   // [B][blocks][D] states before each block of 64 tokens: written (may be NULL), or read
    float *part;                    // backward: [B tiles][D] sums of -s dl (may be NULL)
    uint64_t *words;                // [chains][tiles][channels]; chains: B cols, column blocks of a batch row
    uint32_t *tickets;              // [groups]
    int B, T, D, tiles, cols, blocks, groups;
};

// ---- decays and gates -----------------------------------------------------------
// Exponents are kept in base 2: k = q log2(e), with log2(e) in the channel's rate.
constexpr float kLog2e = 1.44269504f;

// a = 2^-k and e = 1 - a.  Where k is small, e is a series and a is 1 - e; elsewhere e is 1 - a, off by the exponential's
// error.  FINE: seven terms up to 1/2 (the first left out is 1.5e-8 of the sum); 1 - a is off by 2e-7 of itself there.  Else
// three up to 1/32 (4e-7), and 1 - a is off by 1.5e-6 just above as measured (2.8e-6 by an ulp of a).  fp32 results take the
// former at no cost (2 x 8192 x 2048 103.5 us with either; errors 1.0e-7 to 1.5e-7 of the results' norm with the latter,
// 0.6e-7 to 1.1e-7 with the former), bf16 ones, whose rounding is 4e-3, the latter (2 x 8192 x 4096: 93 us, with the former
// 97; gradients 184 and 193).
template <bool FINE>
struct Decay {
    float e, a;
    __device__ __forceinline__ explicit Decay(float k) {
        float p = 0.0555041087f;
        if constexpr (FINE) {
            p = fmaf(k, 1.52527338e-5f, -1.54035304e-4f);
            p = fmaf(k, p, 1.33335581e-3f);
            p = fmaf(k, p, -9.61812911e-3f);
            p = fmaf(k, p, 0.0555041087f);
        }
        p = k * fmaf(k, fmaf(k, p, -0.240226507f), 0.693147181f);
        const float f = __builtin_amdgcn_exp2f(-k);
        const bool small = k < (FINE ? 0.5f : 0.03125f);
        e = small ? p : 1.f - f;
        a = small ? 1.f - p : f;
    }
};

__device__ __forceinline__ float factor(float k) {
    const float f = __builtin_amdgcn_exp2f(-k);
    return f < 0.5f ? -f : Decay<true>(k).e;
}

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * g)); }

// The gradients need s (1 - s) too, and 1 - s formed of an s next to 1 has few digits (0.5% off at g = 12, none left from 17
// on): with c the lesser of s and 1 - s, both formed of exp(-|g|), it is c (1 - c).  Where the registers allow (bf16 in rows
// of aligned groups: 252 of them), s and s (1 - s) are kept from one pass over a tile to the other (2 x 8192 x 4096: 184 us,
// with c alone 196); elsewhere c is, with a sign that says which it is (-0: s = 1).
template <bool BOTH>
struct Gated;
template <>
struct Gated<true> {
    float s, p;
    __device__ __forceinline__ float set(float g) {
        const float t = __builtin_amdgcn_exp2f(-kLog2e * fabsf(g)), r = __builtin_amdgcn_rcpf(1.f + t), c = t * r;
        p = r * c, s = g < 0.f ? c : r;
        asm volatile("" : "+v"(s), "+v"(p));  // keeps the compiler from holding what they are formed of
        return s;
    }
    __device__ __forceinline__ float sigmoid() const { return s; }
    __device__ __forceinline__ float slope() const { return p; }
    __device__ __forceinline__ void forget() {}
};
template <>
struct Gated<false> {
    float w;  // s, or s - 1
    __device__ __forceinline__ float set(float g) {
        const float t = __builtin_amdgcn_exp2f(-kLog2e * fabsf(g));
        w = copysignf(t * __builtin_amdgcn_rcpf(1.f + t), -g);
        forget();
        return sigmoid();
    }
    __device__ __forceinline__ float sigmoid() const { return far(w) ? 1.f + w : w; }
    __device__ __forceinline__ float slope() const { return fmaf(-w, w, fabsf(w)); }
    // the same for w and what is formed of it
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(w)); }
};

// Tokens past the last: a gate of -infinity, whose decay is 1 and whose input counts for nothing.
template <int ROWS>
__device__ __forceinline__ void close_gate(Raw8<uint16_t, ROWS> &r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.u[i] = 0xff80ff80u;
    if constexpr (ROWS == kAny) r.down = 0;
}
template <int ROWS>
__device__ __forceinline__ void close_gate(Raw8<float, ROWS> &r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.a[i] = r.b[i] = -__builtin_inff();
    if constexpr (ROWS == kAny) r.down = 0;
}

// ---- words between tiles (msr_lookback.hpp) ---------------------------------------
__device__ __forceinline__ void store(uint64_t *w, uint64_t v) {
    __hip_atomic_store(w, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(uint64_t *w, float z, float h) { store(w, pair_word(z, h)); }
__device__ __forceinline__ void publish(uint64_t *w, float state) { store(w, pack(kState, state)); }

constexpr int kSpins = 1 << 22;  // polls: seconds, far beyond any wait; an end for callers who share a workspace
constexpr int kLook = 8;         // tiles looked at: 93 and 239 us (loops as above); with four 89 and 257, with 16 98 and 246
constexpr int kSleep = 8;        // between polls, in 64 clocks: with two 93.5 and 240 us

// the state that tile n of a chain starts from (w: tile 0's word; a tile's words are CH apart)
template <int CH>
__device__ __forceinline__ float state_before(const uint64_t *w, int n) {
    return look_back<kLook>(
        kSpins,
        [&](int i) {
            return __hip_atomic_load(w + (int64_t)max(n - 1 - i, 0) * CH, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        },
        [] { __builtin_amdgcn_s_sleep(kSleep); });
}

// The tiles are dealt out in order of time by `groups` counters: ticket q of a group's n chains is tile q / n of its chain
// q % n.  Workgroups go to the XCDs in turn: with eight groups or more, a chain stays on one.
struct Deal {
    uint32_t group, n;
    uint32_t *counter;
    __device__ __forceinline__ explicit Deal(const GateArgs &a) {
        n = (uint32_t)a.B * a.cols / a.groups;
        group = blockIdx.x % a.groups;
        counter = a.tickets + group;
    }
    __device__ __forceinline__ uint32_t take(const GateArgs &a, uint32_t *slot) const {  // by all threads of a workgroup
        if (a.tiles == 1) return blockIdx.x / a.groups;  // no tile waits for another
        if (threadIdx.x == 0) *slot = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        return __builtin_amdgcn_readfirstlane(*slot);
    }
};

// the tile that ticket q of a group is
struct Place {
    int tile, b, c0;
    uint32_t chain;
    __device__ __forceinline__ Place(const GateArgs &a, const Deal &d, uint32_t q, int channels) {
        tile = (int)(q / d.n);
        chain = d.group + a.groups * (q - tile * d.n);
        b = (int)(chain / a.cols);
        c0 = (int)(chain - b * a.cols) * channels;
    }
};

// ---- the forward pass -----------------------------------------------------------
// a slice's tokens: a and m x of each, their sum of k, and the state that they make of 0.  raw(t, x, g) gives a
// token's eight channels
template <bool FINE, int S, bool NORM, typename Raw>
__device__ __forceinline__ void slice(const Raw &raw, const float (&rate)[8], float (&keep)[S][8], float (&u)[S][8],
                                      float (&k)[8], float (&h)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = h[i] = 0.f;
#pragma unroll
    for (int t = 0; t < S; ++t) {
        float g[8];
        raw(t, u[t], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float kt = rate[i] * sigmoid(g[i]);
            const Decay<FINE> d(kt);
            if constexpr (NORM) u[t][i] *= __builtin_amdgcn_sqrtf(fmaf(-d.e, d.e, d.e + d.e));
            keep[t][i] = d.a;
            k[i] += kt;
            h[i] = fmaf(keep[t][i], h[i], u[t][i]);
        }
    }
}

// What one thread does per channel c between a tile's barriers: from the slices' k and ends to the states that they
// start from (in hs), by way of the tile's own.
template <int NS, int S, int CH>
__device__ __forceinline__ void join_slices(const GateArgs &a, const Place &pl, float (&ks)[NS][CH], float (&hs)[NS][CH],
                                            int c) {
    const bool live = pl.c0 + c < a.D;
    const int64_t at = (int64_t)pl.b * a.D + pl.c0 + c;
    uint64_t *w = a.words + (uint64_t)pl.chain * a.tiles * CH + c;
    float k = 0.f, h = 0.f, p = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        k += ks[i][c];
        h = fmaf(__builtin_amdgcn_exp2f(-ks[i][c]), h, hs[i][c]);
    }
    const float z = factor(k);
    if (pl.tile == 0) {
        if (a.state_in && live) p = a.state_in[at];
    } else {
        if (pl.tile + 1 < a.tiles) publish(w + (int64_t)pl.tile * CH, z, h);
        p = state_before<CH>(w, pl.tile);
    }
    const float last = apply(z, p) + h;
    if (pl.tile + 1 < a.tiles)
        publish(w + (int64_t)pl.tile * CH, last);
    else if (a.state_out && live)
        a.state_out[at] = last;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int64_t t = (int64_t)pl.tile * (NS * S) + i * S;
        if (i * S % MSR_GATE_BLOCK == 0 && a.carry && live && t < a.T)
            a.carry[((int64_t)pl.b * a.blocks + t / MSR_GATE_BLOCK) * a.D + pl.c0 + c] = p;
        const float end = hs[i][c];
        hs[i][c] = p;
        p = fmaf(__builtin_amdgcn_exp2f(-ks[i][c]), p, end);
    }
}

template <typename T, int ROWS, int LX, int W, int S, bool NORM>
__global__ __launch_bounds__(64 * W) void gate_kernel(GateArgs a) {
    constexpr int NS = 64 / LX * W, TILE = S * NS, CH = 8 * LX;
    static_assert(TILE % MSR_GATE_BLOCK == 0 && MSR_GATE_BLOCK % S == 0, "");
    __shared__ float ks[NS][CH], hs[NS][CH];
    __shared__ uint32_t slot;
    const Deal deal(a);
    const uint32_t q = deal.take(a, &slot);
    if (q >= deal.n * a.tiles) return;  // calls at once that share a workspace: wrong results, but nothing outside it
    const Place pl(a, deal, q, CH);
    const int sl = threadIdx.x / LX, e0 = 8 * (threadIdx.x % LX), left = a.D - pl.c0 - e0;
    const int64_t t0 = (int64_t)pl.tile * TILE + sl * S;
    const int mine = (int)min(max((int64_t)a.T - t0, (int64_t)0), (int64_t)S);  // tokens of this slice
    const int64_t at = ((int64_t)pl.b * a.T + t0) * a.D + pl.c0 + e0;
    const bool whole = (int64_t)(pl.tile + 1) * TILE <= a.T && pl.c0 + CH <= a.D;
    float keep[S][8], u[S][8];
    {
        Raw8<T, ROWS> rx[S], rg[S];
        float rate[8], k[8], h[8];
        const T *px = static_cast<const T *>(a.x) + at, *pg = static_cast<const T *>(a.g) + at;
        if (whole) {
#pragma unroll
            for (int t = 0; t < S; ++t, px += a.D, pg += a.D) rx[t].load(px, 8), rg[t].load(pg, 8);
        } else {
#pragma unroll
            for (int t = 0; t < S; ++t, px += a.D, pg += a.D) {
                const int l = t < mine ? left : 0;
                rx[t].load(px, l), rg[t].load(pg, l);
            }
        }
        load8<ROWS>(a.rate + pl.c0 + e0, left, rate);
#pragma unroll
        for (int i = 0; i < 8; ++i) rate[i] *= kLog2e;
        if (mine < S) {
#pragma unroll
            for (int t = 0; t < S; ++t)
                if (t >= mine) close_gate(rg[t]);
        }
        slice<sizeof(T) == 4, S, NORM>([&](int t, float (&x)[8], float (&g)[8]) { rx[t].get(x), rg[t].get(g); }, rate, keep, u,
                                       k, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) ks[sl][e0 + i] = k[i], hs[sl][e0 + i] = h[i];
    }
    __syncthreads();
    if (threadIdx.x < CH) join_slices<NS, S, CH>(a, pl, ks, hs, threadIdx.x);
    if (!a.y) return;
    __syncthreads();
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = hs[sl][e0 + i];
    T *y = static_cast<T *>(a.y) + at;
#pragma unroll
    for (int t = 0; t < S; ++t, y += a.D) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = fmaf(keep[t][i], h[i], u[t][i]);
        if (whole)
            store8<ROWS>(y, 8, h);
        else if (t < mine)
            store8<ROWS>(y, left, h);
    }
}

// The tiles from the last to the first: h again from the state before the
// tile's first token, mu by looking back over the later tiles.
template <typename T, int ROWS, int LX, int W, int S, bool NORM>
__global__ __launch_bounds__(64 * W) void gate_backward_kernel(GateArgs a) {
    constexpr int NS = 64 / LX * W, TILE = S * NS, CH = 8 * LX;
    static_assert(TILE % MSR_GATE_BLOCK == 0 && 2 * CH <= 64 * W, "");
    __shared__ float ks[NS][CH], hs[NS][CH], ms[NS][CH];
    __shared__ uint32_t slot;
    const Deal deal(a);
    const uint32_t q = deal.take(a, &slot);
    if (q >= deal.n * a.tiles) return;  // calls at once that share a workspace: wrong results, but nothing outside it
    const Place pl(a, deal, q, CH);
    const int n = pl.tile, tile = a.tiles - 1 - n, b = pl.b, c0 = pl.c0;
    const int sl = threadIdx.x / LX, e0 = 8 * (threadIdx.x % LX), left = a.D - c0 - e0;
    const int64_t t0 = (int64_t)tile * TILE;
    const int mine = (int)min(max((int64_t)a.T - t0 - sl * S, (int64_t)0), (int64_t)S);
    const int64_t at = ((int64_t)b * a.T + t0 + sl * S) * a.D + c0 + e0;
    const bool whole = t0 + TILE <= a.T && c0 + CH <= a.D;
    float start = 0.f;  // the state before the tile, for the thread that needs it
    if (threadIdx.x >= CH && threadIdx.x < 2 * CH && c0 + (int)threadIdx.x - CH < a.D)
        start = a.carry[((int64_t)b * a.blocks + t0 / MSR_GATE_BLOCK) * a.D + c0 + threadIdx.x - CH];
    Raw8<T, ROWS> rd[S];
    float rate[8], keep[S][8], m[S][8], u[S][8];
    Gated<sizeof(T) == 2 && ROWS != kAny> sg[S][8];
    {
        Raw8<T, ROWS> rx[S], rg[S];
        const T *px = static_cast<const T *>(a.x) + at, *pg = static_cast<const T *>(a.g) + at;
        const T *pd = static_cast<const T *>(a.dh) + at;
        if (whole) {
#pragma unroll
            for (int t = 0; t < S; ++t, px += a.D, pg += a.D, pd += a.D)
                rx[t].load(px, 8), rg[t].load(pg, 8), rd[t].load(pd, 8);
        } else {
#pragma unroll
            for (int t = 0; t < S; ++t, px += a.D, pg += a.D, pd += a.D) {
                const int l = t < mine ? left : 0;
                rx[t].load(px, l), rg[t].load(pg, l), rd[t].load(pd, l);
            }
        }
        load8<ROWS>(a.rate + c0 + e0, left, rate);
        if (mine < S) {
#pragma unroll
            for (int t = 0; t < S; ++t)
                if (t >= mine) close_gate(rg[t]);
        }
        float k[8], h[8], mu[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = h[i] = mu[i] = 0.f;
#pragma unroll
        for (int t = 0; t < S; ++t) {
            float g[8];
            rx[t].get(u[t]);
            rg[t].get(g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float kt = rate[i] * kLog2e * sg[t][i].set(g[i]);
                const Decay<sizeof(T) == 4> d(kt);
                if constexpr (NORM) {
                    m[t][i] = __builtin_amdgcn_sqrtf(fmaf(-d.e, d.e, d.e + d.e));
                    u[t][i] *= m[t][i];
                }
                keep[t][i] = d.a;
                k[i] += kt;
                h[i] = fmaf(keep[t][i], h[i], u[t][i]);
            }
        }
#pragma unroll
        for (int t = S - 1; t >= 0; --t) {
            float d[8];
            rd[t].get(d);
#pragma unroll
            for (int i = 0; i < 8; ++i) mu[i] = keep[t][i] * (d[i] + mu[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ks[sl][e0 + i] = k[i];
            hs[sl][e0 + i] = h[i];
            ms[sl][e0 + i] = mu[i];
        }
    }
    __syncthreads();
    if (threadIdx.x < CH) {
        const int c = threadIdx.x;
        const bool live = c0 + c < a.D;
        uint64_t *w = a.words + (uint64_t)pl.chain * a.tiles * CH + c;
        float k = 0.f, m = 0.f, p = 0.f;
#pragma unroll
        for (int i = NS - 1; i >= 0; --i) {
            k += ks[i][c];
            m = fmaf(__builtin_amdgcn_exp2f(-ks[i][c]), m, ms[i][c]);
        }
        const float z = factor(k);
        if (n == 0) {
            if (a.state_in && live) p = a.state_in[(int64_t)b * a.D + c0 + c];
        } else {
            if (tile > 0) publish(w + (int64_t)n * CH, z, m);
            p = state_before<CH>(w, n);
        }
        const float last = apply(z, p) + m;
        if (tile > 0)
            publish(w + (int64_t)n * CH, last);
        else if (a.state_out && live)
            a.state_out[(int64_t)b * a.D + c0 + c] = last;
#pragma unroll
        for (int i = NS - 1; i >= 0; --i) {
            const float end = ms[i][c];
            ms[i][c] = p;
            p = fmaf(__builtin_amdgcn_exp2f(-ks[i][c]), p, end);
        }
    } else if (threadIdx.x - CH < CH) {  // the states, from the one before the tile, in the other waves
        const int c = threadIdx.x - CH;
        float p = start;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const float end = hs[i][c];
            hs[i][c] = p;
            p = fmaf(__builtin_amdgcn_exp2f(-ks[i][c]), p, end);
        }
    }
    __syncthreads();
    // what was formed of these is formed again: kept across the barriers, it would not fit the registers
#pragma unroll
    for (int t = 0; t < S; ++t) {
        rd[t].forget();
#pragma unroll
        for (int i = 0; i < 8; ++i) sg[t][i].forget();
    }
    float before[S][8], mu[8], dr[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) before[0][i] = hs[sl][e0 + i], mu[i] = ms[sl][e0 + i], dr[i] = 0.f;
#pragma unroll
    for (int t = 0; t + 1 < S; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) before[t + 1][i] = fmaf(keep[t][i], before[t][i], u[t][i]);
    const int64_t row = (int64_t)(S - 1) * a.D;
    T *dxp = static_cast<T *>(a.y) + at + row, *dgp = static_cast<T *>(a.dg) + at + row;
#pragma unroll
    for (int t = S - 1; t >= 0; --t, dxp -= a.D, dgp -= a.D) {
        float dx[8], dg[8], dl[8];
        rd[t].get(dx);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float lam = dx[i] + mu[i];
            mu[i] = keep[t][i] * lam;
            dx[i] = lam;
            float by = before[t][i];
            if constexpr (NORM) {
                // u = m x: x / m = u / m^2, and u is 0 where m is (an m that is not 0 is above 1e-23)
                const float r = __builtin_amdgcn_rcpf(fmaxf(m[t][i], 1e-30f));
                dx[i] = lam * m[t][i];
                by = fmaf(-keep[t][i], u[t][i] * r * r, by);
            }
            dl[i] = mu[i] * by;
            dg[i] = -sg[t][i].slope() * (rate[i] * dl[i]);
        }
        if (whole || t < mine) {  // past the last token s is 0, but dl is not where the last state is not finite
#pragma unroll
            for (int i = 0; i < 8; ++i) dr[i] = fmaf(-sg[t][i].sigmoid(), dl[i], dr[i]);
        }
        if (whole) {
            store8<ROWS>(dxp, 8, dx);
            store8<ROWS>(dgp, 8, dg);
        } else if (t < mine) {
            store8<ROWS>(dxp, left, dx);
            store8<ROWS>(dgp, left, dg);
        }
    }
    if (!a.part) return;
    // ks is free: it was read before the last barrier
#pragma unroll
    for (int i = 0; i < 8; ++i) ks[sl][e0 + i] = dr[i];
    __syncthreads();
    if (threadIdx.x < CH && c0 + threadIdx.x < a.D) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) s += ks[i][threadIdx.x];
        a.part[((int64_t)b * a.tiles + tile) * a.D + c0 + threadIdx.x] = s;
    }
}

// One token: h = a state + m x, bound by its launch where it is small (64 x 4096 bf16 3.5 us in a graph) and by memory (512
// x 8192 bf16 11 us, 5.3 TB/s).  Where a >= 1/2 it is taken as two numbers, 1 - e rounded and the rest that this left out,
// so that the state's roundings are those of the two sums alone; below, where 1 - e has few digits or none, it is the
// exponential itself.
template <typename T, int ROWS, bool NORM>
__global__ __launch_bounds__(256) void gate_step_kernel(GateArgs a, int groups) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i0 >= (int64_t)a.B * groups) return;
    const int b = (int)(i0 / groups), e0 = (int)(i0 - (int64_t)b * groups) * 8, left = a.D - e0;
    const int64_t at = (int64_t)b * a.D + e0;
    float x[8], g[8], rate[8], st[8], y[8];
    load8<ROWS>(static_cast<const T *>(a.x) + at, left, x);
    load8<ROWS>(static_cast<const T *>(a.g) + at, left, g);
    load8<ROWS>(a.state_in + at, left, st);
    load8<ROWS>(a.rate + e0, left, rate);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const Decay<true> d(kLog2e * rate[i] * sigmoid(g[i]));
        const float e = d.e;
        const float m = NORM ? __builtin_amdgcn_sqrtf(fmaf(-e, e, e + e)) : 1.f, f = 1.f - e;
        const bool strong = e > 0.5f;
        const float rest = strong ? 0.f : (1.f - f) - e;
        // the rest of an infinite state is a number
        const float add = fmaf(m, x[i], rest * __builtin_amdgcn_fmed3f(st[i], -3.40282347e38f, 3.40282347e38f));
        y[i] = fmaf(strong ? d.a : f, st[i], add);
    }
    store8<ROWS>(a.state_out + at, left, y);
    store8<ROWS>(static_cast<T *>(a.y) + at, left, y);
}

// no word published, no tile taken: n words, then the tickets
__global__ __launch_bounds__(256) void gate_clear_kernel(uint64_t *words, int64_t n, int64_t tickets) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    uint32_t *z = reinterpret_cast<uint32_t *>(words + n);
    for (int64_t i = i0; i < n; i += step) words[i] = ~0ull;
    for (int64_t i = i0; i < tickets; i += step) z[i] = 0;
}

__global__ __launch_bounds__(256) void gate_copy_kernel(const float *from, float *to, int64_t n) {  // from NULL: zeros
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : 0.f;
}

template <int N>
using C = std::integral_constant<int, N>;

template <typename F>
hipError_t by_type(int dtype, int D, bool norm, F f) {
    auto rows = [&](auto t, auto n) {
        if (D % 8 == 0) return f(t, C<kAligned>(), n);
        if (D > 8) return f(t, C<kAny>(), n);
        return f(t, C<kTiny>(), n);
    };
    if (dtype == MSR_BF16) return norm ? rows(uint16_t(), std::true_type()) : rows(uint16_t(), std::false_type());
    return norm ? rows(float(), std::true_type()) : rows(float(), std::false_type());
}

constexpr int kWaves = 4, kLanes = 16, kChannels = 8 * kLanes;  // of a tile: lanes across, channels

// Tokens of a lane.  bf16 forward: 93 us (2 x 8192 x 4096) and 239 (131072 x 1024) with eight, 101 and 386 with four.
// Gradients, whose registers hold more of each token: 184 us with four, 224 with eight.  fp32 holds twice the bits.
constexpr int tokens_of(int dtype, bool backward) { return dtype == MSR_BF16 && !backward ? 8 : 4; }
constexpr int tile_of(int dtype, bool backward) { return 64 / kLanes * kWaves * tokens_of(dtype, backward); }

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m; }

hipError_t copy(const float *from, float *to, int64_t n, hipStream_t st) {
    if (!to || n == 0) return hipSuccess;
    hipLaunchKernelGGL(gate_copy_kernel, dim3((unsigned)up(n, 256)), dim3(256), 0, st, from, to, n);
    return hipGetLastError();
}

// what the chains need: [words][tickets]
struct Plan {
    int tiles, cols, blocks, groups;
    int64_t chains, words;
    size_t bytes;
};

constexpr int kGroups = 64;  // counters at most

Plan plan(int B, int T, int D, int dtype, bool backward) {
    Plan p;
    p.tiles = (int)up(T, tile_of(dtype, backward)), p.cols = (int)up(D, kChannels), p.blocks = (int)up(T, MSR_GATE_BLOCK);
    p.chains = (int64_t)B * p.cols, p.words = p.tiles > 1 ? p.chains * p.tiles * kChannels : 0;
    for (p.groups = kGroups; p.chains % p.groups; p.groups /= 2) {}
    p.bytes = (size_t)p.words * 8 + kGroups * 4;
    return p;
}

hipError_t fill(GateArgs &a, const Plan &p, char *ws, hipStream_t st) {
    a.tiles = p.tiles, a.cols = p.cols, a.blocks = p.blocks, a.groups = p.groups;
    a.words = reinterpret_cast<uint64_t *>(ws);
    a.tickets = reinterpret_cast<uint32_t *>(ws + p.words * 8);
    if (p.tiles == 1) return hipSuccess;  // neither is used: 7.5 us for 10.0 (8 x 100 x 4096 bf16)
    const int64_t g = std::min<int64_t>(up(p.words, 1024), 2048);
    hipLaunchKernelGGL(gate_clear_kernel, dim3((unsigned)g), dim3(256), 0, st, a.words, p.words, (int64_t)kGroups);
    return hipGetLastError();
}

}  // namespace

// enough for either type
size_t gate_workspace(int B, int T, int D, bool backward, bool carry_given) {
    if (B == 0 || T == 0 || D == 0) return 0;
    size_t most = 0;
    for (int dtype : {MSR_F32, MSR_BF16}) {
        const Plan f = plan(B, T, D, dtype, false), p = plan(B, T, D, dtype, true);
        size_t n = f.bytes;
        if (backward) {
            n = up(std::max(p.bytes, carry_given ? 0 : f.bytes), 256) * 256 + up((int64_t)B * p.tiles * D * 4, 256) * 256;
            if (!carry_given) n += up((int64_t)B * p.blocks * D * 4, 256) * 256;
        }
        most = std::max(most, n);
    }
    return most;
}

hipError_t launch_gate(const Gate &q, char *ws, hipStream_t st) {
    GateArgs a{};
    a.x = q.x, a.g = q.g, a.rate = q.rate, a.state_in = q.state_in, a.y = q.h, a.state_out = q.state_out, a.carry = q.carry;
    a.B = q.B, a.T = q.T, a.D = q.D;
    if (q.T == 0) return copy(q.state_in, q.state_out, (int64_t)q.B * q.D, st);
    const Plan p = plan(q.B, q.T, q.D, q.dtype, false);
    hipError_t e = fill(a, p, ws, st);
    if (e != hipSuccess) return e;
    return by_type(q.dtype, q.D, q.normalize, [&](auto t, auto rows, auto norm) {
        constexpr int S = tokens_of(sizeof(t) == 2 ? MSR_BF16 : MSR_F32, false);
        hipLaunchKernelGGL((gate_kernel<decltype(t), rows.value, kLanes, kWaves, S, norm.value>),
                           dim3((unsigned)(p.chains * p.tiles)), dim3(64 * kWaves), 0, st, a);
        return hipGetLastError();
    });
}

hipError_t launch_gate_step(const Gate &q, hipStream_t st) {
    GateArgs a{};
    a.x = q.x, a.g = q.g, a.rate = q.rate, a.state_in = q.state_in, a.y = q.h, a.state_out = q.state_out, a.B = q.B, a.D = q.D;
    const int groups = (q.D + 7) / 8;
    return by_type(q.dtype, q.D, q.normalize, [&](auto t, auto rows, auto norm) {
        hipLaunchKernelGGL((gate_step_kernel<decltype(t), rows.value, norm.value>),
                           dim3((unsigned)up((int64_t)q.B * groups, 256)), dim3(256), 0, st, a, groups);
        return hipGetLastError();
    });
}

hipError_t launch_gate_backward(const Gate &q, char *ws, hipStream_t st) {
    hipError_t e;
    if (q.T == 0) {
        if ((e = copy(q.dstate_out, q.dstate_in, (int64_t)q.B * q.D, st)) != hipSuccess) return e;
        return copy(nullptr, q.drate, q.D, st);
    }
    const Plan p = plan(q.B, q.T, q.D, q.dtype, true);
    // past the words of this pass and of the forward one
    char *w = ws + up(q.carry ? p.bytes : std::max(p.bytes, plan(q.B, q.T, q.D, q.dtype, false).bytes), 256) * 256;
    float *part = reinterpret_cast<float *>(w);
    w += up((int64_t)q.B * p.tiles * q.D * 4, 256) * 256;
    GateArgs a{};
    a.x = q.x, a.g = q.g, a.rate = q.rate, a.B = q.B, a.T = q.T, a.D = q.D;
    float *carry = q.carry;
    if (!carry) {  // the forward pass again, for its states alone
        carry = reinterpret_cast<float *>(w);
        Gate f = q;
        f.h = nullptr, f.state_out = nullptr, f.carry = carry;
        if ((e = launch_gate(f, ws, st)) != hipSuccess) return e;
    }
    a.state_in = q.dstate_out, a.state_out = q.dstate_in, a.dh = q.dh, a.y = q.dx, a.dg = q.dg, a.carry = carry;
    a.part = q.drate ? part : nullptr;
    if ((e = fill(a, p, ws, st)) != hipSuccess) return e;
    e = by_type(q.dtype, q.D, q.normalize, [&](auto t, auto rows, auto norm) {
        constexpr int S = tokens_of(sizeof(t) == 2 ? MSR_BF16 : MSR_F32, true);
        hipLaunchKernelGGL((gate_backward_kernel<decltype(t), rows.value, kLanes, kWaves, S, norm.value>),
                           dim3((unsigned)(p.chains * p.tiles)), dim3(64 * kWaves), 0, st, a);
        return hipGetLastError();
    });
    if (e == hipSuccess && q.drate) e = launch_column_sum(part, q.drate, nullptr, q.B * p.tiles, q.D, st);
    return e;
}
