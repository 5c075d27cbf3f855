// k_gate.hip -- the gated recurrence, its single step and its gradients.  Per
// batch row and channel, s_t = sigmoid(g_t), q_t = rate s_t:
//   a_t = exp(-q_t),  m_t = sqrt(1 - a_t^2) (or 1),  h_t = a_t h_{t-1} + m_t x_t
//   lam_t = dh_t + mu_{t+1},  mu_t = a_t lam_t,  dx_t = m_t lam_t,
//   dl_t = mu_t h_{t-1} - lam_t x_t a_t^2 / m_t   (the gradient of log a_t)
//   dg_t = -rate s_t (1 - s_t) dl_t,  drate = -sum s_t dl_t
// Everything is fp32 between the loads and the stores.  A step takes away
// e_t h with e_t = 1 - a_t = -expm1(-q_t) formed without cancellation, and
// 1 - a^2 = e (2 - e): a decay next to 1, rounded, would be off by the same
// amount at every token, 3e-5 of the state after 1000 tokens.
//
// A workgroup takes a tile of kTile tokens by 128 channels: 16 lanes hold a
// token's channels (eight each), and each such group a slice of S tokens.
// A stretch of tokens maps the state p before it to f p + H; the slices'
// factors and ends meet in LDS, one thread per channel folds them into the
// tile's, and every slice then runs again from the state it starts with.
//
// Tiles of one channel block follow each other by looking back: a workgroup
// publishes its tile's (f, H) at once, goes back over the words of the tiles
// before it to the latest that holds an end state (f = 0), applies the pairs
// since to it, and publishes its own end state.  The input is read once.  A
// pair travels in one 64-bit atomic word, so no fence is needed.  Workgroups take tiles in order from a counter
// per channel block and wait for earlier ones alone: of the tiles under way
// the first never waits, so every wait ends.
#include <algorithm>

#include "msr_quant.hpp"

namespace {

using namespace msr;

constexpr int kChannels = 128;  // of a tile
constexpr uint32_t kUnset = 0xffffffffu;  // factor bits of a word that is not published yet,
constexpr uint32_t kState = 0x80000000u;  // and of one that holds a state: f = 0

struct GateArgs {
    const void *x, *g, *dh;         // dh: backward only
    const float *rate, *state_in;   // state_in: the state before token 0 (forward), the gradient of the last state (backward)
    void *y, *dg;                   // y: h (may be NULL), or dx
    float *state_out;               // the last state, or the gradient of state_in (may be NULL)
    float *carry;                   // [B][blocks][D] states before each block of 64 tokens: written (may be NULL), or read
    float *part;                    // backward: [B tiles][D] sums of -s dl (may be NULL)
    uint64_t *words;                // [B column blocks][tiles][128]
    uint32_t *tickets;              // [B column blocks]
    int B, T, D, tiles, cols, blocks;  // cols: blocks of 128 channels
};

// ---- factors ----------------------------------------------------------------
// A factor f in [0, 1] is held as 1 - f where f >= 1/2 and as -f below (the
// sign bit tells them apart), so that neither a state that hardly decays nor
// one that is nearly gone loses accuracy.  -0 is f = 0.
__device__ __forceinline__ bool far(float z) { return (int)__float_as_uint(z) < 0; }
__device__ __forceinline__ float apply(float z, float p) { return fmaf(-z, p, far(z) ? 0.f : p); }
__device__ __forceinline__ float both(float y, float z) {  // the product of two factors
    const float ey = far(y) ? 1.f + y : y, ez = far(z) ? 1.f + z : z;
    const float f = (far(y) ? -y : 1.f - y) * (far(z) ? -z : 1.f - z);
    return f < 0.5f ? -f : fmaf(-ey, ez, ey) + ez;
}

constexpr float kLog2e = 1.44269504f;

// 1 - exp(-q): the series where it is small (the first term left out is 5e-8 of the sum at 1/4)
__device__ __forceinline__ float lost(float q) {
    const float p = q * fmaf(q, fmaf(q, fmaf(q, fmaf(q, fmaf(q, -1.f / 720.f, 1.f / 120.f), -1.f / 24.f), 1.f / 6.f), -0.5f), 1.f);
    const float d = 1.f - __builtin_amdgcn_exp2f(-kLog2e * q);
    return q < 0.25f ? p : d;
}

__device__ __forceinline__ float factor(float q) {
    const float f = __builtin_amdgcn_exp2f(-kLog2e * q);
    return f < 0.5f ? -f : lost(q);
}

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * g)); }

// ---- words between tiles ------------------------------------------------------
__device__ __forceinline__ void publish(uint64_t *w, float z, float h) {
    const uint32_t u = z != z ? 0x7fc00000u : __float_as_uint(z);  // no NaN that looks unpublished
    __hip_atomic_store(w, (uint64_t)u << 32 | __float_as_uint(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that tile n of a chain starts from: back over the words of tiles n - 1, n - 2, ... (kChannels apart) to the
// latest state, then forward again over the pairs since.  Where that state lies depends on how far the other workgroups
// are; the result does not, since every tile's end state is formed from its start state by the same pair.
__device__ __forceinline__ float look_back(const uint64_t *w, int n) {
    constexpr int N = 8;  // words under way at a time
    uint64_t v[N];
    float p = 0.f;
    int j = n - 1;
    auto fetch = [&] {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = __hip_atomic_load(w + (int64_t)max(j - i, 0) * kChannels, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    auto forward = [&] {
#pragma unroll
        for (int i = N - 1; i >= 0; --i) {
            const uint32_t u = (uint32_t)(v[i] >> 32);
            const float h = __uint_as_float((uint32_t)v[i]);
            p = u == kState ? h : apply(__uint_as_float(u), p) + h;
        }
    };
    for (int idle = 0; idle < (1 << 22);) {  // far beyond any wait (seconds): an end for a caller who shares the workspace
        fetch();
        bool found = false, open = false;  // a state; a word that is not published, after any state
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t u = (uint32_t)(v[i] >> 32);
            open = open || (!found && u == kUnset);
            found = found || u == kState;
        }
        if (!open && found) break;
        if (!open)
            j -= N, idle = 0;
        else
            ++idle;
    }
    // an older word than the latest state may not be published yet: it is not used
#pragma unroll
    for (int i = 0; i < N; ++i)
        if ((uint32_t)(v[i] >> 32) == kUnset) v[i] = (uint64_t)kState << 32;
    forward();
    while (j < n - 1) {
        j += N;
        fetch();
        forward();
    }
    return p;
}

// the next tile of this workgroup's channel block
__device__ __forceinline__ int take_tile(const GateArgs &a, uint32_t chain, int *slot) {
    if (a.tiles == 1) return 0;
    if (threadIdx.x == 0)
        *slot = (int)__hip_atomic_fetch_add(a.tickets + chain, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    return *slot;
}

template <typename T, int ROWS, int W, int S, bool NORM>
__global__ __launch_bounds__(64 * W) void gate_kernel(GateArgs a) {
    constexpr int NS = 4 * W, TILE = S * NS;
    static_assert(TILE % MSR_GATE_BLOCK == 0 && MSR_GATE_BLOCK % S == 0, "");
    __shared__ float zs[NS][kChannels], hs[NS][kChannels];
    __shared__ int slot;
    const uint32_t chains = (uint32_t)a.B * a.cols, chain = blockIdx.x % chains;
    const int tile = take_tile(a, chain, &slot);
    const int b = chain / a.cols, c0 = chain % a.cols * kChannels;
    const int sl = threadIdx.x >> 4, e0 = 8 * (threadIdx.x & 15), left = a.D - c0 - e0;
    const int64_t t0 = (int64_t)tile * TILE;
    const int mine = (int)min(max((int64_t)a.T - t0 - sl * S, (int64_t)0), (int64_t)S);  // tokens of this slice
    const int64_t at = ((int64_t)b * a.T + t0 + sl * S) * a.D + c0 + e0;
    float rate[8], lo[S][8], u[S][8];
    {
        Raw8<T, ROWS> rx[S], rg[S];
#pragma unroll
        for (int t = 0; t < S; ++t) {
            rx[t].load(static_cast<const T *>(a.x) + at + (int64_t)t * a.D, t < mine ? left : 0);
            rg[t].load(static_cast<const T *>(a.g) + at + (int64_t)t * a.D, t < mine ? left : 0);
        }
        load8<ROWS>(a.rate + c0 + e0, left, rate);
        float q[8], h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = h[i] = 0.f;
#pragma unroll
        for (int t = 0; t < S; ++t) {
            float gt[8];
            rx[t].get(u[t]);
            rg[t].get(gt);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float qt = t < mine ? rate[i] * sigmoid(gt[i]) : 0.f, e = lost(qt);  // past the last token: kept
                if constexpr (NORM) u[t][i] *= __builtin_amdgcn_sqrtf(fmaf(-e, e, 2.f * e));
                lo[t][i] = e;
                q[i] += qt;
                h[i] = fmaf(-e, h[i], h[i] + u[t][i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            zs[sl][e0 + i] = factor(q[i]);
            hs[sl][e0 + i] = h[i];
        }
    }
    __syncthreads();
    if (threadIdx.x < kChannels) {
        const int c = threadIdx.x;
        const bool live = c0 + c < a.D;
        uint64_t *w = a.words + (uint64_t)chain * a.tiles * kChannels + c;
        float z = 0.f, h = 0.f, p = 0.f;
        for (int i = 0; i < NS; ++i) {
            z = both(z, zs[i][c]);
            h = apply(zs[i][c], h) + hs[i][c];
        }
        if (tile > 0) {
            if (tile + 1 < a.tiles) publish(w + (int64_t)tile * kChannels, z, h);
            p = look_back(w, tile);
        } else if (a.state_in && live) {
            p = a.state_in[(int64_t)b * a.D + c0 + c];
        }
        const float last = apply(z, p) + h;
        if (tile + 1 < a.tiles)
            publish(w + (int64_t)tile * kChannels, -0.f, last);
        else if (a.state_out && live)
            a.state_out[(int64_t)b * a.D + c0 + c] = last;
        for (int i = 0; i < NS; ++i) {
            if (i * S % MSR_GATE_BLOCK == 0 && a.carry && live && t0 + i * S < a.T)
                a.carry[((int64_t)b * a.blocks + (t0 + i * S) / MSR_GATE_BLOCK) * a.D + c0 + c] = p;
            const float end = hs[i][c];
            hs[i][c] = p;
            p = apply(zs[i][c], p) + end;
        }
    }
    if (!a.y) return;
    __syncthreads();
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = hs[sl][e0 + i];
#pragma unroll
    for (int t = 0; t < S; ++t) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = fmaf(-lo[t][i], h[i], h[i] + u[t][i]);
        if (t < mine) store8<ROWS>(static_cast<T *>(a.y) + at + (int64_t)t * a.D, left, h);
    }
}

// The tiles from the last to the first: h again from the state before the
// tile's first token, mu by looking back over the later tiles.
template <typename T, int ROWS, int W, int S, bool NORM>
__global__ __launch_bounds__(64 * W) void gate_backward_kernel(GateArgs a) {
    constexpr int NS = 4 * W, TILE = S * NS;
    static_assert(TILE % MSR_GATE_BLOCK == 0, "");
    __shared__ float zs[NS][kChannels], hs[NS][kChannels], ms[NS][kChannels];
    __shared__ int slot;
    const uint32_t chains = (uint32_t)a.B * a.cols, chain = blockIdx.x % chains;
    const int n = take_tile(a, chain, &slot), tile = a.tiles - 1 - n;
    const int b = chain / a.cols, c0 = chain % a.cols * kChannels;
    const int sl = threadIdx.x >> 4, e0 = 8 * (threadIdx.x & 15), left = a.D - c0 - e0;
    const int64_t t0 = (int64_t)tile * TILE;
    const int mine = (int)min(max((int64_t)a.T - t0 - sl * S, (int64_t)0), (int64_t)S);
    const int64_t at = ((int64_t)b * a.T + t0 + sl * S) * a.D + c0 + e0;
    Raw8<T, ROWS> rx[S], rd[S];
    float rate[8], lo[S][8], sg[S][8];
    {
        Raw8<T, ROWS> rg[S];
#pragma unroll
        for (int t = 0; t < S; ++t) {
            rx[t].load(static_cast<const T *>(a.x) + at + (int64_t)t * a.D, t < mine ? left : 0);
            rg[t].load(static_cast<const T *>(a.g) + at + (int64_t)t * a.D, t < mine ? left : 0);
            rd[t].load(static_cast<const T *>(a.dh) + at + (int64_t)t * a.D, t < mine ? left : 0);
        }
        load8<ROWS>(a.rate + c0 + e0, left, rate);
        float q[8], h[8], mu[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = h[i] = mu[i] = 0.f;
#pragma unroll
        for (int t = 0; t < S; ++t) {
            float x[8];
            rx[t].get(x);
            rg[t].get(sg[t]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sg[t][i] = t < mine ? sigmoid(sg[t][i]) : 0.f;
                const float qt = rate[i] * sg[t][i], e = lost(qt);
                if constexpr (NORM) x[i] *= __builtin_amdgcn_sqrtf(fmaf(-e, e, 2.f * e));
                lo[t][i] = e;
                q[i] += qt;
                h[i] = fmaf(-e, h[i], h[i] + x[i]);
            }
        }
#pragma unroll
        for (int t = S - 1; t >= 0; --t) {
            float d[8];
            rd[t].get(d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float lam = d[i] + mu[i];
                mu[i] = fmaf(-lo[t][i], lam, lam);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            zs[sl][e0 + i] = factor(q[i]);
            hs[sl][e0 + i] = h[i];
            ms[sl][e0 + i] = mu[i];
        }
    }
    __syncthreads();
    if (threadIdx.x < kChannels) {
        const int c = threadIdx.x;
        const bool live = c0 + c < a.D;
        uint64_t *w = a.words + (uint64_t)chain * a.tiles * kChannels + c;
        float z = 0.f, m = 0.f, p = 0.f;
        for (int i = NS - 1; i >= 0; --i) {
            z = both(z, zs[i][c]);
            m = apply(zs[i][c], m) + ms[i][c];
        }
        if (n > 0 && tile > 0) publish(w + (int64_t)n * kChannels, z, m);
        if (live) p = a.carry[((int64_t)b * a.blocks + t0 / MSR_GATE_BLOCK) * a.D + c0 + c];
        for (int i = 0; i < NS; ++i) {
            const float end = hs[i][c];
            hs[i][c] = p;
            p = apply(zs[i][c], p) + end;
        }
        p = 0.f;
        if (n > 0)
            p = look_back(w, n);
        else if (a.state_in && live)
            p = a.state_in[(int64_t)b * a.D + c0 + c];
        const float last = apply(z, p) + m;
        if (tile > 0)
            publish(w + (int64_t)n * kChannels, -0.f, last);
        else if (a.state_out && live)
            a.state_out[(int64_t)b * a.D + c0 + c] = last;
        for (int i = NS - 1; i >= 0; --i) {
            const float end = ms[i][c];
            ms[i][c] = p;
            p = apply(zs[i][c], p) + end;
        }
    }
    __syncthreads();
    float before[S][8], mu[8], dr[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) before[0][i] = hs[sl][e0 + i], mu[i] = ms[sl][e0 + i], dr[i] = 0.f;
#pragma unroll
    for (int t = 0; t + 1 < S; ++t) {
        float x[8];
        rx[t].get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = lo[t][i];
            if constexpr (NORM) x[i] *= __builtin_amdgcn_sqrtf(fmaf(-e, e, 2.f * e));
            before[t + 1][i] = fmaf(-e, before[t][i], before[t][i] + x[i]);
        }
    }
#pragma unroll
    for (int t = S - 1; t >= 0; --t) {
        float x[8], dx[8], dg[8];
        rx[t].get(x);
        rd[t].get(dx);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = lo[t][i], lam = dx[i] + mu[i];
            mu[i] = fmaf(-e, lam, lam);
            float dl = mu[i] * before[t][i];
            dx[i] = lam;
            if constexpr (NORM) {
                const float m2 = fmaf(-e, e, 2.f * e), r = m2 > 1e-36f ? __builtin_amdgcn_rsqf(m2) : 0.f;
                dx[i] = lam * (m2 * r);
                dl = fmaf(-(mu[i] * x[i]), r * (1.f - e), dl);
            }
            const float sd = sg[t][i] * dl;
            dr[i] -= sd;
            dg[i] = (sg[t][i] - 1.f) * (rate[i] * sd);
        }
        if (t < mine) {
            store8<ROWS>(static_cast<T *>(a.y) + at + (int64_t)t * a.D, left, dx);
            store8<ROWS>(static_cast<T *>(a.dg) + at + (int64_t)t * a.D, left, dg);
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) zs[sl][e0 + i] = dr[i];
    __syncthreads();
    if (threadIdx.x < kChannels && c0 + threadIdx.x < a.D) {
        float s = 0.f;
        for (int i = 0; i < NS; ++i) s += zs[i][threadIdx.x];
        a.part[((int64_t)b * a.tiles + tile) * a.D + c0 + threadIdx.x] = s;
    }
}

// One token: h = a state + m x.
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
        const float e = lost(rate[i] * sigmoid(g[i]));
        if constexpr (NORM) x[i] *= __builtin_amdgcn_sqrtf(fmaf(-e, e, 2.f * e));
        y[i] = fmaf(-e, st[i], st[i] + x[i]);
    }
    store8<ROWS>(a.state_out + at, left, y);
    store8<ROWS>(static_cast<T *>(a.y) + at, left, y);
}

// no pair published, no tile taken
__global__ __launch_bounds__(256) void gate_clear_kernel(uint64_t *words, int64_t n, uint32_t *tickets, int64_t chains) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = i0; i < n; i += step) words[i] = ~0ull;
    for (int64_t i = i0; i < chains; i += step) tickets[i] = 0;
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

constexpr int kWaves = 4, kTokens = 4, kTile = 4 * kWaves * kTokens;

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m; }

hipError_t copy(const float *from, float *to, int64_t n, hipStream_t st) {
    if (!to || n == 0) return hipSuccess;
    hipLaunchKernelGGL(gate_copy_kernel, dim3((unsigned)up(n, 256)), dim3(256), 0, st, from, to, n);
    return hipGetLastError();
}

// what the chains need: [words][tickets]
struct Plan {
    int tiles, cols, blocks;
    int64_t chains, words;
    size_t bytes;
};

Plan plan(int B, int T, int D) {
    Plan p;
    p.tiles = (int)up(T, kTile), p.cols = (int)up(D, kChannels), p.blocks = (int)up(T, MSR_GATE_BLOCK);
    p.chains = (int64_t)B * p.cols, p.words = p.tiles > 1 ? p.chains * p.tiles * kChannels : 0;
    p.bytes = p.tiles > 1 ? (size_t)(p.words * 8 + up(p.chains * 4, 256) * 256) : 0;
    return p;
}

hipError_t fill(GateArgs &a, const Plan &p, char *ws, hipStream_t st) {
    a.tiles = p.tiles, a.cols = p.cols, a.blocks = p.blocks;
    if (p.tiles <= 1) return hipSuccess;
    a.words = reinterpret_cast<uint64_t *>(ws);
    a.tickets = reinterpret_cast<uint32_t *>(ws + p.words * 8);
    const int64_t g = std::min<int64_t>(up(p.words, 1024), 2048);
    hipLaunchKernelGGL(gate_clear_kernel, dim3((unsigned)g), dim3(256), 0, st, a.words, p.words, a.tickets, p.chains);
    return hipGetLastError();
}

}  // namespace

size_t gate_workspace(int B, int T, int D, bool backward, bool carry_given) {
    const Plan p = plan(B, T, D);
    size_t n = p.bytes;
    if (backward) {
        n += up((int64_t)B * p.tiles * D * 4, 256) * 256;
        if (!carry_given) n += up((int64_t)B * p.blocks * D * 4, 256) * 256;
    }
    return n;
}

hipError_t launch_gate(const Gate &q, char *ws, hipStream_t st) {
    GateArgs a{};
    a.x = q.x, a.g = q.g, a.rate = q.rate, a.state_in = q.state_in, a.y = q.h, a.state_out = q.state_out, a.carry = q.carry;
    a.B = q.B, a.T = q.T, a.D = q.D;
    if (q.T == 0) return copy(q.state_in, q.state_out, (int64_t)q.B * q.D, st);
    const Plan p = plan(q.B, q.T, q.D);
    hipError_t e = fill(a, p, ws, st);
    if (e != hipSuccess) return e;
    return by_type(q.dtype, q.D, q.normalize, [&](auto t, auto rows, auto norm) {
        hipLaunchKernelGGL((gate_kernel<decltype(t), rows.value, kWaves, kTokens, norm.value>),
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
    const Plan p = plan(q.B, q.T, q.D);
    char *w = ws + p.bytes;
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
        hipLaunchKernelGGL((gate_backward_kernel<decltype(t), rows.value, kWaves, kTokens, norm.value>),
                           dim3((unsigned)(p.chains * p.tiles)), dim3(64 * kWaves), 0, st, a);
        return hipGetLastError();
    });
    if (e == hipSuccess && q.drate) e = launch_column_sum(part, q.drate, nullptr, q.B * p.tiles, q.D, st);
    return e;
}
