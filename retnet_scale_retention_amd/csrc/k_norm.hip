// k_norm.hip -- the residual's addition with a root-mean-square norm, its
// output in the input's type and / or in 8 bits with scales, and the
// gradients.  Per row of d values:
//   h = x + r,  rstd = 1 / sqrt(mean(h^2) + eps),  n = h rstd w
//   g = w dn,   dx = rstd (g - h rstd^2 mean(g h)) + dh,  dw = sum_rows dn h rstd
// Everything is fp32 between the loads and the stores; n is taken from the
// unrounded h, so the stored sum's rounding does not reach it.
//
// A row is held in registers by W waves, V groups of 8 elements per lane (but
// for the gradients of rows beyond 16384, or beyond 8192 of a width that is no
// multiple of 8, which are read twice):
// group v of lane l of wave w starts at element 8 (64 (v W + w) + l), so a
// wave reads contiguous kilobytes and a block of 128 is one row of 16 lanes
// (its largest magnitude needs four lane-row rotations, no LDS).  Rows of up
// to 128 (256) elements, a head's for one, take L = 16 (32) lanes, four (two)
// of them to a wave.
//
// Bound by memory: 16384 x 4096 bf16 with the residual's addition and 8-bit
// output 79 us a call on changing inputs (6.0 TB/s of the 472 MB; 69 us in a
// loop over one set, part of it then in the last-level cache; a 1 GiB copy
// reaches 5.1 TB/s), its gradients 95 us (5.7 TB/s; 94 in a loop).  fp32
// 16384 x 2048: 95 us with the residual (537 MB), 41 without (268 MB), in
// a loop.  Times of variants below are of such loops.
#include <algorithm>

#include "msr_quant.hpp"

namespace {

using namespace msr;

struct NormArgs {
    const void *x, *r, *w;  // r, w may be NULL
    void *sum, *y;          // may be NULL
    uint8_t *q;             // may be NULL; [rows][dpad]
    float *qs;              // [rows][dpad / 128]
    int64_t row0, rows;     // first row of this launch
    int d, dpad, w_bf16;
    float eps;
};

// the sum over the L lanes of a wave that share a row
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
    if constexpr (L == 64) return wave_sum_dpp(x);
    x = row16_sum(x);
    if constexpr (L == 32) {
        const uint32_t u = __float_as_uint(x);
        const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return x;
}

// the sum over the W waves (of L lanes) that share a row (team `tm` of the workgroup)
template <int W, int L>
__device__ __forceinline__ float team_sum(float x, float *red, int tm, int w) {
    x = lanes_sum<L>(x);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) red[tm * W + w] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) x += red[tm * W + i];
    }
    return x;
}

template <typename T, int ROWS, int W, int V, int L>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void add_rmsnorm_kernel(NormArgs a) {
    constexpr int TEAMS = W < 4 ? 4 / W : 1;
    static_assert(L == 64 || W * V == 1, "");
    __shared__ float red[TEAMS * W];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tm = wave / W, w = wave % W;
    const int64_t row_raw = a.row0 + ((int64_t)blockIdx.x * TEAMS + tm) * (64 / L) + lane / L;
    const int e0 = 8 * (64 * w + lane % L);  // group v starts at e0 + 512 W v
    const bool live = row_raw < a.rows;
    const int64_t row = live ? row_raw : a.rows - 1;  // a team past the end repeats the last row and stores nothing
    const T *x = static_cast<const T *>(a.x) + row * a.d;
    const T *r = a.r ? static_cast<const T *>(a.r) + row * a.d : nullptr;
    float h[V][8];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = e0 + 512 * W * v;
        load8<ROWS>(x + e, a.d - e, h[v]);
    }
    if (r) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = e0 + 512 * W * v;
            float t[8];
            load8<ROWS>(r + e, a.d - e, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[v][i] += t[i];
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[v][i], h[v][i], ss);
    if (a.sum && live) {
        T *s = static_cast<T *>(a.sum) + row * a.d;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = e0 + 512 * W * v;
            store8<ROWS>(s + e, a.d - e, h[v]);
        }
    }
    const float rstd = 1.f / sqrtf(team_sum<W, L>(ss, red, tm, w) / (float)a.d + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = e0 + 512 * W * v;
        float g[8];
        load_weight8<ROWS>(a.w, a.w_bf16, e, a.d - e, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * rstd * g[i];
        if (a.y && live) store8<ROWS>(static_cast<T *>(a.y) + row * a.d + e, a.d - e, h[v]);
        if (a.q) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, abs_bits(h[v][i]));
            const float s = block_scale(row16_max(m));
            if (live && e < a.dpad) {
                stream_out(a.q + row * a.dpad + e, pack8(h[v], s));
                if ((lane & 15) == 0) a.qs[row * (a.dpad / kBlock) + e / kBlock] = s;
            }
        }
    }
}

struct NormBackArgs {
    const void *h, *w, *dy, *dsum;  // w, dsum may be NULL
    void *dx;
    float *part;                    // [gridDim.x][d], or NULL: no weight gradient
    int64_t rows;
    int d, w_bf16;
    float eps;
};

// Each team walks over rows team, team + teams, ... with the next row's loads
// under way (where the registers allow), and keeps the weight and its
// gradient over those rows in registers (the row's values as loaded: held as
// floats across the barrier, 512 workgroups took 118 us instead of 101 for
// 16384 x 4096; without the loads ahead 216);
// the workgroup's teams add up in LDS, its sum goes to `part`, and
// column_sum_kernel adds the parts in a fixed order (no atomics).
template <typename T, int ROWS, int W, int V, int L>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void rmsnorm_backward_kernel(NormBackArgs a) {
    constexpr int TEAMS = W < 4 ? 4 / W : 1, PER = 64 / L;  // teams of a workgroup, rows of a team at a time
    static_assert(L == 64 || W * V == 1, "");
    __shared__ float red[2][2 * TEAMS * W];
    __shared__ float dws[TEAMS > 1 ? TEAMS - 1 : 1][TEAMS > 1 ? 512 * W * V : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tm = wave / W, w = wave % W;
    const int64_t team = ((int64_t)blockIdx.x * TEAMS + tm) * PER + lane / L, teams = (int64_t)gridDim.x * TEAMS * PER;
    const int64_t turns = (a.rows + teams - 1) / teams;  // the same for every team: the barriers match
    const int e0 = 8 * (64 * w + lane % L);              // group v starts at e0 + 512 W v
    // the longest rows are read a second time instead of kept, and their weight gradient stays in LDS (all in registers,
    // 276 of them spilled: 1024 x 32768 bf16 231 us)
    constexpr bool keep = W * V <= (ROWS == kAligned ? 32 : 16);
    __shared__ __attribute__((aligned(16))) float4 dwl[keep ? 1 : 128 * W * V];
    Raw8<T, ROWS> hr[V], gr[V], dr[V];
    auto fetch = [&](int64_t t) {  // past the last row: that row again, not used
        const int64_t r = t * teams + team, row = r < a.rows ? r : a.rows - 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = e0 + 512 * W * v;
            hr[v].load(static_cast<const T *>(a.h) + row * a.d + e, a.d - e);
            gr[v].load(static_cast<const T *>(a.dy) + row * a.d + e, a.d - e);
            if (a.dsum) dr[v].load(static_cast<const T *>(a.dsum) + row * a.d + e, a.d - e);
        }
    };
    constexpr bool early = keep && V * sizeof(T) <= 8;
    float wt[V][8], dw[V][8];
    if (keep) fetch(0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = e0 + 512 * W * v;
        if constexpr (keep) {
            load_weight8<ROWS>(a.w, a.w_bf16, e, a.d - e, wt[v]);
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[v][i] = 0.f;
        } else {
            dwl[64 * (2 * (v * W + w)) + lane] = dwl[64 * (2 * (v * W + w) + 1) + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    const float dims = (float)a.d;
    for (int64_t t = 0; t < turns; ++t) {
        const int64_t row = t * teams + team;
        const int64_t at = (row < a.rows ? row : a.rows - 1) * a.d;
        Raw8<T, ROWS> hc[V], gc[V], dc[V];
        if constexpr (keep) {
#pragma unroll
            for (int v = 0; v < V; ++v) hc[v] = hr[v], gc[v] = gr[v], dc[v] = dr[v];
        }
        if (early && t + 1 < turns) fetch(t + 1);
        float ss = 0.f, gh = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float h[8], g[8];
            if constexpr (!keep) {
                const int e = e0 + 512 * W * v;
                __builtin_amdgcn_sched_barrier(0);  // a group's loads at a time
                hc[v].load(static_cast<const T *>(a.h) + at + e, a.d - e);
                gc[v].load(static_cast<const T *>(a.dy) + at + e, a.d - e);
                load_weight8<ROWS>(a.w, a.w_bf16, e, a.d - e, wt[v]);
            }
            hc[v].get(h);
            gc[v].get(g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = fmaf(h[i], h[i], ss);
                gh = fmaf(h[i], g[i] * wt[v][i], gh);
            }
        }
        ss = lanes_sum<L>(ss);
        gh = lanes_sum<L>(gh);
        if constexpr (W > 1) {
            float *rd = red[t & 1];  // two areas: one barrier per turn separates a turn's reads from its writes
            if (lane == 0) {
                rd[2 * (tm * W + w)] = ss;
                rd[2 * (tm * W + w) + 1] = gh;
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the next row's loads stay under way
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            ss = gh = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                ss += rd[2 * (tm * W + i)];
                gh += rd[2 * (tm * W + i) + 1];
            }
        }
        // rstd^2 = d / (sum(h^2) + d eps): no mean is formed, since a product with 1 / d, rounded itself, shifts every row of
        // a width alike, and a division by d takes longer (16384 x 4096 bf16 94.5 us, 94.1 so)
        const float t2 = fmaf(a.eps, dims, ss);
        const float rstd = sqrtf(dims / t2);
        const float c = rstd == 0.f ? 0.f : gh / t2;  // squares past fp32: n is 0, whatever gh came to
        if (row >= a.rows) continue;  // the last turn of this team
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = e0 + 512 * W * v;
            float h[8], g[8], ds[8], o[8];
            if constexpr (keep) {
                hc[v].forget();
                gc[v].forget();
            } else {
                __builtin_amdgcn_sched_barrier(0);
                hc[v].load(static_cast<const T *>(a.h) + at + e, a.d - e);
                gc[v].load(static_cast<const T *>(a.dy) + at + e, a.d - e);
                if (a.dsum) dc[v].load(static_cast<const T *>(a.dsum) + at + e, a.d - e);
                load_weight8<ROWS>(a.w, a.w_bf16, e, a.d - e, wt[v]);
            }
            hc[v].get(h);
            gc[v].get(g);
            if (a.dsum) {
                dc[v].get(ds);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) ds[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = fmaf(rstd, g[i] * wt[v][i] - h[i] * c, ds[i]);
                if constexpr (keep) dw[v][i] = fmaf(g[i], h[i] * rstd, dw[v][i]);
            }
            if constexpr (!keep) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {  // this lane's own numbers: no barrier
                    float4 &x = dwl[64 * (2 * (v * W + w) + b) + lane];
                    float4 y = x;
                    y.x = fmaf(g[4 * b], h[4 * b] * rstd, y.x);
                    y.y = fmaf(g[4 * b + 1], h[4 * b + 1] * rstd, y.y);
                    y.z = fmaf(g[4 * b + 2], h[4 * b + 2] * rstd, y.z);
                    y.w = fmaf(g[4 * b + 3], h[4 * b + 3] * rstd, y.w);
                    x = y;
                }
            }
            store8<ROWS>(static_cast<T *>(a.dx) + row * a.d + e, a.d - e, o);
        }
        if (keep && !early && t + 1 < turns) fetch(t + 1);
    }
    if (a.part) {
        if constexpr (PER > 1) {  // the rows of a team
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t u = __float_as_uint(dw[0][i]);
                if constexpr (PER == 4) {
                    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
                    u = __float_as_uint(__uint_as_float(r[0]) + __uint_as_float(r[1]));
                }
                const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
                dw[0][i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
            }
        }
        if constexpr (TEAMS > 1) {
            if (tm > 0) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < 8; ++i) dws[tm - 1][(v * W + w) * 512 + i * 64 + lane] = dw[v][i];
            }
            __syncthreads();
            if (tm > 0) return;
#pragma unroll
            for (int q = 0; q < TEAMS - 1; ++q)
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < 8; ++i) dw[v][i] += dws[q][(v * W + w) * 512 + i * 64 + lane];
        }
        if (lane >= L) return;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = e0 + 512 * W * v;
            if constexpr (!keep) {
                const float4 x = dwl[64 * (2 * (v * W + w)) + lane], y = dwl[64 * (2 * (v * W + w) + 1) + lane];
                const float z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                store8<ROWS>(a.part + (int64_t)blockIdx.x * a.d + e, a.d - e, z);
            } else {
                store8<ROWS>(a.part + (int64_t)blockIdx.x * a.d + e, a.d - e, dw[v]);
            }
        }
    }
}

// out[c] = sum_p part[p][c] for 32 columns: p in order within each of 64
// slices (eight loads of four columns under way), the slices in pairs, pairs
// of pairs, ... (one after the other, the last sums' roundings were most of
// the weight gradient's error: 1.7e-7 of its norm for 3001 x 1000 fp32, not 1.0e-7)
__global__ __launch_bounds__(512) void column_sum_kernel(const float *part, float *out, int parts, int d) {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    __shared__ float red[64][33];
    const int q = 4 * (threadIdx.x & 7), c = (int)blockIdx.x * 32 + q, sl = threadIdx.x >> 3;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (c + 4 <= d) {
        for (int p0 = sl; p0 < parts; p0 += 512) {
            f32x4 x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {  // zeros past the last part
                x[u] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (p0 + 64 * u < parts) x[u] = load_any<f32x4>(part + (size_t)(p0 + 64 * u) * d + c);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) s += x[u];
        }
    } else {
        for (int p = sl; p < parts; p += 64)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < d) s[i] += part[(size_t)p * d + c + i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[sl][q + i] = s[i];
    __syncthreads();
    if (threadIdx.x < 32) {
        float t[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) t[i] = red[i][threadIdx.x];
#pragma unroll
        for (int n = 32; n > 0; n /= 2)
#pragma unroll
            for (int i = 0; i < n; ++i) t[i] += t[i + n];
        const int o = (int)blockIdx.x * 32 + threadIdx.x;
        if (o < d) out[o] = t[0];
    }
}

template <int N>
using C = std::integral_constant<int, N>;

// (waves, groups per lane, lanes of a wave) that hold a row of d <= 8 L W V
// values.  Twice the waves with one group each (ONE) suit the gradients (16384
// x 4096: 93 us against 98, f32 16384 x 2048 94 against 101) and f32 forwards
// (16384 x 2048 with 8-bit output 77 against 79), whose lanes have 32 bytes of
// each array under way all the same; bf16 forwards want two (70 against 76).
template <bool ONE, typename F>
hipError_t by_width(int d, F f) {
    constexpr int m = ONE ? 2 : 1;
    if (d <= 128) return f(C<1>(), C<1>(), C<16>());
    if (d <= 256) return f(C<1>(), C<1>(), C<32>());
    if (d <= 512) return f(C<1>(), C<1>(), C<64>());
    if (d <= 1024) return f(C<m>(), C<2 / m>(), C<64>());
    if (d <= 2048) return f(C<2 * m>(), C<2 / m>(), C<64>());
    if (d <= 4096) return f(C<4 * m>(), C<2 / m>(), C<64>());
    if (d <= 8192) return f(C<8 * m>(), C<2 / m>(), C<64>());
    if (d <= 16384) return f(C<8>(), C<4>(), C<64>());
    return f(C<16>(), C<4>(), C<64>());
}

template <bool ONE, typename T, typename F>
hipError_t by_rows(int d, F f) {
    if (d % 8 == 0) return by_width<ONE>(d, [&](auto... c) { return f(T(), C<kAligned>(), c...); });
    if (d > 8) return by_width<ONE>(d, [&](auto... c) { return f(T(), C<kAny>(), c...); });
    return f(T(), C<kTiny>(), C<1>(), C<1>(), C<16>());
}

// Workgroups of the backward pass: each writes one partial weight gradient.
// At most 512 of them where a workgroup's rows are up to 4 KiB, 256 where
// they are longer: about 6 MB under way in both cases (512 x bf16: 43 us
// against 52 for 65536 rows, but 4096 x bf16 100 against 93 for 16384); about
// one per eight rows but no fewer than the CUs (few rows: the parts' own bytes
// count), evened out so that all walk over equally many rows.  A few turns of
// one workgroup go straight into the weight gradient instead of a second
// launch (bf16, 32 x 512 7.1 us against 11.5, 8 x 4096 9.6 against 11.7, but
// 12 x 4096 13.3 and 8 x 16384 21).
constexpr int kBackGroups = 512;

int back_groups(int64_t rows, int d, int dtype) {
    if (rows == 0) return 0;
    const int64_t teams = d <= 128 ? 16 : d <= 256 ? 8 : d <= 512 ? 4 : d <= 1024 ? 2 : 1;  // rows at a time, by_width
    if (rows <= std::min(8, std::max(MSR_MAX_NORM_DIM / d, 1)) * teams) return 1;
    const int64_t most = teams * d * (dtype == MSR_BF16 ? 2 : 4) <= 4096 ? kBackGroups : kBackGroups / 2;
    const int64_t g = std::min((rows + teams - 1) / teams, std::min(std::max<int64_t>(rows / 8, 256), most));
    const int64_t turns = std::max<int64_t>((rows + g * teams / 2) / (g * teams), 1);
    return (int)std::min<int64_t>((rows + turns * teams - 1) / (turns * teams), kBackGroups);
}

}  // namespace

hipError_t launch_add_rmsnorm(int64_t rows, int d, int dtype, const void *x, const void *r, const void *w, int w_dtype,
                              float eps, void *sum, void *y, void *q, float *qs, hipStream_t st) {
    NormArgs a{x, r, w, sum, y, static_cast<uint8_t *>(q), qs, 0, rows, d, (int)round128(d), w_dtype == MSR_BF16, eps};
    auto launch = [&](auto t, auto rw, auto W, auto V, auto L) {
        constexpr int teams = (W.value < 4 ? 4 / W.value : 1) * (64 / L.value), nt = W.value < 4 ? 256 : 64 * W.value;
        constexpr int64_t most = (int64_t)1 << 21;  // workgroups of a launch: its threads stay below 2^32
        hipError_t e = hipSuccess;
        for (a.row0 = 0; a.row0 < rows && e == hipSuccess; a.row0 += most * teams) {
            const int64_t g = std::min<int64_t>((rows - a.row0 + teams - 1) / teams, most);
            hipLaunchKernelGGL((add_rmsnorm_kernel<decltype(t), rw.value, W.value, V.value, L.value>), dim3((unsigned)g),
                               dim3(nt), 0, st, a);
            e = hipGetLastError();
        }
        return e;
    };
    return dtype == MSR_BF16 ? by_rows<false, uint16_t>(d, launch) : by_rows<true, float>(d, launch);
}

// enough for either type; none for a single part, which is the weight gradient itself
size_t rmsnorm_backward_workspace(int64_t rows, int d) {
    const int parts = std::max(back_groups(rows, d, MSR_BF16), back_groups(rows, d, MSR_F32));
    return parts > 1 ? (size_t)parts * d * sizeof(float) : 0;
}

hipError_t launch_rmsnorm_backward(int64_t rows, int d, int dtype, const void *h, const void *w, int w_dtype, float eps,
                                   const void *dy, const void *dsum, void *dx, float *dw, float *part, hipStream_t st) {
    const int parts = back_groups(rows, d, dtype);
    const NormBackArgs a{h, w, dy, dsum, dx, dw ? (parts > 1 ? part : dw) : nullptr, rows, d, w_dtype == MSR_BF16, eps};
    auto launch = [&](auto t, auto rw, auto W, auto V, auto L) {
        constexpr int nt = W.value < 4 ? 256 : 64 * W.value;
        hipLaunchKernelGGL((rmsnorm_backward_kernel<decltype(t), rw.value, W.value, V.value, L.value>), dim3(parts),
                           dim3(nt), 0, st, a);
        return hipGetLastError();
    };
    hipError_t e = hipSuccess;
    if (parts > 0) e = dtype == MSR_BF16 ? by_rows<true, uint16_t>(d, launch) : by_rows<true, float>(d, launch);
    if (e == hipSuccess && dw && parts != 1) {
        hipLaunchKernelGGL(column_sum_kernel, dim3((d + 31) / 32), dim3(512), 0, st, part, dw, parts, d);
        e = hipGetLastError();
    }
    return e;
}
