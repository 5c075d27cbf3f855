// k_qknorm.hip -- root-mean-square norms of the query and key heads with the
// position rotation in the same pass, and their gradients.  Per row x of d_k
// values (a token's head) at position p, s = 1 for Q and the scale for K:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w,   y = s R(p theta) n
//   u = s R(-p theta) dy,  g = w u,  dx = r (g - x r^2 mean(g x)),
//   dw = sum over rows of u x r
// R turns the pairs (x[2i], x[2i+1]).  Everything is fp32 between the loads
// and the stores (the angles in fp64, rot_cos_sin).
//
// A wave takes a token.  L lanes hold a head's row, eight values each, and a
// wave 64 / L heads at a time: a lane meets the same four pairs in every head,
// so their angles, most of the arithmetic of a row, are formed once per token.
//
// Bound by memory: Q and K of 16384 tokens, 16 heads of 256, bf16 84 us in a
// loop over one set (537 MB; 100 us on changing inputs, 5.4 TB/s), their
// gradients 151 us (805 MB, 5.3 TB/s); a 1 GiB copy reaches 5.1 TB/s.
#include <algorithm>

#include "msr_quant.hpp"

namespace {

using namespace msr;

struct QkArgs {
    const void *x[2], *dy[2];  // Q, K; dy: backward only
    void *y[2];                // results: y, or dx
    const void *w[2];          // may be NULL
    int64_t xs[2], ys[2];      // elements from a token of x (of y) to the next
    float *part;               // backward: [2][parts][dk], or NULL
    const int64_t *pos_rows;
    int64_t pos0, tokens;
    int H[2], dk, T, w_bf16, rotate, per;  // per: head groups that a wave takes of a token
    float scale, eps;
    float theta[MSR_MAX_DK / 2];
};

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}

// the sum over each group of L lanes: neighbours, pairs, then mirrored halves of 8 and 16 (all of whose quads, then
// eights, hold one number by then), then the lane rows
template <int L>
__device__ __forceinline__ float group_sum(float x) {
    if constexpr (L >= 2) x += dpp<0xb1>(x);   // quad_perm 1 0 3 2
    if constexpr (L >= 4) x += dpp<0x4e>(x);   // quad_perm 2 3 0 1
    if constexpr (L >= 8) x += dpp<0x141>(x);  // row_half_mirror
    if constexpr (L >= 16) x += dpp<0x140>(x);  // row_mirror
    if constexpr (L >= 32) {
        const uint32_t u = __float_as_uint(x);
        const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (L >= 64) {
        const uint32_t u = __float_as_uint(x);
        const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return x;
}

// cos and sin of a lane's four pairs at the token's position
__device__ __forceinline__ void angles(const QkArgs &a, int64_t tok, const float (&th)[4], float (&cs)[4], float (&sn)[4]) {
    const uint32_t b = (uint32_t)tok / (uint32_t)a.T, t = (uint32_t)tok - b * (uint32_t)a.T;
    const int64_t p = (a.pos_rows ? a.pos_rows[b] : a.pos0) + t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (a.rotate)
            rot_cos_sin(p, th[i], cs[i], sn[i]);
        else
            cs[i] = 1.f, sn[i] = 0.f;
    }
}

template <typename T, int ROWS, int L>
__global__ __launch_bounds__(256) void qk_norm_kernel(QkArgs a) {
    constexpr int G = 64 / L, U = sizeof(T) == 2 ? 4 : 2;  // head rows of a wave at a time, and of these under way
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int e0 = 8 * (lane % L), sub = lane / L, left = a.dk - e0;
    const int n0 = (a.H[0] + G - 1) / G, n1 = (a.H[1] + G - 1) / G;
    const int it0 = blockIdx.y * a.per, it1 = min(it0 + a.per, n0 + n1);
    float w[2][8], th[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) th[i] = 2 * i < left ? a.theta[e0 / 2 + i] : 0.f;
    load_weight8<ROWS>(a.w[0], a.w_bf16, e0, left, w[0]);
    load_weight8<ROWS>(a.w[1], a.w_bf16, e0, left, w[1]);
    const float dims = (float)a.dk;
    for (int64_t tok = (int64_t)blockIdx.x * 4 + wave; tok < a.tokens; tok += (int64_t)gridDim.x * 4) {
        float cs[4], sn[4];
        angles(a, tok, th, cs, sn);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int base = k ? n0 : 0, lo = max(it0, base), hi = min(it1, k ? n0 + n1 : n0), H = a.H[k];
            const T *x = static_cast<const T *>(a.x[k]) + tok * a.xs[k] + e0;
            T *y = static_cast<T *>(a.y[k]) + tok * a.ys[k] + e0;
            const float s = k ? a.scale : 1.f;
            for (int it = lo; it < hi; it += U) {
                Raw8<T, ROWS> raw[U];
#pragma unroll
                for (int u = 0; u < U; ++u)  // past the last head: that head again, not stored
                    raw[u].load(x + (int64_t)min((it + u - base) * G + sub, H - 1) * a.dk, left);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int head = (it + u - base) * G + sub;
                    if (it + u >= hi) break;
                    float v[8], ss = 0.f;
                    raw[u].get(v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
                    const float ms = group_sum<L>(ss) / dims + a.eps, r = ms == 0.f ? 0.f : s / sqrtf(ms);  // NaN stays
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = v[2 * i] * r * w[k][2 * i], q = v[2 * i + 1] * r * w[k][2 * i + 1];
                        v[2 * i] = p * cs[i] - q * sn[i];
                        v[2 * i + 1] = q * cs[i] + p * sn[i];
                    }
                    if (head < H) store8<ROWS>(y + (int64_t)head * a.dk, left, v);
                }
            }
        }
    }
}

// The weight gradients of a workgroup's rows stay in registers until its last
// row; its waves add up in LDS, its sum goes to `part`, and the parts are
// added in a fixed order afterwards (no atomics).
template <typename T, int ROWS, int L>
__global__ __launch_bounds__(256) void qk_norm_backward_kernel(QkArgs a) {
    constexpr int G = 64 / L, U = sizeof(T) == 2 ? 2 : 1;
    __shared__ float red[3][2][8][L];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int e0 = 8 * (lane % L), sub = lane / L, left = a.dk - e0;
    const int n0 = (a.H[0] + G - 1) / G, n1 = (a.H[1] + G - 1) / G;
    const int it0 = blockIdx.y * a.per, it1 = min(it0 + a.per, n0 + n1);
    float w[2][8], dw[2][8], th[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) th[i] = 2 * i < left ? a.theta[e0 / 2 + i] : 0.f;
    load_weight8<ROWS>(a.w[0], a.w_bf16, e0, left, w[0]);
    load_weight8<ROWS>(a.w[1], a.w_bf16, e0, left, w[1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
    const float dims = (float)a.dk;
    for (int64_t tok = (int64_t)blockIdx.x * 4 + wave; tok < a.tokens; tok += (int64_t)gridDim.x * 4) {
        float cs[4], sn[4];
        angles(a, tok, th, cs, sn);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int base = k ? n0 : 0, lo = max(it0, base), hi = min(it1, k ? n0 + n1 : n0), H = a.H[k];
            const T *x = static_cast<const T *>(a.x[k]) + tok * a.xs[k] + e0;
            const T *dy = static_cast<const T *>(a.dy[k]) + tok * ((int64_t)H * a.dk) + e0;
            T *y = static_cast<T *>(a.y[k]) + tok * a.ys[k] + e0;
            const float s = k ? a.scale : 1.f;
            for (int it = lo; it < hi; it += U) {
                Raw8<T, ROWS> rx[U], rg[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t at = (int64_t)min((it + u - base) * G + sub, H - 1) * a.dk;
                    rx[u].load(x + at, left);
                    rg[u].load(dy + at, left);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int head = (it + u - base) * G + sub;
                    if (it + u >= hi) break;
                    float v[8], g[8], ss = 0.f, gx = 0.f;
                    rx[u].get(v);
                    rg[u].get(g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = g[2 * i], q = g[2 * i + 1];
                        g[2 * i] = s * (p * cs[i] + q * sn[i]);
                        g[2 * i + 1] = s * (q * cs[i] - p * sn[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        ss = fmaf(v[i], v[i], ss);
                        gx = fmaf(v[i], g[i] * w[k][i], gx);
                    }
                    // r^2 = d / (sum(x^2) + d eps), which overflows where the sum is subnormal: there it is scaled first
                    const float t2 = fmaf(a.eps, dims, group_sum<L>(ss));
                    const bool low = t2 < 0x1p-96f;
                    const float root = sqrtf(dims / (low ? t2 * 0x1p64f : t2)), r = t2 == 0.f ? 0.f : low ? root * 0x1p32f : root;
                    gx = group_sum<L>(gx);
                    const float c = r == 0.f ? 0.f : gx / t2;  // squares past fp32: n is 0, whatever the sum came to
                    if (head < H) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            dw[k][i] = fmaf(g[i], v[i] * r, dw[k][i]);
                            v[i] = r * (g[i] * w[k][i] - v[i] * c);
                        }
                        store8<ROWS>(y + (int64_t)head * a.dk, left, v);
                    }
                }
            }
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int o = L; o < 64; o *= 2) dw[k][i] += __shfl_xor(dw[k][i], o, 64);
            if (wave > 0 && sub == 0) red[wave - 1][k][i][lane] = dw[k][i];
        }
    __syncthreads();
    if (wave > 0 || sub > 0) return;
    const size_t parts = (size_t)gridDim.x * gridDim.y, p = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[k][i] += red[0][k][i][lane] + red[1][k][i][lane] + red[2][k][i][lane];
        store8<ROWS>(a.part + (k * parts + p) * a.dk + e0, left, dw[k]);
    }
}

template <int N>
using C = std::integral_constant<int, N>;

template <typename T, int ROWS, typename F>
hipError_t by_lanes(int dk, F f) {
    if (dk <= 8) return f(T(), C<ROWS>(), C<1>());
    if (dk <= 16) return f(T(), C<ROWS>(), C<2>());
    if (dk <= 32) return f(T(), C<ROWS>(), C<4>());
    if (dk <= 64) return f(T(), C<ROWS>(), C<8>());
    if (dk <= 128) return f(T(), C<ROWS>(), C<16>());
    if (dk <= 256) return f(T(), C<ROWS>(), C<32>());
    return f(T(), C<ROWS>(), C<64>());
}

template <typename F>
hipError_t by_type(int dtype, int dk, bool aligned, F f) {
    if (dk < 8) return dtype == MSR_BF16 ? f(uint16_t(), C<kTiny>(), C<1>()) : f(float(), C<kTiny>(), C<1>());
    if (aligned) return dtype == MSR_BF16 ? by_lanes<uint16_t, kAligned>(dk, f) : by_lanes<float, kAligned>(dk, f);
    return dtype == MSR_BF16 ? by_lanes<uint16_t, kAny>(dk, f) : by_lanes<float, kAny>(dk, f);
}

int lanes_of(int dk) {
    int l = 1;
    while (8 * l < dk) l *= 2;
    return l;
}

// Workgroups (four waves, a token each) along the tokens, and the ways a
// token's head groups are split where there are few tokens.
struct Split {
    int x, y, per;
};

Split split(int64_t tokens, int H, int Hk, int dk, int64_t most) {
    const int g = 64 / lanes_of(dk), groups = (H + g - 1) / g + (Hk + g - 1) / g;
    const int64_t x = std::min<int64_t>((tokens + 3) / 4, most);
    const int64_t ways = std::min<int64_t>(std::max<int64_t>(512 / std::max<int64_t>(x, 1), 1), groups);
    const int per = (int)((groups + ways - 1) / ways);
    return {(int)x, (groups + per - 1) / per, per};
}

// Workgroups along the tokens.  Results: 4096 (16384 tokens of 2 x 16 heads of 256 bf16 84 us; 1024 85).  Gradients of short
// tokens, which a wave has done after a few rows, three on a CU, of long ones two (more rows apart at a time cost more than
// they hide), by the bytes of Q and K in a token.  With 768 and with 512, 16384 tokens: bf16 2 x 4 heads of 64 24.3 and 28.5
// us, 2 x 16 of 128 73.4 and 73.9, 32 + 8 of 128 95 and 94, 2 x 16 of 256 159 and 153; fp32 2 x 4 of 128 38.2 and 39.1, 2 x 4
// of 256 79.1 and 79.9, 32 + 8 of 64 100 and 99, 2 x 8 of 256 155.5 and 152.2.
constexpr int kForward = 4096;
int backward_groups(int H, int Hk, int dk, size_t e) { return (H + Hk) * dk * e <= 8192 ? 768 : 512; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

size_t qk_norm_backward_workspace(int64_t tokens, int H, int Hk, int dk) {
    const Split s = split(tokens, H, Hk, dk, backward_groups(H, Hk, dk, 2));  // of either type: fp32 takes no more
    return (size_t)2 * s.x * s.y * dk * sizeof(float);
}

hipError_t launch_qk_norm(const QkNorm &q, bool backward, hipStream_t st) {
    QkArgs a{};
    const size_t e = q.dtype == MSR_BF16 ? 2 : 4;
    bool al = q.dk % 8 == 0;
    for (int k = 0; k < 2; ++k) {
        a.x[k] = q.x[k], a.dy[k] = q.dy[k], a.y[k] = q.y[k], a.w[k] = q.w[k];
        a.xs[k] = q.xs[k], a.ys[k] = q.ys[k], a.H[k] = q.H[k];
        al = al && aligned16(q.x[k]) && aligned16(q.y[k]) && q.xs[k] * e % 16 == 0 && q.ys[k] * e % 16 == 0;
    }
    a.pos_rows = q.pos_rows, a.pos0 = q.pos0, a.tokens = q.tokens;
    a.dk = q.dk, a.T = q.T, a.w_bf16 = q.w_dtype == MSR_BF16, a.rotate = q.rotate, a.scale = q.scale, a.eps = q.eps;
    for (int i = 0; i < q.dk / 2; ++i) a.theta[i] = q.theta[i];
    const int most = backward ? backward_groups(q.H[0], q.H[1], q.dk, e) : kForward;
    const Split s = split(q.tokens, q.H[0], q.H[1], q.dk, most);
    const int parts = s.x * s.y;
    a.per = s.per;
    a.part = backward && (q.dw[0] || q.dw[1]) ? q.part : nullptr;
    hipError_t err = hipSuccess;
    if (q.tokens > 0) {
        err = by_type(q.dtype, q.dk, al, [&](auto t, auto rows, auto l) {
            if (backward)
                hipLaunchKernelGGL((qk_norm_backward_kernel<decltype(t), rows.value, l.value>), dim3(s.x, s.y), dim3(256), 0,
                                   st, a);
            else
                hipLaunchKernelGGL((qk_norm_kernel<decltype(t), rows.value, l.value>), dim3(s.x, s.y), dim3(256), 0, st, a);
            return hipGetLastError();
        });
    }
    if (err == hipSuccess && backward && (q.dw[0] || q.dw[1]))
        err = launch_column_sum(q.part, q.dw[0], q.dw[1], parts, q.dk, st);
    return err;
}
