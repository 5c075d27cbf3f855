// k_matmul.hip -- the matrix product of 8-bit operands with one fp32 scale
// per block of 128 along the contraction:
//   C[m][n] = sum_kb sa[m][kb] sb[n'][kb] sum_{k in kb} a[m][k] b[n][k],
// n' = n (B scaled by rows) or n / 128 (B scaled in 128 x 128 squares).
// Both operands are rows of contraction-contiguous e4m3 bytes, so a step of
// the contraction is one block, 128 bytes per row: it is multiplied by the
// matrix cores into a fresh fp32 tile, which is then folded into the running
// fp32 sum with its scales.
//
// Two ways to multiply a block, by the output's type:
//   bf16 output: the 8-bit instruction (16x16x128).  It aligns each 8
//     consecutive products before adding them and drops what lies more than
//     13 bits below the largest's exponent (measured); the loss, about
//     1.5e-5 of the result for normal values, is far below bf16's 2^-9.
//   fp32 output: the values widened to bf16 (exact) and the bf16 instruction
//     (16x16x32), whose products and sums keep fp32's accuracy.
#include "msr_quant.hpp"

namespace {

using namespace msr;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct MatArgs {
    const uint8_t *a, *b;
    const float *sa, *sb;
    void *out;
    int M, N, K, nkb;  // nkb = K / 128 (K is padded to whole blocks)
    int mt, nt;
};

constexpr int kUnitScale = 0x7f7f7f7f;  // the instruction's own block scales, all 2^0

struct Frag {  // 32 contraction bytes of one row per lane: a 16-row operand of one block
    i32x4 lo, hi;
};

__device__ __forceinline__ bf16x8 widen(int lo, int hi) {
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
    return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

__device__ __forceinline__ f32x4 block_product(const Frag &x, const Frag &y) {
    const i32x8 a = {x.lo[0], x.lo[1], x.lo[2], x.lo[3], x.hi[0], x.hi[1], x.hi[2], x.hi[3]};
    const i32x8 b = {y.lo[0], y.lo[1], y.lo[2], y.lo[3], y.hi[0], y.hi[1], y.hi[2], y.hi[3]};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, kUnitScale, 0,
                                                            kUnitScale);
}

struct WideFrag {  // the same operand as bf16: four contraction steps of 32
    bf16x8 s[4];
};

__device__ __forceinline__ WideFrag widen(const Frag &f) {
    return {{widen(f.lo[0], f.lo[1]), widen(f.lo[2], f.lo[3]), widen(f.hi[0], f.hi[1]), widen(f.hi[2], f.hi[3])}};
}

__device__ __forceinline__ f32x4 block_product(const WideFrag &x, const WideFrag &y) {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.s[i], y.s[i], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ void load_lds16(const void *gptr, void *lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)gptr,
                                     (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}

// Four consecutive output features of one token (n < N for the first).
template <typename OUT>
__device__ __forceinline__ void store_row4(OUT *row, int n, int N, f32x4 v) {
    if ((N & 3) == 0) {
        if constexpr (sizeof(OUT) == 2)
            *reinterpret_cast<uint2 *>(row + n) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        else
            *reinterpret_cast<float4 *>(row + n) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < N) store(row, n + r, v[r]);
    }
}

// A workgroup of WM x WN waves computes a tile of BM tokens by BN features.
// B's rows are the instruction's first operand: lane (l16, g) of a 16 x 16
// result holds token l16 and features 4 g .. 4 g + 3, so A's scale is one
// number per lane and the four results are neighbours in the output row.
// Each block's bytes go straight into LDS (direct 16-byte loads, one block
// ahead into the other of two buffers); rows are 128 bytes, their 16-byte
// chunks XOR-swizzled by row through the choice of each lane's source chunk.
template <int BM, int BN, int WM, int WN, typename OUT, bool BROW>
__global__ __launch_bounds__(64 * WM * WN) void matmul_tile_kernel(MatArgs a) {
    constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr bool WIDE = sizeof(OUT) == 4;
    constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // 1 KiB loads per wave and block
    __shared__ __attribute__((aligned(1024))) char As[2][BM * 128];
    __shared__ __attribute__((aligned(1024))) char Bs[2][BN * 128];

    const int total = a.mt * a.nt, per = (total + 7) / 8;
    const int id = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
    if ((int)(blockIdx.x / 8) >= per || id >= total) return;
    const int grp = id / (8 * a.nt), in = id % (8 * a.nt), gm = min(8, a.mt - grp * 8);
    const int m0 = (grp * 8 + in % gm) * BM, n0 = in / gm * BN;

    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4, wm = wv / WN, wn = wv % WN;

    const uint8_t *ag[LA], *bg[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int r = 8 * (wv + NW * i) + (lane >> 3);
        ag[i] = a.a + (size_t)min(m0 + r, a.M - 1) * a.K + 16 * ((lane & 7) ^ (r & 7));
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int r = 8 * (wv + NW * i) + (lane >> 3);
        bg[i] = a.b + (size_t)min(n0 + r, a.N - 1) * a.K + 16 * ((lane & 7) ^ (r & 7));
    }
    auto issue = [&](int kb, int buf) {
#pragma unroll
        for (int i = 0; i < LA; ++i) load_lds16(ag[i] + (size_t)kb * 128, As[buf] + (wv + NW * i) * 1024);
#pragma unroll
        for (int i = 0; i < LB; ++i) load_lds16(bg[i] + (size_t)kb * 128, Bs[buf] + (wv + NW * i) * 1024);
    };
    auto frag = [&](const char *base, int row) {
        Frag f;
        f.lo = *reinterpret_cast<const i32x4 *>(base + row * 128 + (((2 * g) ^ (row & 7)) << 4));
        f.hi = *reinterpret_cast<const i32x4 *>(base + row * 128 + (((2 * g + 1) ^ (row & 7)) << 4));
        return f;
    };
    const int mw = m0 + wm * (BM / WM), nw = n0 + wn * (BN / WN);  // the wave's corner

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (a.nkb > 0) issue(0, 0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int kb = 0; kb < a.nkb; ++kb) {
        const int buf = kb & 1;
        float sa[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = a.sa[(size_t)min(mw + 16 * i + l16, a.M - 1) * a.nkb + kb];
        if (kb + 1 < a.nkb) issue(kb + 1, buf ^ 1);
        using F = std::conditional_t<WIDE, WideFrag, Frag>;
        auto conv = [](const Frag &f) -> F {
            if constexpr (WIDE) return widen(f);
            else return f;
        };
        F fa[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[i] = conv(frag(As[buf], wm * (BM / WM) + 16 * i + l16));
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const F fb = conv(frag(Bs[buf], wn * (BN / WN) + 16 * j + l16));
            f32x4 sb;
            if constexpr (BROW) {
#pragma unroll
                for (int r = 0; r < 4; ++r) sb[r] = a.sb[(size_t)min(nw + 16 * j + 4 * g + r, a.N - 1) * a.nkb + kb];
            } else {
                const float s = a.sb[(size_t)(min(nw + 16 * j, a.N - 1) >> 7) * a.nkb + kb];
                sb = f32x4{s, s, s, s};
            }
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const f32x4 p = block_product(fb, fa[i]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(p[r], sa[i] * sb[r], acc[i][j][r]);
            }
        }
        __builtin_amdgcn_s_waitcnt(0);  // the next block has landed
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = mw + 16 * i + l16;
        if (m >= a.M) continue;
        OUT *row = static_cast<OUT *>(a.out) + (size_t)m * a.N;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int n = nw + 16 * j + 4 * g;
            if (n < a.N) store_row4(row, n, a.N, acc[i][j]);
        }
    }
}

template <typename OUT, bool BROW>
hipError_t matmul(MatArgs a, hipStream_t st) {
    constexpr int BM = 128, BN = 128;
    a.mt = (a.M + BM - 1) / BM;
    a.nt = (a.N + BN - 1) / BN;
    const unsigned grid = (unsigned)((a.mt * a.nt + 7) / 8 * 8);
    hipLaunchKernelGGL((matmul_tile_kernel<BM, BN, 2, 2, OUT, BROW>), dim3(grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace

size_t scaled_matmul_workspace(int64_t m, int64_t n, int64_t k, int out_dtype) { return 0; }

hipError_t launch_scaled_matmul(int m, int n, int k, const void *A, const float *sa, const void *B, const float *sb,
                                int b_rows, int out_dtype, void *out, void *ws, hipStream_t st) {
    const MatArgs a{static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(B), sa, sb, out, m, n, k, k / 128, 0, 0};
    if (out_dtype == MSR_BF16) return b_rows == 1 ? matmul<uint16_t, true>(a, st) : matmul<uint16_t, false>(a, st);
    return b_rows == 1 ? matmul<float, true>(a, st) : matmul<float, false>(a, st);
}
