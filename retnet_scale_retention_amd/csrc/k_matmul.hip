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

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}

// 16 (or 4) bytes per lane from a buffer straight into LDS, lane l's at dst + 16 l (4 l; dst wave-uniform); past the
// buffer's end zeros arrive
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, char *dst, int lane_off, int off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)dst, 16, lane_off, off, 0, 0);
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, char *dst, int lane_off, int off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)dst, 4, lane_off, off, 0, 0);
}

// vmcnt(N) and lgkmcnt(0), then a barrier
template <int N>
__device__ __forceinline__ void wait_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// a number that is the same for the whole wave, through the scalar cache
__device__ __forceinline__ float uniform_load(const float *p) {
    return *(const __attribute__((address_space(4))) float *)p;
}

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

template <typename OUT>
using OperandOf = std::conditional_t<sizeof(OUT) == 4, WideFrag, Frag>;

template <typename OUT>
__device__ __forceinline__ OperandOf<OUT> operand(const Frag &f) {
    if constexpr (sizeof(OUT) == 4) return widen(f);
    else return f;
}

// Rows of a block in LDS are 128 bytes, their 16-byte chunks XOR-swizzled by
// half the row number.  Lane (l16, g) of a 16-row operand takes chunks g and
// g + 4 of row l16 (any split of the 128 will do that both operands share):
// each quarter of the lanes that LDS serves together then touches all 64
// banks once (no conflicts measured; keyed by the row number itself, half
// the cycles were conflicts).
struct LaneRow {
    int lo, hi;
    __device__ __forceinline__ explicit LaneRow(int lane) {
        const int l16 = lane & 15, g = lane >> 4, key = l16 >> 1;
        lo = l16 * 128 + ((g ^ key) << 4);
        hi = l16 * 128 + (((g + 4) ^ key) << 4);
    }
    __device__ __forceinline__ Frag load(const char *rows) const {
        return {*reinterpret_cast<const i32x4 *>(rows + lo), *reinterpret_cast<const i32x4 *>(rows + hi)};
    }
};

// Where lane l of a 1 KiB load of rows 8 q .. 8 q + 7 (128 bytes each, K
// apart) finds the bytes that the swizzle puts at its place.
__device__ __forceinline__ int swizzled_source(int lane, int q, int K) {
    return (lane >> 3) * K + 16 * ((lane & 7) ^ ((4 * (q & 1) + (lane >> 4)) & 7));
}

// Four consecutive output features of one token (n < N for the first), at an element's own alignment.
template <typename OUT>
__device__ __forceinline__ void store_row4(OUT *row, int n, int N, f32x4 v) {
    if (n + 4 <= N) {
        if constexpr (sizeof(OUT) == 2)
            store_any(row + n, (uint64_t)pack_bf16(v[2], v[3]) << 32 | pack_bf16(v[0], v[1]));
        else
            store_any(row + n, v);
    } else {
#pragma unroll
        for (int r = 0; r < 3; ++r)
            if (n + r < N) store(row, n + r, v[r]);
    }
}

// Results v, w of two neighbouring column tiles as bf16: lanes of even g get eight features of the first tile, of odd g
// of the second, 8 (g / 2) .. + 7.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4 pack_pair(f32x4 v, f32x4 w) {
    const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16(v[0], v[1]), pack_bf16(w[0], w[1]), false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16(v[2], v[3]), pack_bf16(w[2], w[3]), false, false);
    return u32x4{lo[0], hi[0], lo[1], hi[1]};
}

// Tile id -> (row tile, column tile).  Ids are dealt round-robin over the 8
// XCDs; each takes a contiguous range of an order in which groups of 8 row
// tiles sweep the column tiles, so what runs together on an XCD shares rows
// of A and B in its L2.
__device__ __forceinline__ bool tile_of(int block, int mt, int nt, int &tm, int &tn) {
    const int total = mt * nt, per = (total + 7) / 8, id = block % 8 * per + block / 8;
    if (block / 8 >= per || id >= total) return false;
    const int grp = id / (8 * nt), in = id % (8 * nt), gm = min(8, mt - grp * 8);
    tm = grp * 8 + in % gm;
    tn = in / gm;
    return true;
}

// A tile of BM tokens by BN features per workgroup of KG x WM x WN waves; the
// KG groups share out the contraction's blocks and add up in LDS at the end.
// B's rows are the instruction's first operand: lane (l16, g) of a 16 x 16
// result holds token l16 and features 4 g .. 4 g + 3, so A's scale is one
// number per lane and the four results are neighbours in the output row.
// Blocks go straight into a ring of ST LDS stages (16-byte direct loads),
// ST - 1 blocks ahead, with one barrier per block.  The stages are separate
// arrays: the compiler then knows that reads of one do not wait for the loads
// into the others (in one array it drained every load before each block's
// first read: 787 us against 645 for 16384 x 8192 x 4096, which take 605 with
// the stores of today; the large kernel below 470).
// With fp32 output the vector instructions bind it: a bf16 matrix instruction
// takes 8 cycles of a SIMD's issue and 16 of its matrix core, a vector
// instruction 4.3, and at 128 x 128 (64 x 64 per wave) each matrix instruction
// comes with two conversions and, B scaled by rows, a scale product and a
// fold: 26 cycles at best, 30 measured (4096 x 4096 x 16384: 505-511 us = 1080
// TFLOP/s in a loop over one set of operands, 525-548 a call on changing ones,
// the clock at 1.94 GHz by the chip's power; in the loop 486 us without the
// conversions, 433 over zeros).  Reading the operands half a block ahead, or
// spreading all vector work evenly between the matrix instructions, won
// nothing (539, 543 us where this took 515).
template <int BM, int BN, int KG, int WM, int WN, int ST, typename OUT, bool BROW>
__device__ __forceinline__ void tile_body(const MatArgs &a) {
    constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int LA = BM / 8, L = (BM + BN) / 8 / NW;  // 1 KiB loads of a block's A, and of a wave
    constexpr int SA = (BM + BN) * 128, SB = SA + (BM < 64 ? 64 : BM) * 4;
    constexpr int STAGE = SB + (BROW ? (BN < 64 ? 64 : BN) * 4 : 0);
    constexpr int NSA = (BM + 63) / 64, NS = NSA + (BROW ? (BN + 63) / 64 : 0);  // loads of 64 scales
    static_assert((BM + BN) / 8 % NW == 0 && NS <= NW && ST >= 2 && ST <= 4, "");
    __shared__ __attribute__((aligned(1024))) char S0[KG * STAGE];
    __shared__ __attribute__((aligned(1024))) char S1[KG * STAGE];
    __shared__ __attribute__((aligned(1024))) char S2[ST > 2 ? KG * STAGE : 16];
    __shared__ __attribute__((aligned(1024))) char S3[ST > 3 ? KG * STAGE : 16];

    int tm, tn;
    if (!tile_of(blockIdx.x, a.mt, a.nt, tm, tn)) return;
    const int m0 = tm * BM, n0 = tn * BN, K = a.K, nkb = a.nkb;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = wave / NW, wv = wave % NW, l16 = lane & 15, g = lane >> 4;
    const int ar = wv / WN * (BM / WM), br = wv % WN * (BN / WN);
    const int steps = (nkb + KG - 1) / KG, k0 = kg * steps, k1 = min(k0 + steps, nkb);

    const auto ra = rsrc(a.a + (size_t)m0 * K, (uint32_t)(min(a.M - m0, BM) * K));
    const auto rb = rsrc(a.b + (size_t)n0 * K, (uint32_t)(min(a.N - n0, BN) * K));
    const int vo[2] = {swizzled_source(lane, wv * L, K), swizzled_source(lane, wv * L + 1, K)};
    // every wave brings 64 scales (those past the last repeat the first), so that all wait for the same count
    const int sw = wv < NS ? wv : 0, srow = sw < NSA ? 64 * sw : 64 * (sw - NSA);
    const auto rs = sw < NSA ? rsrc(a.sa + (size_t)m0 * nkb, (uint32_t)(min(a.M - m0, BM) * nkb * 4))
                             : rsrc(a.sb + (size_t)n0 * nkb, (uint32_t)(min(a.N - n0, BN) * nkb * 4));
    const int so = (srow + lane) * nkb * 4, sdst = (sw < NSA ? SA : SB) + srow * 4;
    auto issue = [&](int i, char *S) __attribute__((always_inline)) {
        const int kb = min(k0 + i, nkb - 1);
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int q = wv * L + j;
            load_lds16(q < LA ? ra : rb, S + kg * STAGE + q * 1024, vo[j & 1], (q < LA ? q : q - LA) * 8 * K + kb * 128);
        }
        load_lds4(rs, S + kg * STAGE + sdst, so, kb * 4);
    };
    const LaneRow rows(lane);
    const float *sb_square = BROW ? nullptr : a.sb + (size_t)(min(n0 + br, a.N - 1) >> 7) * nkb;

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    float sbn = 1.f;
    if (nkb > 0) {
        if (!BROW) sbn = uniform_load(sb_square + min(k0, nkb - 1));
        issue(0, S0);
        if (ST > 2) issue(1, S1);
        if (ST > 3) issue(2, S2);
    }
    // block i of the group, in S; D is the stage that the block before it has left
    auto step = [&](int i, const char *S, char *D) __attribute__((always_inline)) {
        wait_barrier<(ST - 2) * (L + 1)>();  // this block has landed for every wave, and all are done with the last one
        issue(i + ST - 1, D);
        if (KG > 1 && k0 + i >= k1) return;  // a group that has one block less
        S += kg * STAGE;
        float sa[TM];
#pragma unroll
        for (int r = 0; r < TM; ++r) sa[r] = *reinterpret_cast<const float *>(S + SA + 4 * (ar + 16 * r + l16)) * sbn;
        if (!BROW) sbn = uniform_load(sb_square + min(k0 + i + 1, nkb - 1));
        OperandOf<OUT> fa[TM];
#pragma unroll
        for (int r = 0; r < TM; ++r) fa[r] = operand<OUT>(rows.load(S + (ar + 16 * r) * 128));
        f32x4 p[2][TM], sb[2];
#pragma unroll
        for (int j = 0; j <= TN; ++j) {  // products one column tile ahead of the folds
            if (j < TN) {
                const OperandOf<OUT> fb = operand<OUT>(rows.load(S + (BM + br + 16 * j) * 128));
                if constexpr (BROW) sb[j & 1] = *reinterpret_cast<const f32x4 *>(S + SB + 4 * (br + 16 * j + 4 * g));
#pragma unroll
                for (int r = 0; r < TM; ++r) p[j & 1][r] = block_product(fb, fa[r]);
            }
            if (j > 0) {
                const int u = (j - 1) & 1;
#pragma unroll
                for (int r = 0; r < TM; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[r][j - 1][e] = fmaf(p[u][r][e], BROW ? sa[r] * sb[u][e] : sa[r], acc[r][j - 1][e]);
            }
        }
    };
    for (int i = 0; i < steps;) {
        if constexpr (ST == 2) {
            step(i, S0, S1);
            if (++i == steps) break;
            step(i, S1, S0);
        } else if constexpr (ST == 3) {
            step(i, S0, S2);
            if (++i == steps) break;
            step(i, S1, S0);
            if (++i == steps) break;
            step(i, S2, S1);
        } else {
            step(i, S0, S3);
            if (++i == steps) break;
            step(i, S1, S0);
            if (++i == steps) break;
            step(i, S2, S1);
            if (++i == steps) break;
            step(i, S3, S2);
        }
        ++i;
    }
    wait_barrier<0>();  // no load into LDS is under way any more
    if constexpr (KG > 1) {
        static_assert((KG - 1) * NW * TM * TN * 1024 <= KG * STAGE, "");
        f32x4 *red = reinterpret_cast<f32x4 *>(S0);
        if (kg > 0) {
#pragma unroll
            for (int t = 0; t < TM * TN; ++t) red[(((kg - 1) * NW + wv) * TM * TN + t) * 64 + lane] = acc[t / TN][t % TN];
        }
        __syncthreads();
        if (kg > 0) return;
#pragma unroll
        for (int q = 0; q < KG - 1; ++q)
#pragma unroll
            for (int t = 0; t < TM * TN; ++t) acc[t / TN][t % TN] += red[((q * NW + wv) * TM * TN + t) * 64 + lane];
    }
    if constexpr (sizeof(OUT) == 2 && TN % 2 == 0) {
        // 16 bytes per lane, 64 of a row, after a lane swap (8 and 32 without: 16384 x 16384 x 256 238 us instead of
        // 181, 2000 x 1544 x 512 7.0 instead of 6.5); no faster where rows start anywhere
        if (a.N % 8 == 0) {
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int m = m0 + ar + 16 * i + l16;
                OUT *row = static_cast<OUT *>(a.out) + (size_t)m * a.N;
#pragma unroll
                for (int j = 0; j < TN; j += 2) {
                    const u32x4 x = pack_pair(acc[i][j], acc[i][j + 1]);
                    const int n = n0 + br + 16 * (j + (g & 1)) + 8 * (g >> 1);
                    if (m < a.M && n < a.N) *reinterpret_cast<u32x4 *>(row + n) = x;
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = m0 + ar + 16 * i + l16;
        if (m >= a.M) continue;
        OUT *row = static_cast<OUT *>(a.out) + (size_t)m * a.N;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int n = n0 + br + 16 * j + 4 * g;
            if (n < a.N) store_row4(row, n, a.N, acc[i][j]);
        }
    }
}

template <int BM, int BN, int KG, int WM, int WN, int ST, typename OUT, bool BROW>
__global__ __launch_bounds__(64 * KG * WM * WN) void matmul_tile_kernel(MatArgs a) {
    tile_body<BM, BN, KG, WM, WN, ST, OUT, BROW>(a);
}

// A few tokens against all of B (a decode step): B is read once, straight
// into registers, two blocks at a time.  A workgroup of eight waves takes 16
// features and up to 16 tokens; the waves split the contraction's blocks and
// their sums meet in LDS, so that 4096 features already give 256 workgroups
// with 2048 waves' loads under way.  1 x 4096 x 4096: 4.6 us, of which 17 MB
// at the caches' 7.2 TB/s are 2.3 and a launch's start and end most of the
// rest (32 x 32 tiles: 6.0).
template <typename OUT, bool BROW>
__global__ __launch_bounds__(512) void matmul_stream_kernel(MatArgs a) {
    constexpr int KW = 8;
    __shared__ __attribute__((aligned(16))) float red[KW][16][20];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4, n0 = blockIdx.x * 16;
    const int k0 = (int)((int64_t)a.nkb * wv / KW), k1 = (int)((int64_t)a.nkb * (wv + 1) / KW);
    const size_t m = min(l16, a.M - 1);
    const uint8_t *ap = a.a + m * a.K + 16 * g, *bp = a.b + (size_t)min(n0 + l16, a.N - 1) * a.K + 16 * g;
    const float *sap = a.sa + m * a.nkb, *sbp[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        sbp[r] = a.sb + (size_t)a.nkb * (BROW ? min(n0 + 4 * g + r, a.N - 1) : min(n0, a.N - 1) >> 7);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    struct Blk {
        Frag a, b;
        float sa, sb[4];
    };
    auto load = [&](int kb) __attribute__((always_inline)) {
        Blk x;
        const size_t o = (size_t)kb * 128;
        x.b.lo = *reinterpret_cast<const i32x4 *>(bp + o);
        x.b.hi = *reinterpret_cast<const i32x4 *>(bp + o + 64);
        x.a.lo = *reinterpret_cast<const i32x4 *>(ap + o);
        x.a.hi = *reinterpret_cast<const i32x4 *>(ap + o + 64);
        x.sa = sap[kb];
#pragma unroll
        for (int r = 0; r < (BROW ? 4 : 1); ++r) x.sb[r] = sbp[r][kb];
        return x;
    };
    auto use = [&](const Blk &x) __attribute__((always_inline)) {
        const f32x4 p = block_product(operand<OUT>(x.b), operand<OUT>(x.a));
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = fmaf(p[r], x.sa * x.sb[BROW ? r : 0], acc[r]);
    };
    if (k0 < k1) {
        Blk x = load(k0);
        for (int kb = k0; kb < k1; kb += 2) {
            const Blk y = load(min(kb + 1, k1 - 1));
            use(x);
            if (kb + 1 >= k1) break;
            x = load(min(kb + 2, k1 - 1));
            use(y);
        }
    }
    *reinterpret_cast<f32x4 *>(&red[wv][l16][4 * g]) = acc;
    __syncthreads();
    if (threadIdx.x < 64) {
        const int row = threadIdx.x >> 2, n = 4 * (threadIdx.x & 3);
        if (row >= a.M || n0 + n >= a.N) return;
        f32x4 s = *reinterpret_cast<const f32x4 *>(&red[0][row][n]);
#pragma unroll
        for (int w = 1; w < KW; ++w) s += *reinterpret_cast<const f32x4 *>(&red[w][row][n]);
        store_row4(static_cast<OUT *>(a.out) + (size_t)row * a.N, n0 + n, a.N, s);
    }
}

// The whole chip on a large product (bf16 output).  256 workgroups of 8
// waves, one per CU, each walk over 256 x 256 tiles; a wave holds 64 tokens x
// 128 features of the tile as 4 x 8 results (128 registers).  Two LDS stages
// of a block (64 KiB each), filled by direct loads; the sequence of blocks
// runs on over the tiles' ends, so a tile's first blocks are under way while
// the last one's results are stored, for any count of blocks from four on.
//   - A block is worked off in four phases of two column tiles.  Each phase
//     starts by reading the next phase's operands into registers, and the
//     last phase the next block's A; the one barrier of a block stands before
//     the last phase, when the block's bytes are all in registers and the
//     next block's have landed.  The loads of the block after that go out
//     behind it, A's between the last phase's products and B's between those
//     of the phase that follows (all of them in the last phase: 500 us).
//   - Results are folded two products behind.
//   - A ninth load per wave and block brings A's scales two blocks ahead (four
//     waves) or pulls lines three blocks ahead into the XCD's L2 (the others:
//     a quarter of A's rows and an eighth of B's, which the 32 workgroups of
//     an XCD share); without it the loads' latency showed (2.2 against 1.7 us
//     per block).  With B scaled by rows every wave does both, scales (A's or
//     B's) and lines.
//   - After a lane swap every lane stores 16 bytes of a row (8 where rows
//     start anywhere; 16 at a time were no faster there).
// 16384 x 8192 x 4096: 470 us = 2340 TFLOP/s in a loop over one set of operands
// (477-501 a call on changing ones).  It is bound by the chip's power:
// the same kernel over zeros takes 388 us, and its blocks without loads 1.05
// us each, the products' own rate (1.6 with random bytes and all).  The
// tiles' ends cost 70 us, 45 of them the 268 MB of results, which all
// workgroups write at the same time.  With B scaled by rows 640 us (128 x 128
// tiles 715): the scales' products double the vector instructions, which then
// take longer than the matrix instructions beside them.
struct BigTile {
    int m0, n0, share;  // share: first of the rows whose lines this wave pulls into L2
};

template <bool BROW>
__device__ __forceinline__ void big_body(const MatArgs &a) {
    constexpr int BM = 256, BN = 256, NW = 8, TM = 4, TN = 8, LAG = 2, AHEAD = 3;
    __shared__ __attribute__((aligned(1024))) char As0[BM * 128];
    __shared__ __attribute__((aligned(1024))) char As1[BM * 128];
    __shared__ __attribute__((aligned(1024))) char Bs0[BN * 128];
    __shared__ __attribute__((aligned(1024))) char Bs1[BN * 128];
    constexpr int SR = BROW ? BM + BN : BM, X = BROW ? 2 : 1;  // scales of a block; extra loads of a wave
    // a ring of blocks' scales (A's, and B's by rows, which slower waves still read in a block's last phase when others
    // load three blocks ahead), and the place where the L2 loads' bytes go
    constexpr int RING = BROW ? 8 : 4;
    __shared__ __attribute__((aligned(16))) float Ss[RING][SR];
    __shared__ float sink[64];

    const int total = a.mt * a.nt, per = (total + 7) / 8, xcd = blockIdx.x % 8, slots = gridDim.x / 8;
    const int tend = min(per, total - xcd * per);
    int t = blockIdx.x / 8;
    if (t >= tend) return;

    const int K = a.K, nkb = a.nkb;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4, ar = wv / 2 * 64, br = wv % 2 * 128;
    const bool scales = !BROW && wv < 4, pulls_a = BROW ? (wv & 2) == 0 : wv < 6;

    // as tile_of, for tile tt of this XCD's range
    auto big_tile = [&](int tt) __attribute__((always_inline)) {
        const int id = xcd * per + tt, grp = id / (8 * a.nt), in = id % (8 * a.nt), gm = min(8, a.mt - grp * 8);
        const int tm = in % gm, tn = in / gm;
        return BigTile{(grp * 8 + tm) * BM, tn * BN, scales ? 0 : pulls_a ? 64 * (tn & 3) : 32 * (tm & 7)};
    };
    const auto ra = rsrc(a.a, (uint32_t)((size_t)a.M * K)), rb = rsrc(a.b, (uint32_t)((size_t)a.N * K));
    const auto rx = scales ? rsrc(a.sa, (uint32_t)((size_t)a.M * nkb * 4)) : pulls_a ? ra : rb;
    const int vo = 8 * wv * K + swizzled_source(lane, wv, K);
    int xo = scales ? (64 * wv + lane) * nkb * 4
                    : (pulls_a ? 32 * (wv & 1) + (lane & 31) : 16 * (wv & 1) + (lane & 15)) * K;
    if (BROW) {
        const int part = (wv & 1) + (wv >> 2) * 2;  // of four waves
        xo = (pulls_a ? 16 * part + (lane & 15) : 8 * part + (lane & 7)) * K;
    }
    const auto ry = wv < 4 ? rsrc(a.sa, (uint32_t)((size_t)a.M * nkb * 4))
                           : rsrc(a.sb, (uint32_t)((size_t)a.N * nkb * 4));
    const int yo = (64 * (wv & 3) + lane) * nkb * 4;
    const int xstep = scales ? 4 : 128, xahead = scales ? 2 : AHEAD;
    auto xbase = [&](const BigTile &x) __attribute__((always_inline)) {
        return scales ? x.m0 * nkb * 4 : ((pulls_a ? x.m0 : x.n0) + x.share) * K;
    };
    auto sbase = [&](const BigTile &x) __attribute__((always_inline)) {
        return BROW ? (wv < 4 ? x.m0 : x.n0) * nkb * 4 : (min(x.n0 + br, a.N - 1) >> 7) * nkb;
    };

    // byte offsets of this tile's and the next one's A, B, extra loads and B scales
    BigTile cur = big_tile(t), nxt = big_tile(min(t + slots, tend - 1));
    int a0 = cur.m0 * K, a1 = nxt.m0 * K, b0 = cur.n0 * K, b1 = nxt.n0 * K, x0 = xbase(cur), x1 = xbase(nxt);
    int s0 = sbase(cur), s1 = sbase(nxt);

    // load i (of 8) of block kb, which may lie past this tile's end: then it is the next tile's
    auto issue = [&](int kb, char *Ad, char *Bd, int i) __attribute__((always_inline)) {
        const bool over = kb >= nkb;
        const int k = (over ? kb - nkb : kb) * 128;
        if (i < 4)
            load_lds16(ra, Ad + (wv + NW * i) * 1024, vo, (over ? a1 : a0) + k + i * 64 * K);
        else
            load_lds16(rb, Bd + (wv + NW * (i - 4)) * 1024, vo, (over ? b1 : b0) + k + (i - 4) * 64 * K);
    };
    // the ninth load, as of block kb, number gs of all blocks
    auto extra = [&](int kb, int gs) __attribute__((always_inline)) {
        const int kk = max(kb + xahead, 0);
        const bool over = kk >= nkb;
        float *dst = scales ? &Ss[(gs + 2) & (RING - 1)][64 * wv] : sink;
        if constexpr (BROW) {
            const int ks = max(kb + 2, 0);
            const bool past = ks >= nkb;
            load_lds4(ry, reinterpret_cast<char *>(&Ss[(gs + 2) & (RING - 1)][64 * wv]), yo,
                      (past ? s1 : s0) + (past ? ks - nkb : ks) * 4);
        }
        load_lds4(rx, reinterpret_cast<char *>(dst), xo, (over ? x1 : x0) + (over ? kk - nkb : kk) * xstep);
    };
    const LaneRow rows(lane);

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    extra(-2, -2);
    extra(-1, -1);
    extra(0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) issue(0, As0, Bs0, i);
    wait_barrier<0>();
#pragma unroll
    for (int i = 0; i < 4; ++i) issue(1, As1, Bs1, i);
    Frag fa[TM], fb[2][2];
    float sa[TM];
    const float sb0 = BROW ? 1.f : uniform_load(a.sb + s0);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        fa[i] = rows.load(As0 + (ar + 16 * i) * 128);
        sa[i] = Ss[0][ar + 16 * i + l16] * sb0;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) fb[0][j] = rows.load(Bs0 + (br + 16 * j) * 128);

    int gs = 0, kb = 0;
    auto step = [&](char *Ac, char *Bc, char *An, char *Bn) __attribute__((always_inline)) {
        f32x4 p[4], sb[2][2];
        float sn[TM], sbn = 1.f;
        // product u of the block is that of column tile 2 (u / 8) + u % 2 and row tile u / 2 % 4
        auto fold = [&](int u) __attribute__((always_inline)) {
            const int j = 2 * (u / (2 * TM)) + (u & 1), i = u / 2 % TM;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[i][j][r] = fmaf(p[u & 3][r], BROW ? sa[i] * sb[u / (2 * TM) & 1][u & 1][r] : sa[i], acc[i][j][r]);
        };
#pragma unroll
        for (int ph = 0; ph < TN / 2; ++ph) {
            const bool last = ph == TN / 2 - 1;
            if (last) {
                wait_barrier<X>();  // the newest load, the ninth, may still be under way
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    if (!BROW) sn[i] *= sbn;
            }
            __builtin_amdgcn_sched_barrier(0);
            if (!BROW && ph == 0) sbn = uniform_load(a.sb + (kb + 1 < nkb ? s0 + kb + 1 : s1));
            const char *bnext = last ? Bn : Bc;
            if constexpr (BROW) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    sb[ph & 1][j] =
                        *reinterpret_cast<const f32x4 *>(&Ss[gs & (RING - 1)][BM + br + 16 * (2 * ph + j) + 4 * g]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                fb[(ph + 1) & 1][j] = rows.load(bnext + (br + 16 * (last ? j : 2 * ph + 2 + j)) * 128);
            if (ph == 0) {
#pragma unroll
                for (int i = 0; i < TM; ++i) sn[i] = Ss[(gs + 1) & (RING - 1)][ar + 16 * i + l16];
            }
#pragma unroll
            for (int i = 0; i < TM; ++i) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int u = ph * TM * 2 + i * 2 + j;
                    p[u & 3] = block_product(fb[ph & 1][j], fa[i]);
                    if (u >= LAG) fold(u - LAG);
                }
                if (last) {
                    fa[i] = rows.load(An + (ar + 16 * i) * 128);
                    issue(kb + 2, Ac, Bc, i);
                }
                if (ph == 0) issue(kb + 1, An, Bn, 4 + i);
                if (ph == 1 && i == 1) extra(kb + 1, gs + 1);
            }
        }
#pragma unroll
        for (int u = TM * TN - LAG; u < TM * TN; ++u) fold(u);
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = sn[i];
        ++gs;
        ++kb;
    };
    auto tile_end = [&]() __attribute__((always_inline)) {
        const auto ro = rsrc(static_cast<uint16_t *>(a.out) + (size_t)cur.m0 * a.N,
                             (uint32_t)(min(BM, a.M - cur.m0) * a.N * 2));
        if (a.N % 8 == 0) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; j += 2) {
                    const u32x4 x = pack_pair(acc[i][j], acc[i][j + 1]);
                    const int m = ar + 16 * i + l16, n = cur.n0 + br + 16 * (j + (g & 1)) + 8 * (g >> 1);
                    const int off = n < a.N ? (m * a.N + n) * 2 : 0x7fffffff;  // rows, columns past the end: dropped
                    __builtin_amdgcn_raw_buffer_store_b128(x, ro, off, 0, 0);
                }
        } else {  // rows that start anywhere
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int m = cur.m0 + ar + 16 * i + l16, n = cur.n0 + br + 4 * g;
                uint16_t *row = static_cast<uint16_t *>(a.out) + (size_t)m * a.N;
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    if (m < a.M && n + 16 * j < a.N) store_row4(row, n + 16 * j, a.N, acc[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        t += slots;
        if (t >= tend) return false;
        kb = 0;
        cur = nxt, a0 = a1, b0 = b1, x0 = x1, s0 = s1;
        nxt = big_tile(min(t + slots, tend - 1));
        a1 = nxt.m0 * K, b1 = nxt.n0 * K, x1 = xbase(nxt), s1 = sbase(nxt);
        return true;
    };
    for (;;) {
        step(As0, Bs0, As1, Bs1);
        if (kb == nkb && !tile_end()) break;
        step(As1, Bs1, As0, Bs0);
        if (kb == nkb && !tile_end()) break;
    }
    __builtin_amdgcn_s_waitcnt(0);  // loads past the last block still write this workgroup's LDS
}

template <bool BROW>
__global__ __launch_bounds__(512, 1) void matmul_big_kernel(MatArgs a) { big_body<BROW>(a); }

// ---- choice of a kernel -------------------------------------------------------
// A kernel's time is close to max(f0 + f1 nkb, T (t0 + t1 nkb)): a lone
// tile's latency, and the chip's throughput over T tiles, T rounded up to
// what fills the CUs evenly.  The constants (us) are least-squares fits to
// times over 600 random sizes (9 .. 16384 tokens, 64 .. 16384 features, a
// contraction of 256 .. 16384; B by rows and by squares alike), for bf16 and
// for fp32 output; taking the smallest costs 1.8% (1.0%) over the best kernel
// of each size.  Groups of waves that share a tile's blocks, and stages
// further ahead, pay where there are few tiles; small LDS, so more workgroups
// per CU, where there are many.  Times in us of that sweep (loops over one set
// of operands), bf16 output (32 x 32 by four groups | by one | 32 x 64 | 64 x
// 64 by two | by one | 128 x 64 | 128 x 128 | 128 x 64 with four stages | 256 x 256):
//   64 x 4096 x 4096        6.7 |  9.2 |  8.3 | 10.7 | 12.9 | 15.6 | 21.9 | 15.4 |  45
//   64 x 8192 x 4096       12.9 | 11.2 |  9.2 | 12.0 | 19.9 | 22.3 | 25.0 | 16.6 |  45
//   100 x 8192 x 4096      21.3 | 16.5 | 13.1 | 12.4 | 19.6 | 23.2 | 25.8 | 17.0 |  45
//   256 x 8192 x 4096      43.6 | 32.5 | 24.2 | 22.9 | 21.8 | 25.6 | 27.1 | 19.0 |  47
//   4096 x 2048 x 2048      113 |   61 |   49 |   50 |   37 |   29 |   23 |   37 |  30
//   4096 x 4096 x 4096      328 |  217 |  164 |  159 |  133 |  102 |   78 |  136 |  65
//   16384 x 8192 x 4096    2609 | 1722 | 1303 | 1273 | 1039 |  834 |  598 | 1052 | 459
struct Fit {
    int rows, cols, threads, round;
    double f0, f1, t0, t1;
};
// the last two are for bf16 output alone
constexpr int kConfigs = 9;
constexpr Fit kFit[2][kConfigs] = {{{32, 32, 512, 256, 3, 0.0938, 0.00793, 0.000448},
                                    {32, 32, 128, 256, 2.55, 0.192, 0.00197, 0.000487},
                                    {32, 64, 256, 256, 2.79, 0.168, 0.00498, 0.000628},
                                    {64, 64, 512, 256, 3.25, 0.213, 0.00868, 0.00107},
                                    {64, 64, 256, 256, 2.5, 0.279, 0.00217, 0.00105},
                                    {128, 64, 256, 256, 2.26, 0.532, 0.00448, 0.00155},
                                    {128, 128, 256, 256, 3.3, 0.737, 0.00873, 0.00229},
                                    {128, 64, 256, 256, 3.14, 0.431, 0.0103, 0.00182},
                                    {256, 256, 512, 256, 9.53, 1.59, 0.0319, 0.00664}},
                                   {{32, 32, 512, 256, 3.03, 0.127, 0.00864, 0.000543},
                                    {32, 32, 128, 512, 2.48, 0.328, 0.00269, 0.000454},
                                    {32, 64, 256, 256, 2.92, 0.249, 0.00615, 0.000716},
                                    {64, 64, 512, 256, 3.3, 0.358, 0.0115, 0.00134},
                                    {64, 64, 256, 256, 2.61, 0.457, 0.00588, 0.00118},
                                    {128, 64, 256, 256, 3.36, 0.713, 0.00979, 0.00203},
                                    {128, 128, 256, 256, 4.84, 1.09, 0.0154, 0.00335},
                                    {},
                                    {}}};

double fitted_us(const Fit &f, int64_t M, int64_t N, int64_t nkb) {
    int64_t T = ((M + f.rows - 1) / f.rows) * ((N + f.cols - 1) / f.cols);
    T = (T + f.round - 1) / f.round * f.round;
    const double lone = f.f0 + f.f1 * nkb, chip = T * (f.t0 + f.t1 * nkb);
    return lone > chip ? lone : chip;
}

template <int BM, int BN, int KG, int WM, int WN, int ST, typename OUT, bool BROW>
void launch_tile(const MatArgs &a, hipStream_t st) {
    const unsigned grid = (unsigned)(((int64_t)a.mt * a.nt + 7) / 8 * 8);
    hipLaunchKernelGGL((matmul_tile_kernel<BM, BN, KG, WM, WN, ST, OUT, BROW>), dim3(grid), dim3(64 * KG * WM * WN), 0,
                       st, a);
}

template <typename OUT, bool BROW>
hipError_t matmul(MatArgs a, hipStream_t st) {
    constexpr bool wide = sizeof(OUT) == 4;
    if (a.M <= 8 && a.N <= 4096 && a.nkb > 0) {
        // few tokens and no more workgroups than CUs: one 16-token operand per wave, B straight from memory
        // (1 x 4096 x 4096: 4.6 us, 32 x 32 tiles 6.0; but 8 x 8192 x 8192 16.7 against 12.2, 16 x 4096 x 4096 6.8
        // against 6.1: every wave reads A's rows again)
        hipLaunchKernelGGL((matmul_stream_kernel<OUT, BROW>), dim3((a.N + 15) / 16), dim3(512), 0, st, a);
        return hipGetLastError();
    }
    int best = 0;
    double us = 1e30;
    for (int i = 0; i < (wide ? kConfigs - 2 : kConfigs); ++i) {
        // the large kernel: 32-bit offsets over the whole of A and B, and four blocks (its loads run that far ahead) or,
        // with rows of results that start anywhere, eight (3465 x 2663 x 512: 20.9 us against 16.5 with 128 x 64 tiles,
        // but 8192 x 8191 x 1024 117 against 130)
        if (i == 8 && (a.nkb < (a.N % 8 ? 8 : 4) || (int64_t)(a.M + 256) * a.K > INT32_MAX ||
                       (int64_t)(a.N + 256) * a.K > INT32_MAX || (int64_t)a.N * 512 > INT32_MAX))
            break;
        const Fit &f = kFit[wide][i];
        // a launch holds fewer than 2^32 threads (the large kernel's is 256 workgroups whatever the size); the caller sees
        // to it that the 32 x 32 tiles of 128 threads fit
        if (i < 8 && ((int64_t)(a.M + f.rows - 1) / f.rows * ((a.N + f.cols - 1) / f.cols) + 7) * f.threads > UINT32_MAX)
            continue;
        const double x = fitted_us(f, a.M, a.N, a.nkb);
        if (x < us) us = x, best = i;
    }
    const Fit &f = kFit[wide][best];
    a.mt = (a.M + f.rows - 1) / f.rows;
    a.nt = (a.N + f.cols - 1) / f.cols;
    switch (best) {
        case 0: launch_tile<32, 32, 4, 2, 1, 3, OUT, BROW>(a, st); break;
        case 1: launch_tile<32, 32, 1, 2, 1, 4, OUT, BROW>(a, st); break;
        case 2: launch_tile<32, 64, 2, 1, 2, 3, OUT, BROW>(a, st); break;
        case 3: launch_tile<64, 64, 2, 2, 2, 3, OUT, BROW>(a, st); break;
        case 4: launch_tile<64, 64, 1, 2, 2, 2, OUT, BROW>(a, st); break;
        case 5: launch_tile<128, 64, 1, 2, 2, 2, OUT, BROW>(a, st); break;
        case 6: launch_tile<128, 128, 1, 2, 2, 2, OUT, BROW>(a, st); break;
        default:
            if constexpr (!wide) {
                if (best == 7) {
                    launch_tile<128, 64, 1, 2, 2, 4, OUT, BROW>(a, st);
                    break;
                }
            }
            if constexpr (!wide) hipLaunchKernelGGL(matmul_big_kernel<BROW>, dim3(256), dim3(512), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scaled_matmul(int m, int n, int k, const void *A, const float *sa, const void *B, const float *sb,
                                int b_rows, int out_dtype, void *out, hipStream_t st) {
    const MatArgs a{static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(B), sa, sb, out, m, n, k, k / 128, 0, 0};
    if (out_dtype == MSR_BF16) return b_rows == 1 ? matmul<uint16_t, true>(a, st) : matmul<uint16_t, false>(a, st);
    return b_rows == 1 ? matmul<float, true>(a, st) : matmul<float, false>(a, st);
}
