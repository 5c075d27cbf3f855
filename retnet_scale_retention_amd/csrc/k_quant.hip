// k_quant.hip -- a matrix into 8 bits (e4m3) with one scale per block of
// 128, in its own order, transposed, or both from one pass over it.  A block
// is 128 values of a row (of a column for the transposed copy), or a square
// of 128 x 128, in which case the transposed copy has the same scales and
// bytes.  Scales, rounding and non-finite values: msr_quant.hpp.
#include "msr_quant.hpp"

namespace {

using namespace msr;

struct QuantArgs {
    const void *x;
    uint8_t *q, *qt;      // NULL: not wanted.  [R][Cp] and [C][Rp]
    float *s, *st;
    int64_t R, C, Cp, Rp;
    int tiles_c;
};

// Own order, blocks within a row: 16 lanes take a block, 8 values each, and
// four blocks one after the other, loaded together.  Bound by memory: 16384 x
// 4096 bf16 32 us in a loop over one buffer (203 MB, 6.4 TB/s; the transposed
// copy alone, by the tile kernel, 33 us).
template <typename T, int ROWS>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a) {
    constexpr int U = 4;
    const uint32_t per_row = (uint32_t)(a.Cp / kBlock);
    const int64_t first = (int64_t)blockIdx.x * (16 * U), row0 = first / per_row;  // the same for the workgroup
    const uint32_t col0 = (uint32_t)(first - row0 * per_row);
    Raw8<T, ROWS> x[U];
    int64_t row[U];
    uint32_t blk[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t at = col0 + 16 * u + (threadIdx.x >> 4);
        row[u] = row0 + at / per_row;
        blk[u] = at % per_row;
        const int64_t c = (int64_t)blk[u] * kBlock + 8 * (threadIdx.x & 15);
        x[u].load(static_cast<const T *>(a.x) + row[u] * a.C + c, row[u] < a.R ? (int)(a.C - c) : 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[8];
        x[u].get(v);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
        const float sc = block_scale(row16_max(m));
        if (row[u] < a.R) {
            stream_out(a.q + row[u] * a.Cp + (int64_t)blk[u] * kBlock + 8 * (threadIdx.x & 15), pack8(v, sc));
            if ((threadIdx.x & 15) == 0) a.s[row[u] * per_row + blk[u]] = sc;
        }
    }
}

// the largest over the lanes l, l ^ 16, l ^ 32, l ^ 48
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    const uint32_t y = max((uint32_t)r[0], (uint32_t)r[1]);
    const auto t = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return max((uint32_t)t[0], (uint32_t)t[1]);
}

// A workgroup takes a 128 x 128 tile: thread t holds the 8 x 8 values of rows
// 8 (t / 16) .., columns 8 (t % 16) .. in registers, as they came, so both
// directions' packs are register work; the transposed bytes pass through LDS
// to leave in whole 128-byte rows.  Bound by memory: 16384 x 4096 bf16 in
// both orders 58 us a call on changing inputs (4.7 TB/s; 48 us, 5.7 TB/s, in
// a loop over one buffer), in squares 42 us (6.4 TB/s) in a loop.  What it took:
// the values kept as loaded, not widened (174 -> 117 registers, 74 -> 59 us;
// the squares' kernel has room for the floats and is faster with them), and
// stores that do not linger in L2 (59 -> 48 us).
template <typename T, int ROWS, bool SQUARE>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantArgs a) {
    __shared__ __attribute__((aligned(16))) uint32_t cmax[4][128];
    __shared__ float cscale[128];
    __shared__ uint32_t tmax[4];
    __shared__ __attribute__((aligned(16))) uint8_t tr[128 * 128];
    const int64_t tr_i = blockIdx.x / a.tiles_c, tc = blockIdx.x % a.tiles_c;
    const int64_t r0 = tr_i * 128, c0 = tc * 128;
    const int rg = threadIdx.x >> 4, cg = threadIdx.x & 15, wave = threadIdx.x >> 6;
    const int64_t c = c0 + 8 * cg;
    Raw8<T, ROWS> x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 8 * rg + i;
        x[i].load(static_cast<const T *>(a.x) + r * a.C + c, r < a.R ? (int)(a.C - c) : 0);
    }
    uint32_t cm[8], all = 0;  // the columns' largest magnitudes, and the tile's
#pragma unroll
    for (int j = 0; j < 8; ++j) cm[j] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        x[i].get(v);
        uint32_t rm = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t m = abs_bits(v[j]);
            rm = max(rm, m);
            cm[j] = max(cm[j], m);
        }
        if constexpr (SQUARE) {
            all = max(all, rm);
        } else if (a.q) {
            const float s = block_scale(row16_max(rm));
            const int64_t r = r0 + 8 * rg + i;
            if (r < a.R) {
                stream_out(a.q + r * a.Cp + c, pack8(v, s));
                if (cg == 0) a.s[r * (a.Cp / kBlock) + tc] = s;
            }
        }
        if (!SQUARE) x[i].forget();
    }
    float square = 0.f;
    if constexpr (SQUARE) {
        all = wave_max(row16_max(all));
        if ((threadIdx.x & 63) == 0) tmax[wave] = all;
        __syncthreads();
        square = block_scale(max(max(tmax[0], tmax[1]), max(tmax[2], tmax[3])));
        if (threadIdx.x == 0) {
            if (a.q) a.s[tr_i * (a.Cp / kBlock) + tc] = square;
            if (a.qt) a.st[tc * (a.Rp / kBlock) + tr_i] = square;
        }
        if (a.q) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t r = r0 + 8 * rg + i;
                float v[8];
                x[i].get(v);
                if (r < a.R) stream_out(a.q + r * a.Cp + c, pack8(v, square));
            }
        }
    } else if (a.qt) {
#pragma unroll
        for (int j = 0; j < 8; ++j) cm[j] = wave_max(cm[j]);
        if ((threadIdx.x & 48) == 0) {
            *reinterpret_cast<uint4 *>(&cmax[wave][8 * cg]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
            *reinterpret_cast<uint4 *>(&cmax[wave][8 * cg + 4]) = make_uint4(cm[4], cm[5], cm[6], cm[7]);
        }
        __syncthreads();
        if (threadIdx.x < 128) {  // one thread per column
            const int k = threadIdx.x;
            const float s = block_scale(max(max(cmax[0][k], cmax[1][k]), max(cmax[2][k], cmax[3][k])));
            cscale[k] = s;
            if (c0 + k < a.C) a.st[(c0 + k) * (a.Rp / kBlock) + tr_i] = s;
        }
        __syncthreads();
    }
    if (a.qt) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float col[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v[8];
                x[i].get(v);
                col[i] = v[j];
            }
            // 8-byte pieces of a row XOR-swizzled by row / 8: the wave's 16 rows per store fall on different banks
            *reinterpret_cast<uint2 *>(tr + (8 * cg + j) * 128 + 8 * (rg ^ cg)) =
                pack8(col, SQUARE ? square : cscale[8 * cg + j]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = 32 * i + (int)(threadIdx.x >> 3), p = threadIdx.x & 7, x = k >> 3;
            uint4 u = *reinterpret_cast<const uint4 *>(tr + k * 128 + 16 * (p ^ (x >> 1)));
            if (x & 1) u = make_uint4(u.z, u.w, u.x, u.y);
            if (c0 + k < a.C) stream_out(a.qt + (c0 + k) * a.Rp + r0 + 16 * p, u);
        }
    }
}

template <typename T, int ROWS>
hipError_t quantize(const QuantArgs &a, int block_rows, hipStream_t st) {
    if (block_rows == 1 && !a.qt) {
        const int64_t g = (a.R * (a.Cp / kBlock) + 63) / 64;
        hipLaunchKernelGGL((quantize_rows_kernel<T, ROWS>), dim3((unsigned)g), dim3(256), 0, st, a);
    } else {
        const unsigned tiles = (unsigned)(a.Rp / 128 * a.tiles_c);
        if (block_rows == 1)
            hipLaunchKernelGGL((quantize_tile_kernel<T, ROWS, false>), dim3(tiles), dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL((quantize_tile_kernel<T, ROWS, true>), dim3(tiles), dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(int64_t R, int64_t C, int dtype, int block_rows, const void *x, void *q, float *s, void *qt,
                           float *s_t, hipStream_t st) {
    const QuantArgs a{x, static_cast<uint8_t *>(q), static_cast<uint8_t *>(qt), s, s_t, R, C, round128(C), round128(R),
                      (int)(round128(C) / 128)};
    if (dtype == MSR_BF16)
        return C % 8 == 0 ? quantize<uint16_t, kAligned>(a, block_rows, st)
               : C > 8    ? quantize<uint16_t, kAny>(a, block_rows, st)
                          : quantize<uint16_t, kTiny>(a, block_rows, st);
    return C % 8 == 0 ? quantize<float, kAligned>(a, block_rows, st)
           : C > 8    ? quantize<float, kAny>(a, block_rows, st)
                      : quantize<float, kTiny>(a, block_rows, st);
}
