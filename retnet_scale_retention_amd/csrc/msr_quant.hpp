// msr_quant.hpp -- device helpers of the 8-bit operators: e4m3 values with
// one fp32 scale for each block of 128, vector loads and stores of eight
// elements, and reductions over a row of 16 lanes.
//
// A block's scale is s = max(amax / 448, 2^-126) (448 is e4m3's largest
// value; the floor keeps 1 / s finite) and its values are rne(v / s), from
// the quotient rounded to fp32 (quotient() below, not a product with 1 / s).
// amax is taken on the bit patterns of |v|, which order as the numbers do,
// with infinity above every number and NaN above infinity: a block that
// holds either gets a NaN scale, and stands for NaN as a whole, zeros of a
// row's padding that lie in it included.
#pragma once

#include "msr_device.hpp"

namespace msr {

constexpr int kBlock = 128;
constexpr float kF8Max = 448.f;
constexpr float kScaleFloor = 1.17549435e-38f;  // 2^-126

__host__ __device__ constexpr int64_t round128(int64_t n) { return (n + 127) / 128 * 128; }

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// v / s, inv = 1 / s within an ulp or two: the product's error is made up for by its remainder (Markstein's step), so
// that a value is rounded to 8 bits from its correctly rounded quotient; v * inv alone moves values that lie between two
// e4m3 numbers, and a division of its own for every value is ten instructions.
__device__ __forceinline__ float quotient(float v, float s, float inv) {
    const float q = v * inv;
    return fmaf(fmaf(-q, s, v), inv, q);
}

__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
    const float s = quotient(__uint_as_float(amax_bits), kF8Max, 1.f / kF8Max);
    return s < kScaleFloor ? kScaleFloor : s;
}

// eight values over s as e4m3 bytes, in order (round to nearest even); s >= 2^-126 and 1 / s are normal numbers
__device__ __forceinline__ uint2 pack8(const float (&v)[8], float s) {
    const float inv = __builtin_amdgcn_rcpf(s);
    int a = 0, b = 0;
    a = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[0], s, inv), quotient(v[1], s, inv), a, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[2], s, inv), quotient(v[3], s, inv), a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4], s, inv), quotient(v[5], s, inv), b, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[6], s, inv), quotient(v[7], s, inv), b, true);
    return make_uint2((uint32_t)a, (uint32_t)b);
}

// lane l of a row of 16 reads lane (l + N) % 16 of it
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 | N, 0xf, 0xf, true);
}

__device__ __forceinline__ uint32_t row16_max(uint32_t x) {
    x = max(x, row_ror<8>(x));
    x = max(x, row_ror<4>(x));
    x = max(x, row_ror<2>(x));
    return max(x, row_ror<1>(x));
}

__device__ __forceinline__ float row16_sum(float x) {
    x += __uint_as_float(row_ror<8>(__float_as_uint(x)));
    x += __uint_as_float(row_ror<4>(__float_as_uint(x)));
    x += __uint_as_float(row_ror<2>(__float_as_uint(x)));
    return x + __uint_as_float(row_ror<1>(__float_as_uint(x)));
}

// the sum over the wave: lane rows by rotation, the four rows by the lane swaps
__device__ __forceinline__ float wave_sum_dpp(float x) {
    const uint32_t a = __float_as_uint(row16_sum(x));
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const uint32_t b = __float_as_uint(__uint_as_float(r[0]) + __uint_as_float(r[1]));
    const auto t = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __uint_as_float(t[0]) + __uint_as_float(t[1]);
}

// Accesses of 4 to 16 bytes at an element's own alignment: rows of a width that is not a multiple of 8 start anywhere,
// and the memory pipeline takes any address (element by element, the norm's gradients of 2941 x 1789 bf16 took 50 us).
template <typename V>
struct __attribute__((packed, aligned(2))) AnyAlign {
    V v;
};
template <typename V>
__device__ __forceinline__ V load_any(const void *p) {
    return static_cast<const AnyAlign<V> *>(p)->v;
}
template <typename V>
__device__ __forceinline__ void store_any(void *p, V v) {
    static_cast<AnyAlign<V> *>(p)->v = v;
}

// How rows lie: of widths that are multiples of 8 (every group of eight aligned to 16 bytes, none cut), of any width
// from 8 on, or of fewer than 8 elements.
enum { kTiny, kAny, kAligned };

// Eight consecutive elements at p as they lie in memory, and as floats: loads go out early this way and are widened
// late.  Elements from index `left` on lie past the row's end, are not read and count as zero.  Where a row of any
// width ends inside the eight, its last eight are read instead and moved down in get(): no lane then waits for its loads
// before the others' (pieces of 4, 2 and 1 in a branch of their own: the norm's gradients of 2941 x 1789 took 24 us).
template <typename T, int ROWS>
struct Raw8;

template <int ROWS>
struct Raw8<uint16_t, ROWS> {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4 u;
    int down;  // kAny: elements to move down by
    __device__ __forceinline__ void load(const uint16_t *p, int left) {
        u = u32x4{0, 0, 0, 0};
        if constexpr (ROWS == kAligned) {
            if (left > 0) u = *reinterpret_cast<const u32x4 *>(p);
        } else if constexpr (ROWS == kTiny) {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < left) u[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
        } else {
            down = left < 8 && left > 0 ? 8 - left : 0;
            if (left > 0) u = load_any<u32x4>(p - down);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        u32x4 x = u;
        if constexpr (ROWS == kAny) {
            if (down & 4) x = u32x4{x[2], x[3], 0, 0};
            if (down & 2) x = u32x4{x[1], x[2], x[3], 0};
            if (down & 1) x = u32x4{x[0] >> 16 | x[1] << 16, x[1] >> 16 | x[2] << 16, x[2] >> 16 | x[3] << 16, x[3] >> 16};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(x[i] << 16);
            v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        }
    }
    // keeps the compiler from holding the floats (twice the registers) from one get() to the next
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(u)); }
};

template <int ROWS>
struct Raw8<float, ROWS> {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    f32x4 a, b;
    int down;
    __device__ __forceinline__ void load(const float *p, int left) {
        a = b = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (ROWS == kAligned) {
            if (left > 0) {
                a = *reinterpret_cast<const f32x4 *>(p);
                b = *reinterpret_cast<const f32x4 *>(p + 4);
            }
        } else if constexpr (ROWS == kTiny) {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < left) (i < 4 ? a : b)[i & 3] = p[i];
        } else {
            down = left < 8 && left > 0 ? 8 - left : 0;
            if (left > 0) {
                a = load_any<f32x4>(p - down);
                b = load_any<f32x4>(p - down + 4);
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        f32x4 x = a, y = b;
        if constexpr (ROWS == kAny) {
            if (down & 4) x = y, y = f32x4{0.f, 0.f, 0.f, 0.f};
            if (down & 2) x = f32x4{x[2], x[3], y[0], y[1]}, y = f32x4{y[2], y[3], 0.f, 0.f};
            if (down & 1) x = f32x4{x[1], x[2], x[3], y[0]}, y = f32x4{y[1], y[2], y[3], 0.f};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = x[i], v[4 + i] = y[i];
    }
    __device__ __forceinline__ void forget() {}
};

template <int ROWS, typename T>
__device__ __forceinline__ void load8(const T *p, int left, float (&v)[8]) {
    Raw8<T, ROWS> r;
    r.load(p, left);
    r.get(v);
}

// Stores of results that this kernel does not read again, past the caches' retention: for instructions that fill whole
// lines (norm 16384 x 4096 bf16: 85 -> 70 us).  Eight floats per lane take two 16-byte stores that each fill half of
// every line; those stay ordinary (streamed, 16384 x 2048 fp32 took 108 us instead of 96).
__device__ __forceinline__ void stream_out(void *p, uint2 v) {
    __builtin_nontemporal_store((uint64_t)v.y << 32 | v.x, static_cast<uint64_t *>(p));
}
__device__ __forceinline__ void stream_out(void *p, uint4 v) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, static_cast<u32x4 *>(p));
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2_t p = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, p);
}

// Stores of eight elements, those from `left` on left out.  Ordinary ones where lanes do not fill whole lines.
template <int ROWS>
__device__ __forceinline__ void store8(uint16_t *p, int left, const float (&v)[8]) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 u = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    if constexpr (ROWS == kAligned) {
        if (left > 0) stream_out(p, make_uint4(u[0], u[1], u[2], u[3]));
    } else if (left >= 8) {
        store_any(p, u);
    } else if (left > 0) {
        if (left & 4) store_any(p, (uint64_t)u[1] << 32 | u[0]);
        if (left & 2) store_any(p + (left & 4), (left & 4) ? u[2] : u[0]);
        if (left & 1) p[left & 6] = (uint16_t)((left & 4) ? ((left & 2) ? u[3] : u[2]) : ((left & 2) ? u[1] : u[0]));
    }
}

template <int ROWS>
__device__ __forceinline__ void store8(float *p, int left, const float (&v)[8]) {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    if constexpr (ROWS == kAligned) {
        if (left > 0) {
            *reinterpret_cast<f32x4 *>(p) = a;
            *reinterpret_cast<f32x4 *>(p + 4) = b;
        }
    } else if (left >= 8) {
        store_any(p, a);
        store_any(p + 4, b);
    } else if (left > 0) {
        if (left & 4) store_any(p, a);
        if (left & 2) store_any(p + (left & 4), (left & 4) ? f32x2{b[0], b[1]} : f32x2{a[0], a[1]});
        if (left & 1) p[left & 6] = (left & 4) ? ((left & 2) ? b[2] : b[0]) : ((left & 2) ? a[2] : a[0]);
    }
}

// the same for a weight row whose type is known at run time only (NULL: ones)
template <int ROWS>
__device__ __forceinline__ void load_weight8(const void *w, int bf16, size_t i, int left, float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 1.f;
    } else if (bf16) {
        load8<ROWS>(static_cast<const uint16_t *>(w) + i, left, v);
    } else {
        load8<ROWS>(static_cast<const float *>(w) + i, left, v);
    }
}

}  // namespace msr
