// msr_quant.hpp -- device helpers of the 8-bit operators: e4m3 values with
// one fp32 scale for each block of 128, vector loads and stores of eight
// elements, and reductions over a row of 16 lanes.
//
// A block's scale is s = max(amax / 448, 2^-126) (448 is e4m3's largest
// value; the floor keeps 1 / s finite) and its values are rne(v * (1 / s)).
// amax is taken on the bit patterns of |v|, which order as the numbers do,
// with infinity above every number and NaN above infinity: a block that
// holds one gets an infinite or NaN scale, and stands for NaN as a whole.
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

// Eight consecutive elements at p (16-byte aligned when VEC) as they lie in
// memory, and as floats: loads go out early this way and are widened late.
// Elements from index `left` on lie past the row's end, are not read and
// count as zero.
template <typename T, bool VEC>
struct Raw8;

template <>
struct Raw8<uint16_t, true> {
    uint4 u;
    __device__ __forceinline__ void load(const uint16_t *p, int left) {
        u = make_uint4(0, 0, 0, 0);
        if (left > 0) u = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // keeps the compiler from holding the floats (twice the registers) from one get() to the next
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(u.x), "+v"(u.y), "+v"(u.z), "+v"(u.w)); }
};

template <>
struct Raw8<float, true> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p, int left) {
        a = b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (left > 0) {
            a = *reinterpret_cast<const float4 *>(p);
            b = *reinterpret_cast<const float4 *>(p + 4);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void forget() {}
};

template <typename T>
struct Raw8<T, false> {
    float x[8];
    __device__ __forceinline__ void load(const T *p, int left) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < left ? msr::load(p, i) : 0.f;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[i];
    }
    __device__ __forceinline__ void forget() {}
};

template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T *p, int left, float (&v)[8]) {
    Raw8<T, VEC> r;
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

template <bool VEC>
__device__ __forceinline__ void store8(uint16_t *p, int left, const float (&v)[8]) {
    if constexpr (VEC) {
        if (left > 0)
            stream_out(p, make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                     pack_bf16(v[6], v[7])));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = f32_to_bf16(v[i]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(float *p, int left, const float (&v)[8]) {
    if constexpr (VEC) {
        if (left > 0) {
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = v[i];
    }
}

// the same for a weight row whose type is known at run time only (NULL: ones)
template <bool VEC>
__device__ __forceinline__ void load_weight8(const void *w, int bf16, size_t i, int left, float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 1.f;
    } else if (bf16) {
        load8<VEC>(static_cast<const uint16_t *>(w) + i, left, v);
    } else {
        load8<VEC>(static_cast<const float *>(w) + i, left, v);
    }
}

}  // namespace msr
