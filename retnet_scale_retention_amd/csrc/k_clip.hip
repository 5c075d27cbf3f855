// k_clip.hip -- the norm of many gradient tensors together, and their
// scaling to a largest norm: norm = sqrt(sum of squares),
// out = g min(1, max / norm).
//
// Tensors travel as a table in the kernel's arguments (kTable of them per
// launch) and are cut into chunks that the workgroups take in turn.  Squares
// are formed and added in fp64, so that no finite gradient overflows or
// vanishes; each workgroup writes one sum, and whoever needs the total adds
// the sums in the same order (no atomics, the same norm on every run).
//
// Bound by memory: two reads and a write where the gradients exceed the
// caches.  Five fp32 tensors of 403 MB together: 222 us in a loop (206 in
// place), 231 on changing inputs (1.2 GB, 5.2 TB/s; a 1 GiB copy reaches
// 5.06); 300 bf16 tensors of 189 MB in place 106 in a loop.  60 bf16
// tensors of 37.8 MB together: 23 us of kernels (8.8 and 15); the call takes
// the host 30 us in place (16 to write the table, 9 the C call) and 41 with
// tensors for the results.
#include <algorithm>

#include "msr_quant.hpp"

namespace {

using namespace msr;

constexpr int kTable = 96, kThreads = 256, kGroups = 4, kChunk = kThreads * 8 * kGroups;

struct Entry {
    const void *g;
    void *out;
    int64_t n;
    int32_t start, bf16;  // first chunk
};

struct ClipArgs {
    Entry t[kTable];
    int count, chunks;
    // norm: where the sums go.  clip: the total is that of `sums` of them, or of *norm where that is given
    double *sums;
    int n_sums;
    const float *norm;
    float *norm_out;
    float max_norm;
};

static_assert(sizeof(ClipArgs) <= 4096 && kTable <= 128, "a kernel's arguments; two tensors to a lane");

// The tensor of chunk c: the starts lie one to a lane (two for the first kTable - 64), and a vote counts those up to c.
// 61 tensors of 21.5 MB: 16.6 us; with a walk along the table, which waits for a scalar load per tensor, 28.3.
struct Find {
    int lo, hi;
    __device__ __forceinline__ explicit Find(const ClipArgs &a) {
        const int l = threadIdx.x & 63;
        lo = l < a.count ? a.t[l].start : INT32_MAX;
        hi = l + 64 < a.count ? a.t[l + 64].start : INT32_MAX;
    }
    __device__ __forceinline__ int operator()(int c) const {
        return __builtin_amdgcn_readfirstlane(__popcll(__ballot(lo <= c)) + __popcll(__ballot(hi <= c)) - 1);
    }
};

__device__ __forceinline__ double block_sum64(double x, double *red) {
#pragma unroll
    for (int o = 32; o > 0; o /= 2) x += __shfl_xor(x, o, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// the total of n sums, the same in every workgroup that forms it
__device__ __forceinline__ double total(const double *sums, int64_t n, double *red) {
    double x = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) x += sums[i];
    return block_sum64(x, red);
}

// A chunk's values, eight to a lane: f(group, values, how many of them exist).  Of a chunk that the tensor's end cuts, the
// last eight are read together and moved down (Raw8), but for tensors of fewer than eight.
template <typename T, typename F>
__device__ __forceinline__ void for_groups(const T *p, int64_t left, bool tiny, const F &f) {
    if (left >= kChunk) {
        Raw8<T, kAny> r[kGroups];
#pragma unroll
        for (int u = 0; u < kGroups; ++u) r[u].load(p + (u * kThreads + threadIdx.x) * 8, 8);
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            float v[8];
            r[u].get(v);
            f((u * kThreads + threadIdx.x) * 8, v, 8);
        }
    } else if (tiny) {
        if (threadIdx.x == 0) {
            float v[8];
            load8<kTiny>(p, (int)left, v);
            f(0, v, (int)left);
        }
    } else {
        Raw8<T, kAny> r[kGroups];
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            const int i = (u * kThreads + threadIdx.x) * 8;
            r[u].load(p + i, (int)left - i);
        }
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            const int i = (u * kThreads + threadIdx.x) * 8;
            float v[8];
            r[u].get(v);
            f(i, v, (int)left - i);
        }
    }
}

template <typename T>
__device__ __forceinline__ double squares(const T *p, int64_t left, bool tiny) {
    double s[2] = {0.0, 0.0};
    for_groups(p, left, tiny, [&](int, const float (&v)[8], int) {  // what does not exist is zero
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i & 1] = fma((double)v[i], (double)v[i], s[i & 1]);
    });
    return s[0] + s[1];
}

template <typename T>
__device__ __forceinline__ void scale(const T *p, T *o, int64_t left, bool tiny, double f) {
    // fp32: one rounding of the product with the fp64 factor; bf16: the fp32 product's rounding is far below its own.  The
    // factor's exponent goes on afterwards, since large gradients and a small limit make factors that fp32 does not hold.
    int e;
    const float m = (float)frexp(f, &e);
    auto one = [&](float v) { return sizeof(T) == 4 ? (float)((double)v * f) : ldexpf(v * m, e); };
    for_groups(p, left, tiny, [&](int at, float (&v)[8], int n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = one(v[i]);
        store8<kAny>(o + at, n, v);
    });
}

__global__ __launch_bounds__(kThreads) void gradient_norm_kernel(ClipArgs a) {
    __shared__ double red[4];
    double s = 0.0;
    const Find find(a);
    for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        const int e = find(c);
        const int64_t at = (int64_t)(c - a.t[e].start) * kChunk, left = a.t[e].n - at;
        const bool tiny = a.t[e].n < 8;
        s += a.t[e].bf16 ? squares(static_cast<const uint16_t *>(a.t[e].g) + at, left, tiny)
                         : squares(static_cast<const float *>(a.t[e].g) + at, left, tiny);
    }
    s = block_sum64(s, red);
    if (threadIdx.x == 0) a.sums[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void gradient_total_kernel(double *sums, int64_t n, double *out, float *norm) {
    __shared__ double red[4];
    const double s = total(sums, n, red);
    if (threadIdx.x == 0) {
        if (out) *out = s;
        if (norm) *norm = (float)sqrt(s);
    }
}

// From the last chunk to the first: what the norm read last may still lie in the caches.
__global__ __launch_bounds__(kThreads) void clip_kernel(ClipArgs a) {
    __shared__ double red[4];
    const double norm = a.norm ? (double)*a.norm : sqrt(total(a.sums, a.n_sums, red));
    if (a.norm_out && blockIdx.x == 0 && threadIdx.x == 0) *a.norm_out = (float)norm;
    const bool clip = norm > (double)a.max_norm && isfinite((float)norm);  // as the caller sees it
    const double f = clip ? (double)a.max_norm / norm : 1.0;
    const Find find(a);
    for (int c = a.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
        const int e = find(c);
        if (!clip && a.t[e].g == a.t[e].out) continue;
        const int64_t at = (int64_t)(c - a.t[e].start) * kChunk, left = a.t[e].n - at;
        const bool tiny = a.t[e].n < 8;
        if (a.t[e].bf16)
            scale(static_cast<const uint16_t *>(a.t[e].g) + at, static_cast<uint16_t *>(a.t[e].out) + at, left, tiny, f);
        else
            scale(static_cast<const float *>(a.t[e].g) + at, static_cast<float *>(a.t[e].out) + at, left, tiny, f);
    }
}

constexpr int kSums = 1024;  // workgroups, and so sums, of a norm launch

// The launches that cover the tensors: f(args) for each, whose chunks are counted in 31 bits.
template <typename F>
hipError_t batches(const msr_gradient *t, int64_t count, F f) {
    ClipArgs a{};
    int64_t chunks = 0;
    auto flush = [&] {
        a.chunks = (int)chunks;
        const hipError_t e = a.count > 0 ? f(a) : hipSuccess;
        a.count = 0, chunks = 0;
        return e;
    };
    for (int64_t i = 0; i < count; ++i) {
        const size_t e = t[i].dtype == MSR_BF16 ? 2 : 4;
        // a tensor of more chunks than a launch counts goes in pieces
        for (int64_t at = 0; at < t[i].n;) {
            constexpr int64_t most = (int64_t)1 << 30;
            const int64_t n = std::min(t[i].n - at, most * kChunk), c = (n + kChunk - 1) / kChunk;
            if (a.count == kTable || chunks + c > most) {
                const hipError_t r = flush();
                if (r != hipSuccess) return r;
            }
            a.t[a.count++] = {static_cast<const char *>(t[i].grad) + at * e,
                              t[i].out ? static_cast<char *>(t[i].out) + at * e : nullptr, n, (int32_t)chunks,
                              t[i].dtype == MSR_BF16};
            chunks += c;
            at += n;
        }
    }
    return flush();
}

hipError_t sum_squares(const msr_gradient *t, int64_t count, double *sums, int64_t &n, hipStream_t st) {
    n = 0;
    return batches(t, count, [&](ClipArgs &a) {
        const int g = std::min(a.chunks, kSums);
        a.sums = sums + n;
        n += g;
        hipLaunchKernelGGL(gradient_norm_kernel, dim3(g), dim3(kThreads), 0, st, a);
        return hipGetLastError();
    });
}

}  // namespace

// one double per workgroup of the norm (its launches end at kTable tensors, or sooner where one is cut), and one for their
// total: at least as many as batches() makes
size_t gradient_norm_workspace(const msr_gradient *t, int64_t count) {
    int64_t chunks = 0, launches = count / kTable + 1;
    for (int64_t i = 0; i < count; ++i) {
        const int64_t c = (t[i].n + kChunk - 1) / kChunk;
        chunks += c;
        launches += c >> 29;
    }
    launches += chunks >> 29;
    return (size_t)(std::min(chunks, launches * kSums) + 1) * sizeof(double);
}

hipError_t launch_gradient_norm(const msr_gradient *t, int64_t count, float *norm, double *ws, hipStream_t st) {
    int64_t n = 0;
    const hipError_t e = sum_squares(t, count, ws + 1, n, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(gradient_total_kernel, dim3(1), dim3(kThreads), 0, st, ws + 1, n, nullptr, norm);
    return hipGetLastError();
}

hipError_t launch_clip_gradients(const msr_gradient *t, int64_t count, float max_norm, const float *norm, float *norm_out,
                                 double *ws, hipStream_t st) {
    int64_t n = 0;
    hipError_t e;
    double *sums = ws + 1;
    if (!norm) {
        if ((e = sum_squares(t, count, sums, n, st)) != hipSuccess) return e;
        // every workgroup adds up to 2048 sums by itself; more of them are added once
        if (n > 2048 || n == 0) {
            hipLaunchKernelGGL(gradient_total_kernel, dim3(1), dim3(kThreads), 0, st, sums, n, ws, n ? nullptr : norm_out);
            if ((e = hipGetLastError()) != hipSuccess || n == 0) return e;
            sums = ws, n = 1;
        }
    }
    return batches(t, count, [&](ClipArgs &a) {
        a.sums = sums, a.n_sums = (int)n, a.norm = norm, a.norm_out = norm_out, a.max_norm = max_norm;
        norm_out = nullptr;  // the first launch writes it
        hipLaunchKernelGGL(clip_kernel, dim3(std::min(a.chunks, 2048)), dim3(kThreads), 0, st, a);
        return hipGetLastError();
    });
}
