// msr_layer.cpp -- the C ABI of the layer around retention (declared in
// include/msr.h): argument checks and dispatch to the norm, the quantiser and
// the matrix product.  Everything is checked before the first launch.
#include <cmath>

#include "msr_internal.hpp"

namespace {

struct Tensor {
    const char *name;
    const void *p;
    size_t bytes;
};

bool bad_dtype(int32_t t) { return t != MSR_F32 && t != MSR_BF16; }
size_t elem(int32_t t) { return t == MSR_BF16 ? 2 : 4; }
int64_t padded(int64_t n) { return (n + MSR_BLOCK - 1) / MSR_BLOCK * MSR_BLOCK; }

// Every given pointer aligned (sizes and the required ones are checked by the caller).
msr_status check_aligned(const Tensor *t, int n) {
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(t[i].p) & 15u)
            return set_error(MSR_ERR_INVALID_ARG, "%s is not 16-byte aligned", t[i].name);
    return MSR_OK;
}

bool overlap(const Tensor &a, const Tensor &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x && y && x < y + b.bytes && y < x + a.bytes;
}

// No output of t[from..n) may overlap any other tensor, except that bit j of
// same[i - from] lets output i BE tensor j (the same address).
msr_status check_overlap(const Tensor *t, int n, int from, const uint32_t *same) {
    for (int i = from; i < n; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && overlap(t[i], t[j]) && !(same && t[i].p == t[j].p && (same[i - from] >> j & 1)))
                return set_error(MSR_ERR_INVALID_ARG, "%s must not overlap %s", t[i].name, t[j].name);
    return MSR_OK;
}

msr_status check_norm(int64_t rows, int32_t d, int32_t dtype, const void *weight, int32_t weight_dtype, float eps) {
    if (bad_dtype(dtype)) return set_error(MSR_ERR_DTYPE, "dtype %d is neither MSR_F32 (0) nor MSR_BF16 (1)", dtype);
    if (weight && bad_dtype(weight_dtype))
        return set_error(MSR_ERR_DTYPE, "weight_dtype %d is neither MSR_F32 (0) nor MSR_BF16 (1)", weight_dtype);
    if (rows < 0 || rows > INT32_MAX) return set_error(MSR_ERR_SHAPE, "rows=%lld outside 0..2^31-1", (long long)rows);
    if (d < 1 || d > MSR_MAX_NORM_DIM) return set_error(MSR_ERR_SHAPE, "d=%d outside 1..%d", d, MSR_MAX_NORM_DIM);
    if (!(eps >= 0.f) || !std::isfinite(eps))
        return set_error(MSR_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", eps);
    return MSR_OK;
}

msr_status done(hipError_t e, const char *what) {
    return e == hipSuccess ? MSR_OK : set_error(MSR_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

}  // namespace

extern "C" {

msr_status msr_add_rmsnorm(int64_t rows, int32_t d, int32_t dtype, const void *x, const void *residual,
                           const void *weight, int32_t weight_dtype, float eps, void *sum, void *y, void *q,
                           float *q_scale, void *hip_stream) {
    msr_status s = check_norm(rows, d, dtype, weight, weight_dtype, eps);
    if (s != MSR_OK) return s;
    if (!q != !q_scale) return set_error(MSR_ERR_INVALID_ARG, "q and q_scale must be given together");
    if (rows == 0) return MSR_OK;
    if (!sum && !y && !q) return set_error(MSR_ERR_INVALID_ARG, "one of sum, y and q must be non-NULL");
    if (!x) return set_error(MSR_ERR_INVALID_ARG, "x is NULL");
    const size_t n = (size_t)rows * d * elem(dtype), nq = (size_t)rows * padded(d);
    const Tensor t[7] = {{"x", x, n}, {"residual", residual, n}, {"weight", weight, (size_t)d * elem(weight_dtype)},
                         {"sum", sum, n}, {"y", y, n}, {"q", q, nq}, {"q_scale", q_scale, nq / MSR_BLOCK * 4}};
    const uint32_t same[4] = {0x3, 0x1, 0, 0};  // sum: x or residual; y: x
    if ((s = check_aligned(t, 7)) != MSR_OK || (s = check_overlap(t, 7, 3, same)) != MSR_OK) return s;
    return done(launch_add_rmsnorm(rows, d, dtype, x, residual, weight, weight_dtype, eps, sum, y, q, q_scale,
                                   static_cast<hipStream_t>(hip_stream)),
                "add rmsnorm");
}

size_t msr_add_rmsnorm_backward_workspace(int64_t rows, int32_t d) {
    if (rows < 0 || rows > INT32_MAX || d < 1 || d > MSR_MAX_NORM_DIM) return 0;
    return rmsnorm_backward_workspace(rows, d);
}

msr_status msr_add_rmsnorm_backward(int64_t rows, int32_t d, int32_t dtype, const void *h, const void *weight,
                                    int32_t weight_dtype, float eps, const void *dy, const void *dsum, void *dx,
                                    float *dweight, void *ws, size_t ws_bytes, void *hip_stream) {
    msr_status s = check_norm(rows, d, dtype, weight, weight_dtype, eps);
    if (s != MSR_OK) return s;
    if (rows > 0 && (!h || !dy || !dx)) return set_error(MSR_ERR_INVALID_ARG, "h, dy and dx must be non-NULL");
    const size_t n = (size_t)rows * d * elem(dtype), need = dweight ? rmsnorm_backward_workspace(rows, d) : 0;
    const Tensor t[7] = {{"h", h, n}, {"weight", weight, (size_t)d * elem(weight_dtype)}, {"dy", dy, n},
                         {"dsum", dsum, n}, {"dx", dx, n}, {"dweight", dweight, (size_t)d * 4}, {"ws", ws, need}};
    const uint32_t same[3] = {0xc, 0, 0};  // dx: dy or dsum
    if ((s = check_aligned(t, 7)) != MSR_OK || (s = check_overlap(t, 7, 4, same)) != MSR_OK) return s;
    if (need > 0 && (!ws || ws_bytes < need))
        return set_error(MSR_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : 0);
    if (rows == 0 && !dweight) return MSR_OK;
    return done(launch_rmsnorm_backward(rows, d, dtype, h, weight, weight_dtype, eps, dy, dsum, dx, dweight,
                                        static_cast<float *>(ws), static_cast<hipStream_t>(hip_stream)),
                "add rmsnorm backward");
}

msr_status msr_quantize(int64_t rows, int64_t cols, int32_t dtype, int32_t block_rows, const void *x, void *q,
                        float *scale, void *qt, float *scale_t, void *hip_stream) {
    if (bad_dtype(dtype)) return set_error(MSR_ERR_DTYPE, "dtype %d is neither MSR_F32 (0) nor MSR_BF16 (1)", dtype);
    if (rows < 0 || cols < 0 || padded(rows) > INT32_MAX || padded(cols) > INT32_MAX)
        return set_error(MSR_ERR_SHAPE, "rows=%lld and cols=%lld must be in 0..2^31-128", (long long)rows,
                         (long long)cols);
    // a launch holds fewer than 2^32 threads, here in workgroups of 256: a 128 x 128 tile each, or (own order alone,
    // blocks within a row) 64 blocks
    const bool by_rows = block_rows == 1 && !qt;
    const int64_t blocks = rows * (padded(cols) / MSR_BLOCK);
    if ((by_rows ? (blocks + 63) / 64 : padded(rows) / MSR_BLOCK * (padded(cols) / MSR_BLOCK)) >= 1 << 24)
        return set_error(MSR_ERR_SHAPE, "rows=%lld x cols=%lld is too large", (long long)rows, (long long)cols);
    if (block_rows != 1 && block_rows != MSR_BLOCK)
        return set_error(MSR_ERR_INVALID_ARG, "block_rows=%d is neither 1 nor %d", block_rows, MSR_BLOCK);
    if (!q != !scale || !qt != !scale_t)
        return set_error(MSR_ERR_INVALID_ARG, "an 8-bit array and its scales must be given together");
    if (rows == 0 || cols == 0) return MSR_OK;
    if (!q && !qt) return set_error(MSR_ERR_INVALID_ARG, "one of q and qt must be non-NULL");
    if (!x) return set_error(MSR_ERR_INVALID_ARG, "x is NULL");
    const size_t nq = (size_t)rows * padded(cols), nt = (size_t)cols * padded(rows);
    const size_t sq = (size_t)(block_rows == 1 ? rows : padded(rows) / MSR_BLOCK) * (padded(cols) / MSR_BLOCK) * 4;
    const size_t sn = (size_t)(block_rows == 1 ? cols : padded(cols) / MSR_BLOCK) * (padded(rows) / MSR_BLOCK) * 4;
    const Tensor t[5] = {{"x", x, (size_t)rows * cols * elem(dtype)}, {"q", q, nq}, {"scale", scale, sq},
                         {"qt", qt, nt}, {"scale_t", scale_t, sn}};
    msr_status s;
    if ((s = check_aligned(t, 5)) != MSR_OK || (s = check_overlap(t, 5, 1, nullptr)) != MSR_OK) return s;
    return done(launch_quantize(rows, cols, dtype, block_rows, x, q, scale, qt, scale_t,
                                static_cast<hipStream_t>(hip_stream)),
                "quantize");
}

msr_status msr_scaled_matmul(int64_t m, int64_t n, int64_t k, const void *a, const float *a_scale, const void *b,
                             const float *b_scale, int32_t b_block_rows, int32_t out_dtype, void *out,
                             void *hip_stream) {
    if (bad_dtype(out_dtype))
        return set_error(MSR_ERR_DTYPE, "out_dtype %d is neither MSR_F32 (0) nor MSR_BF16 (1)", out_dtype);
    if (m < 0 || n < 0 || k < 0 || m > INT32_MAX - 1024 || n > INT32_MAX - 1024 || k > INT32_MAX)
        return set_error(MSR_ERR_SHAPE, "m=%lld, n=%lld, k=%lld outside 0..2^31-1025", (long long)m, (long long)n,
                         (long long)k);
    // 32-bit offsets within a tile
    if (k > (1 << 24) - MSR_BLOCK) return set_error(MSR_ERR_SHAPE, "k=%lld exceeds 2^24 - 128", (long long)k);
    if (k % MSR_BLOCK) return set_error(MSR_ERR_SHAPE, "k=%lld must be a multiple of %d", (long long)k, MSR_BLOCK);
    if (b_block_rows != 1 && b_block_rows != MSR_BLOCK)
        return set_error(MSR_ERR_INVALID_ARG, "b_block_rows=%d is neither 1 nor %d", b_block_rows, MSR_BLOCK);
    // the smallest tiles are 32 x 32, of 128 threads: a launch holds fewer than 2^32 threads
    if (((m + 31) / 32) * ((n + 31) / 32) > (1 << 25) - 8)
        return set_error(MSR_ERR_SHAPE, "m=%lld x n=%lld is too large", (long long)m, (long long)n);
    if (m == 0 || n == 0) return MSR_OK;
    if (!out || (k > 0 && (!a || !a_scale || !b || !b_scale)))
        return set_error(MSR_ERR_INVALID_ARG, "a, a_scale, b, b_scale and out must be non-NULL");
    const size_t kb = (size_t)k / MSR_BLOCK;
    const Tensor t[5] = {{"a", a, (size_t)m * k}, {"a_scale", a_scale, (size_t)m * kb * 4}, {"b", b, (size_t)n * k},
                         {"b_scale", b_scale, (size_t)(b_block_rows == 1 ? n : padded(n) / MSR_BLOCK) * kb * 4},
                         {"out", out, (size_t)m * n * elem(out_dtype)}};
    msr_status s;
    if ((s = check_aligned(t, 5)) != MSR_OK || (s = check_overlap(t, 5, 4, nullptr)) != MSR_OK) return s;
    return done(launch_scaled_matmul((int)m, (int)n, (int)k, a, a_scale, b, b_scale, b_block_rows, out_dtype, out,
                                     static_cast<hipStream_t>(hip_stream)),
                "scaled matmul");
}

}  // extern "C"
