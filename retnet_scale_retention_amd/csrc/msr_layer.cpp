// msr_layer.cpp -- the C ABI of the layer around retention and of the
// operators next to it (declared in include/msr.h): argument checks and
// dispatch to the norms, the quantiser, the matrix product, the gated
// recurrence and the gradients' clipping.  Everything is checked before the
// first launch.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

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

// ---- head norms with the rotation ----
msr_status check_qk(const msr_problem *p, int32_t key_heads, float eps, const void *wq, const void *wk,
                    int32_t weight_dtype) {
    if (!p) return set_error(MSR_ERR_INVALID_ARG, "problem pointer is NULL");
    if (bad_dtype(p->dtype))
        return set_error(MSR_ERR_DTYPE, "dtype %d is neither MSR_F32 (0) nor MSR_BF16 (1)", p->dtype);
    if ((wq || wk) && bad_dtype(weight_dtype))
        return set_error(MSR_ERR_DTYPE, "weight_dtype %d is neither MSR_F32 (0) nor MSR_BF16 (1)", weight_dtype);
    if (p->B < 0 || p->T < 0 || (int64_t)p->B * p->T > INT32_MAX)
        return set_error(MSR_ERR_SHAPE, "B=%d and T=%d must be >= 0 and B*T at most 2^31-1", p->B, p->T);
    if (p->H < 1 || p->H > MSR_MAX_HEADS) return set_error(MSR_ERR_SHAPE, "H=%d outside 1..%d", p->H, MSR_MAX_HEADS);
    if (key_heads < 0 || key_heads > MSR_MAX_HEADS)
        return set_error(MSR_ERR_SHAPE, "key_heads=%d outside 0..%d", key_heads, MSR_MAX_HEADS);
    if (p->dk < 2 || p->dk > MSR_MAX_DK || (p->dk & 1))
        return set_error(MSR_ERR_SHAPE, "dk=%d must be even and in 2..%d", p->dk, MSR_MAX_DK);
    if (!(eps >= 0.f) || !std::isfinite(eps))
        return set_error(MSR_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", eps);
    if (!std::isfinite(p->scale)) return set_error(MSR_ERR_INVALID_ARG, "scale is not finite");
    if (p->theta)
        for (int i = 0; i < p->dk / 2; ++i)
            if (!std::isfinite(p->theta[i])) return set_error(MSR_ERR_INVALID_ARG, "theta[%d] is not finite", i);
    if (p->pos0 < 0) return set_error(MSR_ERR_INVALID_ARG, "pos0=%lld must be >= 0", (long long)p->pos0);
    if (p->pos0 > ((int64_t)1 << 40) - p->T)
        return set_error(MSR_ERR_INVALID_ARG, "positions beyond 2^40 are not supported");
    if (p->pos_rows && (reinterpret_cast<uintptr_t>(p->pos_rows) & 7u))
        return set_error(MSR_ERR_INVALID_ARG, "pos_rows is not 8-byte aligned");
    if (p->flags & ~(uint32_t)MSR_FLAG_NO_ROTATE)
        return set_error(MSR_ERR_INVALID_ARG, "flags 0x%x: MSR_FLAG_NO_ROTATE alone is allowed", p->flags);
    return MSR_OK;
}

// elements from a token to the next
msr_status check_stride(const char *name, int64_t &stride, int heads, int dk) {
    const int64_t row = (int64_t)heads * dk;
    if (stride == 0) stride = row;
    if (stride < row || stride > (int64_t)1 << 31)
        return set_error(MSR_ERR_SHAPE, "%s=%lld is less than heads * dk = %lld, or beyond 2^31", name, (long long)stride,
                         (long long)row);
    return MSR_OK;
}

size_t extent(const msr_problem *p, int64_t stride, int heads) {
    const int64_t tokens = (int64_t)p->B * p->T;
    return tokens > 0 && heads > 0 ? (size_t)((tokens - 1) * stride + (int64_t)heads * p->dk) * elem(p->dtype) : 0;
}

msr_status check_element_aligned(const Tensor *t, int n, size_t e) {
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(t[i].p) % e)
            return set_error(MSR_ERR_INVALID_ARG, "%s is not aligned to its type", t[i].name);
    return MSR_OK;
}

// frequencies: the problem's, or the default ones, formed once per width and host thread
const float *frequencies(const msr_problem *p) {
    if (p->theta) return p->theta;
    static thread_local int dk = 0;
    static thread_local float theta[MSR_MAX_DK / 2];
    if (dk != p->dk)
        for (int i = 0; i < p->dk / 2; ++i) theta[i] = (float)std::pow(10000.0, -2.0 * (double)i / (double)p->dk);
    dk = p->dk;
    return theta;
}

QkNorm qk_norm(const msr_problem *p, int32_t key_heads, float eps, int32_t weight_dtype) {
    QkNorm q{};
    q.pos_rows = p->pos_rows, q.pos0 = p->pos0, q.tokens = (int64_t)p->B * p->T;
    q.H[0] = p->H, q.H[1] = key_heads, q.dk = p->dk, q.T = p->T, q.dtype = p->dtype, q.w_dtype = weight_dtype;
    q.rotate = !(p->flags & MSR_FLAG_NO_ROTATE), q.eps = eps;
    q.scale = p->scale != 0.f ? p->scale : (float)(1.0 / std::sqrt((double)p->dk));
    q.theta = frequencies(p);
    return q;
}

// ---- gated recurrence ----
msr_status check_gate(int64_t B, int64_t T, int64_t D, int32_t dtype) {
    if (bad_dtype(dtype)) return set_error(MSR_ERR_DTYPE, "dtype %d is neither MSR_F32 (0) nor MSR_BF16 (1)", dtype);
    if (B < 0 || T < 0 || D < 0 || B > INT32_MAX || T > INT32_MAX || D > INT32_MAX)
        return set_error(MSR_ERR_SHAPE, "B=%lld, T=%lld and D=%lld must be in 0..2^31-1", (long long)B, (long long)T,
                         (long long)D);
    // workgroups of 256 threads, each 64 tokens or more by 128 channels: fewer than 2^32 threads in a launch
    const int64_t tiles = std::max<int64_t>((T + 63) / 64, 1), cols = std::max<int64_t>((D + 127) / 128, 1);
    if (B * tiles >= 1 << 24 || B * tiles * cols >= 1 << 24)
        return set_error(MSR_ERR_SHAPE, "B=%lld x T=%lld x D=%lld is too large", (long long)B, (long long)T, (long long)D);
    return MSR_OK;
}

msr_status check_ws(const void *ws, size_t given, size_t need) {
    if (need > 0 && (!ws || given < need))
        return set_error(MSR_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? given : 0);
    return MSR_OK;
}

// ---- gradients ----
msr_status check_gradients(const msr_gradient *t, int64_t count, bool outputs) {
    if (count < 0 || count > INT32_MAX)
        return set_error(MSR_ERR_SHAPE, "count=%lld outside 0..2^31-1", (long long)count);
    if (count > 0 && !t) return set_error(MSR_ERR_INVALID_ARG, "grads is NULL");
    for (int64_t i = 0; i < count; ++i) {
        if (t[i].dtype != MSR_F32 && t[i].dtype != MSR_BF16)
            return set_error(MSR_ERR_DTYPE, "grads[%lld]: dtype %lld is neither MSR_F32 (0) nor MSR_BF16 (1)", (long long)i,
                             (long long)t[i].dtype);
        const size_t e = elem((int32_t)t[i].dtype);
        if (t[i].n < 0 || t[i].n > (int64_t)1 << 56)
            return set_error(MSR_ERR_SHAPE, "grads[%lld]: n=%lld outside 0..2^56", (long long)i, (long long)t[i].n);
        if (t[i].n == 0) continue;
        if (!t[i].grad || (outputs && !t[i].out))
            return set_error(MSR_ERR_INVALID_ARG, "grads[%lld]: a pointer is NULL", (long long)i);
        if (reinterpret_cast<uintptr_t>(t[i].grad) % e || (outputs && reinterpret_cast<uintptr_t>(t[i].out) % e))
            return set_error(MSR_ERR_INVALID_ARG, "grads[%lld] is not aligned to its type", (long long)i);
    }
    if (!outputs) return MSR_OK;
    // no output may overlap another tensor: by address, each against what began before it
    struct Span {
        uintptr_t from, to;
        bool out;
    };
    std::vector<Span> s;
    s.reserve(2 * (size_t)count);
    for (int64_t i = 0; i < count; ++i) {
        if (t[i].n == 0) continue;
        const uintptr_t g = reinterpret_cast<uintptr_t>(t[i].grad), o = reinterpret_cast<uintptr_t>(t[i].out);
        const size_t n = (size_t)t[i].n * elem((int32_t)t[i].dtype);
        if (g != o) s.push_back({g, g + n, false});
        s.push_back({o, o + n, true});
    }
    std::sort(s.begin(), s.end(), [](const Span &a, const Span &b) { return a.from < b.from; });
    uintptr_t any = 0, out = 0;  // where the spans so far, and the outputs among them, end
    for (const Span &x : s) {
        if (x.from < out || (x.out && x.from < any))
            return set_error(MSR_ERR_INVALID_ARG, "an output of the gradients overlaps another tensor");
        any = std::max(any, x.to);
        if (x.out) out = std::max(out, x.to);
    }
    return MSR_OK;
}

// no gradient or output may overlap what the calls write besides
msr_status check_apart(const msr_gradient *t, int64_t count, bool outputs, const Tensor &w) {
    for (int64_t i = 0; i < count; ++i) {
        const size_t n = (size_t)t[i].n * elem((int32_t)t[i].dtype);
        if (n > 0 && (overlap(w, {"", t[i].grad, n}) || (outputs && overlap(w, {"", t[i].out, n}))))
            return set_error(MSR_ERR_INVALID_ARG, "%s must not overlap grads[%lld]", w.name, (long long)i);
    }
    return MSR_OK;
}

// f() with what it may throw (the host's memory running out) as a status
template <typename F>
msr_status guarded(F f) {
    try {
        return f();
    } catch (const std::bad_alloc &) {
        return set_error(MSR_ERR_INVALID_ARG, "out of host memory");
    }
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

msr_status msr_qk_norm_rotate(const msr_problem *p, int32_t key_heads, float eps, const void *Q, int64_t q_stride,
                              const void *K, int64_t k_stride, const void *wq, const void *wk, int32_t weight_dtype,
                              void *QO, void *KO, void *hip_stream) {
    msr_status s = check_qk(p, key_heads, eps, wq, wk, weight_dtype);
    if (s != MSR_OK) return s;
    if ((s = check_stride("q_stride", q_stride, p->H, p->dk)) != MSR_OK ||
        (s = check_stride("k_stride", k_stride, key_heads, p->dk)) != MSR_OK)
        return s;
    if (key_heads == 0 && (K || KO || wk))
        return set_error(MSR_ERR_INVALID_ARG, "K, KO and wk must be NULL where key_heads is 0");
    if ((int64_t)p->B * p->T == 0) return MSR_OK;
    if (!Q || !QO || (key_heads > 0 && (!K || !KO)))
        return set_error(MSR_ERR_INVALID_ARG, "Q, QO, K and KO must be non-NULL");
    const int64_t qo = (int64_t)p->H * p->dk, ko = (int64_t)key_heads * p->dk;
    const size_t nw = (size_t)p->dk * elem(weight_dtype);
    const Tensor t[6] = {{"Q", Q, extent(p, q_stride, p->H)}, {"K", K, extent(p, k_stride, key_heads)}, {"wq", wq, nw},
                         {"wk", wk, nw}, {"QO", QO, extent(p, qo, p->H)}, {"KO", KO, extent(p, ko, key_heads)}};
    const uint32_t same[2] = {q_stride == qo ? 1u : 0u, k_stride == ko ? 2u : 0u};
    if ((s = check_element_aligned(t, 2, elem(p->dtype))) != MSR_OK || (s = check_aligned(t + 2, 4)) != MSR_OK ||
        (s = check_overlap(t, 6, 4, same)) != MSR_OK)
        return s;
    QkNorm q = qk_norm(p, key_heads, eps, weight_dtype);
    q.x[0] = Q, q.x[1] = K, q.w[0] = wq, q.w[1] = wk, q.y[0] = QO, q.y[1] = KO;
    q.xs[0] = q_stride, q.xs[1] = k_stride, q.ys[0] = qo, q.ys[1] = ko;
    return done(launch_qk_norm(q, false, static_cast<hipStream_t>(hip_stream)), "qk norm rotate");
}

size_t msr_qk_norm_rotate_backward_workspace(int64_t tokens, int32_t heads, int32_t key_heads, int32_t dk) {
    if (tokens < 0 || tokens > INT32_MAX || heads < 1 || heads > MSR_MAX_HEADS || key_heads < 0 ||
        key_heads > MSR_MAX_HEADS || dk < 2 || dk > MSR_MAX_DK || (dk & 1))
        return 0;
    return qk_norm_backward_workspace(tokens, heads, key_heads, dk);
}

msr_status msr_qk_norm_rotate_backward(const msr_problem *p, int32_t key_heads, float eps, const void *Q,
                                       int64_t q_stride, const void *K, int64_t k_stride, const void *wq,
                                       const void *wk, int32_t weight_dtype, const void *dQO, const void *dKO, void *dQ,
                                       int64_t dq_stride, void *dK, int64_t dk_stride, float *dwq, float *dwk, void *ws,
                                       size_t ws_bytes, void *hip_stream) {
    msr_status s = check_qk(p, key_heads, eps, wq, wk, weight_dtype);
    if (s != MSR_OK) return s;
    if ((s = check_stride("q_stride", q_stride, p->H, p->dk)) != MSR_OK ||
        (s = check_stride("k_stride", k_stride, key_heads, p->dk)) != MSR_OK ||
        (s = check_stride("dq_stride", dq_stride, p->H, p->dk)) != MSR_OK ||
        (s = check_stride("dk_stride", dk_stride, key_heads, p->dk)) != MSR_OK)
        return s;
    if (key_heads == 0 && (K || dKO || dK || wk || dwk))
        return set_error(MSR_ERR_INVALID_ARG, "K, dKO, dK, wk and dwk must be NULL where key_heads is 0");
    const int64_t tokens = (int64_t)p->B * p->T;
    if (tokens > 0 && (!Q || !dQO || !dQ || (key_heads > 0 && (!K || !dKO || !dK))))
        return set_error(MSR_ERR_INVALID_ARG, "Q, dQO, dQ, K, dKO and dK must be non-NULL");
    const int64_t qo = (int64_t)p->H * p->dk, ko = (int64_t)key_heads * p->dk;
    const size_t nw = (size_t)p->dk * elem(weight_dtype), ng = (size_t)p->dk * 4;
    const size_t need = dwq || dwk ? qk_norm_backward_workspace(tokens, p->H, key_heads, p->dk) : 0;
    const Tensor t[11] = {{"Q", Q, extent(p, q_stride, p->H)}, {"K", K, extent(p, k_stride, key_heads)},
                          {"dQ", dQ, extent(p, dq_stride, p->H)}, {"dK", dK, extent(p, dk_stride, key_heads)},
                          {"dQO", dQO, extent(p, qo, p->H)}, {"dKO", dKO, extent(p, ko, key_heads)}, {"wq", wq, nw},
                          {"wk", wk, nw}, {"dwq", dwq, ng}, {"dwk", dwk, ng}, {"ws", ws, need}};
    if ((s = check_element_aligned(t, 4, elem(p->dtype))) != MSR_OK || (s = check_aligned(t + 4, 7)) != MSR_OK) return s;
    // dQ and dK side by side in rows of one stride: no head of one reaches into the other
    bool side = false;
    if (dQ && dK && dq_stride == dk_stride) {
        const intptr_t e = (intptr_t)elem(p->dtype);
        intptr_t apart = reinterpret_cast<intptr_t>(dK) - reinterpret_cast<intptr_t>(dQ);
        if (apart % e == 0) {
            apart = apart / e % dq_stride;
            if (apart < 0) apart += dq_stride;
            side = apart >= qo && apart + ko <= dq_stride;
        }
    }
    for (int i : {2, 3, 8, 9, 10})
        for (int j = 0; j < 11; ++j) {
            if (i == j || !overlap(t[i], t[j])) continue;
            if (side && ((i == 2 && j == 3) || (i == 3 && j == 2))) continue;
            if (t[i].p == t[j].p && ((i == 2 && j == 4 && dq_stride == qo) || (i == 3 && j == 5 && dk_stride == ko))) continue;
            return set_error(MSR_ERR_INVALID_ARG, "%s must not overlap %s", t[i].name, t[j].name);
        }
    if ((s = check_ws(ws, ws_bytes, need)) != MSR_OK) return s;
    QkNorm q = qk_norm(p, key_heads, eps, weight_dtype);
    q.x[0] = Q, q.x[1] = K, q.w[0] = wq, q.w[1] = wk, q.y[0] = dQ, q.y[1] = dK, q.dy[0] = dQO, q.dy[1] = dKO;
    q.xs[0] = q_stride, q.xs[1] = k_stride, q.ys[0] = dq_stride, q.ys[1] = dk_stride;
    q.dw[0] = dwq, q.dw[1] = dwk, q.part = static_cast<float *>(ws);
    return done(launch_qk_norm(q, true, static_cast<hipStream_t>(hip_stream)), "qk norm rotate backward");
}

msr_status msr_gated_recurrence(int64_t B, int64_t T, int64_t D, int32_t dtype, int32_t normalize, const void *x,
                                const void *g, const float *rate, const float *state_in, void *h, float *state_out,
                                float *carry, void *ws, size_t ws_bytes, void *hip_stream) {
    msr_status s = check_gate(B, T, D, dtype);
    if (s != MSR_OK) return s;
    if (B == 0 || D == 0) return MSR_OK;
    if (T > 0 && (!x || !g || !rate)) return set_error(MSR_ERR_INVALID_ARG, "x, g and rate must be non-NULL");
    if (T > 0 && !h && !state_out && !carry)
        return set_error(MSR_ERR_INVALID_ARG, "one of h, state_out and carry must be non-NULL");
    const size_t n = (size_t)B * T * D * elem(dtype), ns = (size_t)B * D * 4;
    const size_t nc = (size_t)B * ((T + MSR_GATE_BLOCK - 1) / MSR_GATE_BLOCK) * D * 4;
    const size_t need = gate_workspace((int)B, (int)T, (int)D, false, true);
    const Tensor t[8] = {{"x", x, n}, {"g", g, n}, {"rate", rate, (size_t)D * 4}, {"state_in", state_in, ns},
                         {"h", h, n}, {"state_out", state_out, ns}, {"carry", carry, nc}, {"ws", ws, need}};
    const uint32_t same[4] = {0, 0x8, 0, 0};  // state_out: state_in
    if ((s = check_aligned(t, 8)) != MSR_OK || (s = check_overlap(t, 8, 4, same)) != MSR_OK ||
        (s = check_ws(ws, ws_bytes, need)) != MSR_OK)
        return s;
    Gate q{};
    q.x = x, q.g = g, q.rate = rate, q.state_in = state_in, q.h = h, q.state_out = state_out, q.carry = carry;
    q.B = (int)B, q.T = (int)T, q.D = (int)D, q.dtype = dtype, q.normalize = normalize != 0;
    return done(launch_gate(q, static_cast<char *>(ws), static_cast<hipStream_t>(hip_stream)), "gated recurrence");
}

size_t msr_gated_recurrence_workspace(int64_t B, int64_t T, int64_t D, int32_t pass) {
    if (pass < 0 || pass > 2 || check_gate(B, T, D, MSR_F32) != MSR_OK || B == 0 || D == 0) return 0;
    return gate_workspace((int)B, (int)T, (int)D, pass != 0, pass == 1);
}

msr_status msr_gated_recurrence_step(int64_t B, int64_t D, int32_t dtype, int32_t normalize, const void *x,
                                     const void *g, const float *rate, const float *state, float *state_out, void *h,
                                     void *hip_stream) {
    msr_status s = check_gate(B, 1, D, dtype);
    if (s != MSR_OK) return s;
    if (B == 0 || D == 0) return MSR_OK;
    if (!x || !g || !rate || !state || !state_out || !h)
        return set_error(MSR_ERR_INVALID_ARG, "x, g, rate, state, state_out and h must be non-NULL");
    const size_t n = (size_t)B * D * elem(dtype), ns = (size_t)B * D * 4;
    const Tensor t[6] = {{"x", x, n}, {"g", g, n}, {"rate", rate, (size_t)D * 4}, {"state", state, ns},
                         {"state_out", state_out, ns}, {"h", h, n}};
    const uint32_t same[2] = {0x8, 0};  // state_out: state
    if ((s = check_aligned(t, 6)) != MSR_OK || (s = check_overlap(t, 6, 4, same)) != MSR_OK) return s;
    Gate q{};
    q.x = x, q.g = g, q.rate = rate, q.state_in = state, q.state_out = state_out, q.h = h;
    q.B = (int)B, q.T = 1, q.D = (int)D, q.dtype = dtype, q.normalize = normalize != 0;
    return done(launch_gate_step(q, static_cast<hipStream_t>(hip_stream)), "gated recurrence step");
}

msr_status msr_gated_recurrence_backward(int64_t B, int64_t T, int64_t D, int32_t dtype, int32_t normalize,
                                         const void *x, const void *g, const float *rate, const float *state_in,
                                         const float *carry, const void *dh, const float *dstate_out, void *dx, void *dg,
                                         float *drate, float *dstate_in, void *ws, size_t ws_bytes, void *hip_stream) {
    msr_status s = check_gate(B, T, D, dtype);
    if (s != MSR_OK) return s;
    if (D == 0 || (B == 0 && !drate)) return MSR_OK;
    if (B == 0) T = 0;  // drate is zero
    if (T > 0 && (!x || !g || !rate || !dh || !dx || !dg))
        return set_error(MSR_ERR_INVALID_ARG, "x, g, rate, dh, dx and dg must be non-NULL");
    const size_t n = (size_t)B * T * D * elem(dtype), ns = (size_t)B * D * 4;
    const size_t nc = (size_t)B * ((T + MSR_GATE_BLOCK - 1) / MSR_GATE_BLOCK) * D * 4;
    const size_t need = gate_workspace((int)B, (int)T, (int)D, true, carry != nullptr);
    const Tensor t[12] = {{"x", x, n}, {"g", g, n}, {"rate", rate, (size_t)D * 4}, {"state_in", state_in, ns},
                          {"carry", carry, nc}, {"dh", dh, n}, {"dstate_out", dstate_out, ns}, {"dx", dx, n}, {"dg", dg, n},
                          {"drate", drate, (size_t)D * 4}, {"dstate_in", dstate_in, ns}, {"ws", ws, need}};
    if ((s = check_aligned(t, 12)) != MSR_OK || (s = check_overlap(t, 12, 7, nullptr)) != MSR_OK ||
        (s = check_ws(ws, ws_bytes, need)) != MSR_OK)
        return s;
    Gate q{};
    q.x = x, q.g = g, q.dh = dh, q.rate = rate, q.state_in = state_in, q.dstate_out = dstate_out;
    q.carry = const_cast<float *>(carry), q.dx = dx, q.dg = dg, q.drate = drate, q.dstate_in = dstate_in;
    q.B = (int)B, q.T = (int)T, q.D = (int)D, q.dtype = dtype, q.normalize = normalize != 0;
    return done(launch_gate_backward(q, static_cast<char *>(ws), static_cast<hipStream_t>(hip_stream)),
                "gated recurrence backward");
}

size_t msr_gradient_norm_workspace(const msr_gradient *grads, int64_t count) {
    if (check_gradients(grads, count, false) != MSR_OK) return 0;
    return gradient_norm_workspace(grads, count);
}

msr_status msr_gradient_norm(const msr_gradient *grads, int64_t count, float *norm, void *ws, size_t ws_bytes,
                             void *hip_stream) {
    msr_status s = check_gradients(grads, count, false);
    if (s != MSR_OK) return s;
    if (!norm) return set_error(MSR_ERR_INVALID_ARG, "norm is NULL");
    const Tensor t[2] = {{"norm", norm, 4}, {"ws", ws, gradient_norm_workspace(grads, count)}};
    if (reinterpret_cast<uintptr_t>(norm) % 4) return set_error(MSR_ERR_INVALID_ARG, "norm is not aligned to its type");
    if ((s = check_aligned(t + 1, 1)) != MSR_OK || (s = check_overlap(t, 2, 1, nullptr)) != MSR_OK ||
        (s = check_apart(grads, count, false, t[0])) != MSR_OK || (s = check_apart(grads, count, false, t[1])) != MSR_OK ||
        (s = check_ws(ws, ws_bytes, t[1].bytes)) != MSR_OK)
        return s;
    return done(launch_gradient_norm(grads, count, norm, static_cast<double *>(ws), static_cast<hipStream_t>(hip_stream)),
                "gradient norm");
}

msr_status msr_clip_gradients(const msr_gradient *grads, int64_t count, float max_norm, const float *norm,
                              float *norm_out, void *ws, size_t ws_bytes, void *hip_stream) {
    return guarded([&] {
        msr_status s = check_gradients(grads, count, true);
        if (s != MSR_OK) return s;
        if (!(max_norm >= 0.f)) return set_error(MSR_ERR_INVALID_ARG, "max_norm=%g must be >= 0", max_norm);
        if (norm && norm_out) return set_error(MSR_ERR_INVALID_ARG, "norm_out is for the norm that the call forms");
        const size_t need = norm ? 0 : gradient_norm_workspace(grads, count);
        const Tensor t[3] = {{"norm", norm, 4}, {"norm_out", norm_out, 4}, {"ws", ws, need}};
        if (reinterpret_cast<uintptr_t>(norm) % 4 || reinterpret_cast<uintptr_t>(norm_out) % 4)
            return set_error(MSR_ERR_INVALID_ARG, "norm or norm_out is not aligned to its type");
        if ((s = check_aligned(t + 2, 1)) != MSR_OK || (s = check_overlap(t, 3, 1, nullptr)) != MSR_OK ||
            (s = check_ws(ws, ws_bytes, need)) != MSR_OK)
            return s;
        for (const Tensor &w : t)
            if (w.p && (s = check_apart(grads, count, true, w)) != MSR_OK) return s;
        return done(launch_clip_gradients(grads, count, max_norm, norm, norm_out, static_cast<double *>(ws),
                                          static_cast<hipStream_t>(hip_stream)),
                    "clip gradients");
    });
}

}  // extern "C"
