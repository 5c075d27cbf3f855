"""CPU checks of the layer around retention: the float64 definitions against
loops and differences, and the refusals of the C ABI, all before any launch."""
import ctypes

import numpy as np
import pytest

import retnet_scale_retention_amd as msr
from oracle import layer as ol
from retnet_scale_retention_amd import msr as m

P = ctypes.c_void_p
NULL = P()
A, B, C, D, E, F = (P(0x1000000 * (i + 1)) for i in range(6))  # far apart, aligned, never dereferenced


def refused(status, code, word):
    assert m.STATUS[status] == code, (m.STATUS[status], msr.load().msr_last_error())
    assert word in msr.load().msr_last_error().decode()


def test_e4m3_table():
    t = ol.E4M3
    assert t[0] == 0 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[0x38] == 1 and t[0x7E] == 448
    assert np.isnan(t[0x7F]) and np.isnan(t[0xFF]) and np.all(t[129:255] == -t[1:127])
    import torch
    c = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(c, t, equal_nan=True)


def test_norm_definition_by_loops_and_differences():
    rng = np.random.default_rng(1)
    x, r, w = rng.standard_normal((3, 6)), rng.standard_normal((3, 6)), rng.standard_normal(6)
    n, h = ol.add_rmsnorm(x, r, w, 1e-3)
    for i in range(3):
        ms = sum((x[i, j] + r[i, j]) ** 2 for j in range(6)) / 6
        for j in range(6):
            assert h[i, j] == x[i, j] + r[i, j]
            assert abs(n[i, j] - w[j] * h[i, j] / (ms + 1e-3) ** 0.5) < 1e-14
    dy, ds = rng.standard_normal((3, 6)), rng.standard_normal((3, 6))
    dx, dw, _, _ = ol.add_rmsnorm_backward(h, w, dy, ds, 1e-3)
    f = lambda hh, ww: (dy * ol.add_rmsnorm(hh, None, ww, 1e-3)[0]).sum() + (ds * hh).sum()
    t = 1e-5  # symmetric differences: t^2 of the third derivative, and 1e-16 / t of rounding
    for i in range(3):
        for j in range(6):
            e = np.zeros((3, 6))
            e[i, j] = t
            assert abs((f(h + e, w) - f(h - e, w)) / (2 * t) - dx[i, j]) < 1e-8
    for j in range(6):
        e = np.zeros(6)
        e[j] = t
        assert abs((f(h, w + e) - f(h, w - e)) / (2 * t) - dw[j]) < 1e-8


def test_block_scales_and_product_by_loops():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((130, 200))
    s1, e1 = ol.block_scales(x, 1)
    s2, e2 = ol.block_scales(x, 128)
    assert s1.shape == (130, 2) and s2.shape == (2, 2) and e1.shape == e2.shape == x.shape
    assert s1[129, 1] == np.abs(x[129, 128:]).max() / 448 and e1[129, 150] == s1[129, 1]
    assert s2[1, 0] == np.abs(x[128:, :128]).max() / 448 and e2[129, 5] == s2[1, 0]
    assert np.all(ol.block_scales(np.zeros((2, 3)), 1)[0] == 2.0 ** -126)
    a, b = rng.integers(0, 127, (2, 256)).astype(np.uint8), rng.integers(0, 127, (130, 256)).astype(np.uint8)
    sa, sb = rng.random((2, 2)), rng.random((2, 2))
    c, _ = ol.matmul(a, sa, b, sb, 128)
    want = sum(ol.E4M3[a[1, k]] * sa[1, k // 128] * ol.E4M3[b[129, k]] * sb[1, k // 128] for k in range(256))
    assert abs(c[1, 129] - want) <= 1e-12 * abs(want)


def test_norm_refusals():
    f = msr.load().msr_add_rmsnorm
    ok = [4, 512, 1, A, NULL, NULL, 0, 1e-6, NULL, B, NULL, NULL, NULL]

    def call(**kw):
        v = list(ok)
        for k, x in kw.items():
            v[int(k[1:])] = x
        return f(*v)

    refused(call(_2=7), "MSR_ERR_DTYPE", "dtype")
    refused(call(_5=C, _6=9), "MSR_ERR_DTYPE", "weight_dtype")
    refused(call(_0=-1), "MSR_ERR_SHAPE", "rows")
    refused(call(_0=1 << 31), "MSR_ERR_SHAPE", "rows")
    for d in (0, -5, 32769):
        refused(call(_1=d), "MSR_ERR_SHAPE", "d=")
    for eps in (-1.0, float("nan"), float("inf")):
        refused(call(_7=eps), "MSR_ERR_INVALID_ARG", "eps")
    refused(call(_10=C), "MSR_ERR_INVALID_ARG", "together")
    refused(call(_11=C), "MSR_ERR_INVALID_ARG", "together")
    refused(call(_9=NULL), "MSR_ERR_INVALID_ARG", "one of")
    refused(call(_3=NULL), "MSR_ERR_INVALID_ARG", "x is NULL")
    refused(call(_3=P(0x1000002)), "MSR_ERR_INVALID_ARG", "x is not 16-byte aligned")
    refused(call(_9=P(0x1000000 + 64)), "MSR_ERR_INVALID_ARG", "y must not overlap x")
    refused(call(_8=B), "MSR_ERR_INVALID_ARG", "overlap")
    refused(call(_4=B), "MSR_ERR_INVALID_ARG", "y must not overlap residual")
    refused(call(_10=C, _11=C), "MSR_ERR_INVALID_ARG", "overlap")
    assert f(*[0, *ok[1:3], NULL, *ok[4:9], NULL, *ok[10:]]) == 0  # no rows: nothing to do


def test_norm_backward_refusals():
    lib = msr.load()
    f = lib.msr_add_rmsnorm_backward
    need = lib.msr_add_rmsnorm_backward_workspace(33, 512)
    assert need > 0 and lib.msr_add_rmsnorm_backward_workspace(33, 0) == 0
    assert lib.msr_add_rmsnorm_backward_workspace(32, 512) == 0  # one workgroup: no partial gradients
    ok = [33, 512, 1, A, NULL, 0, 1e-6, B, NULL, C, D, E, need, NULL]

    def call(**kw):
        v = list(ok)
        for k, x in kw.items():
            v[int(k[1:])] = x
        return f(*v)

    refused(call(_2=2), "MSR_ERR_DTYPE", "dtype")
    refused(call(_1=40000), "MSR_ERR_SHAPE", "d=")
    refused(call(_6=-1.0), "MSR_ERR_INVALID_ARG", "eps")
    for i in (3, 7, 9):
        refused(call(**{f"_{i}": NULL}), "MSR_ERR_INVALID_ARG", "non-NULL")
    refused(call(_9=A), "MSR_ERR_INVALID_ARG", "dx must not overlap h")
    refused(call(_10=C), "MSR_ERR_INVALID_ARG", "overlap")
    refused(call(_8=P(8)), "MSR_ERR_INVALID_ARG", "dsum is not 16-byte aligned")
    refused(call(_11=NULL), "MSR_ERR_WORKSPACE", "workspace")
    refused(call(_12=need - 1), "MSR_ERR_WORKSPACE", "workspace")


def test_quantize_refusals():
    f = msr.load().msr_quantize
    ok = [200, 300, 1, 1, A, B, C, NULL, NULL, NULL]

    def call(**kw):
        v = list(ok)
        for k, x in kw.items():
            v[int(k[1:])] = x
        return f(*v)

    refused(call(_2=5), "MSR_ERR_DTYPE", "dtype")
    for i in (0, 1):
        for n in (-1, (1 << 31) - 1, 1 << 40):
            refused(call(**{f"_{i}": n}), "MSR_ERR_SHAPE", "rows=")
    refused(call(_0=(1 << 31) - 256, _1=(1 << 31) - 256), "MSR_ERR_SHAPE", "too large")
    for b in (0, 2, 64, 256):
        refused(call(_3=b), "MSR_ERR_INVALID_ARG", "block_rows")
    refused(call(_5=NULL), "MSR_ERR_INVALID_ARG", "together")
    refused(call(_7=D), "MSR_ERR_INVALID_ARG", "together")
    refused(call(_5=NULL, _6=NULL), "MSR_ERR_INVALID_ARG", "one of")
    refused(call(_4=NULL), "MSR_ERR_INVALID_ARG", "x is NULL")
    refused(call(_6=P(0x3000004)), "MSR_ERR_INVALID_ARG", "scale is not 16-byte aligned")
    refused(call(_5=A), "MSR_ERR_INVALID_ARG", "q must not overlap x")
    refused(call(_7=B, _8=D), "MSR_ERR_INVALID_ARG", "overlap")
    assert call(_0=0, _4=NULL) == 0 and call(_1=0) == 0


def test_matmul_refusals():
    lib = msr.load()
    f = lib.msr_scaled_matmul
    ok = [200, 300, 256, A, B, C, D, 128, 1, E, NULL]

    def call(**kw):
        v = list(ok)
        for k, x in kw.items():
            v[int(k[1:])] = x
        return f(*v)

    refused(call(_8=3), "MSR_ERR_DTYPE", "out_dtype")
    for i in (0, 1, 2):
        for n in (-1, 1 << 31):
            refused(call(**{f"_{i}": n}), "MSR_ERR_SHAPE", "m=")
    refused(call(_2=200), "MSR_ERR_SHAPE", "multiple of 128")
    refused(call(_2=1 << 24), "MSR_ERR_SHAPE", "2^24")
    refused(call(_0=1 << 30, _1=1 << 30), "MSR_ERR_SHAPE", "too large")
    for b in (0, 64, 129):
        refused(call(_7=b), "MSR_ERR_INVALID_ARG", "b_block_rows")
    for i in (3, 4, 5, 6, 9):
        refused(call(**{f"_{i}": NULL}), "MSR_ERR_INVALID_ARG", "non-NULL")
    refused(call(_5=P(0x3000008)), "MSR_ERR_INVALID_ARG", "b is not 16-byte aligned")
    refused(call(_9=A), "MSR_ERR_INVALID_ARG", "out must not overlap a")
    assert call(_0=0) == 0 and call(_1=0, _9=NULL) == 0


def test_binding_refuses_what_it_cannot_pass_on():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    for call in (lambda: msr.msr_add_rmsnorm(x), lambda: msr.msr_add_rmsnorm_backward(x, None, x),
                 lambda: msr.msr_quantize(x), lambda: msr.msr_scaled_matmul(x, x, x, x)):
        with pytest.raises(ValueError):  # host tensors
            call()


def test_quantize_refuses_what_a_launch_cannot_hold():
    # workgroups of 256 threads, fewer than 2^32 threads in a launch; what is just small enough gets to the next check
    f = msr.load().msr_quantize
    misaligned = P(0x3000004)

    def rows_only(rows, cols):
        return f(rows, cols, 1, 1, A, B, misaligned, NULL, NULL, NULL)

    def tiles(rows, cols, block_rows):
        return f(rows, cols, 1, block_rows, A, NULL, NULL, B, misaligned, NULL)

    for cols in (1, 8, 128):
        refused(rows_only((1 << 30) - 63, cols), "MSR_ERR_SHAPE", "too large")
        refused(rows_only((1 << 30) - 64, cols), "MSR_ERR_INVALID_ARG", "scale is not 16-byte aligned")
    refused(rows_only(1 << 20, 129 * 1024), "MSR_ERR_SHAPE", "too large")
    refused(rows_only(1 << 20, 127 * 1024), "MSR_ERR_INVALID_ARG", "scale is not 16-byte aligned")
    for block_rows in (1, 128):
        refused(tiles(129, (1 << 31) - 128, block_rows), "MSR_ERR_SHAPE", "too large")
        refused(tiles(128, (1 << 31) - 128, block_rows), "MSR_ERR_INVALID_ARG", "scale_t is not 16-byte aligned")
        refused(tiles(1 << 19, 1 << 19, block_rows), "MSR_ERR_SHAPE", "too large")
        refused(tiles(1 << 19, (1 << 19) - 128, block_rows), "MSR_ERR_INVALID_ARG", "scale_t is not 16-byte aligned")


def test_matmul_refuses_what_a_launch_cannot_hold():
    # at most 2^25 - 8 tiles of 32 x 32; what is just small enough gets to the next check
    f = msr.load().msr_scaled_matmul
    misaligned = P(0x3000008)
    for big, small in ((1 << 30, 32), (1 << 29, 64), (1 << 18, 1 << 17)):
        for m_, n_, swap in ((big, small, False), (small, big, True)):
            call = lambda m, n: f(*((n, m) if swap else (m, n)), 256, A, B, misaligned, D, 128, 1, E, NULL)
            m_, n_ = (n_, m_) if swap else (m_, n_)
            refused(call(m_, n_), "MSR_ERR_SHAPE", "too large")
            refused(call(m_ - 256, n_), "MSR_ERR_INVALID_ARG", "b is not 16-byte aligned")
