"""CPU checks of the operators next to retention: the float64 definitions
against loops and differences, the refusals of the C ABI and of the binding, all
before any launch."""
import ctypes

import numpy as np
import pytest

import retnet_scale_retention_amd as msr
from oracle import step_ops as so
from retnet_scale_retention_amd import msr as m

P = ctypes.c_void_p
NULL = P()
A, B, C, D, E, F, G, H, I, J, K, L = (P(0x1000000 * (i + 1)) for i in range(12))  # far apart, aligned, never dereferenced


def refused(status, code, word):
    assert m.STATUS[status] == code, (m.STATUS[status], msr.load().msr_last_error())
    assert word in msr.load().msr_last_error().decode(), msr.load().msr_last_error()


def caller(f, ok):
    def call(**kw):
        v = list(ok)
        for k, x in kw.items():
            v[int(k[1:])] = x
        return f(*v)
    return call


# ---- definitions -----------------------------------------------------------------
def test_qk_norm_definition_by_loops_and_differences():
    rng = np.random.default_rng(1)
    x, w, th = rng.standard_normal((2, 3, 2, 6)), rng.standard_normal(6), so.default_theta(6)
    pos = np.array([[0, 1, 2], [9, 10, 11]])
    y, size = so.qk_norm(x, w, pos, th, 1e-3, 0.5)
    for b in range(2):
        for t in range(3):
            for h in range(2):
                r = x[b, t, h]
                n = r / np.sqrt((r * r).sum() / 6 + 1e-3) * w
                for i in range(3):
                    a = pos[b, t] * float(th[i])
                    want = (0.5 * (n[2 * i] * np.cos(a) - n[2 * i + 1] * np.sin(a)),
                            0.5 * (n[2 * i + 1] * np.cos(a) + n[2 * i] * np.sin(a)))
                    assert np.allclose(y[b, t, h, 2 * i:2 * i + 2], want, rtol=0, atol=1e-14)
    assert np.all(size >= np.abs(y) - 1e-15)
    dy = rng.standard_normal(x.shape)
    dx, dw, mx, mw = so.qk_norm_backward(x, w, dy, pos, th, 1e-3, 0.5)
    loss = lambda xx, ww: (dy * so.qk_norm(xx, ww, pos, th, 1e-3, 0.5)[0]).sum()
    t = 1e-5
    for _ in range(5):
        v, vw = rng.standard_normal(x.shape), rng.standard_normal(6)
        assert abs((loss(x + t * v, w) - loss(x - t * v, w)) / (2 * t) - (dx * v).sum()) < 1e-8
        assert abs((loss(x, w + t * vw) - loss(x, w - t * vw)) / (2 * t) - (dw * vw).sum()) < 1e-8
    assert np.all(mx >= np.abs(dx) - 1e-15) and np.all(mw >= np.abs(dw) - 1e-15)


@pytest.mark.parametrize("normalize", [True, False])
def test_gate_definition_by_loops_and_differences(normalize):
    rng = np.random.default_rng(2)
    x, g, dh = (rng.standard_normal((2, 7, 3)) for _ in range(3))
    r, s, ds = np.array([0.01, 0.4, 2.0]), rng.standard_normal((2, 3)), rng.standard_normal((2, 3))
    h, bound = so.gate(x, g, r, s, normalize)
    p = s.copy()
    for t in range(7):
        for b in range(2):
            for d in range(3):
                a = np.exp(-r[d] / (1 + np.exp(-g[b, t, d])))
                p[b, d] = a * p[b, d] + (np.sqrt(1 - a * a) if normalize else 1.0) * x[b, t, d]
        assert np.allclose(h[:, t], p, rtol=0, atol=1e-12)
    assert np.all(bound > 0)
    got, bounds = so.gate_backward(x, g, r, s, dh, ds, normalize)
    loss = lambda x, g, r, s: (dh * so.gate(x, g, r, s, normalize)[0]).sum() + (ds * so.gate(x, g, r, s, normalize)[0][:, -1]).sum()
    args, t = [x, g, r, s], 1e-6
    for i, d in enumerate(got):
        assert bounds[i].shape == d.shape and np.all(bounds[i] >= 0)
        for _ in range(3):
            v = rng.standard_normal(d.shape) * (0.1 * r if i == 2 else 1.0)
            plus, minus = list(args), list(args)
            plus[i], minus[i] = args[i] + t * v, args[i] - t * v
            assert abs((loss(*plus) - loss(*minus)) / (2 * t) - (d * v).sum()) < 1e-7 * (1 + np.abs(d * v).sum())


def test_the_gate_bounds_hold_for_an_fp32_recurrence():
    # the definition in fp32, token by token, stays within the bounds that the GPU tests use; with a step left out it does not
    rng = np.random.default_rng(3)
    f = np.float32
    x, g = rng.standard_normal((1, 400, 40)).astype(f), rng.standard_normal((1, 400, 40)).astype(f)
    r = np.exp(rng.uniform(np.log(1e-3), np.log(2), 40)).astype(f)
    want, bound = so.gate(x, g, r, None)

    def run(skip):
        h, out = np.zeros((1, 40), f), []
        for t in range(400):
            q = r * (f(1) / (f(1) + np.exp(-g[:, t])))
            e = -np.expm1(-q)
            if t != skip:
                h = (h - e * h) + np.sqrt(e * (f(2) - e)) * x[:, t]
            out.append(h)
        return np.abs(np.stack(out, 1) - want)

    assert np.all(run(-1) <= bound) and not np.all(run(100) <= 10 * bound)


@pytest.mark.parametrize("lost", [False, True])
def test_the_gate_bounds_hold_for_strong_decays_and_for_nothing_less(lost):
    # fp32, token by token, rates up to 40, a third of the inputs 0: a decay as its exponential stays within the bounds, one
    # as 1 - (1 - a), of which few digits are left, does not
    rng = np.random.default_rng(4)
    f = np.float32
    B, T, D = 3, 60, 50
    x, dh = ((rng.standard_normal((B, T, D)) * (rng.random((B, T, D)) < 0.7)).astype(f) for _ in range(2))
    g = (2 + 2 * rng.standard_normal((B, T, D))).astype(f)
    r = np.exp(rng.uniform(np.log(2), np.log(40), D)).astype(f)
    st, ds = (rng.standard_normal((B, D)).astype(f) for _ in range(2))
    t = np.exp(-np.abs(g))
    c = t / (f(1) + t)
    s, slope = np.where(g < 0, c, f(1) / (f(1) + t)), c * (f(1) - c)
    q = r * s
    e = -np.expm1(-q)
    a, m = f(1) - e if lost else np.exp(-q), np.sqrt(e * (f(2) - e))
    h, before = st, []
    for i in range(T):
        before.append(h)
        h = a[:, i] * h + m[:, i] * x[:, i]
    want, bound = so.gate(x, g, r, st)
    inside = [np.abs(np.stack(before[1:] + [h], 1) - want) <= bound + 1e-37]  # below 2^-126 fp32 has no more digits
    mu, dx, dg, dr = ds, np.empty_like(x), np.empty_like(x), np.zeros(D, f)
    for i in reversed(range(T)):
        lam = dh[:, i] + mu
        mu = a[:, i] * lam
        dl = mu * (before[i] - a[:, i] * x[:, i] / m[:, i])
        dx[:, i], dg[:, i] = m[:, i] * lam, -(r * slope[:, i]) * dl
        dr -= (s[:, i] * dl).sum(0, dtype=f)
    want, bounds = so.gate_backward(x, g, r, st, dh, ds)
    inside += [np.abs(z - w) <= b + 1e-37 for z, w, b in zip((dx, dg, dr, mu), want, bounds)]
    if not lost:
        assert all(i.all() for i in inside), [int((~i).sum()) for i in inside]
    else:
        assert not any(inside[i].all() for i in (0, 2, 3, 4)), [int((~i).sum()) for i in inside]


def test_the_gate_bounds_reject_results_of_zero():
    # one token without input, of q = 10, 20, 30 and 60: what is left of the state, and the gradients, are within 1% at most
    g, one = np.full((1, 1, 4), 0.5), np.ones((1, 1, 4))
    r = np.array([10.0, 20.0, 30.0, 60.0]) * (1 + np.exp(-0.5))
    h, bound = so.gate(0 * one, g, r, one[0])
    assert np.all(bound < 0.01 * h)
    got, bounds = so.gate_backward(0 * one, g, r, one[0], one, one[0])
    for i in (1, 2, 3):
        assert np.all(bounds[i] < 0.01 * np.abs(got[i])), i


def test_clip_definition():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    out, n = so.clip(g, 1.0)
    assert n == 5 and np.allclose(out[0], [0.6, 0]) and np.allclose(out[1], [[0.8]])
    assert np.array_equal(so.clip(g, 6.0)[0][1], g[1]) and np.array_equal(so.clip(g, 0.0)[0][0], [0, 0])
    out, n = so.clip([np.array([np.inf, 1.0])], 1.0)
    assert np.isinf(n) and np.array_equal(out[0], [np.inf, 1.0])


# ---- head norms ------------------------------------------------------------------
def problem(B=2, T=8, H=4, dk=16, dtype=1, theta=None, scale=0.0, pos0=0, flags=0, pos_rows=None):
    return m._head_problem(B, T, H, dk, dtype, theta, scale, pos0, flags, None, None)[0]


def test_the_binding_packs_msr_problem_as_ctypes_does():
    th = np.arange(8, dtype=np.float32)
    raw = problem(3, 5, 7, 16, 1, th, 0.25, 1 << 33, 1)
    d = m.Problem.from_buffer_copy(raw)
    assert len(raw) == ctypes.sizeof(m.Problem)
    assert (d.B, d.T, d.H, d.dk, d.dtype, d.scale, d.pos0, d.flags) == (3, 5, 7, 16, 1, 0.25, 1 << 33, 1)
    assert not d.gamma and not d.pos_rows and [d.theta[i] for i in range(8)] == list(range(8))


BAD_PROBLEMS = [(dict(dtype=7), "MSR_ERR_DTYPE", "dtype"), (dict(B=-1), "MSR_ERR_SHAPE", "B="), (dict(T=-1), "MSR_ERR_SHAPE", "T="),
                (dict(B=1 << 16, T=1 << 15), "MSR_ERR_SHAPE", "B*T"), (dict(H=0), "MSR_ERR_SHAPE", "H="),
                (dict(H=129), "MSR_ERR_SHAPE", "H="), (dict(dk=15), "MSR_ERR_SHAPE", "dk="), (dict(dk=0), "MSR_ERR_SHAPE", "dk="),
                (dict(dk=514), "MSR_ERR_SHAPE", "dk="), (dict(scale=float("nan")), "MSR_ERR_INVALID_ARG", "scale"),
                (dict(pos0=-1), "MSR_ERR_INVALID_ARG", "pos0"), (dict(pos0=(1 << 40) - 7), "MSR_ERR_INVALID_ARG", "2^40"),
                (dict(flags=2), "MSR_ERR_INVALID_ARG", "flags"),
                (dict(theta=np.full(8, np.inf, np.float32)), "MSR_ERR_INVALID_ARG", "theta")]


def test_qk_norm_refusals():
    ok = [problem(), 4, 1e-6, A, 0, B, 0, NULL, NULL, 0, C, D, NULL]
    call = caller(msr.load().msr_qk_norm_rotate, ok)
    refused(call(_0=NULL), "MSR_ERR_INVALID_ARG", "problem")
    for kw, code, word in BAD_PROBLEMS:
        refused(call(_0=problem(**kw)), code, word)
    for n in (-1, 129):
        refused(call(_1=n), "MSR_ERR_SHAPE", "key_heads")
    refused(call(_1=0), "MSR_ERR_INVALID_ARG", "NULL")
    for eps in (-1.0, float("nan"), float("inf")):
        refused(call(_2=eps), "MSR_ERR_INVALID_ARG", "eps")
    for i in (3, 5, 10, 11):
        refused(call(**{f"_{i}": NULL}), "MSR_ERR_INVALID_ARG", "non-NULL")
    for i in (4, 6):
        for n in (63, -64, 1 << 40):
            refused(call(**{f"_{i}": n}), "MSR_ERR_SHAPE", "stride")
    refused(call(_7=E, _9=5), "MSR_ERR_DTYPE", "weight_dtype")
    refused(call(_3=P(0x1000001)), "MSR_ERR_INVALID_ARG", "aligned")
    refused(call(_10=P(0x3000008)), "MSR_ERR_INVALID_ARG", "16-byte")
    refused(call(_10=D), "MSR_ERR_INVALID_ARG", "overlap")
    refused(call(_10=B), "MSR_ERR_INVALID_ARG", "overlap")
    refused(call(_10=A, _4=128), "MSR_ERR_INVALID_ARG", "overlap")  # in place needs packed rows
    refused(call(_8=C), "MSR_ERR_INVALID_ARG", "overlap")
    assert call(_0=problem(T=0), _3=NULL, _5=NULL, _10=NULL, _11=NULL) == 0


def test_qk_norm_backward_refusals():
    lib = msr.load()
    need = lib.msr_qk_norm_rotate_backward_workspace(16, 4, 4, 16)
    assert need > 0
    for bad in ((-1, 4, 4, 16), (1 << 31, 4, 4, 16), (16, 0, 4, 16), (16, 4, 129, 16), (16, 4, 4, 15)):
        assert lib.msr_qk_norm_rotate_backward_workspace(*bad) == 0
    ok = [problem(), 4, 1e-6, A, 0, B, 0, NULL, NULL, 0, C, D, E, 0, F, 0, G, H, I, need, NULL]
    call = caller(lib.msr_qk_norm_rotate_backward, ok)
    for kw, code, word in BAD_PROBLEMS:
        refused(call(_0=problem(**kw)), code, word)
    for i in (3, 5, 10, 11, 12, 14):
        refused(call(**{f"_{i}": NULL}), "MSR_ERR_INVALID_ARG", "non-NULL")
    for i in (4, 6, 13, 15):
        refused(call(**{f"_{i}": 63}), "MSR_ERR_SHAPE", "stride")
    refused(call(_1=0), "MSR_ERR_INVALID_ARG", "NULL")
    refused(call(_18=NULL), "MSR_ERR_WORKSPACE", "workspace")
    refused(call(_19=need - 1), "MSR_ERR_WORKSPACE", "workspace")
    refused(call(_18=P(0x9000004)), "MSR_ERR_INVALID_ARG", "ws")
    refused(call(_12=A), "MSR_ERR_INVALID_ARG", "dQ must not overlap Q")
    refused(call(_12=D), "MSR_ERR_INVALID_ARG", "overlap")
    refused(call(_12=C, _13=128), "MSR_ERR_INVALID_ARG", "overlap")
    refused(call(_17=G), "MSR_ERR_INVALID_ARG", "overlap")
    # side by side in rows of 128 elements (256 bytes): heads of 64 elements fit twice, not when they reach into each other
    refused(call(_13=128, _15=128, _14=P(E.value + 126)), "MSR_ERR_INVALID_ARG", "overlap")
    refused(call(_13=128, _15=128, _14=P(E.value + 130)), "MSR_ERR_INVALID_ARG", "overlap")
    refused(call(_13=128, _15=128, _14=P(E.value + 128), _18=NULL), "MSR_ERR_WORKSPACE", "workspace")  # got past it
    refused(call(_13=128, _15=256, _14=P(E.value + 128)), "MSR_ERR_INVALID_ARG", "overlap")


# ---- gated recurrence ------------------------------------------------------------
def test_gate_refusals():
    lib = msr.load()
    ws = lib.msr_gated_recurrence_workspace(2, 3000, 200, 0)
    assert ws > 0 and lib.msr_gated_recurrence_workspace(2, 3000, 200, 2) > lib.msr_gated_recurrence_workspace(2, 3000, 200, 1) > 0
    for bad in ((-1, 5, 5, 0), (5, 1 << 31, 5, 0), (5, 5, -1, 0), (1 << 20, 1 << 20, 5, 0), (2, 5, 5, 3), (2, 5, 5, -1), (0, 5, 5, 0)):
        assert lib.msr_gated_recurrence_workspace(*bad) == 0
    ok = [2, 3000, 200, 1, 1, A, B, C, D, E, F, G, H, ws, NULL]
    call = caller(lib.msr_gated_recurrence, ok)
    refused(call(_3=2), "MSR_ERR_DTYPE", "dtype")
    for i in range(3):
        for n in (-1, 1 << 31):
            refused(call(**{f"_{i}": n}), "MSR_ERR_SHAPE", "B=")
    refused(call(_0=1 << 24, _1=1, _2=1), "MSR_ERR_SHAPE", "too large")
    refused(call(_0=1 << 10, _1=1 << 20, _2=1 << 10), "MSR_ERR_SHAPE", "too large")
    refused(call(_0=(1 << 31) - 1, _1=(1 << 31) - 1, _2=(1 << 31) - 1), "MSR_ERR_SHAPE", "too large")
    for i in (5, 6, 7):
        refused(call(**{f"_{i}": NULL}), "MSR_ERR_INVALID_ARG", "non-NULL")
    refused(call(_9=NULL, _10=NULL, _11=NULL), "MSR_ERR_INVALID_ARG", "one of")
    refused(call(_5=P(0x1000004)), "MSR_ERR_INVALID_ARG", "x is not 16-byte aligned")
    refused(call(_9=A), "MSR_ERR_INVALID_ARG", "h must not overlap x")
    refused(call(_10=P(D.value + 16)), "MSR_ERR_INVALID_ARG", "overlap")
    refused(call(_11=E), "MSR_ERR_INVALID_ARG", "overlap")
    refused(call(_12=NULL), "MSR_ERR_WORKSPACE", "workspace")
    refused(call(_13=ws - 1), "MSR_ERR_WORKSPACE", "workspace")
    refused(call(_10=D, _13=0), "MSR_ERR_WORKSPACE", "workspace")  # the state in place is allowed
    assert call(_0=0) == 0 and call(_2=0) == 0


def test_a_launch_of_the_gate_has_fewer_than_2_32_threads():
    """A workgroup of 256 threads takes 64 tokens (128 of bf16 forward) by 128 channels."""
    lib = msr.load()
    count = lib.msr_gated_recurrence_workspace
    most = (1 << 24) - 1
    for most_size, more in (((1, 64 * most, 1), (1, 64 * most + 1, 1)), ((1, 1, 128 * most), (1, 1, 128 * most + 1)),
                            ((most, 1, 1), (most + 1, 1, 1)), ((1 << 12, 64 * 4095, 128), (1 << 12, 64 * 4095 + 1, 129))):
        assert all(count(*most_size, i) > 0 and count(*more, i) == 0 for i in (0, 1, 2)), (most_size, more)
        call = caller(lib.msr_gated_recurrence, [*more, 1, 1, A, B, C, D, E, F, G, H, 0, NULL])
        refused(call(), "MSR_ERR_SHAPE", "too large")


def test_gate_step_and_backward_refusals():
    lib = msr.load()
    call = caller(lib.msr_gated_recurrence_step, [4, 200, 1, 1, A, B, C, D, E, F, NULL])
    refused(call(_2=9), "MSR_ERR_DTYPE", "dtype")
    refused(call(_0=-1), "MSR_ERR_SHAPE", "B=")
    for i in range(4, 10):
        refused(call(**{f"_{i}": NULL}), "MSR_ERR_INVALID_ARG", "non-NULL")
    refused(call(_9=A), "MSR_ERR_INVALID_ARG", "h must not overlap x")
    refused(call(_8=P(D.value + 32)), "MSR_ERR_INVALID_ARG", "overlap")
    assert call(_0=0) == 0
    ws = lib.msr_gated_recurrence_workspace(2, 3000, 200, 1)
    ok = [2, 3000, 200, 1, 1, A, B, C, D, E, F, G, H, I, J, K, L, ws, NULL]
    call = caller(lib.msr_gated_recurrence_backward, ok)
    refused(call(_3=2), "MSR_ERR_DTYPE", "dtype")
    refused(call(_1=-5), "MSR_ERR_SHAPE", "T=")
    for i in (5, 6, 7, 10, 12, 13):
        refused(call(**{f"_{i}": NULL}), "MSR_ERR_INVALID_ARG", "non-NULL")
    for i in (12, 13, 14, 15):
        refused(call(**{f"_{i}": A}), "MSR_ERR_INVALID_ARG", "overlap")
    refused(call(_12=F), "MSR_ERR_INVALID_ARG", "dx must not overlap dh")
    refused(call(_16=NULL), "MSR_ERR_WORKSPACE", "workspace")
    refused(call(_17=ws - 1), "MSR_ERR_WORKSPACE", "workspace")
    refused(call(_9=NULL), "MSR_ERR_WORKSPACE", "workspace")  # without the carry it takes more
    assert call(_2=0) == 0 and call(_0=0, _14=NULL) == 0


# ---- gradients -------------------------------------------------------------------
def table(*rows):
    return (ctypes.c_int64 * (4 * len(rows)))(*[getattr(x, "value", x) or 0 for r in rows for x in r])


def test_gradient_refusals():
    lib = msr.load()
    good = table((A, B, 100, 0), (C, C, 9000, 1))
    need = lib.msr_gradient_norm_workspace(good, 2)
    assert need > 0 and lib.msr_gradient_norm_workspace(table((A, B, 1, 5)), 1) == 0
    norm = caller(lib.msr_gradient_norm, [good, 2, D, E, need, NULL])
    clip = caller(lib.msr_clip_gradients, [good, 2, 1.0, NULL, D, E, need, NULL])
    for call in (norm, clip):
        refused(call(_1=-1), "MSR_ERR_SHAPE", "count")
        refused(call(_0=NULL), "MSR_ERR_INVALID_ARG", "grads")
        refused(call(_0=table((A, B, 100, 2)), _1=1), "MSR_ERR_DTYPE", "dtype")
        refused(call(_0=table((A, B, -1, 0)), _1=1), "MSR_ERR_SHAPE", "n=")
        refused(call(_0=table((NULL, B, 1, 0)), _1=1), "MSR_ERR_INVALID_ARG", "NULL")
        refused(call(_0=table((P(0x1000002), B, 1, 0)), _1=1), "MSR_ERR_INVALID_ARG", "aligned")
    refused(norm(_2=NULL), "MSR_ERR_INVALID_ARG", "norm is NULL")
    refused(norm(_2=P(0x4000002)), "MSR_ERR_INVALID_ARG", "aligned")
    refused(norm(_2=P(A.value + 4)), "MSR_ERR_INVALID_ARG", "norm must not overlap grads[0]")
    refused(norm(_3=P(C.value + 16)), "MSR_ERR_INVALID_ARG", "ws must not overlap grads[1]")
    refused(norm(_3=D), "MSR_ERR_INVALID_ARG", "overlap")
    refused(norm(_3=NULL), "MSR_ERR_WORKSPACE", "workspace")
    refused(norm(_4=need - 1), "MSR_ERR_WORKSPACE", "workspace")
    for bad in (-1.0, float("nan")):
        refused(clip(_2=bad), "MSR_ERR_INVALID_ARG", "max_norm")
    refused(clip(_0=table((A, NULL, 1, 0)), _1=1), "MSR_ERR_INVALID_ARG", "NULL")
    refused(clip(_3=F), "MSR_ERR_INVALID_ARG", "norm_out")
    refused(clip(_5=NULL), "MSR_ERR_WORKSPACE", "workspace")
    refused(clip(_4=P(C.value + 400)), "MSR_ERR_INVALID_ARG", "norm_out must not overlap grads[1]")
    refused(clip(_3=P(B.value + 4), _4=NULL), "MSR_ERR_INVALID_ARG", "norm must not overlap grads[0]")
    over = lambda *rows: refused(clip(_0=table(*rows), _1=len(rows)), "MSR_ERR_INVALID_ARG", "overlaps another")
    over((A, A, 100, 0), (A, A, 100, 0))                          # the same tensor twice, in place
    over((A, P(A.value + 4), 100, 0))
    over((A, B, 100, 0), (C, P(B.value + 396), 100, 0))
    over((A, B, 100, 0), (P(B.value + 200), C, 100, 0))
    over((A, B, 100, 0), (P(B.value + 200), P(B.value + 200), 100, 0))
    # inputs alone may share memory: past the overlap check
    refused(clip(_0=table((A, B, 100, 0), (A, C, 100, 0)), _5=NULL), "MSR_ERR_WORKSPACE", "workspace")


def test_workspace_covers_the_sums_of_all_launches():
    # one sum per workgroup, 1024 at most of each launch of 96 tensors, and the total's
    ws = msr.load().msr_gradient_norm_workspace
    for n, sizes in ((1, [1]), (2, [8192] * 1), (1025, [8192 * 5000]), (2 * 1024 + 1, [8192 * 2000] * 97)):
        assert ws(table(*[(A, A, s, 0) for s in sizes]), len(sizes)) >= 8 * n


# ---- the binding -----------------------------------------------------------------
def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x, h = torch.zeros(2, 4, 8), torch.zeros(2, 4, 2, 8)
    for call in (lambda: msr.msr_qk_norm_rotate(h, h), lambda: msr.msr_qk_norm_rotate_backward(h, h, None, None, h, h),
                 lambda: msr.msr_gated_recurrence(x, x, x[0, 0]), lambda: msr.msr_gated_recurrence_step(x[0], x[0], x[0], x[0, 0]),
                 lambda: msr.msr_gated_recurrence_backward(x, x, x[0, 0], x), lambda: msr.msr_gradient_norm([x]),
                 lambda: msr.msr_clip_gradients([x], 1.0), lambda: msr.msr_gradient_norm([])):
        with pytest.raises(ValueError):
            call()


def test_heads_as_views():
    torch = pytest.importorskip("torch")
    from tests.test_binding_cpu import OnDevice
    t = torch.zeros(3, 5, 40, dtype=torch.bfloat16).as_subclass(OnDevice)
    heads = lambda v: m._heads("q", v, torch.bfloat16, 0)
    v = t[..., 8:24].unflatten(-1, (2, 8))
    assert heads(v)[:4] == (3, 5, 2, 8) and heads(v)[5] == 40 and heads(v)[4] == t.data_ptr() + 16
    assert heads(v[:, 0])[:4] == (3, 1, 2, 8) and heads(v[:, 0])[5] == 200      # one token of each row
    assert heads(v[:, 1:2])[5] == 200 and heads(v[:1])[5] == 40
    assert heads(v.contiguous())[5] == 16
    for bad in (v[:, 1:3], v[:, ::2], v.transpose(1, 2), v[..., ::2], v[:, :, :, :7], v[:, 0].unsqueeze(1).expand(3, 4, 2, 8),
                t[:1, :1, :16].unflatten(-1, (2, 8)).expand(3, 5, 2, 8)):
        with pytest.raises(ValueError):
            heads(bad)
    with pytest.raises(ValueError):
        m._heads("q", v, torch.float32, 0)
    with pytest.raises(ValueError):
        m._heads("q", v, torch.bfloat16, 1)
    with pytest.raises(ValueError):
        heads(v[0, 0])
