"""The gated recurrence, its step and its gradients where a decay is strong, a
gate wide open or hardly open, a state infinite or a tile cut by the sequence's
end, against the formulas in float64.

Tolerances, relative to each term (u = 2^-24).  The kernels' sigmoid is off by
es = (8 + 2 |g|) u (the argument's rounding, an exponential and a reciprocal of
1 ulp), the exponent q = rate s by es + 4 u, a decay a = exp(-q) by
q (es + 4 u) + 4 u of itself, and m by es + 8 u at most (half of es of its
square).  What a result is stored in adds 2^-8 (bf16) or u (fp32)."""
import numpy as np
import pytest

from oracle import step_ops as so
from tests.gpu_util import down, note, torch_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
STORED = {"f32": U, "bf16": 2.0 ** -8}


def _msr():
    import retnet_scale_retention_amd as msr
    return msr


def tensor(torch, dev, a, dtype="f32"):
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dev)
    t = t.to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
    return t, down(t)


def parts(g, rate, normalize):
    s = 1 / (1 + np.exp(-g))
    q = rate * s
    return s, q, np.exp(-q), np.sqrt(-np.expm1(-2 * q)) if normalize else np.ones_like(q), (8 + 2 * np.abs(g)) * U


def near(t, want, room, dtype, name):
    got = down(t)
    assert got.shape == want.shape, name
    bad = ~(np.abs(got - want) <= room + STORED[dtype] * np.abs(want) * (1 + 1e-6) + 1e-37)
    worst = float(np.max(np.abs(got - want) / (np.abs(want) + 1e-37)))
    assert not bad.any(), (name, int(bad.sum()), worst)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [0.01, 0.5, 5.0, 12.0, 20.0, 30.0, 60.0])
def test_a_step_keeps_what_a_strong_decay_leaves(rate, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    rng = np.random.default_rng([51, int(100 * rate)])
    B, D = 7, 301
    x, xf = tensor(torch, dev, rng.standard_normal((B, D)) * (rng.random((B, D)) < 0.7), dtype)
    g, gf = tensor(torch, dev, 2 + 2 * rng.standard_normal((B, D)), dtype)
    r, rf = tensor(torch, dev, np.full(D, rate))
    st, sf = tensor(torch, dev, 10 ** rng.uniform(0, 8, (B, D)) * rng.choice([-1, 1], (B, D)))
    for normalize in (True, False):
        s, q, a, m, es = parts(gf, rf, normalize)
        want = a * sf + m * xf
        room = (q * (es + 4 * U) + 4 * U) * np.abs(a * sf) + (es + 10 * U) * np.abs(m * xf) + U * np.abs(want)
        room += 1.2e-38 * np.abs(sf)  # a below 2^-126 counts as 0
        out = torch.empty_like(st)
        h = msr.msr_gated_recurrence_step(x, g, st, r, normalize=normalize, state_out=out)
        near(out, want, room, "f32", "state")
        near(h, want, room, dtype, "h")


def mostly_closed(rng, T, D, opens):
    """Gates open at a few tokens, closed (decay 1) at the others."""
    g = np.full((1, T, D), -60.0)
    for t in opens:
        g[:, t] = rng.uniform(1, 5, D)
    return g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,opens", [(1, [0]), (3, [0, 1, 2]), (130, [2, 71, 129]), (700, [0, 130, 600])])
@pytest.mark.parametrize("rate", [10.0, 15.0, 20.0])
def test_a_prompt_keeps_what_a_strong_decay_leaves(rate, T, opens, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    rng = np.random.default_rng([52, T, int(rate)])
    D = 70
    g, gf = tensor(torch, dev, mostly_closed(rng, T, D, opens), dtype)
    r, rf = tensor(torch, dev, np.full(D, rate))
    st, sf = tensor(torch, dev, 1e6 * rng.standard_normal((1, D)))
    x = torch.zeros_like(g)
    _, q, _, _, es = parts(gf, rf, True)
    want = np.exp(-np.cumsum(q, 1)) * sf[:, None]
    # each open token's decay, a rounding of the state; at closed ones the state stays.  Slices' sums of exponents: at most
    # 24 additions in a row; a slice's and a tile's factor: 2 ulp each
    per = np.where(gf > 0, q * (es + 4 * U) + 8 * U, 0)
    room = (np.cumsum(per, 1) + 24 * U * np.cumsum(q, 1) + 4 * U * (2 + np.arange(1, T + 1) / 4)[None, :, None]) * np.abs(want)
    for normalize in (True, False):
        h, last, _ = msr.msr_gated_recurrence(x, g, r, normalize=normalize, state_in=st)
        near(last, want[:, -1], room[:, -1], "f32", "state")
        near(h, want, room, dtype, "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [5.0, 12.0, 20.0, 30.0])
def test_gradients_keep_what_a_strong_decay_leaves(rate, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    rng = np.random.default_rng([53, int(rate)])
    D = 1001
    x, xf = tensor(torch, dev, rng.standard_normal((1, 1, D)) * (rng.random(D) < 0.5), dtype)
    g, gf = tensor(torch, dev, rng.uniform(0, 4, (1, 1, D)), dtype)
    dh, dhf = tensor(torch, dev, rng.standard_normal((1, 1, D)), dtype)
    r, rf = tensor(torch, dev, np.full(D, rate))
    st, sf = tensor(torch, dev, rng.standard_normal((1, D)))
    ds, dsf = tensor(torch, dev, rng.standard_normal((1, D)))
    for normalize in (True, False):
        s, q, a, m, es = parts(gf, rf, normalize)
        lam, ra = dhf + dsf[:, None], q * (es + 4 * U) + 6 * U
        lroom = U * np.abs(lam)
        old = a * lam * sf[:, None]
        new = lam * xf * a * a / m if normalize else np.zeros_like(a)
        dl = old - new
        droom = (ra + 8 * U) * np.abs(old) + (2 * ra + es + 12 * U) * np.abs(new)
        k = rate * s * (1 - s)
        got = msr.msr_gated_recurrence_backward(x, g, r, dh, normalize=normalize, state_in=st, grad_state=ds)
        near(got[0], m * lam, lroom + (es + 8 * U) * np.abs(m * lam), dtype, "dx")
        # 1 - s as the difference: es of s
        near(got[1], -k * dl, k * droom + (2 * es + 8 * U + (es + 2 * U) * s / (1 - s)) * k * np.abs(dl), dtype, "dg")
        near(got[2], -(s * dl)[0, 0], (s * droom + (es + 8 * U) * s * np.abs(dl))[0, 0], "f32", "drate")
        # formed as f dstate + (a dh), f and a each within ra of exp(-q): relative to the two terms, which may cancel
        near(got[3], (a * lam)[:, 0], ((ra + 4 * U) * a * (np.abs(dhf) + np.abs(dsf[:, None])))[:, 0], "f32", "dstate")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_gradient_of_a_gate_that_is_wide_open(dtype):
    # 1 - s = exp(-g) / (1 + exp(-g)), off by es of itself, not of 1
    torch, dev = torch_dev()
    msr = _msr()
    rng = np.random.default_rng(54)
    D = 801
    g, gf = tensor(torch, dev, np.linspace(-10, 80, D)[None, None], dtype)
    x, xf = tensor(torch, dev, rng.standard_normal((1, 1, D)) * (rng.random(D) < 0.5), dtype)
    dh, dhf = tensor(torch, dev, rng.standard_normal((1, 1, D)), dtype)
    r, rf = tensor(torch, dev, np.full(D, 0.5))
    st, sf = tensor(torch, dev, rng.standard_normal((1, D)))
    for normalize in (True, False):
        s, q, a, m, es = parts(gf, rf, normalize)
        c = np.exp(-gf) / (1 + np.exp(-gf))
        old = a * dhf * sf[:, None]
        new = dhf * xf * a * a / m if normalize else np.zeros_like(a)
        k = 0.5 * s * c
        room = k * ((3 * es + 24 * U) * np.abs(old) + (5 * es + 32 * U) * np.abs(new))
        dg = msr.msr_gated_recurrence_backward(x, g, r, dh, normalize=normalize, state_in=st)[1]
        near(dg, -k * (old - new), room, dtype, "dg")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["gate", "rate"])
def test_gradients_where_the_input_hardly_counts(kind, dtype):
    # m^2 = 2 q down to 4e-38: dx = m lam, and the input's share of dl, lam x / m
    torch, dev = torch_dev()
    msr = _msr()
    rng = np.random.default_rng(55)
    D = 203
    gates = np.linspace(-60, -86, D) if kind == "gate" else np.zeros(D)
    rates = np.ones(D) if kind == "gate" else 10 ** np.linspace(-30, -37, D)
    g, gf = tensor(torch, dev, gates[None, None], dtype)
    r, rf = tensor(torch, dev, rates)
    x, xf = tensor(torch, dev, rng.standard_normal((1, 1, D)), dtype)
    dh, dhf = tensor(torch, dev, rng.standard_normal((1, 1, D)), dtype)
    s, q, a, m, es = parts(gf, rf, True)
    dl = -dhf * xf * a * a / m
    dx, dg, dr, _ = msr.msr_gated_recurrence_backward(x, g, r, dh)
    near(dx, m * dhf, (es + 8 * U) * np.abs(m * dhf), dtype, "dx")
    near(dg, -rf * s * (1 - s) * dl, (3 * es + 24 * U) * np.abs(rf * s * dl), dtype, "dg")
    near(dr, -(s * dl)[0, 0], ((2 * es + 16 * U) * s * np.abs(dl))[0, 0], "f32", "drate")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 64, 70, 129, 192])
def test_the_last_input_without_normalize_is_in_no_gradient(T, dtype):
    # h_T alone holds x_T, and no gradient holds h_T: tokens behind the sequence's end count for nothing
    torch, dev = torch_dev()
    msr = _msr()
    gen = torch.Generator(device=dev).manual_seed(T)
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    x, g, dh = (torch.randn(2, T, 40, generator=gen, device=dev).to(kind) for _ in range(3))
    r, st = torch.rand(40, generator=gen, device=dev), torch.randn(2, 40, generator=gen, device=dev)
    x[:, -1] = 0
    want = msr.msr_gated_recurrence_backward(x, g, r, dh, normalize=False, state_in=st, grad_state=st)
    assert all(bool(torch.isfinite(t).all()) for t in want)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[0, -1, 3] = bad
        got = msr.msr_gated_recurrence_backward(y, g, r, dh, normalize=False, state_in=st, grad_state=st)
        for name, a, b in zip(("dx", "dg", "drate", "dstate"), got, want):
            assert torch.equal(a, b), (name, bad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_an_infinity_stays_one(dtype):
    # a inf + m x = inf while a is not 0: 700 tokens at 0.1 leave e^-70 at least
    torch, dev = torch_dev()
    msr = _msr()
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    T, D, inf = 700, 40, float("inf")
    gen = torch.Generator(device=dev).manual_seed(56)
    x, g, dh = (torch.randn(2, T, D, generator=gen, device=dev).to(kind) for _ in range(3))
    r, st = torch.full((D,), 0.1, device=dev), torch.randn(2, D, generator=gen, device=dev)
    x[0, 10, ::2], st[1, 1::2] = inf, -inf
    for normalize in (True, False):
        h, last, carry = msr.msr_gated_recurrence(x, g, r, normalize=normalize, state_in=st, want_carry=True)
        assert bool((h[0, 10:, ::2] == inf).all()) and bool((last[0, ::2] == inf).all()) and bool((carry[0, 1:, ::2] == inf).all())
        assert bool((h[1, :, 1::2] == -inf).all()) and bool((last[1, 1::2] == -inf).all())
        for t in (h[0, :10], h[0, :, 1::2], h[1, :, ::2], last[0, 1::2], last[1, ::2]):
            assert bool(torch.isfinite(t).all())
        s = st.clone()
        for t in range(9, 14):
            msr.msr_gated_recurrence_step(x[:, t].contiguous(), g[:, t].contiguous(), s, r, normalize=normalize)
        assert bool((s[0, ::2] == inf).all()) and bool((s[1, 1::2] == -inf).all()) and bool(torch.isfinite(s[0, 1::2]).all())
        x2, s2, d2 = torch.zeros_like(x), torch.zeros_like(st), dh.clone()
        d2[0, 600, ::2] = inf
        dx, _, _, ds = msr.msr_gated_recurrence_backward(x2, g, r, d2, normalize=normalize, state_in=s2)
        assert bool((dx[0, :601, ::2] == inf).all()) and bool((ds[0, ::2] == inf).all())
        assert bool(torch.isfinite(dx[0, 601:]).all()) and bool(torch.isfinite(dx[1]).all()) and bool(torch.isfinite(ds[1]).all())


def test_long_memory_around_where_a_decay_takes_its_series():
    # the same gate at every token: a relative error of 1 - a moves the state 1 / (1 - a) by as much
    torch, dev = torch_dev()
    msr = _msr()
    T, D = 3000, 128
    x, g = torch.ones(1, T, D, device=dev), torch.zeros(1, T, D, device=dev)
    r, rf = tensor(torch, dev, 2 * np.log(2) * np.linspace(0.02, 0.2, D))
    q = 0.5 * rf
    h, last, _ = msr.msr_gated_recurrence(x, g, r, normalize=False)
    want = -np.expm1(-q * T) / -np.expm1(-q)
    err = np.abs(down(last)[0] / want - 1).max()
    note(f"largest {err:.1e}")
    # 1 - a: 2.8e-6 of itself at most; q: 4 u; roundings of h, u of it at each of the 1 / (1 - a) = 72 tokens that it holds
    assert err < 2.8e-6 + 4 * U + 72 * U


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", [(2, 1, 40), (1, 70, 24), (2, 300, 33), (1, 2000, 8)])
def test_strong_decays_over_tiles(B, T, D, dtype):
    # against the oracle's bounds, whose decays are off relative to themselves; twice them as in test_gpu_gate.py
    torch, dev = torch_dev()
    msr = _msr()
    rng = np.random.default_rng([57, B, T, D])
    some = lambda: rng.standard_normal((B, T, D)) * (rng.random((B, T, D)) < 0.7)
    (x, xf), (dh, dhf) = tensor(torch, dev, some(), dtype), tensor(torch, dev, some(), dtype)
    g, gf = tensor(torch, dev, 2 + 2 * rng.standard_normal((B, T, D)), dtype)
    r, rf = tensor(torch, dev, np.exp(rng.uniform(np.log(2), np.log(40), D)))
    (st, sf), (ds, dsf) = (tensor(torch, dev, rng.standard_normal((B, D))) for _ in range(2))
    for normalize in (True, False):
        want, bound = so.gate(xf, gf, rf, sf, normalize)
        h, last, carry = msr.msr_gated_recurrence(x, g, r, normalize=normalize, state_in=st, want_carry=True)
        near(h, want, 2 * bound, dtype, "h")
        near(last, want[:, -1], 2 * bound[:, -1], "f32", "state")
        s = st.clone()
        for t in range(min(T, 20)):
            one = msr.msr_gated_recurrence_step(x[:, t].contiguous(), g[:, t].contiguous(), s, r, normalize=normalize)
            near(one, want[:, t], 2 * bound[:, t], dtype, "step")
        got = msr.msr_gated_recurrence_backward(x, g, r, dh, normalize=normalize, state_in=st, carry=carry, grad_state=ds)
        want, bound = so.gate_backward(xf, gf, rf, sf, dhf, dsf, normalize)
        for name, a, b, c in zip(("dx", "dg", "drate", "dstate"), got, want, bound):
            near(a, b, 2 * c, dtype if name in ("dx", "dg") else "f32", name)


def test_fp32_inputs_keep_their_accuracy_at_every_decay():
    # h = m x of one token, dx = m lam.  A gate of 0 is 1/2 exactly; q is off by 3 u (two products, log2 e), 1 - a by that
    # and 4 u (a series' roundings, or an ulp of a >= 1/2 in a difference >= 0.29), 1 - a^2 by 2 u more, m by half of
    # these and 2 u (the root), the product by u: 8 u
    torch, dev = torch_dev()
    msr = _msr()
    D = 20000
    r, rf = tensor(torch, dev, 2 * np.log(2) * np.geomspace(1e-4, 3, D))
    m = np.sqrt(-np.expm1(-rf))
    x, g = torch.ones(1, 1, D, device=dev), torch.zeros(1, 1, D, device=dev)
    h, last, _ = msr.msr_gated_recurrence(x, g, r)
    step = msr.msr_gated_recurrence_step(x[0], g[0], torch.zeros(1, D, device=dev), r)
    dx = msr.msr_gated_recurrence_backward(x, g, r, x)[0]
    for name, t in (("h", h), ("state", last), ("step", step), ("dx", dx)):
        err = np.abs(down(t).ravel() / m - 1).max()
        note(f"{name} {err:.1e}")
        assert err <= 8 * U, name
