"""GPU parity of the gated recurrence, its step and its gradients against the
float64 definitions of oracle/step_ops.py.

Tolerances: the oracle's bounds of an fp32 computation (each step's relative
errors run through the recurrence themselves), times 2 for the slices and
tiles, whose factors and ends add roundings of the same sizes once per 4 and
per 64 tokens, plus the rounding of the type that a result is stored in
(2^-8 bf16, 2^-24 fp32, relative).  These take every rounding's worst side; of
1000 fp32 results together the norm is held to 8e-6: 11 u of a typical
sigmoid's error, and 2 u sqrt(2000) for the roundings of a state's memory of up
to 2000 tokens, whose signs differ."""
import numpy as np
import pytest

from oracle import step_ops as so
from tests.gpu_util import down, note, torch_dev

pytestmark = pytest.mark.gpu
STORED = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _msr():
    import retnet_scale_retention_amd as msr
    return msr


def tensor(torch, dev, a, dtype="f32"):
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dev)
    t = t.to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
    return t, down(t)


def problem(torch, dev, B, T, D, dtype, seed, state=True):
    rng = np.random.default_rng([31, seed, B, T, D])
    x = tensor(torch, dev, rng.standard_normal((B, T, D)), dtype)
    g = tensor(torch, dev, 1.5 * rng.standard_normal((B, T, D)), dtype)
    rate = tensor(torch, dev, np.exp(rng.uniform(np.log(1e-3), np.log(2.0), D)))
    st = tensor(torch, dev, rng.standard_normal((B, D))) if state else (None, None)
    dh = tensor(torch, dev, rng.standard_normal((B, T, D)), dtype)
    ds = tensor(torch, dev, rng.standard_normal((B, D))) if state else (None, None)
    return x, g, rate, st, dh, ds


def close(t, ref, bound, dtype, name):
    got = down(t)
    room = 2 * bound + STORED[dtype] * np.abs(ref) + 1e-37
    bad = ~(np.abs(got - ref) <= room)
    assert got.shape == ref.shape and not bad.any(), (name, int(bad.sum()), float((np.abs(got - ref) / room).max()))
    if dtype == "f32" and ref.size >= 1000 and np.isfinite(ref).all():
        assert np.linalg.norm(got - ref) <= 8e-6 * np.linalg.norm(ref), name


def blocks_of(h, state, B, D):
    first = np.zeros((B, 1, D)) if state is None else state[:, None]
    return np.concatenate([first, h], 1)[:, :-1][:, ::64]


SIZES = [(1, 1, 1), (2, 3, 5), (1, 2, 8), (1, 64, 8), (3, 65, 7), (2, 63, 128), (1, 129, 130), (2, 200, 1000), (1, 1000, 16), (1, 2500, 72), (9, 1100, 40),
         (3, 777, 257), (1, 5000, 33), (64, 16, 512), (2, 2048, 128), (5, 100, 9), (1, 1025, 12), (7, 1, 300), (1, 4099, 100)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D", SIZES)
def test_gated_recurrence(B, T, D, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    for normalize, state in ((True, True), (False, False)):
        note(f"gate {B}x{T}x{D} {dtype} {normalize}")
        (x, xf), (g, gf), (r, rf), (s, sf), _, _ = problem(torch, dev, B, T, D, dtype, 1, state)
        h, last, carry = msr.msr_gated_recurrence(x, g, r, normalize=normalize, state_in=s, want_carry=True)
        want, bound = so.gate(xf, gf, rf, sf, normalize)
        close(h, want, bound, dtype, "h")
        close(last, want[:, -1], bound[:, -1], "f32", "state")
        close(carry, blocks_of(want, sf, B, D), blocks_of(bound, None, B, D), "f32", "carry")
        again = msr.msr_gated_recurrence(x, g, r, normalize=normalize, state_in=s, want_carry=True)
        assert all(torch.equal(a, b) for a, b in zip(again, (h, last, carry)))
        h2, none, none2 = msr.msr_gated_recurrence(x, g, r, normalize=normalize, state_in=s, return_state=False)
        assert none is None and none2 is None and torch.equal(h2, h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D", SIZES)
def test_gated_recurrence_backward(B, T, D, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    for normalize, state in ((True, True), (False, False)):
        note(f"gate backward {B}x{T}x{D} {dtype} {normalize}")
        (x, xf), (g, gf), (r, rf), (s, sf), (dh, dhf), (ds, dsf) = problem(torch, dev, B, T, D, dtype, 2, state)
        _, _, carry = msr.msr_gated_recurrence(x, g, r, normalize=normalize, state_in=s, want_carry=True)
        got = msr.msr_gated_recurrence_backward(x, g, r, dh, normalize=normalize, state_in=s, carry=carry, grad_state=ds)
        want, bound = so.gate_backward(xf, gf, rf, sf, dhf, dsf, normalize)
        for name, t, w, b in zip(("dx", "dg", "drate", "dstate"), got, want, bound):
            close(t, w, b, dtype if name in ("dx", "dg") else "f32", name)
        again = msr.msr_gated_recurrence_backward(x, g, r, dh, normalize=normalize, state_in=s, grad_state=ds)
        assert all(torch.equal(a, b) for a, b in zip(again, got))  # without the carry: the same
        only = msr.msr_gated_recurrence_backward(x, g, r, dh, normalize=normalize, state_in=s, carry=carry, grad_state=ds,
                                                 want_rate_grad=False, want_state_grad=False)
        assert only[2] is None and only[3] is None and torch.equal(only[0], got[0]) and torch.equal(only[1], got[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 7), (2, 8), (64, 512), (5, 1001), (130, 130)])
def test_step(B, D, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    for normalize in (True, False):
        (x, xf), (g, gf), (r, rf), (s, sf), _, _ = problem(torch, dev, B, 1, D, dtype, 3)
        want, bound = so.gate(xf, gf, rf, sf, normalize)
        keep = s.clone()
        out = torch.empty_like(s)
        h = msr.msr_gated_recurrence_step(x[:, 0].contiguous(), g[:, 0].contiguous(), s, r, normalize=normalize, state_out=out)
        assert torch.equal(s, keep)
        close(h, want[:, 0], bound[:, 0], dtype, "h")
        close(out, want[:, 0], bound[:, 0], "f32", "state")
        h2 = msr.msr_gated_recurrence_step(x[:, 0].contiguous(), g[:, 0].contiguous(), s, r, normalize=normalize)
        assert torch.equal(h2, h) and torch.equal(s, out)


def test_a_sequence_in_pieces_and_token_by_token():
    torch, dev = torch_dev()
    msr = _msr()
    (x, xf), (g, gf), (r, rf), (s, sf), _, _ = problem(torch, dev, 2, 300, 72, "f32", 4)
    want, bound = so.gate(xf, gf, rf, sf, True)
    state, parts = s.clone(), []
    for a, b in ((0, 1), (1, 130), (130, 131), (131, 300)):
        h, out, _ = msr.msr_gated_recurrence(x[:, a:b].contiguous(), g[:, a:b].contiguous(), r, state_in=state,
                                             out=(None, state, None))
        assert out is state
        parts.append(h)
    close(torch.cat(parts, 1), want, 2 * bound, "f32", "pieces")
    state = s.clone()
    for t in range(300):
        h = msr.msr_gated_recurrence_step(x[:, t].contiguous(), g[:, t].contiguous(), state, r)
        close(h, want[:, t], bound[:, t], "f32", f"token {t}")


def test_long_memory_keeps_its_accuracy():
    # a decay of 1 - 5e-4 a token over 20000 tokens, the same at each: a rounded once would be off by 2^-25 / 5e-4 = 6e-5
    torch, dev = torch_dev()
    msr = _msr()
    T = 20000
    x, g = torch.ones(1, T, 8, device=dev), torch.zeros(1, T, 8, device=dev)
    r = torch.full((8,), 1e-3, device=dev)
    h, last, _ = msr.msr_gated_recurrence(x, g, r, normalize=False)
    q = float(np.float32(1e-3)) * 0.5
    want = -np.expm1(-q * np.arange(1, T + 1)) / -np.expm1(-q)
    # errors of q relative to it (8 u) move h by as much; roundings of h add up over 1 / q tokens at random
    err = np.abs(down(h)[0, :, 0] / want - 1).max()
    note(f"long memory error {err:.1e}")
    assert err < 5e-6


@pytest.mark.parametrize("T", [5, 64, 300])
def test_no_tokens_no_rows_and_nothing_outside(T):
    torch, dev = torch_dev()
    msr = _msr()
    (x, _), (g, _), (r, _), (s, _), _, _ = problem(torch, dev, 2, T, 77, "bf16", 5)
    e = x[:, :0].contiguous()
    h, last, carry = msr.msr_gated_recurrence(e, e, r, state_in=s, want_carry=True)
    assert h.shape == (2, 0, 77) and carry.shape == (2, 0, 77) and torch.equal(last, s)
    dx, dg, dr, d0 = msr.msr_gated_recurrence_backward(e, e, r, e, grad_state=s, out=(None, None, torch.ones(77, device=dev), None))
    assert dx.shape == (2, 0, 77) and not dr.any() and torch.equal(d0, s)
    e = x[:0].contiguous()
    assert msr.msr_gated_recurrence(e, e, r)[0].shape == (0, T, 77)
    dr = msr.msr_gated_recurrence_backward(e, e, r, e, out=(None, None, torch.ones(77, device=dev), None))[2]
    assert not dr.any()
    # memory around the outputs stays as it was
    n, room = 2 * T * 77, 4096
    flat = torch.full((n + 2 * room,), 7.0, device=dev, dtype=torch.bfloat16)
    out = flat[room:room + n].view(2, T, 77)
    sflat = torch.full((2 * 77 + 256,), 7.0, device=dev)
    so_ = sflat[128:128 + 154].view(2, 77)
    h, _, _ = msr.msr_gated_recurrence(x, g, r, state_in=s, out=(out, so_, None))
    ref = msr.msr_gated_recurrence(x, g, r, state_in=s)
    assert torch.equal(h, ref[0]) and torch.equal(so_, ref[1])
    assert bool((flat[:room] == 7).all()) and bool((flat[room + n:] == 7).all())
    assert bool((sflat[:128] == 7).all()) and bool((sflat[128 + 154:] == 7).all())
    dx, dg = (torch.full((n + 2 * room,), 7.0, device=dev, dtype=torch.bfloat16) for _ in range(2))
    msr.msr_gated_recurrence_backward(x, g, r, x.clone(), state_in=s,
                                      out=(dx[room:room + n].view(2, T, 77), dg[room:room + n].view(2, T, 77), None, None))
    for f in (dx, dg):
        assert bool((f[:room] == 7).all()) and bool((f[room + n:] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_non_finite_values_reach_what_follows_and_nothing_else(dtype):
    torch, dev = torch_dev()
    msr = _msr()
    (x, _), (g, _), (r, _), (s, _), _, _ = problem(torch, dev, 2, 400, 130, dtype, 6)
    clean, last, carry = msr.msr_gated_recurrence(x, g, r, state_in=s, want_carry=True)
    x2, g2 = x.clone(), g.clone()
    x2[0, 70, 3] = float("nan")
    g2[0, 200, 7] = float("nan")
    x2[1, 100, 129] = float("inf")
    h, last2, carry2 = msr.msr_gated_recurrence(x2, g2, r, state_in=s, want_carry=True)
    bad = torch.zeros_like(h, dtype=torch.bool)
    bad[0, 70:, 3], bad[0, 200:, 7], bad[1, 100:, 129] = True, True, True
    assert torch.equal(h[~bad], clean[~bad]) and not bool(torch.isfinite(h[bad]).any())
    assert bool(torch.isnan(h[0, 70:, 3]).all()) and bool(torch.isnan(h[0, 200:, 7]).all())
    assert float(h[1, 100, 129]) == float("inf")
    assert not bool(torch.isfinite(last2[0, 3])) and not bool(torch.isfinite(last2[0, 7]))
    # every bit set is a NaN too, and not mistaken for a word that is not published
    bits = torch.full((1,), -1, dtype=torch.int32, device=dev).view(torch.float32)
    if dtype == "f32":
        g3 = g.clone()
        g3[0, 10, 5] = bits
        h3 = msr.msr_gated_recurrence(x, g3, r, state_in=s)[0]
        assert bool(torch.isnan(h3[0, 10:, 5]).all()) and torch.equal(h3[1], clean[1])
        s3 = s.clone()
        s3[0, 5] = bits
        h3 = msr.msr_gated_recurrence(x, g, r, state_in=s3)[0]
        assert bool(torch.isnan(h3[0, :, 5]).all()) and torch.equal(h3[1], clean[1])
    # gates without bound: a closed one keeps the state, an open one decays by the rate
    g4 = torch.full_like(g, float("-inf"))
    h4, l4, _ = msr.msr_gated_recurrence(x, g4, r, state_in=s)
    assert torch.equal(l4, s)
    g4 = torch.full_like(g, float("inf"))
    want, bound = so.gate(down(x), np.full(x.shape, 100.0), down(r), down(s), True)
    close(msr.msr_gated_recurrence(x, g4, r, state_in=s)[0], want, bound, dtype, "open")
    dx, dg, dr, d0 = msr.msr_gated_recurrence_backward(x, torch.full_like(g, float("-inf")), r, x.clone(), state_in=s)
    assert not dx.any() and not dg.any() and not dr.any()


@pytest.mark.parametrize("rate", [0.1, 4.0, 60.0])
def test_a_nan_reaches_every_token_after_it(rate):
    # also through stretches whose decay is 0 in fp32 (0 NaN is NaN), in every call
    torch, dev = torch_dev()
    msr = _msr()
    T, D = 5000, 300
    x, g, dh = (torch.randn(2, T, D, device=dev) for _ in range(3))
    r = torch.full((D,), rate, device=dev)
    x[0, 10], dh[1, T - 10] = float("nan"), float("nan")
    clean = torch.nan_to_num(x, 0.0)
    for _ in range(10):
        h, last, _ = msr.msr_gated_recurrence(x, g, r)
        assert bool(torch.isnan(h[0, 10:]).all()) and bool(torch.isnan(last[0]).all())
        assert bool(torch.isfinite(h[0, :10]).all()) and bool(torch.isfinite(h[1]).all())
        dx, dg, _, ds = msr.msr_gated_recurrence_backward(clean, g, r, dh)
        assert bool(torch.isnan(dx[1, :T - 9]).all()) and bool(torch.isnan(ds[1]).all())
        assert bool(torch.isfinite(dx[1, T - 9:]).all()) and bool(torch.isfinite(dx[0]).all())


@pytest.mark.parametrize("rate", [0.0, 1e-12, 50.0])
def test_rates_at_the_ends(rate):
    torch, dev = torch_dev()
    msr = _msr()
    (x, xf), (g, gf), _, (s, sf), (dh, dhf), (ds, dsf) = problem(torch, dev, 1, 200, 24, "f32", 7)
    r = torch.full((24,), rate, device=dev)
    want, bound = so.gate(xf, gf, down(r), sf)
    close(msr.msr_gated_recurrence(x, g, r, state_in=s)[0], want, bound, "f32", "h")
    got = msr.msr_gated_recurrence_backward(x, g, r, dh, state_in=s, grad_state=ds)
    want, bound = so.gate_backward(xf, gf, down(r), sf, dhf, dsf)
    for name, t, w, b in zip(("dx", "dg", "drate", "dstate"), got, want, bound):
        close(t, w, b, "f32", name)


def test_gradients_against_differences():
    # along a direction v, the symmetric difference of the float64 definition with step t is off by about t^2 of its third
    # derivative: t = 1e-4 leaves 1e-8 of the sums, far below fp32's own error
    torch, dev = torch_dev()
    msr = _msr()
    (x, xf), (g, gf), (r, rf), (s, sf), (dh, dhf), (ds, dsf) = problem(torch, dev, 2, 150, 20, "f32", 8)
    got = [down(t) for t in msr.msr_gated_recurrence_backward(x, g, r, dh, state_in=s, grad_state=ds)]

    def loss(x, g, r, s):
        h, _ = so.gate(x, g, r, s)
        return float((dhf * h).sum() + (dsf * h[:, -1]).sum())

    rng = np.random.default_rng(9)
    args, t = [xf, gf, rf, sf], 1e-4
    for i, d in enumerate(got):
        v = rng.standard_normal(d.shape) * (rf if i == 2 else 1.0)
        plus, minus = list(args), list(args)
        plus[i], minus[i] = args[i] + t * v, args[i] - t * v
        num = (loss(*plus) - loss(*minus)) / (2 * t)
        assert abs((d * v).sum() - num) <= 1e-5 * np.abs(d * v).sum(), i


def test_offsets_past_32_bits():
    torch, dev = torch_dev()
    msr = _msr()
    T, D, n = (1 << 21) + 67, 1030, 150
    rng = np.random.default_rng(10)
    x = torch.zeros(1, T, D, dtype=torch.bfloat16, device=dev)
    g = torch.zeros(1, T, D, dtype=torch.bfloat16, device=dev)
    tail, tf = tensor(torch, dev, rng.standard_normal((1, n, D)), "bf16")
    x[:, -n:] = tail
    r, rf = tensor(torch, dev, np.full(D, 0.25))
    h, last, carry = msr.msr_gated_recurrence(x, g, r, want_carry=True)
    want, bound = so.gate(tf, np.zeros_like(tf), rf, None)
    assert not h[:, :-n].any()
    close(h[:, -n:], want, bound, "bf16", "tail")
    close(last, want[:, -1], bound[:, -1], "f32", "state")
    dx, dg, dr, _ = msr.msr_gated_recurrence_backward(x, g, r, x, carry=carry, out=(None, None, None, None))
    (wx, wg, wr, _), (bx, bg, br, _) = so.gate_backward(tf, np.zeros_like(tf), rf, None, tf, None)
    close(dx[:, -n:], wx, bx, "bf16", "dx")
    close(dg[:, -n:], wg, bg, "bf16", "dg")
    del x, g, h, dx, dg


def test_more_channels_than_a_launch_of_the_sums_holds():
    # 2^28 channels and some: 2^23 workgroups of 512 threads in one launch of the rates' sums would be 2^32 threads
    torch, dev = torch_dev()
    msr = _msr()
    D = (1 << 28) + 1000
    x, g, dh = (torch.randn(1, 2, D, device=dev, dtype=torch.bfloat16) for _ in range(3))
    r = torch.rand(D, device=dev) * 2
    h, last, carry = msr.msr_gated_recurrence(x, g, r, want_carry=True)
    got = msr.msr_gated_recurrence_backward(x, g, r, dh, carry=carry)
    for c in (0, (1 << 26) - 70, (1 << 27) - 5, (1 << 28) - 60, D - 100):
        n = slice(c, c + 100)
        xf, gf, df, rf = down(x[..., n].contiguous()), down(g[..., n].contiguous()), down(dh[..., n].contiguous()), down(r[n])
        want, bound = so.gate(xf, gf, rf, None)
        close(h[..., n].contiguous(), want, bound, "bf16", "h")
        close(last[..., n].contiguous(), want[:, -1], bound[:, -1], "f32", "state")
        (wx, wg, wr, _), (bx, bg, br, _) = so.gate_backward(xf, gf, rf, None, df, None)
        close(got[0][..., n].contiguous(), wx, bx, "bf16", "dx")
        close(got[1][..., n].contiguous(), wg, bg, "bf16", "dg")
        close(got[2][n].contiguous(), wr, br, "f32", "drate")


@pytest.mark.parametrize("B,T,D,dtype", [(2, 1000, 200, "bf16"), (1, 3000, 64, "f32")])
def test_in_a_graph_and_on_two_streams(B, T, D, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    sets = [problem(torch, dev, B, T, D, dtype, 20 + i) for i in range(3)]
    run = lambda p: msr.msr_gated_recurrence(p[0][0], p[1][0], p[2][0], state_in=p[3][0], want_carry=True)
    back = lambda p, c: msr.msr_gated_recurrence_backward(p[0][0], p[1][0], p[2][0], p[4][0], state_in=p[3][0], carry=c,
                                                          grad_state=p[5][0])
    eager = []
    for p in sets:
        f = run(p)
        eager.append((*f, *back(p, f[2])))
    buf = [[t.clone() for t, _ in (p[0], p[1], p[2], p[3], p[4], p[5])] for p in sets[:1]][0]
    live = [(t, None) for t in buf]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        f = run(live)
        back(live, f[2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = run(live)
        out = (*f, *back(live, f[2]))
    for i in (1, 2, 0, 1):
        for t, (s, _) in zip(buf, sets[i]):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager[i])), i
        run(sets[0])  # eager work between the replays
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for p, s in zip(sets, streams):
        with torch.cuda.stream(s):
            f = run(p)
            got.append((*f, *back(p, f[2])))
    torch.cuda.synchronize()
    for a, b in zip(got, eager):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
