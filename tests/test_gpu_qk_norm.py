"""GPU parity of the head norms with the rotation and their gradients against
the float64 definitions of oracle/step_ops.py.

Tolerances, from the arithmetic (u = 2^-24): a norm's sum of squares runs over
at most 8 additions per lane and 6 across lanes, halved by the square root,
plus the square root, a division and four products; cos and sin are off by at
most 8 u (an argument of at most pi/4 rounded twice, five terms of a series
each).  64 u of the sum of the magnitudes covers both, plus the rounding of the
stored type (2^-8 bf16, 2^-24 fp32).  dx: two such sums and their products,
128 u of the sum of its terms' magnitudes.  dw: those, and as many u as a
lane's rows, the lanes, waves and parts make additions in a row."""
import numpy as np
import pytest

from oracle import oracle as orc
from oracle import step_ops as so
from tests.gpu_util import TOL, down, note, out_err, torch_dev

pytestmark = pytest.mark.gpu
U = so.U
STORED = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS = 1e-6


def _msr():
    import retnet_scale_retention_amd as msr
    return msr


def tensor(torch, dev, a, dtype):
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dev)
    t = t.to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
    return t, down(t)


def heads(torch, dev, B, T, H, dk, dtype, seed):
    rng = np.random.default_rng([37, seed, B, T, H, dk])
    return tensor(torch, dev, rng.standard_normal((B, T, H, dk)) * np.exp(0.5 * rng.standard_normal(dk)), dtype)


def positions(B, T, pos0=0, rows=None):
    base = np.full(B, pos0, np.float64) if rows is None else np.asarray(rows, np.float64)
    return base[:, None] + np.arange(T)


def near(t, ref, room, dtype, name):
    got = down(t)
    assert got.shape == ref.shape, name
    bad = ~(np.abs(got - ref) <= room + STORED[dtype] * np.abs(ref) * (1 + 1e-6) + 1e-37)
    assert not bad.any(), (name, int(bad.sum()), float(np.abs(got - ref).max()))


SIZES = [(1, 1, 1, 1, 2), (2, 3, 2, 2, 6), (1, 5, 3, 1, 8), (2, 7, 4, 2, 10), (3, 5, 5, 5, 80), (1, 17, 2, 2, 16),
         (2, 9, 3, 3, 34), (2, 33, 16, 16, 64), (1, 65, 8, 8, 128), (2, 40, 16, 4, 256), (1, 9, 3, 2, 512), (4, 1, 128, 128, 32),
         (64, 1, 16, 16, 256), (1, 700, 1, 1, 24), (5, 3, 7, 0, 48), (2, 5, 2, 6, 510), (1, 3, 1, 127, 4), (2, 3000, 2, 1, 130)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,Hk,dk", SIZES)
def test_qk_norm_rotate(B, T, H, Hk, dk, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"qk {B}x{T}x{H}/{Hk}x{dk} {dtype}")
    q, qf = heads(torch, dev, B, T, H, dk, dtype, 1)
    k, kf = heads(torch, dev, B, T, Hk, dk, dtype, 2) if Hk else (None, None)
    rng = np.random.default_rng(dk)
    wt = "f32" if dk % 3 else "bf16"
    wq, wqf = tensor(torch, dev, 1 + 0.2 * rng.standard_normal(dk), wt)
    wk, wkf = tensor(torch, dev, 1 + 0.2 * rng.standard_normal(dk), wt)
    rows = rng.integers(0, 200000, B)
    th = so.default_theta(dk)
    for kind in range(3):
        kw = [dict(pos0=3), dict(pos_rows=torch.from_numpy(rows).to(dev)), dict(flags=msr.MSR_FLAG_NO_ROTATE, scale=0.75)][kind]
        pos = positions(B, T, 3) if kind == 0 else positions(B, T, rows=rows)
        ws = (wq, wk) if kind else (None, None)
        wf = (wqf, wkf) if kind else (None, None)
        s = 0.75 if kind == 2 else dk ** -0.5
        qo, ko = msr.msr_qk_norm_rotate(q, k, *ws, eps=EPS, theta=th if kind else None, **kw)
        want, size = so.qk_norm(qf, wf[0], pos, th, EPS, 1.0, kind < 2)
        near(qo, want, 64 * U * size, dtype, "q")
        if Hk:
            want, size = so.qk_norm(kf, wf[1], pos, th, EPS, s, kind < 2)
            near(ko, want, 64 * U * size, dtype, "k")
        else:
            assert ko is None
        again = msr.msr_qk_norm_rotate(q, k, *ws, eps=EPS, theta=th if kind else None, **kw)
        assert torch.equal(again[0], qo) and (not Hk or torch.equal(again[1], ko))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,Hk,dk", SIZES)
def test_qk_norm_rotate_backward(B, T, H, Hk, dk, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"qk backward {B}x{T}x{H}/{Hk}x{dk} {dtype}")
    q, qf = heads(torch, dev, B, T, H, dk, dtype, 1)
    k, kf = heads(torch, dev, B, T, Hk, dk, dtype, 2) if Hk else (None, None)
    dq, dqf = heads(torch, dev, B, T, H, dk, dtype, 3)
    dkk, dkf = heads(torch, dev, B, T, Hk, dk, dtype, 4) if Hk else (None, None)
    rng = np.random.default_rng(dk)
    wt = "f32" if dk % 3 else "bf16"
    wq, wqf = tensor(torch, dev, 1 + 0.2 * rng.standard_normal(dk), wt)
    wk, wkf = tensor(torch, dev, 1 + 0.2 * rng.standard_normal(dk), wt)
    th = so.default_theta(dk)
    chain = max(H, Hk) * (B * T / 4096 + 1) + 64
    for kind in range(2):
        ws = (wq, wk) if kind else (None, None)
        wf = (wqf, wkf) if kind else (None, None)
        kw = dict(pos0=11) if kind else dict(flags=msr.MSR_FLAG_NO_ROTATE)
        got = msr.msr_qk_norm_rotate_backward(q, k, *ws, dq, dkk, eps=EPS, **kw)
        for i, (x, w, dy, s) in enumerate(((qf, wf[0], dqf, 1.0), (kf, wf[1], dkf, dk ** -0.5))):
            if x is None:
                assert got[1] is None and got[3] is None
                continue
            dx, dw, mx, mw = so.qk_norm_backward(x, w, dy, positions(B, T, 11), th, EPS, s, bool(kind))
            near(got[i], dx, 128 * U * mx, dtype, "dx")
            near(got[2 + i], dw, (chain + 128) * U * mw, "f32", "dw")
        again = msr.msr_qk_norm_rotate_backward(q, k, *ws, dq, dkk, eps=EPS, **kw)
        assert all(a is None if b is None else torch.equal(a, b) for a, b in zip(again, got))
        only = msr.msr_qk_norm_rotate_backward(q, k, *ws, dq, dkk, eps=EPS, want_weight_grad=False, **kw)
        assert only[2] is None and only[3] is None and torch.equal(only[0], got[0]) and (not Hk or torch.equal(only[1], got[1]))
        ip, ik = dq.clone(), None if dkk is None else dkk.clone()
        msr.msr_qk_norm_rotate_backward(q, k, *ws, ip, ik, eps=EPS, out=(ip, ik, None, None), **kw)
        assert torch.equal(ip, got[0]) and (not Hk or torch.equal(ik, got[1]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,Hk,dk", [(2, 5, 3, 3, 10), (3, 4, 4, 2, 80), (64, 1, 16, 16, 256), (2, 33, 2, 2, 34), (1, 1, 2, 1, 6)])
def test_views_of_a_fused_projection(B, T, H, Hk, dk, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    gen = torch.Generator(device=dev).manual_seed(dk)
    width = (H + 2 * Hk) * dk
    fused = torch.randn(B, T, width, generator=gen, device=dev).to(t)
    view = lambda a, i, n: a[..., i * dk:(i + n) * dk].unflatten(-1, (n, dk))
    q, k = view(fused, 0, H), view(fused, H, Hk)
    qc, kc = q.contiguous(), k.contiguous()
    keep = fused.clone()
    a, b = msr.msr_qk_norm_rotate(q, k, pos0=7), msr.msr_qk_norm_rotate(qc, kc, pos0=7)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[0].is_contiguous()
    g = torch.randn(B, T, H, dk, generator=gen, device=dev).to(t), torch.randn(B, T, Hk, dk, generator=gen, device=dev).to(t)
    ref = msr.msr_qk_norm_rotate_backward(qc, kc, None, None, *g, pos0=7)
    out = torch.full_like(fused, 7.0)
    dq, dkk = view(out, 0, H), view(out, H, Hk)
    got = msr.msr_qk_norm_rotate_backward(q, k, None, None, *g, pos0=7, out=(dq, dkk, None, None))
    assert torch.equal(dq, ref[0]) and torch.equal(dkk, ref[1]) and torch.equal(got[2], ref[2]) and torch.equal(got[3], ref[3])
    assert bool((out[..., (H + Hk) * dk:] == 7).all()) and torch.equal(fused, keep)
    if T == 1:  # one token each, without the token dimension
        c = msr.msr_qk_norm_rotate(q[:, 0], k[:, 0], pos0=7)
        assert c[0].shape == (B, H, dk) and torch.equal(c[0], b[0][:, 0]) and torch.equal(c[1], b[1][:, 0])


def test_in_place_and_no_tokens():
    torch, dev = torch_dev()
    msr = _msr()
    for dk in (64, 36):
        q, _ = heads(torch, dev, 2, 50, 6, dk, "bf16", 5)
        k, _ = heads(torch, dev, 2, 50, 3, dk, "bf16", 6)
        want = msr.msr_qk_norm_rotate(q, k)
        got = msr.msr_qk_norm_rotate(q, k, out=(q, k))
        assert got[0] is q and got[1] is k and torch.equal(q, want[0]) and torch.equal(k, want[1])
    e = torch.empty(2, 0, 4, 16, device=dev)
    qo, ko = msr.msr_qk_norm_rotate(e, e)
    assert qo.shape == ko.shape == e.shape
    ones = torch.ones(16, device=dev)
    r = msr.msr_qk_norm_rotate_backward(e, e, None, None, e, e, out=(None, None, ones, ones.clone()))
    assert not r[2].any() and not r[3].any()


def test_zero_tiny_huge_and_non_finite_rows():
    torch, dev = torch_dev()
    msr = _msr()
    q, _ = heads(torch, dev, 1, 8, 2, 96, "f32", 7)
    q[0, 1] = 0.0
    q[0, 2] *= 1e-30
    q[0, 3] *= 1e25                  # squares past fp32: the norm is 0
    q[0, 4, 0, 5] = float("nan")
    q[0, 5, 1, 7] = float("inf")
    y, _ = msr.msr_qk_norm_rotate(q, eps=EPS)
    want, size = so.qk_norm(down(q)[:, :3], None, positions(1, 3), so.default_theta(96), EPS, 1.0)
    near(y[:, :3], want, 64 * U * size, "f32", "rows")
    assert not y[0, 1].any() and not y[0, 3].any()
    assert bool(torch.isnan(y[0, 4, 0]).all()) and bool(torch.isfinite(y[0, 4, 1]).all())
    assert bool(torch.isfinite(y[0, 5, 0]).all()) and bool(torch.isnan(y[0, 5, 1, 6:8]).all())
    dy = torch.ones_like(q)
    dq, _, dw, _ = msr.msr_qk_norm_rotate_backward(q[:, :4].contiguous(), None, None, None, dy[:, :4].contiguous(), None, eps=EPS)
    dx, rdw, mx, mw = so.qk_norm_backward(down(q)[:, :3], None, down(dy)[:, :3], positions(1, 3), so.default_theta(96), EPS, 1.0)
    near(dq[:, :3], dx, 128 * U * mx, "f32", "dx")
    assert not dq[0, 3].any()
    near(dw, rdw, 256 * U * mw, "f32", "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_eps(dtype):
    torch, dev = torch_dev()
    msr = _msr()
    q, _ = heads(torch, dev, 2, 3, 3, 40, dtype, 20)
    q[0, 1] = 0.0
    q[1, 2, 1] = 1e-30  # its squares are 0 in fp32
    q[1, 0, 0, 3] = float("nan")
    dy, _ = heads(torch, dev, 2, 3, 3, 40, dtype, 21)
    y, _ = msr.msr_qk_norm_rotate(q, eps=0.0)
    dq, _, dw, _ = msr.msr_qk_norm_rotate_backward(q, None, None, None, dy, None, eps=0.0)
    for t in (y, dq):
        assert not t[0, 1].any() and not t[1, 2, 1].any()
        assert bool(torch.isnan(t[1, 0, 0]).all()) and int(torch.isnan(t).sum()) == 40
    th = so.default_theta(40)
    for b, t in ((0, 0), (0, 2), (1, 1)):
        one = lambda x: down(x[b:b + 1, t:t + 1].contiguous())
        want, size = so.qk_norm(one(q), None, positions(1, 1, t), th, 0.0, 1.0)
        near(y[b:b + 1, t:t + 1].contiguous(), want, 64 * U * size, dtype, "y")
        dx, _, mx, _ = so.qk_norm_backward(one(q), None, one(dy), positions(1, 1, t), th, 0.0, 1.0)
        near(dq[b:b + 1, t:t + 1].contiguous(), dx, 128 * U * mx, dtype, "dx")
    clean = torch.nan_to_num(q, 0.0)
    assert bool(torch.isfinite(msr.msr_qk_norm_rotate_backward(clean, None, None, None, dy, None, eps=0.0)[2]).all())


def test_far_positions():
    torch, dev = torch_dev()
    msr = _msr()
    p0 = (1 << 40) - 64
    q, qf = heads(torch, dev, 1, 4, 2, 32, "f32", 8)
    # the angle in quarter turns is off by 2^-52 of itself: 2^40 theta 2^-52 at most, 1.6 times that in radians
    y, _ = msr.msr_qk_norm_rotate(q, pos0=p0)
    want, size = so.qk_norm(qf, None, positions(1, 4, p0), so.default_theta(32), EPS, 1.0)
    near(y, want, (64 * U + 4 * 2.0 ** -12) * size, "f32", "far")
    p0 = 131072
    y, _ = msr.msr_qk_norm_rotate(q, pos0=p0)
    want, size = so.qk_norm(qf, None, positions(1, 4, p0), so.default_theta(32), EPS, 1.0)
    near(y, want, 64 * U * size, "f32", "131072")


def test_gradients_against_differences():
    torch, dev = torch_dev()
    msr = _msr()
    B, T, H, dk, th = 2, 5, 3, 20, so.default_theta(20)
    q, qf = heads(torch, dev, B, T, H, dk, "f32", 9)
    dy, dyf = heads(torch, dev, B, T, H, dk, "f32", 10)
    rng = np.random.default_rng(11)
    w, wf = tensor(torch, dev, 1 + 0.2 * rng.standard_normal(dk), "f32")
    dq, _, dw, _ = msr.msr_qk_norm_rotate_backward(q, None, w, None, dy, None, eps=EPS, pos0=2)
    loss = lambda x, ww: float((dyf * so.qk_norm(x, ww, positions(B, T, 2), th, EPS, 1.0)[0]).sum())
    t = 1e-4  # symmetric: t^2 of the third derivative, about 1e-8
    for _ in range(3):
        v, vw = rng.standard_normal(qf.shape), rng.standard_normal(dk)
        num = (loss(qf + t * v, wf) - loss(qf - t * v, wf)) / (2 * t)
        assert abs((down(dq) * v).sum() - num) <= 1e-5 * np.abs(down(dq) * v).sum()
        num = (loss(qf, wf + t * vw) - loss(qf, wf - t * vw)) / (2 * t)
        assert abs((down(dw) * vw).sum() - num) <= 1e-5 * np.abs(down(dw) * vw).sum()


def test_the_forms_take_its_results():
    # normed and rotated heads through retention equal retention of the normed heads, which rotates them itself
    torch, dev = torch_dev()
    msr = _msr()
    B, T, H, dk, dv = 2, 192, 4, 64, 64
    q, qf = heads(torch, dev, B, T, H, dk, "bf16", 12)
    k, kf = heads(torch, dev, B, T, H, dk, "bf16", 13)
    v, vf = heads(torch, dev, B, T, H, dv, "bf16", 14)
    gamma = np.linspace(0.9, 0.99, H).astype(np.float32)
    th = so.default_theta(dk)
    qn, kn = msr.msr_qk_norm_rotate(q, k, theta=th, pos0=5)
    o, s = msr.msr_chunkwise(qn, kn, v, gamma, 64, flags=msr.MSR_FLAG_NO_ROTATE, scale=1.0)
    norm = lambda x: so.qk_norm(x, None, positions(B, T), th, EPS, 1.0, False)[0].astype(np.float32)
    ro, rs = orc.chunkwise(norm(qf), norm(kf), vf.astype(np.float32), gamma, 64, theta=th, pos0=5)
    assert out_err(down(o), ro) < TOL["bf16"] and out_err(down(s)[:, None], np.asarray(rs)[:, None]) < TOL["bf16"]


def test_offsets_past_32_bits():
    # rows do not depend on where they lie: the same bits as in a short call
    torch, dev = torch_dev()
    msr = _msr()
    T, H, dk, n = 65600, 128, 256, 40
    assert T * H * dk > 1 << 31
    tail, _ = heads(torch, dev, 1, n, H, dk, "bf16", 15)
    grad, _ = heads(torch, dev, 1, n, H, dk, "bf16", 16)
    q = torch.zeros(1, T, H, dk, dtype=torch.bfloat16, device=dev)
    dy = torch.zeros_like(q)
    q[:, -n:], dy[:, -n:] = tail, grad
    y, _ = msr.msr_qk_norm_rotate(q)
    want, _ = msr.msr_qk_norm_rotate(tail, pos0=T - n)
    assert torch.equal(y[:, -n:], want) and not y[:, :-n].any()
    del y
    dx, _, dw, _ = msr.msr_qk_norm_rotate_backward(q, None, None, None, dy, None)
    wx, _, ww, _ = msr.msr_qk_norm_rotate_backward(tail, None, None, None, grad, None, pos0=T - n)
    assert torch.equal(dx[:, -n:], wx) and not dx[:, :-n].any()
    # sums of the same 5120 rows in two orders: each within 5120 roundings of the sum of the terms' magnitudes, which over
    # a row are at most |u x r| <= |dy| sqrt(dk), u being dy turned and x r of mean square 1
    room = 2 * 5120 * U * float(grad.double().square().sum(-1).sqrt().sum()) * dk ** 0.5
    assert float((dw - ww).abs().max()) <= room
    del dx, q, dy
    # three tokens, 2^30 + 24 elements from one to the next
    step = (1 << 30) + 24
    flat = torch.zeros(2 * step + 32, dtype=torch.bfloat16, device=dev)
    view = torch.as_strided(flat, (1, 3, 2, 16), (3 * step, step, 16, 1))
    x, _ = heads(torch, dev, 1, 3, 2, 16, "bf16", 17)
    view.copy_(x)
    out = torch.zeros_like(flat)
    dv = torch.as_strided(out, view.shape, view.stride())
    assert torch.equal(msr.msr_qk_norm_rotate(view)[0], msr.msr_qk_norm_rotate(x)[0])
    gx, _ = heads(torch, dev, 1, 3, 2, 16, "bf16", 18)
    msr.msr_qk_norm_rotate_backward(view, None, None, None, gx, None, out=(dv, None, None, None))
    assert torch.equal(dv, msr.msr_qk_norm_rotate_backward(x, None, None, None, gx, None)[0])


def test_in_a_graph_and_on_another_stream():
    torch, dev = torch_dev()
    msr = _msr()
    mk = lambda seed: [heads(torch, dev, 2, 200, 4, 80, "bf16", seed + i)[0] for i in range(4)]
    sets = [mk(100 * i) for i in range(3)]
    rows = torch.tensor([5, 90000], device=dev)
    run = lambda p: (*msr.msr_qk_norm_rotate(p[0], p[1], pos_rows=rows),
                     *msr.msr_qk_norm_rotate_backward(p[0], p[1], None, None, p[2], p[3], pos_rows=rows))
    eager = [run(p) for p in sets]
    live = [t.clone() for t in sets[0]]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        other = run(live)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, eager[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(live)
    for i in (1, 0, 2, 1):
        for t, s in zip(live, sets[i]):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager[i])), i
        run(sets[0])
