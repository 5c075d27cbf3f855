"""The operators next to retention as they are used together: a layer's step
from the projection's Q, K and V on -- norms and rotation of the heads,
retention, a gated recurrence over its output, and back, the gradients clipped
to a common norm -- against float64 autograd of the same composition; and
the example layer with norms of its heads.

Tolerances.  fp32: every operator's own error is below 1e-4 of its largest
value (the framework's fp32 tolerance); a gradient passes five of them in a
row, so 5e-4 of the largest value.  The example's 8-bit projections: as in
test_gpu_layer_example.py, a norm of the difference of 0.18 forward; the
head norms' weights see the same roundings as the projections' gradients, 0.23."""
import numpy as np
import pytest

from oracle import grad as og
from oracle import layer as ol
from oracle import oracle as orc
from oracle import step_ops as so
from tests.gpu_util import down, note, torch_dev
from tests.test_gpu_layer_example import BACKWARD, FORWARD, example, rel

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _reference(q, k, v, wq, wk, g, rate, gamma, theta, pos0, dy):
    """Gradients of sum(y dy), y the gated recurrence over retention's output, and y (torch, float64, CPU)."""
    import torch
    leaves = [torch.tensor(np.asarray(a, np.float64), requires_grad=True) for a in (q, k, v, wq, wk, g, rate)]
    q, k, v, wq, wk, g, rate = leaves
    B, T, H, dk = q.shape
    pos = torch.full((B,), float(pos0), dtype=torch.float64)
    th = torch.tensor(np.asarray(theta, np.float64))
    norm = lambda x, w: x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    qr, kr = og._rotate(norm(q, wq), th, pos), og._rotate(norm(k, wk), th, pos) * dk ** -0.5
    ga = torch.tensor(np.asarray(gamma, np.float64))
    o, _ = og._forward(qr, kr, v, None, ga, th, 1.0, 1e-5, pos, False, True)
    x = o.flatten(2)
    a = torch.exp(-rate * torch.sigmoid(g))
    u = torch.sqrt(-torch.expm1(-2 * rate * torch.sigmoid(g))) * x
    h, out = torch.zeros_like(u[:, 0]), []
    for t in range(T):
        h = a[:, t] * h + u[:, t]
        out.append(h)
    y = torch.stack(out, 1)
    (y * torch.tensor(np.asarray(dy, np.float64))).sum().backward()
    return y.detach().numpy(), [t.grad.numpy() for t in leaves]


@pytest.mark.parametrize("B,T,H,dk,dv,chunk", [(2, 96, 2, 32, 32, 32), (1, 150, 3, 16, 24, 64)])
def test_a_layers_step(B, T, H, dk, dv, chunk):
    torch, dev = torch_dev()
    import retnet_scale_retention_amd as msr
    rng = np.random.default_rng([41, T])
    f = lambda *s, scale=1.0: (scale * rng.standard_normal(s)).astype(np.float32)
    q, k, v, g, dy = f(B, T, H, dk), f(B, T, H, dk), f(B, T, H, dv), f(B, T, H * dv), f(B, T, H * dv)
    wq, wk = 1 + f(dk, scale=0.2), 1 + f(dk, scale=0.2)
    rate = np.exp(rng.uniform(np.log(1e-2), np.log(2.0), H * dv)).astype(np.float32)
    gamma, theta = np.linspace(0.93, 0.99, H).astype(np.float32), so.default_theta(dk)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    # Q, K and V side by side, as one projection writes them
    fused = torch.cat([up(a).flatten(2) for a in (q, k, v)], -1)
    qd, kd, vd = (t.unflatten(-1, (H, -1)) for t in fused.split([H * dk, H * dk, H * dv], -1))
    vd, gd, dyd, wqd, wkd, rd = vd.contiguous(), up(g), up(dy), up(wq), up(wk), up(rate)
    form = dict(flags=msr.MSR_FLAG_NO_ROTATE, scale=1.0)
    qn, kn = msr.msr_qk_norm_rotate(qd, kd, wqd, wkd, eps=EPS, theta=theta, pos0=7)
    o, _ = msr.msr_chunkwise(qn, kn, vd, gamma, chunk, **form)
    x = o.flatten(2)
    y, state, carry = msr.msr_gated_recurrence(x, gd, rd, want_carry=True)
    dx, dg, drate, _ = msr.msr_gated_recurrence_backward(x, gd, rd, dyd, carry=carry, want_state_grad=False)
    dqn, dkn, dv_, _ = msr.msr_chunkwise_backward(qn, kn, vd, gamma, chunk, dx.view(o.shape), want_state_grad=False, **form)
    back = torch.zeros_like(fused)  # the fused projection's gradient
    parts = [t.unflatten(-1, (H, -1)) for t in back.split([H * dk, H * dk, H * dv], -1)]
    parts[2].copy_(dv_)
    _, _, dwq, dwk = msr.msr_qk_norm_rotate_backward(qd, kd, wqd, wkd, dqn, dkn, eps=EPS, theta=theta, pos0=7,
                                                     out=(parts[0], parts[1], None, None))
    grads = [back, dwq, dwk, dg, drate]
    plain = [t.clone() for t in grads]
    ry, ref = _reference(q, k, v, wq, wk, g, rate, gamma, theta, 7, dy)
    err = lambda a, b: float(np.abs(down(a) - b).max() / np.abs(b).max())
    errs = [err(y, ry), *(err(p, ref[i]) for i, p in enumerate(parts)), err(dwq, ref[3]), err(dwk, ref[4]), err(dg, ref[5]),
            err(drate, ref[6])]
    note("step", T, " ".join(f"{e:.1e}" for e in errs))
    assert max(errs) < 5e-4
    # token by token the recurrence ends in the same state
    s = torch.zeros(B, H * dv, device=dev)
    for t in range(T):
        last = msr.msr_gated_recurrence_step(x[:, t].contiguous(), gd[:, t].contiguous(), s, rd)
    assert err(s, down(state)) < 1e-4 and err(last, down(y[:, -1])) < 1e-4
    # all gradients clipped to half of their common norm
    n = float(np.sqrt(sum((down(t) ** 2).sum() for t in plain)))
    _, norm = msr.msr_clip_gradients(grads, n / 2)
    assert abs(float(norm) / n - 1) < 1e-6
    for a, b in zip(grads, plain):
        assert np.all(np.abs(down(a) - down(b) / 2) <= 1e-6 * np.abs(down(b)))


@pytest.mark.parametrize("B,T,H,dk,dv,d,chunk", [(2, 192, 4, 64, 128, 256, 64), (1, 77, 2, 32, 32, 192, 64)])
def test_the_example_layer_with_norms_of_its_heads(B, T, H, dk, dv, d, chunk):
    torch, dev = torch_dev()
    layer, w, (wq, wk, wv, wo) = example().make(H, dk, dv, d, chunk, seed=5, qk_norm=True)
    g = torch.Generator(device=dev).manual_seed(6)
    x, r = (torch.randn((B, T + 1, d), generator=g, device=dev).bfloat16() for _ in range(2))
    n, _ = ol.add_rmsnorm(down(x), down(r), down(w), layer.eps)
    th = so.default_theta(dk)
    pos = np.tile(np.arange(T + 1), (B, 1))
    heads = lambda m, wt, s: so.qk_norm((n @ down(m).T).reshape(B, T + 1, H, dk), down(wt), pos, th, layer.eps, s)[0]
    q, k = heads(wq, layer.qk_norm[0], 1.0), heads(wk, layer.qk_norm[1], dk ** -0.5)
    v = (n @ down(wv).T).reshape(B, T + 1, H, dv)
    # already rotated and scaled: the definition without its own rotation
    o, _ = og.forward(q, k, v, layer.gamma, scale=1.0, rotate=False)
    want = o.reshape(B, T + 1, H * dv) @ down(wo).T
    y, _, state = layer.prompt(x[:, :T].contiguous(), r[:, :T].contiguous())
    yt, _ = layer.token(x[:, T].contiguous(), r[:, T].contiguous(), state, T)
    rows = torch.full((B,), T, dtype=torch.int64, device=dev)
    _, _, state2 = layer.prompt(x[:, :T].contiguous(), r[:, :T].contiguous())
    yr, _ = layer.token(x[:, T].contiguous(), r[:, T].contiguous(), state2, rows)
    assert torch.equal(yr, yt)
    err, et = rel(down(y), want[:, :T]), rel(down(yt), want[:, T])
    note(f"prompt {err:.3f} token {et:.3f}")
    assert err < FORWARD and et < FORWARD
    xs, rs = x[:, :T].contiguous(), r[:, :T].contiguous()
    gy, gh = (torch.randn((B, T, d), generator=g, device=dev).bfloat16() for _ in range(2))
    yt2, _, grads = layer.train(xs, rs, gy, gh)
    assert len(grads) == 8 and rel(down(yt2), want[:, :T]) < FORWARD
    # the head norms' gradients against autograd of the plain composition
    leaves = [torch.tensor(down(t), requires_grad=True) for t in layer.qk_norm]
    raw = [torch.tensor((n[:, :T] @ down(m).T).reshape(B, T, H, dk)) for m in (wq, wk)]
    zero = torch.zeros(B, dtype=torch.float64)
    tt = torch.tensor(th.astype(np.float64))
    rot = lambda z, wt: og._rotate(z / torch.sqrt((z * z).mean(-1, keepdim=True) + layer.eps) * wt, tt, zero)
    oo, _ = og._forward(rot(raw[0], leaves[0]), rot(raw[1], leaves[1]) * dk ** -0.5, torch.tensor(v[:, :T]), None,
                        torch.tensor(layer.gamma.astype(np.float64)), tt, 1.0, float(np.float32(1e-5)), zero, False, True)
    (oo.reshape(B, T, H * dv) @ torch.tensor(down(wo)).T * torch.tensor(down(gy))).sum().backward()
    errs = [rel(down(a), b.grad.numpy()) for a, b in zip(grads[6:], leaves)]
    note("head norms' gradients", " ".join(f"{e:.3f}" for e in errs))
    assert max(errs) < BACKWARD
    before = [t.clone() for t in grads]
    norm = float(layer.clip(grads, 1.0))
    assert torch.equal(grads[0], before[0]) and norm > 1
    for a, b in zip(grads[1:], before[1:]):
        assert np.all(np.abs(down(a) - down(b) / norm) <= 2.0 ** -22 * np.abs(down(b) / norm) + 1e-30)


def test_the_example_runs(capsys):
    torch_dev()
    ex = example()
    layer, _, _ = ex.make(2, 32, 32, 64, 32, qk_norm=True)
    assert layer.form and ex.make(2, 32, 32, 64, 32)[0].form == {}
