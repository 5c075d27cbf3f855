"""The retention sub-layer of examples/retention_layer.py (norm, 8-bit
projections, retention, output projection) as one: a prompt, a token after
it, and a training step, against the plain composition in float64
(oracle/layer.py's norm, the oracle's retention and its gradients, matrix
products of the unquantised bf16 weights).

Tolerance.  Rounding to e4m3 is off by at most half a step, 2^-4 of the value,
rms 2^-4 / sqrt(3) = 3.6% where values spread evenly over the steps.  A
product's two operands and what comes after add in quadrature: the forward
pass has up to 6 such roundings one after the other (n, three weights, O, wo:
9%), a gradient up to 10 (those, dy, and dQ, dK, dV: 11%); the norms per head
that they pass through are taken as a factor of two.  So 0.18 and 0.23, as the
norm of the difference over that of the result."""
import importlib.util
from pathlib import Path

import numpy as np
import pytest

from oracle import layer as ol
from oracle import oracle as orc
from tests.gpu_util import down, note, torch_dev

pytestmark = pytest.mark.gpu
FORWARD, BACKWARD = 0.18, 0.23


def example():
    path = Path(__file__).resolve().parents[1] / "examples" / "retention_layer.py"
    spec = importlib.util.spec_from_file_location("retention_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(x, r):
    return float(np.linalg.norm(np.asarray(x, np.float64) - r) / np.linalg.norm(r))


CASES = [(2, 192, 4, 64, 128, 256, 64), (1, 77, 2, 32, 32, 192, 64), (1, 256, 2, 128, 256, 320, 128)]


@pytest.mark.parametrize("B,T,H,dk,dv,d,chunk", CASES)
def test_prompt_and_token(B, T, H, dk, dv, d, chunk):
    torch, dev = torch_dev()
    ex = example()
    layer, w, (wq, wk, wv, wo) = ex.make(H, dk, dv, d, chunk, seed=3)
    g = torch.Generator(device=dev).manual_seed(4)
    x = torch.randn((B, T + 1, d), generator=g, device=dev).bfloat16()
    r = torch.randn((B, T + 1, d), generator=g, device=dev).bfloat16()
    n, h = ol.add_rmsnorm(down(x), down(r), down(w), layer.eps)
    q, k, v = ((n @ down(m).T).reshape(B, T + 1, H, -1) for m in (wq, wk, wv))
    o, _ = orc.parallel(q, k, v, layer.gamma)
    want = o.reshape(B, T + 1, H * dv) @ down(wo).T
    y, hs, state = layer.prompt(x[:, :T].contiguous(), r[:, :T].contiguous())
    err = rel(down(y), want[:, :T])
    yt, ht = layer.token(x[:, T].contiguous(), r[:, T].contiguous(), state, T)
    et = rel(down(yt), want[:, T])
    note(f"prompt {err:.3f} token {et:.3f}")
    assert err < FORWARD and et < FORWARD
    assert np.all(np.abs(down(hs) - h[:, :T]) <= 2.0 ** -8 * np.abs(h[:, :T]))
    assert np.all(np.abs(down(ht) - h[:, T]) <= 2.0 ** -8 * np.abs(h[:, T]))


@pytest.mark.parametrize("B,T,H,dk,dv,d,chunk", CASES)
def test_training_step(B, T, H, dk, dv, d, chunk):
    torch, dev = torch_dev()
    from oracle import grad as og
    ex = example()
    layer, w, ws = ex.make(H, dk, dv, d, chunk, seed=5)
    g = torch.Generator(device=dev).manual_seed(6)
    x, r, gy, gh = (torch.randn((B, T, d), generator=g, device=dev).bfloat16() for _ in range(4))
    y, h, grads = layer.train(x, r, gy, gh)
    # the same in float64 on the CPU, differentiated by autograd at the Q, K, V that the layer's forward pass computed:
    # where a row of O nearly vanishes, GroupNorm's gradient turns with the smallest change of its scores, so that the
    # gradient at other, unquantised Q, K, V is another one (rows of spread 0.01 moved dwq by half of its norm)
    T64 = lambda t: t.detach().double().cpu()
    leaves = [T64(t).requires_grad_(True) for t in (x, w, *ws)]
    xl, wl, wq, wk, wv, wo = leaves
    hl = xl + T64(r)
    n = wl * hl / (hl.square().mean(-1, keepdim=True) + layer.eps).sqrt()
    import retnet_scale_retention_amd as msr
    _, _, n8, s8 = msr.msr_add_rmsnorm(x, w, r, eps=layer.eps, want_y=False, want_q=True)
    at = [T64(t).requires_grad_(True) for t in layer._project(n8, s8)]
    gamma, theta, scale, eps, pos = og._args(at[0].detach().numpy(), layer.gamma, None, None, 1e-5, 0, None)
    o, _ = og._forward(*at, None, gamma, theta, scale, eps, pos, True, True)
    yl = o.flatten(-2) @ wo.t()
    *d_qkv, d_wo = torch.autograd.grad((yl * T64(gy)).sum(), at + [wo])
    through = sum(((n @ m.t()) * g.flatten(-2)).sum() for m, g in zip((wq, wk, wv), d_qkv)) + (hl * T64(gh)).sum()
    ref = (*torch.autograd.grad(through, (xl, wl, wq, wk, wv)), d_wo)
    errs = [rel(down(y), yl.detach().numpy())] + [rel(down(a), b.numpy()) for a, b in zip(grads, ref)]
    note("y, dx, dw, dwq, dwk, dwv, dwo: " + " ".join(f"{e:.3f}" for e in errs))
    assert errs[0] < FORWARD and max(errs[1:]) < BACKWARD
    for a, b in zip(grads, ref):
        assert a.shape == b.shape
