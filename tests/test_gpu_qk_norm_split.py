"""Gradients of the head norms around where the workgroups along the tokens
change (8192 bytes of Q and K in a token), over more tokens than workgroups
take at once, with a workspace of exactly the bytes that are asked for.

Tolerances as in test_gpu_qk_norm.py."""
import pytest

from oracle import step_ops as so
from tests.gpu_util import torch_dev
from tests.test_gpu_qk_norm import EPS, U, heads, near, positions

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,Hk,dk", [(2100, 8, 8, 128), (3001, 16, 16, 128), (2500, 17, 16, 128), (2100, 9, 8, 128), (3001, 4, 4, 34)])
def test_gradients_around_the_split(T, H, Hk, dk, dtype):
    torch, dev = torch_dev()
    import retnet_scale_retention_amd as msr
    from retnet_scale_retention_amd import msr as m
    (q, qf), (k, kf), (dq, dqf), (dk_, dkf) = (heads(torch, dev, 1, T, h, dk, dtype, 80 + i) for i, h in enumerate((H, Hk, H, Hk)))
    need, room = m.load().msr_qk_norm_rotate_backward_workspace(T, H, Hk, dk), 4096
    flat = torch.full((need + 2 * room,), 0x5a, dtype=torch.uint8, device=dev)
    got = msr.msr_qk_norm_rotate_backward(q, k, None, None, dq, dk_, eps=EPS, pos0=11, workspace=flat[room:room + need])
    assert bool((flat[:room] == 0x5a).all()) and bool((flat[room + need:] == 0x5a).all())
    th, chain = so.default_theta(dk), max(H, Hk) * (T / 2048 + 1) + 64
    for i, (x, dy, s) in enumerate(((qf, dqf, 1.0), (kf, dkf, dk ** -0.5))):
        dx, dw, mx, mw = so.qk_norm_backward(x, None, dy, positions(1, T, 11), th, EPS, s)
        near(got[i], dx, 128 * U * mx, dtype, "dx")
        near(got[2 + i], dw, (chain + 128) * U * mw, "f32", "dw")
    again = msr.msr_qk_norm_rotate_backward(q, k, None, None, dq, dk_, eps=EPS, pos0=11)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
