"""Head norms and their gradients without an eps, for rows whose squares are
subnormal in fp32 (a mean square below 2^-126): the norm of a row does not
depend on its size.

Tolerances: those of test_gpu_qk_norm.py (64 u forward, 128 u backward), and
what subnormal squares lose: at most dk + 64 additions, each off by 2^-150, of
a sum dk ms, and a mean off by 2^-150, together (1 + 64 / dk + 1) 2^-150 / ms of
the mean square ms, which enters forward by half and backward in four places
by once at most."""
import numpy as np
import pytest

from oracle import step_ops as so
from tests.gpu_util import down, torch_dev
from tests.test_gpu_qk_norm import U, heads, near, positions, tensor

pytestmark = pytest.mark.gpu
SCALES = [1e-17, 1e-18, 1e-19, 6e-20, 5e-20, 3e-20, 1e-20, 3e-21]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [6, 40, 96, 256])
def test_rows_with_subnormal_squares(dk, dtype):
    torch, dev = torch_dev()
    import retnet_scale_retention_amd as msr
    T, H = len(SCALES), 3
    rng = np.random.default_rng([61, dk])
    # every value well away from 0, so that no square vanishes
    x, xf = tensor(torch, dev, rng.uniform(0.5, 1.5, (1, T, H, dk)) * rng.choice([-1, 1], (1, T, H, dk)) *
                   np.array(SCALES)[None, :, None, None], dtype)
    dy, dyf = heads(torch, dev, 1, T, H, dk, dtype, 62)
    w, wf = tensor(torch, dev, 1 + 0.2 * rng.standard_normal(dk), "f32")
    th = so.default_theta(dk)
    ms = (xf * xf).mean(-1, keepdims=True)
    lost = (2 + 64 / dk) * 2.0 ** -150 / ms
    y, _ = msr.msr_qk_norm_rotate(x, None, w, eps=0.0)
    want, size = so.qk_norm(xf, wf, positions(1, T), th, 0.0, 1.0)
    near(y, want, (64 * U + lost) * size, dtype, "y")
    dx, _, dw, _ = msr.msr_qk_norm_rotate_backward(x, None, w, None, dy, None, eps=0.0)
    rx, rw, mx, mw = so.qk_norm_backward(xf, wf, dyf, positions(1, T), th, 0.0, 1.0)
    near(dx, rx, (128 * U + 4 * lost) * mx, dtype, "dx")
    terms = np.abs(so._pairs(dyf)) * np.abs(xf) / np.sqrt(ms)
    near(dw, rw, 256 * U * mw + (4 * lost * terms).sum((0, 1, 2)), "f32", "dw")
