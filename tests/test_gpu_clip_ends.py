"""Clipping at the ends of fp32's range: factors too small for fp32, and a norm
between its largest number and the border to infinity.

Tolerances: those of test_gpu_clip.py; values below 2^-126 count as zero."""
import numpy as np
import pytest

from oracle import step_ops as so
from tests.gpu_util import down, torch_dev
from tests.test_gpu_clip import ROOM

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", [1e2, 1.0, 1e-2, 1e-5, 1e-7, 1e-10, 1e-20, 1e-30])
def test_factors_too_small_for_fp32(limit):
    # gradients of 1e35, whose norm is 2.6e37: max_norm / norm goes down to 4e-68, and the results are of max_norm's size
    torch, dev = torch_dev()
    import retnet_scale_retention_amd as msr
    gen = torch.Generator(device=dev).manual_seed(71)
    grads = [1e35 * torch.randn(n, generator=gen, device=dev) for n in (3, 8, 30000, 8193)]
    grads = [g.bfloat16() if i % 2 else g for i, g in enumerate(grads)] + [grads[2].bfloat16()]
    want, n = so.clip([down(g) for g in grads], float(np.float32(limit)))
    norm = msr.msr_gradient_norm(grads)
    assert np.isfinite(float(norm))
    out, got = msr.msr_clip_gradients(grads, limit, out=[torch.empty_like(g) for g in grads])
    given, _ = msr.msr_clip_gradients(grads, limit, norm=norm, out=[torch.empty_like(g) for g in grads])
    for a, c, b, g in zip(out, given, want, grads):
        room = ROOM["bf16" if g.dtype == torch.bfloat16 else "f32"]
        assert np.all(np.abs(down(a) - b) <= room * np.abs(b) + 2.0 ** -126)
        assert np.all(np.abs(down(c) - b) <= (room + 2.0 ** -24 * (1 + 1e-6)) * np.abs(b) + 2.0 ** -126)


def test_a_norm_that_rounds_to_the_largest_number():
    # F + 6e30 and F + 3e30 (F = 2^128 - 2^104, half a step 1.0e31) are F in fp32: the norm is finite, and clips
    torch, dev = torch_dev()
    import retnet_scale_retention_amd as msr
    F = torch.finfo(torch.float32).max
    for small in (0.0, 4.5e34, 6.4e34):
        g = [torch.tensor([F, small], device=dev)]
        out, norm = msr.msr_clip_gradients(g, 1.0, out=[torch.empty_like(g[0])])
        assert float(norm) == F
        given, _ = msr.msr_clip_gradients(g, 1.0, norm=norm, out=[torch.empty_like(g[0])])
        want = down(g[0]) / F
        for t in (out[0], given[0]):
            assert np.all(np.abs(down(t) - want) <= 2.0 ** -22 * want), small
    g = [torch.tensor([F, 1.5e35], device=dev)]  # F + 3.3e31: infinite
    out, norm = msr.msr_clip_gradients(g, 1.0, out=[torch.empty_like(g[0])])
    assert float(norm) == float("inf") and torch.equal(out[0], g[0])
