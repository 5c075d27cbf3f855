"""Edges of the layer around retention that the sizes of test_gpu_layer.py do not
reach, against the float64 definitions of oracle/layer.py; tolerances as there
unless stated."""
import numpy as np
import pytest

from oracle import layer as ol
from tests.gpu_util import down, note, torch_dev
from tests.test_gpu_layer import EPS, U, _msr, check_product, operands, product64, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,d", [(3001, 1000), (2048, 256)])
def test_weight_gradient_rounding(rows, d):
    """The size of dweight's rounding, not its bound.  One fp32 rounding is uniform over +-2^-24 of the binade, rms
    s = 2^-24 / sqrt(3) * 0.74 = 2.5e-8 of a value spread evenly over it in the logarithm.  Of N random terms a partial sum
    of k has k / N of the result's square, so in units of s^2 the variance is: a term's product 1 and its row's rstd 3
    (mean 4 / 4, root, reciprocal); a team's turns 3.5 (6 of them, 502 teams, 3001 rows; 1 for 2048 x 256), the teams of
    a workgroup 1 (3.3), four parts in a slice 2.3, 64 slices in pairs 6: 16.8 (16.6).  That is 4.1 s = 1.04e-7; a quarter
    more is allowed.  A chain over the slices has 32 in place of 6: 1.7e-7."""
    torch, dev = torch_dev()
    msr = _msr()
    h, hf = values(torch, dev, (rows, d), "f32", 61, spread=False)
    dy, dyf = values(torch, dev, (rows, d), "f32", 62, spread=False)
    _, dw = msr.msr_add_rmsnorm_backward(h, None, dy, eps=EPS)
    want = ol.add_rmsnorm_backward(hf, None, dyf, None, EPS)[1]
    err = np.linalg.norm(down(dw) - want) / np.linalg.norm(want)
    note(f"dweight {rows}x{d}: {err:.3g} of its norm")
    assert err <= 1.3e-7


@pytest.mark.parametrize("rows,d", [(6, 96), (40, 512), (9, 4096), (4, 9001), (5, 20000)])
def test_gradients_of_rows_whose_squares_overflow(rows, d):
    # the forward pass gives n = 0 for such a row, whatever h: its gradient is the residual stream's alone, and the other
    # rows' gradients are those without it
    torch, dev = torch_dev()
    msr = _msr()
    note(f"overflowing rows {rows}x{d}")
    h, _ = values(torch, dev, (rows, d), "f32", 63, spread=False)
    dy, _ = values(torch, dev, (rows, d), "f32", 64, spread=False)
    ds, _ = values(torch, dev, (rows, d), "f32", 65, spread=False)
    h[1] *= 1e25                      # its squares overflow
    h[2], dy[2] = 3e38, 4.0           # and so does the sum of h dy
    h[3] = 3e38
    h[3, ::2], dy[3] = -3e38, 4.0     # as a difference of infinities
    y, _, _, _ = msr.msr_add_rmsnorm(h, eps=EPS)
    assert not y[1:4].any()
    dx, dw = msr.msr_add_rmsnorm_backward(h, None, dy, grad_sum=ds, eps=EPS)
    assert torch.equal(dx[1:4], ds[1:4])
    keep = [0, *range(4, rows)]
    rdx, rdw, mx, mw = ol.add_rmsnorm_backward(down(h)[keep], None, down(dy)[keep], down(ds)[keep], EPS)
    assert np.all(np.abs(down(dx)[keep] - rdx) <= 64 * U["f32"] * mx + U["f32"] * np.abs(rdx))
    assert np.all(np.abs(down(dw) - rdw) <= (rows + 192) * U["f32"] * mw)


# few tokens: eight waves share the contraction's blocks, so these have 4, 3, 2 or 3, 5 or 6, 16 and 1 or 2 blocks per wave
FEW = [(1, 4096, 4096), (8, 1000, 3072), (3, 130, 2176), (7, 4095, 5248), (2, 17, 16384), (5, 33, 1152)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("m,n,k", FEW)
def test_few_tokens_over_many_blocks(m, n, k, block, out):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"few tokens {m}x{n}x{k} block {block} {out}")
    dt = torch.float32 if out == "f32" else torch.bfloat16
    ops = operands(torch, dev, msr, m, n, k, block, 66)
    c = msr.msr_scaled_matmul(*ops, out_dtype=dt)
    check_product(c, *ops, block, "product")
    # whole quarters that fp32 holds exactly, rounded once: any misplaced row, block or scale shows
    g = torch.Generator(device=dev).manual_seed(k)
    pick = lambda *s: torch.randint(-1, 2, s, generator=g, device=dev).float()
    qa, qb = pick(m, k).to(torch.float8_e4m3fn), pick(n, k).to(torch.float8_e4m3fn)
    sa, sb = torch.exp2(pick(m, k // 128)), torch.exp2(pick(n if block == 1 else -(-n // 128), k // 128))
    assert torch.equal(msr.msr_scaled_matmul(qa, sa, qb, sb, out_dtype=dt), product64(qa, sa, qb, sb, block)[0].float().to(dt))
    # a NaN in the last block stays in its row and its column
    qa.view(torch.uint8)[m - 1, k - 1], sb[0, k // 128 - 1] = 0x7F, float("nan")
    c2 = msr.msr_scaled_matmul(qa, sa, qb, sb, out_dtype=dt)
    columns = 1 if block == 1 else min(n, 128)
    assert torch.isnan(c2[m - 1]).all() and torch.isnan(c2[:, :columns]).all()
    assert torch.isfinite(c2[:m - 1, columns:]).all()
