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
    want = product64(qa, sa, qb, sb, block)[0].float().to(dt)
    assert torch.equal(msr.msr_scaled_matmul(qa, sa, qb, sb, out_dtype=dt), want)
    # a NaN in the last block stays in its row and its column
    qa.view(torch.uint8)[m - 1, k - 1], sb[0, k // 128 - 1] = 0x7F, float("nan")
    c2 = msr.msr_scaled_matmul(qa, sa, qb, sb, out_dtype=dt)
    columns = 1 if block == 1 else min(n, 128)
    assert torch.isnan(c2[m - 1]).all() and torch.isnan(c2[:, :columns]).all()
    assert torch.isfinite(c2[:m - 1, columns:]).all()


# an odd count of blocks shared by two groups of waves (64 x 64 and 32 x 64 tiles), in rings of three and four stages;
# the large kernel at the fewest blocks it takes; one token more, or one feature more, than the few-token kernel takes
TILES = [(903, 655, 9344), (560, 1384, 11904), (20, 10756, 3968), (486, 2790, 2944), (3291, 272, 4096), (199, 12850, 4480),
         (5000, 8200, 512), (9, 4096, 4096), (8, 4097, 4096), (1, 5248, 768), (64, 64, 16384)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("m,n,k", TILES)
def test_product_tiles_and_uneven_groups(m, n, k, block, out):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"product {m}x{n}x{k} block {block} {out}")
    dt = torch.float32 if out == "f32" else torch.bfloat16
    ops = operands(torch, dev, msr, m, n, k, block, 67)
    d = msr.msr_scaled_matmul(*ops, out_dtype=dt).double()
    r, mag = product64(*ops, block)
    d = (d - r).abs()
    if out == "f32":
        assert bool((d <= (16 * k // 128 + 64) * U["f32"] * mag).all())
    else:
        assert bool((d <= U["bf16"] * r.abs() + 2.0 ** -10 * mag).all())
        if r.numel() > 4000:
            assert float(d.norm()) <= (U["bf16"] / np.sqrt(3) + 2.0 ** -12) * float(r.norm())
    g = torch.Generator(device=dev).manual_seed(k)
    pick = lambda *s: torch.randint(-1, 2, s, generator=g, device=dev).float()
    qa, qb = pick(m, k).to(torch.float8_e4m3fn), pick(n, k).to(torch.float8_e4m3fn)
    sa, sb = torch.exp2(pick(m, k // 128)), torch.exp2(pick(n if block == 1 else -(-n // 128), k // 128))
    want = product64(qa, sa, qb, sb, block)[0].float().to(dt)
    assert torch.equal(msr.msr_scaled_matmul(qa, sa, qb, sb, out_dtype=dt), want)


# rows too long for registers (beyond 16384, or 8192 where the width is no multiple of 8) over several turns of every
# workgroup, the last of them uneven; and two turns of a single workgroup
LONG = [(600, 16392), (1030, 20001), (520, 9001), (1024, 32768), (2, 16381), (5, 17000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", LONG)
def test_gradients_of_long_rows_over_several_turns(rows, d, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"long rows {rows}x{d} {dtype}")
    g = torch.Generator(device=dev).manual_seed(d)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    gain = torch.exp(torch.randn(d, generator=g, device=dev))
    h = (torch.randn(rows, d, generator=g, device=dev) * gain).to(t)
    dy, ds = (torch.randn(rows, d, generator=g, device=dev).to(t) for _ in range(2))
    w = torch.randn(d, generator=g, device=dev)
    dx, dw = msr.msr_add_rmsnorm_backward(h, w, dy, grad_sum=ds, eps=EPS)
    # oracle/layer.py's formulas in 64 bits on the card (these sizes are slow on the host)
    h6, dy6, ds6 = h.double(), dy.double(), ds.double()
    g6, rstd = dy6 * w.double(), 1 / ((h6 * h6).mean(1, keepdim=True) + EPS).sqrt()
    mean = (g6 * h6).mean(1, keepdim=True)
    want = rstd * g6 - h6 * rstd ** 3 * mean + ds6
    mag = rstd * g6.abs() + h6.abs() * rstd ** 3 * (g6 * h6).abs().mean(1, keepdim=True) + ds6.abs()
    assert bool(((dx.double() - want).abs() <= 64 * U["f32"] * mag + U[dtype] * want.abs()).all())
    t6 = dy6 * h6 * rstd
    chain = (rows + 63) // 64 + 64 + 64
    assert bool(((dw.double() - t6.sum(0)).abs() <= (chain + 64) * U["f32"] * t6.abs().sum(0)).all())
    # the same into dy's and into dsum's place
    for i in (0, 1):
        a = [dy.clone(), ds.clone()]
        x2, w2 = msr.msr_add_rmsnorm_backward(h, w, a[0], grad_sum=a[1], eps=EPS, out=(a[i], None))
        assert x2 is a[i] and torch.equal(x2, dx) and torch.equal(w2, dw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(7, 5), (300, 86), (67, 256), (130, 517), (40, 1024), (33, 2047), (600, 4096),
                                    (9, 6006)])
def test_gradients_in_the_place_of_dy(rows, d, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"in place {rows}x{d} {dtype}")
    h, _ = values(torch, dev, (rows, d), dtype, 68)
    dy, _ = values(torch, dev, (rows, d), dtype, 69, spread=False)
    w, _ = values(torch, dev, (d,), "f32", 70, spread=False)
    for ds in (None, values(torch, dev, (rows, d), dtype, 71, spread=False)[0]):
        dx, dw = msr.msr_add_rmsnorm_backward(h, w, dy, grad_sum=ds, eps=EPS)
        a = dy.clone()
        x2, w2 = msr.msr_add_rmsnorm_backward(h, w, a, grad_sum=ds, eps=EPS, out=(a, None))
        assert x2 is a and torch.equal(a, dx) and torch.equal(w2, dw)


@pytest.mark.parametrize("rows,d", [(8, 96), (40, 512), (300, 1000), (9, 4096), (8, 9001), (300, 20000)])
def test_gradients_of_zero_and_non_finite_rows(rows, d):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"non-finite gradients {rows}x{d}")
    h, _ = values(torch, dev, (rows, d), "f32", 72, spread=False)
    dy, _ = values(torch, dev, (rows, d), "f32", 73, spread=False)
    w, wf = values(torch, dev, (d,), "f32", 74, spread=False)
    h[1] = 0.0                          # rstd = eps^-1/2, dx = rstd w dy
    h[2] *= 1e-30                       # squares vanish: the same
    clean = [i for i in range(rows) if i not in (3, 4, 5)]
    dx, dw = msr.msr_add_rmsnorm_backward(h[clean], w, dy[clean], eps=EPS)
    rdx, rdw, mx, mw = ol.add_rmsnorm_backward(down(h)[clean], wf, down(dy)[clean], None, EPS)
    assert np.all(np.abs(down(dx) - rdx) <= 64 * U["f32"] * mx + U["f32"] * np.abs(rdx))
    assert np.all(np.abs(down(dw) - rdw) <= (rows + 192) * U["f32"] * mw)
    h[3, 7] = float("nan")
    dy[4, 70] = float("nan")
    h[5, 50] = float("inf")
    d2, w2 = msr.msr_add_rmsnorm_backward(h, w, dy, eps=EPS)
    # a row's NaN reaches all of that row and no other; an infinity leaves n = 0 beside it, so 0, and is NaN itself
    assert torch.isnan(d2[3]).all() and torch.isnan(d2[4]).all() and torch.isnan(d2[5, 50])
    beside = torch.arange(d, device=dev) != 50
    assert not d2[5, beside].any()
    assert np.all(np.abs(down(d2)[clean] - rdx) <= 64 * U["f32"] * mx + U["f32"] * np.abs(rdx))
    # the weight's gradient: every column has a NaN from row 3
    assert torch.isnan(w2).all()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_padding_of_finite_and_non_finite_blocks(block_rows):
    # a block with a NaN or an infinity stands for NaN, its padding too; every other block's padding is zero
    torch, dev = torch_dev()
    msr = _msr()
    x, _ = values(torch, dev, (150, 200), "f32", 75)
    x[5, 190], x[140, 3] = float("nan"), float("inf")
    q, s, qt, st = msr.msr_quantize(x, block_rows=block_rows, want_transposed=True)
    for a, sc, rows, cols in ((q, s, 150, 200), (qt, st, 200, 150)):
        stands = ol.E4M3[a.view(torch.uint8).cpu().numpy()] * ol.spread(down(sc), rows, block_rows)
        bad = np.isnan(ol.spread(down(sc), rows, block_rows))
        assert bad.any() and np.all(np.isnan(stands[bad])) and np.all(np.isfinite(stands[~bad]))
        assert not np.any(np.nan_to_num(stands[:, cols:], nan=0.0)[~bad[:, cols:]])
    # and the product over that padding is NaN in those rows alone
    b, _, _, _ = msr.msr_quantize(values(torch, dev, (40, 200), "f32", 76)[0])
    if block_rows == 1:
        c = msr.msr_scaled_matmul(q, s, b, torch.ones(40, 2, device=dev), out_dtype=torch.float32)
        keep = [i for i in range(150) if i not in (5, 140)]
        assert torch.isnan(c[[5, 140]]).all() and torch.isfinite(c[keep]).all()
