"""GPU parity of the layer around retention (msr_add_rmsnorm and its gradients,
msr_quantize, msr_scaled_matmul) against the float64 definitions of
oracle/layer.py.

Tolerances, from the arithmetic (u = 2^-24 fp32, 2^-8 bf16 relative rounding):
  - a norm's value: its row's sum of squares runs over at most 40 fp32
    additions in a row (32 per lane, then trees), halved by the square root,
    plus a handful of products: 64 u32, and one bf16 rounding where stored so;
  - an 8-bit value: half the e4m3 step at it, plus the fp32 error of what is
    rounded; a scale: the fp32 error of the block's largest value;
  - dx: 64 u32 of the sum of its terms' magnitudes (+ bf16 rounding); dweight:
    as many u32 of the sum of magnitudes as the longest chain of additions;
  - a product with fp32 output: (16 K / 128 + 64) u32 of the sum of its
    products' magnitudes; with bf16 output the bf16 rounding, and 2^-10 of that
    sum for the bits the 8-bit instruction drops (2^-13 of the largest of each
    8 products, 8 times)."""
import numpy as np
import pytest

from oracle import layer as ol
from tests.gpu_util import down, note, torch_dev

pytestmark = pytest.mark.gpu
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS = 1e-6


def _msr():
    import retnet_scale_retention_amd as msr
    return msr


def values(torch, dev, shape, dtype, seed, spread=True):
    """Activations of unlike channels, on the device; and the same numbers in float64."""
    rng = np.random.default_rng([17, seed])
    x = rng.standard_normal(shape)
    if spread:
        x = x * np.exp(rng.standard_normal(shape[-1]))
    t = torch.from_numpy(x.astype(np.float32)).to(dev).to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
    return t, down(t)


def codes(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


def check_blocks(q, s, x, block_rows, err, name):
    """q, s (device) against x (float64, each value known within err): values, scales, padding."""
    R, C = x.shape
    want, sp = ol.block_scales(x, block_rows)
    got = down(s)
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= (err + 4 * U["f32"]) * want), name
    c = codes(q)
    assert c.shape == (R, ol.padded(C)) and not np.any(c[:, C:]), name
    d = ol.E4M3[c[:, :C]]
    v = x / sp
    room = ol.half_step(v) * (1 + 2.0 ** -10) + (err + 8 * U["f32"]) * np.abs(v)
    assert np.all(np.abs(d - v) <= room), name


SIZES = [(1, 1), (1, 64), (3, 128), (5, 136), (64, 200), (7, 511), (130, 512), (9, 1000), (33, 1024), (6, 2047),
         (17, 2048), (5, 4096), (3, 4100), (4, 8192), (2, 16384), (2, 20001), (1, 32768),
         # rows that end 2, 3, 5 or 6 past a group of eight, and rows that share a wave
         (9, 2), (10, 6), (11, 517), (300, 1002), (5, 2067), (4, 6006), (3, 16381), (1001, 128), (67, 256), (1003, 86),
         (21, 130)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", SIZES)
def test_add_rmsnorm(rows, d, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"norm {rows}x{d} {dtype}")
    x, xf = values(torch, dev, (rows, d), dtype, 1)
    r, rf = values(torch, dev, (rows, d), dtype, 2)
    w, wf = values(torch, dev, (d,), "f32" if d % 3 else "bf16", 3, spread=False)
    n, h = ol.add_rmsnorm(xf, rf, wf, EPS)
    y, total, q, s = msr.msr_add_rmsnorm(x, w, r, eps=EPS, want_q=True)
    err = 64 * U["f32"]
    stored = U["bf16"] if dtype == "bf16" else U["f32"]
    assert np.all(np.abs(down(total) - h) <= (stored + U["f32"]) * np.abs(h))
    assert np.all(np.abs(down(y) - n) <= (err + stored) * np.abs(n))
    check_blocks(q, s, n, 1, err, "q")
    # the outputs do not depend on which of them are asked for
    y2, t2, q2, s2 = msr.msr_add_rmsnorm(x, w, r, eps=EPS)
    assert q2 is None and s2 is None and torch.equal(y2, y) and torch.equal(t2, total)
    y3, _, q3, s3 = msr.msr_add_rmsnorm(x, w, r, eps=EPS, want_y=False, want_q=True)
    assert y3 is None and np.array_equal(codes(q3), codes(q)) and torch.equal(s3, s)
    # without a residual and without a weight
    y4, t4, _, _ = msr.msr_add_rmsnorm(x, eps=EPS)
    n4, _ = ol.add_rmsnorm(xf, None, None, EPS)
    assert t4 is None and np.all(np.abs(down(y4) - n4) <= (err + stored) * np.abs(n4))


def test_add_rmsnorm_in_place_and_leading_dimensions():
    torch, dev = torch_dev()
    msr = _msr()
    x, _ = values(torch, dev, (3, 5, 640), "bf16", 4)
    r, _ = values(torch, dev, (3, 5, 640), "bf16", 5)
    y, total, q, s = msr.msr_add_rmsnorm(x, None, r, want_q=True)
    assert q.shape == (3, 5, 640) and s.shape == (3, 5, 5)
    x2, r2 = x.clone(), r.clone()
    y2, t2, _, _ = msr.msr_add_rmsnorm(x2, None, r2, out=(x2, r2, None, None))
    assert y2 is x2 and t2 is r2 and torch.equal(x2, y) and torch.equal(r2, total)
    x3 = x.clone()
    msr.msr_add_rmsnorm(x3, None, r, want_y=False, want_q=True, out=(None, x3, None, None))
    assert torch.equal(x3, total)


@pytest.mark.parametrize("d", [96, 512, 4096])
def test_add_rmsnorm_zero_tiny_and_non_finite_rows(d):
    torch, dev = torch_dev()
    msr = _msr()
    x, _ = values(torch, dev, (6, d), "f32", 6)
    x[1] = 0.0                      # n = 0: scale at its floor, values 0
    x[2] *= 1e-30                   # squares vanish: eps rules
    x[3, 7] = float("nan")
    x[4, 70] = float("inf")
    x[5] *= 1e25                    # squares overflow: n = 0
    y, _, q, s = msr.msr_add_rmsnorm(x, eps=EPS, want_q=True)
    n, _ = ol.add_rmsnorm(down(x), None, None, EPS)
    y, s, v = down(y), down(s), ol.E4M3[codes(q)[:, :d]]
    for i in (0, 2):
        assert np.all(np.abs(y[i] - n[i]) <= 64 * U["f32"] * np.abs(n[i]))
    assert not y[1].any() and not v[1].any() and np.all(s[1] == ol.TINY)
    assert np.all(np.isnan(y[3])) and np.all(np.isnan(s[3]))
    stands = v * ol.spread(s, 6, 1)[:, :d]
    assert np.all(np.isnan(stands[3]))
    # x / inf is 0, inf / inf is NaN; the 8-bit block that holds it stands for NaN as a whole
    assert np.isnan(y[4, 70]) and not np.delete(y[4], 70).any()
    assert np.all(np.isnan(stands[4, :min(d, 128)])) and not stands[4, 128:].any()
    assert not y[5].any() and not v[5].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", SIZES + [(2500, 64), (1200, 520), (700, 4096), (64, 100), (65, 128), (33, 129),
                                            (32, 256), (3001, 256), (5001, 86), (16, 300), (17, 512), (4, 4096),
                                            (8, 1024), (9, 1024)])
def test_add_rmsnorm_backward(rows, d, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"norm backward {rows}x{d} {dtype}")
    h, hf = values(torch, dev, (rows, d), dtype, 11)
    dy, dyf = values(torch, dev, (rows, d), dtype, 12, spread=False)
    ds, dsf = values(torch, dev, (rows, d), dtype, 13, spread=False)
    w, wf = values(torch, dev, (d,), "bf16" if d % 3 else "f32", 14, spread=False)
    chain = (rows + 63) // 64 + 64 + 64  # a team's rows, the teams' slices, the slices
    for weight, grad_sum in ((w, ds), (None, None)):
        dx, dw = msr.msr_add_rmsnorm_backward(h, weight, dy, grad_sum=grad_sum, eps=EPS)
        rdx, rdw, mx, mw = ol.add_rmsnorm_backward(hf, None if weight is None else wf, dyf,
                                                   None if grad_sum is None else dsf, EPS)
        stored = U["bf16"] if dtype == "bf16" else U["f32"]
        assert np.all(np.abs(down(dx) - rdx) <= 64 * U["f32"] * mx + stored * np.abs(rdx))
        assert np.all(np.abs(down(dw) - rdw) <= (chain + 64) * U["f32"] * mw)
        again = msr.msr_add_rmsnorm_backward(h, weight, dy, grad_sum=grad_sum, eps=EPS)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
        only, none = msr.msr_add_rmsnorm_backward(h, weight, dy, grad_sum=grad_sum, eps=EPS, want_weight_grad=False)
        assert none is None and torch.equal(only, dx)
    inplace = ds.clone()
    dx, _ = msr.msr_add_rmsnorm_backward(h, w, dy, grad_sum=ds, eps=EPS)
    msr.msr_add_rmsnorm_backward(h, w, dy, grad_sum=inplace, eps=EPS, out=(inplace, None))
    assert torch.equal(inplace, dx)


def test_add_rmsnorm_gradient_against_differences():
    # dL/dx of L = <dy, n> + <ds, h> along a direction v: the symmetric difference of the float64 definition with step
    # t is off by t^2/6 of the third derivative; t = 1e-4 leaves about 1e-8, far below fp32's own error
    torch, dev = torch_dev()
    msr = _msr()
    h, hf = values(torch, dev, (4, 200), "f32", 21, spread=False)
    dy, dyf = values(torch, dev, (4, 200), "f32", 22, spread=False)
    ds, dsf = values(torch, dev, (4, 200), "f32", 23, spread=False)
    w, wf = values(torch, dev, (200,), "f32", 24, spread=False)
    dx, dw = msr.msr_add_rmsnorm_backward(h, w, dy, grad_sum=ds, eps=EPS)
    rng = np.random.default_rng(25)
    loss = lambda x, ww: float((dyf * ol.add_rmsnorm(x, None, ww, EPS)[0]).sum() + (dsf * x).sum())
    t = 1e-4
    for _ in range(4):
        v, vw = rng.standard_normal(hf.shape), rng.standard_normal(200)
        num = (loss(hf + t * v, wf) - loss(hf - t * v, wf)) / (2 * t)
        mag = np.abs(down(dx) * v).sum()
        assert abs((down(dx) * v).sum() - num) <= 1e-5 * mag
        num = (loss(hf, wf + t * vw) - loss(hf, wf - t * vw)) / (2 * t)
        assert abs((down(dw) * vw).sum() - num) <= 1e-5 * np.abs(down(dw) * vw).sum()


def test_add_rmsnorm_backward_without_rows_gives_a_zero_weight_gradient():
    torch, dev = torch_dev()
    msr = _msr()
    e = torch.empty(0, 96, device=dev)
    dx, dw = msr.msr_add_rmsnorm_backward(e, None, e, out=(None, torch.full((96,), 7.0, device=dev)))
    assert dx.shape == (0, 96) and not dw.any()
    y, _, q, s = msr.msr_add_rmsnorm(e, want_q=True)
    assert y.shape == (0, 96) and q.shape == (0, 128) and s.shape == (0, 1)


QSIZES = [(1, 1), (1, 128), (128, 1), (5, 77), (127, 129), (128, 128), (130, 264), (300, 1000), (257, 512), (64, 4096),
          (129, 258), (40, 1003), (131, 518), (7, 2047)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", QSIZES)
def test_quantize(rows, cols, block_rows, dtype):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"quantize {rows}x{cols} {block_rows} {dtype}")
    x, xf = values(torch, dev, (rows, cols), dtype, 31)
    q, s, qt, st = msr.msr_quantize(x, block_rows=block_rows, want_transposed=True)
    check_blocks(q, s, xf, block_rows, 0.0, "rows")
    check_blocks(qt, st, np.ascontiguousarray(xf.T), block_rows, 0.0, "transposed")
    if block_rows == 128:
        assert torch.equal(s.t(), st) and np.array_equal(codes(q)[:, :cols], codes(qt)[:, :rows].T)
    q1, s1, n1, n2 = msr.msr_quantize(x, block_rows=block_rows)
    assert n1 is None and n2 is None and np.array_equal(codes(q1), codes(q)) and torch.equal(s1, s)
    n1, n2, qt1, st1 = msr.msr_quantize(x, block_rows=block_rows, want_rows=False, want_transposed=True)
    assert n1 is None and n2 is None and np.array_equal(codes(qt1), codes(qt)) and torch.equal(st1, st)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_zero_tiny_and_non_finite_blocks(block_rows):
    torch, dev = torch_dev()
    msr = _msr()
    x, _ = values(torch, dev, (384, 384), "f32", 32)
    x[:128, :128] = 0.0
    x[:128, 128:256] *= 1e-38       # below 448 x 2^-126: the scale's floor
    x[200, 10] = float("nan")
    x[300, 300] = float("-inf")
    x[130, 256:384] = 3e38          # the largest numbers
    xf = down(x)
    q, s, qt, st = msr.msr_quantize(x, block_rows=block_rows, want_transposed=True)
    for a, sc, ref in ((q, s, xf), (qt, st, xf.T)):
        got = ol.E4M3[codes(a)] * ol.spread(down(sc), 384, block_rows)
        good = np.isfinite(ol.block_scales(ref, block_rows)[1])
        assert np.all(np.isnan(got[~good])) and np.all(np.isfinite(got[good]))
        sp = ol.block_scales(np.where(np.isfinite(ref), ref, 0.0), block_rows)[1]
        v = ref / sp
        room = (ol.half_step(np.where(good, v, 0)) * (1 + 2.0 ** -10) + 16 * U["f32"] * np.abs(v)) * sp
        assert np.all(np.abs(got - ref)[good] <= room[good])


def test_quantize_beyond_two_to_the_32():
    # 8-bit and scale offsets past 32 bits: the last rows of a matrix of 2^32 + elements
    torch, dev = torch_dev()
    msr = _msr()
    rows, cols = (1 << 21) + 5, 2176
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=dev)
    tail, tf = values(torch, dev, (7, cols), "bf16", 33)
    x[-7:] = tail
    q, s, _, _ = msr.msr_quantize(x)
    check_blocks(q[-7:], s[-7:], tf, 1, 0.0, "tail")
    assert float(s[:-7].max()) == ol.TINY
    y, _, q2, s2 = msr.msr_add_rmsnorm(x, eps=EPS, want_y=False, want_q=True, out=(None, None, q, s))
    check_blocks(q2[-7:], s2[-7:], ol.add_rmsnorm(tf, None, None, EPS)[0], 1, 64 * U["f32"], "norm tail")


def test_add_rmsnorm_more_rows_than_one_launch_takes():
    torch, dev = torch_dev()
    msr = _msr()
    rows = (1 << 25) + 11  # launches of 2^21 workgroups of sixteen rows
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device=dev)
    tail, tf = values(torch, dev, (29, 8), "bf16", 34)
    x[-29:] = tail
    y, _, q, s = msr.msr_add_rmsnorm(x, eps=EPS, want_q=True)
    n = ol.add_rmsnorm(tf, None, None, EPS)[0]
    assert np.all(np.abs(down(y[-29:]) - n) <= (64 * U["f32"] + U["bf16"]) * np.abs(n)) and not y[:-29].any()
    check_blocks(q[-29:], s[-29:], n, 1, 64 * U["f32"], "tail")


# m, n, k (padded): single tokens, ragged edges of every tile, one block and many
MSIZES = [(1, 1, 128), (1, 64, 256), (2, 200, 1024), (5, 4096, 512), (16, 48, 384), (17, 130, 128), (33, 1000, 2048),
          (64, 256, 4096), (65, 257, 640), (100, 96, 16384), (127, 129, 256), (128, 512, 1152), (200, 72, 8192),
          (255, 1028, 256), (257, 515, 384), (300, 2048, 512), (513, 260, 1024)]


def operands(torch, dev, msr, m, n, k, block, seed):
    a, _ = values(torch, dev, (m, k), "bf16", seed)
    b, _ = values(torch, dev, (n, k), "bf16", seed + 1, spread=False)
    qa, sa, _, _ = msr.msr_quantize(a)
    qb, sb, _, _ = msr.msr_quantize(b, block_rows=block)
    return qa, sa, qb, sb


def check_product(out, qa, sa, qb, sb, block, name):
    import torch
    k = qa.shape[-1]
    r, mag = ol.matmul(codes(qa), down(sa), codes(qb), down(sb), block)
    d = np.abs(down(out) - r)
    if out.dtype == torch.float32:
        assert np.all(d <= (16 * k // 128 + 64) * U["f32"] * mag), name
    else:
        assert np.all(d <= U["bf16"] * np.abs(r) + 2.0 ** -10 * mag), name
        # over many values the roundings' mean square is a third of their largest square, the dropped bits' far less
        if r.size > 4000:
            assert np.linalg.norm(d) <= (U["bf16"] / np.sqrt(3) + 2.0 ** -12) * np.linalg.norm(r), name


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("m,n,k", MSIZES)
def test_scaled_matmul(m, n, k, block, out):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"matmul {m}x{n}x{k} block {block} {out}")
    ops = operands(torch, dev, msr, m, n, k, block, 41)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    c = msr.msr_scaled_matmul(*ops, out_dtype=dt)
    assert c.shape == (m, n) and c.dtype == dt
    check_product(c, *ops, block, "product")
    assert torch.equal(msr.msr_scaled_matmul(*ops, out_dtype=dt), c)


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_scaled_matmul_positions(out):
    # small whole numbers with scales that are powers of two: every product and sum is exact, so any misplaced row,
    # block or scale shows
    torch, dev = torch_dev()
    msr = _msr()
    dt = torch.float32 if out == "f32" else torch.bfloat16
    for m, n, k in ((40, 100, 512), (300, 300, 1024), (520, 264, 256)):
        g = torch.Generator(device="cpu").manual_seed(m)
        a = torch.randint(-1, 2, (m, k), generator=g).to(dev).to(torch.float32)
        b = torch.randint(-1, 2, (n, k), generator=g).to(dev).to(torch.float32)
        qa, qb = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
        for block in (1, 128):
            sa = torch.exp2(torch.randint(-1, 2, (m, k // 128), generator=g).float()).to(dev)
            sb = torch.exp2(torch.randint(-1, 2, (n if block == 1 else -(-n // 128), k // 128), generator=g).float()).to(dev)
            c = msr.msr_scaled_matmul(qa, sa, qb, sb, out_dtype=dt)
            r, _ = ol.matmul(codes(qa), down(sa), codes(qb), down(sb), block)
            want = torch.from_numpy(r.astype(np.float32)).to(dt)
            assert torch.equal(c.cpu(), want), (m, n, k, block)


# the larger tiles: 32 x 64, 64 x 64, 128 x 64 (four stages, two stages), 128 x 128, 256 x 256, with ends inside a tile
LSIZES = [(700, 701, 2048), (704, 704, 2048), (90, 8190, 1152), (70, 8190, 2048), (70, 8192, 2048), (1000, 1100, 4096),
          (300, 6001, 512), (1025, 1990, 256), (1025, 1992, 256), (250, 8184, 4096), (2040, 1545, 640), (2040, 1544, 640),
          (4101, 4100, 512), (4101, 4104, 512), (2561, 2050, 1024), (3001, 4100, 256), (3000, 5003, 640),
          (4010, 8200, 640), (5000, 8200, 640), (3000, 8200, 1024), (3001, 8195, 2176), (8300, 8203, 1152)]


def product64(qa, sa, qb, sb, block):
    # the product and the sum of its terms' sizes in 64 bits on the card (these sizes are slow on the host)
    import torch
    a = qa.to(torch.float32).double() * sa.double().repeat_interleave(128, 1)
    rows = sb if block == 1 else sb.repeat_interleave(128, 0)[:qb.shape[0]]
    b = (qb.to(torch.float32).double() * rows.double().repeat_interleave(128, 1)).t().contiguous()
    return a @ b, a.abs() @ b.abs()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("m,n,k", LSIZES)
def test_scaled_matmul_large_tiles(m, n, k, block, out):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"matmul {m}x{n}x{k} block {block} {out}")
    ops = operands(torch, dev, msr, m, n, k, block, 53)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    c = msr.msr_scaled_matmul(*ops, out_dtype=dt)
    assert torch.equal(msr.msr_scaled_matmul(*ops, out_dtype=dt), c)
    r, mag = product64(*ops, block)
    d = (c.double() - r).abs()
    if out == "f32":
        assert bool((d <= (16 * k // 128 + 64) * U["f32"] * mag).all())
    else:
        assert bool((d <= U["bf16"] * r.abs() + 2.0 ** -10 * mag).all())
        assert float(d.norm()) <= (U["bf16"] / np.sqrt(3) + 2.0 ** -12) * float(r.norm())


@pytest.mark.parametrize("m,n,k", LSIZES)
def test_scaled_matmul_large_tiles_positions(m, n, k):
    # as above: sums of whole quarters that fp32 holds exactly, rounded once
    torch, dev = torch_dev()
    msr = _msr()
    note(f"matmul positions {m}x{n}x{k}")
    g = torch.Generator(device=dev).manual_seed(m)
    pick = lambda *s: torch.randint(-1, 2, s, generator=g, device=dev).float()
    qa, qb = pick(m, k).to(torch.float8_e4m3fn), pick(n, k).to(torch.float8_e4m3fn)
    for block in (1, 128):
        sa, sb = torch.exp2(pick(m, k // 128)), torch.exp2(pick(n if block == 1 else -(-n // 128), k // 128))
        r, _ = product64(qa, sa, qb, sb, block)
        for dt in (torch.float32, torch.bfloat16):
            assert torch.equal(msr.msr_scaled_matmul(qa, sa, qb, sb, out_dtype=dt), r.float().to(dt)), (block, dt)


@pytest.mark.parametrize("m,n,k", [(2040, 1545, 640), (2561, 2050, 1024), (5000, 8200, 512), (3001, 8195, 1152)])
def test_scaled_matmul_large_tiles_non_finite(m, n, k):
    torch, dev = torch_dev()
    msr = _msr()
    note(f"matmul non-finite {m}x{n}x{k}")
    qa, sa, qb, sb = operands(torch, dev, msr, m, n, k, 128, 55)
    clean = msr.msr_scaled_matmul(qa, sa, qb, sb)
    sa[m - 1, 1], sa[m - 2, 0] = float("nan"), float("inf")
    qb.view(torch.uint8)[n - 1, 5] = 0x7F
    c = msr.msr_scaled_matmul(qa, sa, qb, sb)
    assert torch.isnan(c[m - 1]).all() and torch.isnan(c[:, n - 1]).all() and not torch.isfinite(c[m - 2]).any()
    assert torch.equal(c[:m - 2, :n - 1], clean[:m - 2, :n - 1])


@pytest.mark.parametrize("m,n,k", [(3, 100, 384), (150, 300, 384)])
def test_scaled_matmul_non_finite_blocks_stay_in_their_row_and_column(m, n, k):
    torch, dev = torch_dev()
    msr = _msr()
    for out in (torch.bfloat16, torch.float32):
        qa, sa, qb, sb = operands(torch, dev, msr, m, n, k, 1, 43)
        clean = msr.msr_scaled_matmul(qa, sa, qb, sb, out_dtype=out)
        sa[1, 1] = float("nan")
        qb.view(torch.uint8)[7, 5] = 0x7F
        c = msr.msr_scaled_matmul(qa, sa, qb, sb, out_dtype=out)
        assert torch.isnan(c[1]).all() and torch.isnan(c[:, 7]).all()
        keep = torch.ones(m, n, dtype=torch.bool, device=dev)
        keep[1], keep[:, 7] = False, False
        assert torch.equal(c[keep], clean[keep])


def test_scaled_matmul_empty_and_leading_dimensions():
    torch, dev = torch_dev()
    msr = _msr()
    f8 = torch.float8_e4m3fn
    z = lambda *s, **kw: torch.zeros(*s, device=dev, **kw)
    assert msr.msr_scaled_matmul(z(0, 128, dtype=f8), z(0, 1), z(9, 128, dtype=f8), z(9, 1)).shape == (0, 9)
    out = torch.full((3, 9), 5.0, device=dev)
    msr.msr_scaled_matmul(z(3, 0, dtype=f8), z(3, 0), z(9, 0, dtype=f8), z(9, 0), out=out)
    assert not out.any()
    qa, sa, qb, sb = operands(torch, dev, msr, 6, 40, 256, 128, 45)
    c = msr.msr_scaled_matmul(qa.view(2, 3, 256), sa.view(2, 3, 2), qb, sb)
    assert c.shape == (2, 3, 40) and torch.equal(c.view(6, 40), msr.msr_scaled_matmul(qa, sa, qb, sb))


def test_another_stream_than_the_current_one():
    torch, dev = torch_dev()
    msr = _msr()
    x, _ = values(torch, dev, (64, 512), "bf16", 47)
    w, _ = values(torch, dev, (256, 512), "bf16", 48)
    qb, sb, _, _ = msr.msr_quantize(w, block_rows=128)
    _, _, q, s = msr.msr_add_rmsnorm(x, want_y=False, want_q=True)
    want = msr.msr_scaled_matmul(q, s, qb, sb)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    q2, s2, o2 = torch.empty_like(q), torch.empty_like(s), torch.empty_like(want)
    msr.msr_add_rmsnorm(x, want_y=False, want_q=True, out=(None, None, q2, s2), stream=st)
    msr.msr_scaled_matmul(q2, s2, qb, sb, out=o2, stream=st)
    st.synchronize()
    assert torch.equal(o2, want)


def test_graph_replays_match_the_eager_calls():
    torch, dev = torch_dev()
    msr = _msr()
    w, _ = values(torch, dev, (1024, 2048), "bf16", 50)
    qb, sb, _, _ = msr.msr_quantize(w, block_rows=128)
    x = torch.zeros(8, 2048, dtype=torch.bfloat16, device=dev)
    y = torch.empty(8, 1024, dtype=torch.bfloat16, device=dev)
    q, s = torch.empty(8, 2048, dtype=torch.float8_e4m3fn, device=dev), torch.empty(8, 16, device=dev)

    def step():
        msr.msr_add_rmsnorm(x, want_y=False, want_q=True, out=(None, None, q, s))
        msr.msr_scaled_matmul(q, s, qb, sb, out=y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(values(torch, dev, (8, 2048), "bf16", 51 + i)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, y)
