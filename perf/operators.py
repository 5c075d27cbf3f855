"""The measured cases of the layer operators around retention: the residual's addition with a root-mean-square norm (its
output in 8 bits with scales, or not) and its gradients, the 8-bit quantiser, and the matrix product of 8-bit operands
with a scale for each block of 128.

A "8-bit" value is e4m3 (torch.float8_e4m3fn, largest value 448); a block's scale is max(largest magnitude / 448, 2^-126).
Rows of 8-bit arrays are padded with zeros to a multiple of 128 columns."""
import math

import torch

own = False

EPS = 1e-6
TINY = 2.0 ** -126
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
F8 = torch.float8_e4m3fn
ROUND = (64, 128, 192, 256, 320, 512, 640, 768, 1024, 1280, 1536, 2048, 2560, 4096, 5120, 6144, 8192, 10240, 12288, 16384)


def up128(n):
    return -(-n // 128) * 128


def listed():
    return [
        # A decode step's pre-norm: 64 sequences of the 4096-wide layer; the 8-bit output feeds the projections.
        dict(name="norm decode 64x4096", op="norm", rows=64, d=4096, dtype="bf16", residual=True, out="q"),
        # The pre-norm of a whole prompt of the 7B-shaped layer (B=2, T=8192, d_model=4096), serving.
        dict(name="norm prompt 16384x4096", op="norm", rows=16384, d=4096, dtype="bf16", residual=True, out="q"),
        # The small layer (B=4, T=2048, d_model=512) in training: the norm in 16 bits and in 8.
        dict(name="norm small 8192x512", op="norm", rows=8192, d=512, dtype="bf16", residual=True, out="both"),
        # The gradient of the 7B-shaped layer's pre-norm, the residual stream's gradient joined in.
        dict(name="norm grad 16384x4096", op="norm_backward", rows=16384, d=4096, dtype="bf16", dsum=True),
        # The gradient of a norm in fp32 over a ragged batch of tokens and a width that is no multiple of 128.
        dict(name="norm grad f32 3001x1000", op="norm_backward", rows=3001, d=1000, dtype="f32", dsum=False),
        # The output gradient of a projection in training: by rows for dX, transposed for dW.
        dict(name="quantize grad 16384x4096", op="quantize", rows=16384, cols=4096, dtype="bf16", block_rows=1, orders="both"),
        # A V-projection weight after an optimiser step: 128 x 128 blocks, both orders.
        dict(name="quantize weight 8192x4096", op="quantize", rows=8192, cols=4096, dtype="bf16", block_rows=128, orders="both"),
        # One token through the Q projection.
        dict(name="matmul token 1x4096x4096", op="matmul", m=1, n=4096, k=4096, b_block=128, out="bf16"),
        # A decode step of 64 sequences through the V projection.
        dict(name="matmul decode 64x8192x4096", op="matmul", m=64, n=8192, k=4096, b_block=128, out="bf16"),
        # The small layer's projection over a ragged batch of prompts.
        dict(name="matmul ragged 2000x1544x512", op="matmul", m=2000, n=1544, k=512, b_block=128, out="bf16"),
        # The V projection of the 7B-shaped layer over a whole prompt.
        dict(name="matmul prompt 16384x8192x4096", op="matmul", m=16384, n=8192, k=4096, b_block=128, out="bf16"),
        # The Q weight's gradient: the contraction runs over the tokens, both operands scaled by rows.
        dict(name="matmul dW 4096x4096x16384", op="matmul", m=4096, n=4096, k=16384, b_block=1, out="f32"),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "quantize", "matmul", "matmul"])

    def width(lo, hi):  # widths are round more often than not
        if rng.random() < 0.3:
            n = log_int(rng, lo, hi - 2)
            return n + 1 if n % 64 == 0 else n
        return rng.choice([w for w in ROUND if lo <= w <= hi])

    if op == "matmul":
        while True:
            m, n, k = log_int(rng, 1, 16384), width(64, 16384), width(64, 16384)
            if 2.0 * m * n * k <= 2.0 * 16384 * 8192 * 4096:
                break
        return dict(op=op, m=m, n=n, k=k, b_block=rng.choice([128, 128, 1]), out=rng.choice(["bf16", "f32"]))
    while True:
        rows, d = log_int(rng, 1, 65536), width(64, 16384)
        if rows * d <= 16384 * 4096 // 2:
            break
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        return dict(op=op, rows=rows, d=d, dtype=dtype, residual=rng.random() < 0.75, out=rng.choice(["q", "y", "both"]))
    if op == "norm_backward":
        return dict(op=op, rows=rows, d=d, dtype=dtype, dsum=rng.random() < 0.75)
    return dict(op=op, rows=rows, cols=d, dtype=dtype, block_rows=rng.choice([1, 1, 128]), orders=rng.choice(["rows", "both", "transposed"]))


# ---- inputs -------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def channels(d):  # activations: channels of unlike size, a few of them large
        gain = torch.exp(0.5 * normal(d))
        return torch.where(normal(d) > 2.5, 10.0 * gain, gain)

    c = dict(case)
    if c["op"] in ("norm", "norm_backward"):
        R, d, t = c["rows"], c["d"], TYPES[c["dtype"]]
        gain = channels(d)
        st = {"w": (1.0 + 0.2 * normal(d)).to(t)}
        if c["op"] == "norm":
            st["x"] = (normal(R, d) * gain).to(t)
            st["r"] = (2.0 * normal(R, d) * gain).to(t) if c["residual"] else None
            both = c["out"] == "both"
            st["bufs"] = (torch.empty(R, d, dtype=t, device="cuda") if both or c["out"] == "y" else None,
                          torch.empty(R, d, dtype=t, device="cuda") if c["residual"] else None,
                          torch.empty(R, up128(d), dtype=F8, device="cuda") if both or c["out"] == "q" else None,
                          torch.empty(R, up128(d) // 128, device="cuda") if both or c["out"] == "q" else None)
        else:
            st["h"] = (2.0 * normal(R, d) * gain).to(t)
            st["dy"] = (1e-2 * normal(R, d)).to(t)
            st["dsum"] = (1e-2 * normal(R, d)).to(t) if c["dsum"] else None
            st["bufs"] = (torch.empty(R, d, dtype=t, device="cuda"), torch.empty(d, device="cuda"))
    elif c["op"] == "quantize":
        R, C = c["rows"], c["cols"]
        st = {"x": (normal(R, C) * channels(C) * 1e-2).to(TYPES[c["dtype"]])}
        sr = R if c["block_rows"] == 1 else up128(R) // 128
        sc = C if c["block_rows"] == 1 else up128(C) // 128
        rows, trans = c["orders"] != "transposed", c["orders"] != "rows"
        st["bufs"] = (torch.empty(R, up128(C), dtype=F8, device="cuda") if rows else None,
                      torch.empty(sr, up128(C) // 128, device="cuda") if rows else None,
                      torch.empty(C, up128(R), dtype=F8, device="cuda") if trans else None,
                      torch.empty(sc, up128(R) // 128, device="cuda") if trans else None)
    else:
        m, n, k = c["m"], c["n"], c["k"]
        st = {}
        st["a"], st["sa"] = blocks_plain(normal(m, k) * channels(k), 1)
        st["b"], st["sb"] = blocks_plain(normal(n, k) / math.sqrt(k), c["b_block"])
        st["bufs"] = torch.empty(m, n, dtype=TYPES[c["out"]], device="cuda")
    st["case"] = c
    return st


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(st):
    return run_own(st) if own else run_plain(st)


def run_own(st):
    import retnet_scale_retention_amd as msr
    c = st["case"]
    if c["op"] == "norm":
        return msr.msr_add_rmsnorm(st["x"], st["w"], st["r"], eps=EPS, want_y=c["out"] != "q", want_q=c["out"] != "y", out=st["bufs"])
    if c["op"] == "norm_backward":
        return msr.msr_add_rmsnorm_backward(st["h"], st["w"], st["dy"], grad_sum=st["dsum"], eps=EPS, out=st["bufs"])
    if c["op"] == "quantize":
        return msr.msr_quantize(st["x"], block_rows=c["block_rows"], want_rows=c["orders"] != "transposed", want_transposed=c["orders"] != "rows", out=st["bufs"])
    return msr.msr_scaled_matmul(st["a"], st["sa"], st["b"], st["sb"], out=st["bufs"])


def blocks_plain(x, block_rows):
    """x [R, C] in 32 bits as 8-bit values, padded to a multiple of 128 columns, and the scales of its blocks."""
    R, C = x.shape
    x = torch.nn.functional.pad(x, (0, up128(C) - C))
    if block_rows == 1:
        g = x.view(R, -1, 128)
        s = (g.abs().amax(2) / 448.0).clamp_min(TINY)
        return (g / s[:, :, None]).reshape(R, -1).to(F8), s
    g = torch.nn.functional.pad(x, (0, 0, 0, up128(R) - R)).view(up128(R) // 128, 128, -1, 128)
    s = (g.abs().amax((1, 3)) / 448.0).clamp_min(TINY)
    return (g / s[:, None, :, None]).reshape(up128(R), -1)[:R].to(F8), s


def run_plain(st):
    c = st["case"]
    if c["op"] == "norm":
        t = st["x"].dtype
        h = st["x"].float()
        if st["r"] is not None:
            h = h + st["r"].float()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * st["w"].float()
        q, s = blocks_plain(y, 1) if c["out"] != "y" else (None, None)
        return (y.to(t) if c["out"] != "q" else None, h.to(t) if st["r"] is not None else None, q, s)
    if c["op"] == "norm_backward":
        t = st["h"].dtype
        h, dy = st["h"].float(), st["dy"].float()
        rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        n = h * rstd
        g = dy * st["w"].float()
        dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
        if st["dsum"] is not None:
            dx = dx + st["dsum"].float()
        return dx.to(t), (dy * n).sum(0)
    if c["op"] == "quantize":
        x = st["x"].float()
        q, s = blocks_plain(x, c["block_rows"]) if c["orders"] != "transposed" else (None, None)
        qt, s_t = blocks_plain(x.t().contiguous(), c["block_rows"]) if c["orders"] != "rows" else (None, None)
        return q, s, qt, s_t
    n = st["b"].shape[0]
    sb = st["sb"] if c["b_block"] == 1 else st["sb"].repeat_interleave(128, 0)[:n]
    a = st["a"].float() * st["sa"].repeat_interleave(128, 1)
    b = st["b"].float() * sb.repeat_interleave(128, 1)
    return (a @ b.t()).to(TYPES[c["out"]])


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        scales = (m + (n if c["b_block"] == 1 else up128(n) // 128)) * up128(k) // 128
        return {"bytes": m * k + n * k + 4 * scales + m * n * BYTES[c["out"]], "flops": 2.0 * m * n * k}
    e = BYTES[c["dtype"]]
    if c["op"] == "quantize":
        R, C = c["rows"], c["cols"]
        b = R * C * e
        small = c["block_rows"]
        if c["orders"] != "transposed":
            b += R * up128(C) + 4 * -(-R // small) * up128(C) // 128
        if c["orders"] != "rows":
            b += C * up128(R) + 4 * -(-C // small) * up128(R) // 128
        return {"bytes": b, "flops": 3.0 * R * C}
    R, d = c["rows"], c["d"]
    if c["op"] == "norm":
        b = R * d * e + d * e
        b += 2 * R * d * e if c["residual"] else 0
        b += R * d * e if c["out"] != "q" else 0
        b += R * up128(d) + R * up128(d) // 128 * 4 if c["out"] != "y" else 0
        return {"bytes": b, "flops": 6.0 * R * d}
    return {"bytes": R * d * e * (4 if c["dsum"] else 3) + d * (e + 4), "flops": 12.0 * R * d}


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] == "matmul":
        k = st["a"].shape[1]
        kb = torch.arange(k, device="cuda") // 128
        rows = torch.arange(c["n"], device="cuda") // c["b_block"]
        a = st["a"].double() * st["sa"].double()[:, kb]
        b = st["b"].double() * st["sb"].double()[rows][:, kb]
        return torch.mm(a, b.t())
    if c["op"] == "quantize":
        x = st["x"].double()
        return (exact_blocks(x, c["block_rows"]) if c["orders"] != "transposed" else (None, None)) + \
            (exact_blocks(x.t(), c["block_rows"]) if c["orders"] != "rows" else (None, None))
    if c["op"] == "norm":
        h = st["x"].double() if st["r"] is None else st["x"].double() + st["r"].double()
        y = exact_norm(h, st["w"].double())
        q, s = exact_blocks(y, 1) if c["out"] != "y" else (None, None)
        return (y if c["out"] != "q" else None, h if st["r"] is not None else None, q, s)
    h, w = st["h"].double().requires_grad_(True), st["w"].double().requires_grad_(True)
    dx, dw = torch.autograd.grad(exact_norm(h, w), (h, w), st["dy"].double())
    return (dx if st["dsum"] is None else dx + st["dsum"].double()), dw


def exact_norm(h, w):
    return w * h / (h.square().sum(-1, keepdim=True) / h.shape[-1] + EPS).sqrt()


def exact_blocks(x, block_rows):
    """The nearest e4m3 values of x over its blocks' scales, ties to even: steps of 2^(e - 3) where 2^e <= |v| < 2^(e + 1), e >= -6."""
    R, C = x.shape
    full = torch.zeros(-(-R // block_rows) * block_rows, up128(C), dtype=torch.float64, device=x.device)
    full[:R, :C] = x
    tiles = full.unflatten(1, (-1, 128)).unflatten(0, (-1, block_rows))
    s = torch.clamp(tiles.abs().amax(dim=(1, 3)) / 448, min=TINY)
    v = (tiles / s[:, None, :, None]).flatten(0, 1).flatten(1, 2)[:R]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (v / step).round() * step, s
