"""The measured cases of the operators that a training or serving step runs next to retention: norms of queries and keys
for each head with the position rotation in the same pass, and its gradients; a recurrence whose decay depends on the data
and the channel (a prompt, a token, the gradients); the norm of all gradients together, and their clipping to it."""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
BLOCK = 64  # tokens from one kept state of the recurrence to the next
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
LARGEST = 131072 * 1024  # elements of the largest recurrence
GRADS = 4096 * 4096 * 6 + 4096  # parameters of the 7B-shaped layer: wq, wk, wv, wo and the norm


def listed():
    return [
        # A decode step of 64 sequences at their own positions, Q and K as the fused projection left them beside V.
        dict(name="qk decode 64x1x16x256", op="qk", B=64, T=1, H=16, Hk=16, dk=256, dtype="bf16", fused=True, weights=True, rows=True),
        # The whole prompt of the 7B-shaped layer (B=2, T=8192, H=16, d_k=256), right behind its projections.
        dict(name="qk prompt 2x8192x16x256", op="qk", B=2, T=8192, H=16, Hk=16, dk=256, dtype="bf16", fused=False, weights=True, rows=False),
        # A training step of the 7B-shaped layer.
        dict(name="qk grad 2x8192x16x256", op="qk_backward", B=2, T=8192, H=16, Hk=16, dk=256, dtype="bf16", fused=False, weights=True, rows=False),
        # Training in fp32 on ragged sizes, heads whose width is no power of two.
        dict(name="qk grad f32 3x777x5x80", op="qk_backward", B=3, T=777, H=5, Hk=5, dk=80, dtype="f32", fused=False, weights=True, rows=False),
        # One token of each of 64 sequences through a 4096-wide recurrence.
        dict(name="gate token 64x4096", op="step", B=64, D=4096, dtype="bf16", normalize=True),
        # A whole prompt, 4096 wide, that continues from a state.
        dict(name="gate prompt 2x8192x4096", op="gate", B=2, T=8192, D=4096, dtype="bf16", normalize=True, state=True, carry=False),
        # One long sequence (T=131072) with few channels: the scan has to be split over time.
        dict(name="gate long 1x131072x1024", op="gate", B=1, T=131072, D=1024, dtype="bf16", normalize=True, state=False, carry=True),
        # The gradients of the 4096-wide recurrence in training.
        dict(name="gate grad 2x8192x4096", op="gate_backward", B=2, T=8192, D=4096, dtype="bf16", normalize=True, state=False),
        # Gradients in fp32 over ragged sizes, a state's gradient among them.
        dict(name="gate grad f32 3x1777x1000", op="gate_backward", B=3, T=1777, D=1000, dtype="f32", normalize=True, state=True),
        # Clipping the gradients of the 7B-shaped layer, as its weight products leave them (fp32).
        dict(name="clip layer f32 5 tensors", op="clip", shape="layer", width=4096, layers=1, dtype="f32", limit=1.0),
        # Twelve small layers (d_model=512) in bf16: many small tensors.
        dict(name="clip small bf16 60 tensors", op="clip", shape="layer", width=512, layers=12, dtype="bf16", limit=1.0),
        # Tensors of any sizes, some of them tiny, of both types; the norm alone is within the limit, nothing is scaled.
        dict(name="clip mixed 61 tensors", op="clip", shape="mixed", width=1000003, layers=61, dtype="mixed", limit=1e9),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "qk_backward", "step", "gate", "gate", "gate_backward", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("qk", "qk_backward"):
        while True:
            B, T, H = log_int(rng, 1, 64), log_int(rng, 1, 32768), log_int(rng, 1, 32)
            dk = rng.choice([32, 64, 80, 96, 128, 128, 256, 256, 512, 2 * log_int(rng, 1, 255)])
            Hk = H if rng.random() < 0.7 else rng.choice([h for h in range(1, H + 1) if H % h == 0])
            if B * T * H * dk <= 2 * 8192 * 16 * 256 // (2 if dtype == "f32" else 1):
                break
        return dict(op=op, B=B, T=T, H=H, Hk=Hk, dk=dk, dtype=dtype, fused=rng.random() < 0.4, weights=rng.random() < 0.8, rows=rng.random() < 0.4)
    if op == "clip":
        if rng.random() < 0.5:
            width = rng.choice([128, 256, 320, 512, 1000, 1024, 2048])
            most = max(1, GRADS // (6 * width * width + width) // 2)
            return dict(op=op, shape="layer", width=width, layers=log_int(rng, 1, min(most, 12)), dtype=dtype, limit=rng.choice([1.0, 0.01, 1e9]))
        return dict(op=op, shape="mixed", width=log_int(rng, 1, 2000000), layers=log_int(rng, 1, 62), dtype="mixed", limit=rng.choice([1.0, 0.01, 1e9]))
    normalize = rng.random() < 0.75
    wide = rng.choice([256, 512, 1000, 1024, 2048, 2560, 4096, 8192, log_int(rng, 1, 8191)])
    if op == "step":
        return dict(op=op, B=log_int(rng, 1, 512), D=wide, dtype=dtype, normalize=normalize)
    while True:
        B, T = log_int(rng, 1, 64), log_int(rng, 1, 131072)
        if B * T * wide <= LARGEST // (4 if op == "gate_backward" else 2):
            break
    if op == "gate":
        return dict(op=op, B=B, T=T, D=wide, dtype=dtype, normalize=normalize, state=rng.random() < 0.5, carry=rng.random() < 0.5)
    return dict(op=op, B=B, T=T, D=wide, dtype=dtype, normalize=normalize, state=rng.random() < 0.5)


# ---- inputs -------------------------------------------------------------------------------------------------------

def sizes_of(case):
    """(elements, type) of each gradient tensor."""
    c = case
    if c["shape"] == "layer":  # wq, wk [w, w], wv [2 w, w], wo [w, 2 w] and the norm's weight
        w = c["width"]
        return [(n, c["dtype"]) for n in (w * w, w * w, 2 * w * w, 2 * w * w, w)] * c["layers"]
    out, z = [], 12345 + c["width"] + 7 * c["layers"]
    for _ in range(c["layers"]):  # sizes from 1 to `width`, even over their logarithm
        z = (z * 1103515245 + 12345) % 2 ** 31
        out.append((max(1, int(math.exp(z / 2 ** 31 * math.log(c["width"] + 1)))), "bf16" if z >> 20 & 1 else "f32"))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def empty(*shape, t=torch.float32):
        return torch.empty(shape, dtype=t, device="cuda")

    c = dict(case)
    st = {"case": c}
    if c["op"] in ("qk", "qk_backward"):
        B, T, H, Hk, dk, t = c["B"], c["T"], c["H"], c["Hk"], c["dk"], TYPES[c["dtype"]]
        gain = torch.exp(0.5 * normal(dk))  # channels of unlike size
        if c["fused"]:  # one array as a fused projection leaves it: Q, K and V of each token side by side
            all_ = normal(B, T, (H + 2 * Hk) * dk).to(t)
            q, k = all_[..., :H * dk].unflatten(-1, (H, dk)), all_[..., H * dk:(H + Hk) * dk].unflatten(-1, (Hk, dk))
            q.copy_(q.float() * gain)
            k.copy_(k.float() * gain)
        else:
            q, k = (normal(B, T, H, dk) * gain).to(t), (normal(B, T, Hk, dk) * gain).to(t)
        st["q"], st["k"] = q, k
        st["wq"], st["wk"] = ((1.0 + 0.2 * normal(dk)).to(t), (1.0 + 0.2 * normal(dk)).to(t)) if c["weights"] else (None, None)
        st["theta"] = (10000.0 ** (-2.0 * np.arange(dk // 2) / dk)).astype(np.float32)  # on the host, as the forms take it
        st["theta_device"] = torch.from_numpy(st["theta"]).cuda()
        st["pos"] = torch.randint(0, 100000, (B,), generator=gen, device="cuda") if c["rows"] else None
        if c["op"] == "qk":
            st["bufs"] = (empty(B, T, H, dk, t=t), empty(B, T, Hk, dk, t=t))
        else:
            st["dq"], st["dk"] = (1e-2 * normal(B, T, H, dk)).to(t), (1e-2 * normal(B, T, Hk, dk)).to(t)
            st["bufs"] = (empty(B, T, H, dk, t=t), empty(B, T, Hk, dk, t=t), *((empty(dk), empty(dk)) if c["weights"] else (None, None)))
    elif c["op"] in ("step", "gate", "gate_backward"):
        B, D, t = c["B"], c["D"], TYPES[c["dtype"]]
        lead = (B,) if c["op"] == "step" else (B, c["T"])
        st["x"] = normal(*lead, D).to(t)
        st["g"] = (1.5 * normal(*lead, D)).to(t)
        # decays from exp(-0.001) to exp(-2) a token where the gate is open
        st["rate"] = torch.exp(torch.empty(D, device="cuda").uniform_(math.log(1e-3), math.log(2.0), generator=gen))
        st["state"] = normal(B, D) if c.get("state", True) else None
        if c["op"] == "step":
            st["bufs"] = (empty(B, D, t=t), empty(B, D))
        elif c["op"] == "gate":
            blocks = -(-c["T"] // BLOCK)
            st["bufs"] = (empty(*lead, D, t=t), empty(B, D), empty(B, blocks, D) if c["carry"] else None)
        else:
            st["dh"] = (1e-2 * normal(*lead, D)).to(t)
            st["dstate"] = 1e-2 * normal(B, D) if c["state"] else None
            # a training step keeps the forward pass's states at the start of each block
            h = states(*coefficients(st["x"], st["g"], st["rate"], c["normalize"]), st["state"])
            st["carry"] = block_states(h, st["state"])
            st["bufs"] = (empty(*lead, D, t=t), empty(*lead, D, t=t), empty(D), empty(B, D) if c["state"] else None)
    else:
        st["grads"] = [(1e-3 * normal(n)).to(TYPES[t]) for n, t in sizes_of(c)]
        st["bufs"] = [torch.empty_like(g) for g in st["grads"]]
        st["norm"] = empty()
    return st


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(st):
    return run_own(st) if own else run_plain(st)


def run_own(st):
    import retnet_scale_retention_amd as msr
    c = st["case"]
    if c["op"] == "qk":
        return msr.msr_qk_norm_rotate(st["q"], st["k"], st["wq"], st["wk"], eps=EPS, theta=st["theta"], pos_rows=st["pos"], out=st["bufs"])
    if c["op"] == "qk_backward":
        return msr.msr_qk_norm_rotate_backward(st["q"], st["k"], st["wq"], st["wk"], st["dq"], st["dk"], eps=EPS, theta=st["theta"], pos_rows=st["pos"],
                                               want_weight_grad=c["weights"], out=st["bufs"])
    if c["op"] == "step":
        h, s = st["bufs"]
        return msr.msr_gated_recurrence_step(st["x"], st["g"], st["state"], st["rate"], normalize=c["normalize"], state_out=s, out=h), s
    if c["op"] == "gate":
        return msr.msr_gated_recurrence(st["x"], st["g"], st["rate"], normalize=c["normalize"], state_in=st["state"], want_carry=c["carry"], out=st["bufs"])
    if c["op"] == "gate_backward":
        return msr.msr_gated_recurrence_backward(st["x"], st["g"], st["rate"], st["dh"], normalize=c["normalize"], state_in=st["state"], carry=st["carry"],
                                                 grad_state=st["dstate"], want_state_grad=c["state"], out=st["bufs"])
    return msr.msr_clip_gradients(st["grads"], c["limit"], out=st["bufs"], norm_out=st["norm"])


def rotation(st):
    """cos and sin [B, T, 1, dk / 2] of the tokens' angles; far positions need 64 bits."""
    c = st["case"]
    p = torch.arange(c["T"], device="cuda", dtype=torch.float64)[None, :]
    if st["pos"] is not None:
        p = p + st["pos"].double()[:, None]
    a = p[:, :, None, None] * st["theta_device"].double()
    return torch.cos(a).float(), torch.sin(a).float()


def turned(x, cs, sn):
    """Pairs (x[2 i], x[2 i + 1]) turned by their angles."""
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cs - b * sn, b * cs + a * sn), -1).flatten(-2)


def coefficients(x, g, rate, normalize):
    """log(a), u [B, T, D] of h_t = a_t h_{t-1} + u_t in 32 bits, 1 - a^2 without its cancellation."""
    log_a = -rate * torch.sigmoid(g.float())
    m = torch.sqrt(-torch.expm1(2.0 * log_a)) if normalize else 1.0
    return log_a, m * x.float()


def states(log_a, u, start):
    """h [B, T, D]: blocks of tokens side by side, one token of each at a time, then the blocks one after the other.  What
    a step takes away, (1 - a) h, is subtracted: a next to 1, rounded, would be off by the same amount at every token."""
    B, T, D = u.shape
    n = max(1, math.isqrt(T))
    blocks = -(-T // n)
    pad = blocks * n - T
    if pad:  # tokens that keep the state
        log_a = torch.cat((log_a, log_a.new_zeros(B, pad, D)), 1)
        u = torch.cat((u, u.new_zeros(B, pad, D)), 1)
    log_a, h = log_a.view(B, blocks, n, D), u.view(B, blocks, n, D).clone()
    lost = -torch.expm1(log_a)
    for t in range(1, n):
        h[:, :, t] += h[:, :, t - 1] - lost[:, :, t] * h[:, :, t - 1]
    decay = torch.exp(torch.cumsum(log_a, 2))
    into = [start if start is not None else u.new_zeros(B, D)]
    for i in range(blocks - 1):
        into.append(h[:, i, -1] + decay[:, i, -1] * into[-1])
    h += decay * torch.stack(into, 1)[:, :, None]
    return h.view(B, blocks * n, D)[:, :T]


def block_states(h, start):
    """The states that each block of 64 tokens starts from."""
    first = (start if start is not None else torch.zeros_like(h[:, 0]))[:, None]
    return torch.cat((first.to(h.dtype), h[:, BLOCK - 1:-1:BLOCK]), 1)


def run_plain(st):
    c = st["case"]
    if c["op"] == "qk":
        cs, sn = rotation(st)

        def one(x, w, s):
            x, t = x.float(), x.dtype
            n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            return (turned(n if w is None else n * w.float(), cs, sn) * s).to(t)

        return one(st["q"], st["wq"], 1.0), one(st["k"], st["wk"], c["dk"] ** -0.5)
    if c["op"] == "qk_backward":
        cs, sn = rotation(st)

        def one(x, w, dy, s):
            x, t = x.float(), x.dtype
            u = turned(dy.float(), cs, -sn) * s
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            n = x * r
            g = u if w is None else u * w.float()
            return (r * (g - n * (g * n).mean(-1, keepdim=True))).to(t), None if w is None else (u * n).sum((0, 1, 2))

        dq, dwq = one(st["q"], st["wq"], st["dq"], 1.0)
        dk, dwk = one(st["k"], st["wk"], st["dk"], c["dk"] ** -0.5)
        return dq, dk, dwq, dwk
    if c["op"] == "step":
        log_a, u = coefficients(st["x"], st["g"], st["rate"], c["normalize"])
        h = torch.exp(log_a) * st["state"] + u
        return h.to(st["x"].dtype), h
    if c["op"] == "gate":
        h = states(*coefficients(st["x"], st["g"], st["rate"], c["normalize"]), st["state"])
        return h.to(st["x"].dtype), h[:, -1].clone(), block_states(h, st["state"]) if c["carry"] else None
    if c["op"] == "gate_backward":
        x, g, dh, rate = st["x"].float(), st["g"].float(), st["dh"].float(), st["rate"]
        log_a, u = coefficients(st["x"], st["g"], rate, c["normalize"])
        h, a = states(log_a, u, st["state"]), torch.exp(log_a)
        before = torch.cat(((st["state"] if st["state"] is not None else torch.zeros_like(h[:, 0]))[:, None], h[:, :-1]), 1)
        # lam_t = dh_t + a_{t+1} lam_{t+1}: the same recurrence, from the last token to the first
        if st["dstate"] is not None:
            dh = torch.cat((dh[:, :-1], (dh[:, -1] + st["dstate"])[:, None]), 1)
        after = torch.cat((log_a[:, 1:], torch.zeros_like(a[:, :1])), 1)
        lam = states(after.flip(1), dh.flip(1), None).flip(1)
        s = torch.sigmoid(g)
        dlog = a * lam * before
        m = torch.ones_like(a)
        if c["normalize"]:
            m = torch.sqrt(-torch.expm1(-2.0 * rate * s))
            dlog = dlog - torch.where(m > 0, lam * x * a * a / m, torch.zeros_like(m))
        dg = -rate * s * (1.0 - s) * dlog
        out = (m * lam).to(st["x"].dtype), dg.to(st["x"].dtype), -(s * dlog).sum((0, 1))
        return *out, a[:, 0] * lam[:, 0] if c["state"] else None
    total = torch.stack([g.double().square().sum() for g in st["grads"]]).sum()
    norm = torch.sqrt(total)
    f = torch.where(norm > c["limit"], c["limit"] / norm, torch.ones_like(norm)).float()
    return [(g.float() * f).to(g.dtype) for g in st["grads"]], norm.float()


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "clip":
        n = sum(2 * n * BYTES[t] for n, t in sizes_of(c))
        return {"bytes": n, "flops": 3.0 * sum(n for n, _ in sizes_of(c))}
    e = BYTES[c["dtype"]]
    if c["op"] in ("qk", "qk_backward"):
        n = c["B"] * c["T"] * (c["H"] + c["Hk"]) * c["dk"]
        back = c["op"] == "qk_backward"
        small = c["dk"] * (2 * e + (8 if back else 0)) if c["weights"] else 0
        return {"bytes": n * e * (3 if back else 2) + small, "flops": (16.0 if back else 9.0) * n}
    B, D = c["B"], c["D"]
    if c["op"] == "step":
        return {"bytes": B * D * (3 * e + 8) + 4 * D, "flops": 12.0 * B * D}
    n = B * c["T"] * D
    blocks = 4 * B * D * -(-c["T"] // BLOCK)
    states_ = 4 * B * D
    if c["op"] == "gate":
        return {"bytes": 3 * n * e + 4 * D + states_ * (2 if c["state"] else 1) + (blocks if c["carry"] else 0), "flops": 12.0 * n}
    return {"bytes": 5 * n * e + blocks + 8 * D + (2 * states_ if c["state"] else 0), "flops": 30.0 * n}


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] in ("qk", "qk_backward"):
        theta = torch.as_tensor(st["theta"], device="cuda", dtype=torch.float64)
        at = torch.zeros(c["B"], dtype=torch.float64, device="cuda") if st["pos"] is None else st["pos"].double()
        angle = (at.view(-1, 1) + torch.arange(c["T"], device="cuda"))[..., None] * theta
        z = torch.polar(torch.ones_like(angle), angle)[:, :, None]  # a pair as a complex number times e^(i angle)

        def head(x, w, s):
            y = x / (x.square().sum(-1, keepdim=True) / c["dk"] + EPS).sqrt()
            y = y if w is None else y * w
            pairs = torch.view_as_complex(y.unflatten(-1, (-1, 2)).contiguous())
            return torch.view_as_real(pairs * z).flatten(-2) * s

        if c["op"] == "qk":
            d = [t if t is None else t.double() for t in (st["q"], st["k"], st["wq"], st["wk"])]
            return head(d[0], d[2], 1.0), head(d[1], d[3], c["dk"] ** -0.5)
        out, dws = [], []
        for x, w, dy, s in ((st["q"], st["wq"], st["dq"], 1.0), (st["k"], st["wk"], st["dk"], c["dk"] ** -0.5)):
            x = x.double().contiguous().requires_grad_(True)
            w = w if w is None else w.double().requires_grad_(True)
            got = torch.autograd.grad(head(x, w, s), [x] if w is None else [x, w], dy.double())
            out.append(got[0])
            dws.append(None if w is None else got[1])
        return *out, *dws
    if c["op"] == "clip":
        norm = sum(float(g.double().square().sum()) for g in st["grads"]) ** 0.5
        f = min(1.0, c["limit"] / norm) if norm > 0 else 1.0
        return [g.double() * f for g in st["grads"]], torch.tensor(norm, dtype=torch.float64, device="cuda")
    x, g, rate = st["x"].double(), st["g"].double(), st["rate"].double()
    if c["op"] == "step":
        x, g = x[:, None], g[:, None]
    B, T, D = x.shape
    s = 1.0 / (1.0 + torch.exp(-g))
    a = torch.exp(-rate * s)
    m = (-torch.special.expm1(-2.0 * rate * s)).sqrt() if c["normalize"] else torch.ones_like(a)
    start = torch.zeros(B, D, dtype=torch.float64, device="cuda") if st["state"] is None else st["state"].double()
    h = torch.empty(T + 1, B, D, dtype=torch.float64, device="cuda")  # token by token
    h[0] = start
    at, ut = a.transpose(0, 1).contiguous(), (m * x).transpose(0, 1).contiguous()
    for t in range(T):
        torch.addcmul(ut[t], at[t], h[t], out=h[t + 1])
    if c["op"] == "step":
        return h[1], h[1]
    if c["op"] == "gate":
        return h[1:].transpose(0, 1), h[T], h[:T:BLOCK].transpose(0, 1) if c["carry"] else None
    lam = torch.empty(T, B, D, dtype=torch.float64, device="cuda")
    dh = st["dh"].double().transpose(0, 1).contiguous()
    lam[T - 1] = dh[T - 1] if st["dstate"] is None else dh[T - 1] + st["dstate"].double()
    for t in range(T - 2, -1, -1):
        torch.addcmul(dh[t], at[t + 1], lam[t + 1], out=lam[t])
    lam, before = lam.transpose(0, 1), h[:T].transpose(0, 1)
    da = lam * before  # the gradient of a_t, through h and through m = sqrt(1 - a^2)
    if c["normalize"]:
        da = da - lam * x * a / m
    ds = da * a * -rate
    return m * lam, ds * s * (1 - s), (da * a * -s).sum((0, 1)), a[:, 0] * lam[:, 0] if c["state"] else None
