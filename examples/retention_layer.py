"""A retention sub-layer from the library's pieces, its projections in 8 bits: prompt, single tokens, and a training step.

    h = x + residual;  n = RMSNorm(h);  Q, K, V = n Wq^T, n Wk^T, n Wv^T;  O = retention(Q, K, V);  y = O Wo^T

With qk_norm the heads of Q and K are normalised and rotated between projection and retention (one pass), and retention
takes them as they are.  A training step's gradients can be clipped to a common norm.
The norm writes n in 8 bits where the projections read it; retention's output is quantised for the output projection.
Weights are quantised once, in 128 x 128 squares and in both orders (the transposed copy serves the input gradients).

    python examples/retention_layer.py        # runs the three on a small layer and times the 7B-shaped one (GPU)
"""
import sys
import time
from pathlib import Path

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))

import torch  # noqa: E402

import msr_inputs as mi  # noqa: E402
import retnet_scale_retention_amd as msr  # noqa: E402


class RetentionLayer:
    """Weights of one sub-layer: wq, wk [H dk, d], wv [H dv, d], wo [d, H dv] and the norm's w [d] (bfloat16, device);
    qk_norm: None, or the weights [dk] of the norms of Q's and K's heads."""

    def __init__(self, w, wq, wk, wv, wo, H, *, chunk=128, eps=1e-6, qk_norm=None):
        self.w, self.H, self.chunk, self.eps, self.qk_norm = w, H, chunk, eps, qk_norm
        # what retention does to Q and K: the rotation and the scale, unless the heads' norms have done both
        self.form = {} if qk_norm is None else dict(flags=msr.MSR_FLAG_NO_ROTATE, scale=1.0)
        self.gamma = mi.gammas(H)
        self.q8 = [msr.msr_quantize(m, block_rows=128, want_transposed=True) for m in (wq, wk, wv, wo)]

    def _project(self, q, s):
        """Q, K, V [..., H, d] from the norm's 8-bit output."""
        return [msr.msr_scaled_matmul(q, s, m[0], m[1]).unflatten(-1, (self.H, -1)) for m in self.q8[:3]]

    def _heads(self, q, k, v, pos):
        """Q, K, V as retention takes them; pos: the first token's position, or one per batch row (int64 tensor)."""
        if self.qk_norm is None:
            return q, k, v
        at = dict(pos_rows=pos) if isinstance(pos, torch.Tensor) else dict(pos0=pos)
        return (*msr.msr_qk_norm_rotate(q, k, *self.qk_norm, eps=self.eps, **at), v)

    def _output(self, o):
        """O [B, T, H, dv] (or [B, H, dv]) through the output projection: [..., d]."""
        flat = o.flatten(-2)
        q, s, _, _ = msr.msr_quantize(flat.flatten(0, -2))
        return msr.msr_scaled_matmul(q, s, self.q8[3][0], self.q8[3][1]).unflatten(0, flat.shape[:-1])

    def prompt(self, x, residual, state=None, pos0=0):
        """x, residual [B, T, d] -> (y, h, state): y [B, T, d], the residual stream h, the state after the prompt."""
        _, h, q, s = msr.msr_add_rmsnorm(x, self.w, residual, eps=self.eps, want_y=False, want_q=True)
        o, state = msr.msr_chunkwise(*self._heads(*self._project(q, s), pos0), self.gamma, self.chunk, state_in=state, pos0=pos0,
                                     **self.form)
        return self._output(o), h, state

    def token(self, x, residual, state, pos):
        """One token per sequence: x, residual [B, d]; the state is updated in place."""
        _, h, q, s = msr.msr_add_rmsnorm(x, self.w, residual, eps=self.eps, want_y=False, want_q=True)
        o = msr.msr_recurrent_step(*self._heads(*self._project(q, s), pos), state, self.gamma, pos, **self.form)
        return self._output(o), h

    def train(self, x, residual, grad_y, grad_h):
        """Forward and backward: (y, h, grads), grads of x (= of the residual), the norm's weight and wq, wk, wv, wo
        (the weights' in float32), and with qk_norm its two weights'."""
        lead, (wq, wk, wv, wo) = x.shape[:-1], self.q8
        n, h, q, s = msr.msr_add_rmsnorm(x, self.w, residual, eps=self.eps, want_q=True)
        raw = self._project(q, s)
        qkv = self._heads(*raw, 0)
        o, _ = msr.msr_chunkwise(*qkv, self.gamma, self.chunk, return_state=False, **self.form)
        rows = lambda t: t.reshape(lead.numel(), -1)  # [B, T, ...] as a matrix of tokens
        both = lambda t, r=True: msr.msr_quantize(rows(t), want_rows=r, want_transposed=True)
        oq, os_, oqt, ost = both(o)
        y = msr.msr_scaled_matmul(oq, os_, wo[0], wo[1]).view(*lead, -1)
        # output projection: dO = dy Wo, dWo = dy^T O
        gq, gs, gqt, gst = both(grad_y)
        d_o = msr.msr_scaled_matmul(gq, gs, wo[2], wo[3]).view(o.shape)
        d_wo = msr.msr_scaled_matmul(gqt, gst, oqt, ost, out_dtype=torch.float32)
        grads = msr.msr_chunkwise_backward(*qkv, self.gamma, self.chunk, d_o, want_state_grad=False, **self.form)[:3]
        d_heads = ()
        if self.qk_norm is not None:
            dq, dk, *d_heads = msr.msr_qk_norm_rotate_backward(*raw[:2], *self.qk_norm, *grads[:2], eps=self.eps,
                                                               out=(*grads[:2], None, None))
            grads = dq, dk, grads[2]
        # the three projections: dn is the sum of their input gradients
        _, _, nqt, nst = both(n, False)
        d_n, d_w = None, []
        for g, m in zip(grads, (wq, wk, wv)):
            gq, gs, gqt, gst = both(g)
            part = msr.msr_scaled_matmul(gq, gs, m[2], m[3], out_dtype=torch.float32)
            d_n = part if d_n is None else d_n.add_(part)
            d_w.append(msr.msr_scaled_matmul(gqt, gst, nqt, nst, out_dtype=torch.float32))
        d_x, d_norm = msr.msr_add_rmsnorm_backward(h, self.w, d_n.to(h.dtype).view(h.shape), grad_sum=grad_h, eps=self.eps)
        return y, h, (d_x, d_norm, *d_w, d_wo, *d_heads)

    def clip(self, grads, max_norm):
        """Scales the weights' gradients of train() to a common norm of max_norm at most, in place; returns the norm."""
        return msr.msr_clip_gradients(grads[1:], max_norm)[1]


def make(H, dk, dv, d, chunk, seed=0, device="cuda", qk_norm=False):
    """A layer with weights ~ N(0, 1 / fan-in), and the plain weights."""
    g = torch.Generator(device=device).manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g, device=device)
    ws = [(normal(o, i) / i ** 0.5).bfloat16() for o, i in ((H * dk, d), (H * dk, d), (H * dv, d), (d, H * dv))]
    w = (1 + 0.1 * normal(d)).bfloat16()
    heads = tuple((1 + 0.1 * normal(dk)).bfloat16() for _ in range(2)) if qk_norm else None
    return RetentionLayer(w, *ws, H, chunk=chunk, qk_norm=heads), w, ws


def main():
    layer, _, _ = make(4, 64, 128, 256, 64)
    x, r = torch.randn(2, 193, 256, device="cuda").bfloat16(), torch.randn(2, 193, 256, device="cuda").bfloat16()
    y, _, _ = layer.prompt(x, r)
    _, _, state = layer.prompt(x[:, :192].contiguous(), r[:, :192].contiguous())
    yt, _ = layer.token(x[:, 192].contiguous(), r[:, 192].contiguous(), state, 192)
    print("token 192 after a prompt of 192, against the prompt of 193: relative difference "
          f"{float((yt - y[:, 192]).float().norm() / y[:, 192].float().norm()):.1e}")
    _, _, grads = layer.train(x, r, torch.randn_like(y), torch.randn_like(y))
    print("gradients:", ", ".join(f"{tuple(t.shape)} {str(t.dtype)[6:]}" for t in grads))
    normed, _, _ = make(4, 64, 128, 256, 64, qk_norm=True)
    _, _, grads = normed.train(x, r, torch.randn_like(y), torch.randn_like(y))
    print(f"with norms of the heads: gradients' norm {float(normed.clip(grads, 1.0)):.1f}, clipped to "
          f"{float(msr.msr_gradient_norm(grads[1:])):.3f}")

    B, T, H, dk, dv, d = 2, 8192, 16, 256, 512, 4096
    layer, _, _ = make(H, dk, dv, d, 128)
    x, r = torch.randn(B, T, d, device="cuda").bfloat16(), torch.randn(B, T, d, device="cuda").bfloat16()
    g = torch.randn(B, T, d, device="cuda").bfloat16()
    xt, rt, st = x[:, 0].contiguous(), r[:, 0].contiguous(), torch.zeros(B, H, dk, dv, device="cuda")
    for name, f, n in (("prompt", lambda: layer.prompt(x, r), B * T), ("token", lambda: layer.token(xt, rt, st, T), B),
                       ("train", lambda: layer.train(x, r, g, g), B * T)):
        for _ in range(3):
            f()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(10):
            f()
        torch.cuda.synchronize()
        ms = (time.perf_counter() - t0) * 100
        print(f"7B-shaped layer, {name}: {ms:.2f} ms, {n / ms * 1e3:.3g} tokens/s")


if __name__ == "__main__":
    main()
