"""float64 definitions of the layer around retention: the residual's addition
with a root-mean-square norm and its gradients, 8-bit blocks, and the product
of 8-bit operands.  numpy only; shares no code with the library."""
import numpy as np

BLOCK = 128
TINY = 2.0 ** -126
E4M3 = np.array([np.nan if c & 127 == 127 else
                 (-1.0) ** (c >> 7) * ((c & 7) / 8 * 2.0 ** -6 if not (c >> 3) & 15 else
                                       (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7)) for c in range(256)])


def padded(n):
    return -(-n // BLOCK) * BLOCK


def add_rmsnorm(x, r, w, eps):
    """(n, h)"""
    h = np.asarray(x, np.float64) + (0.0 if r is None else np.asarray(r, np.float64))
    with np.errstate(invalid="ignore", over="ignore"):
        n = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
        return (n if w is None else n * np.asarray(w, np.float64)), h


def add_rmsnorm_backward(h, w, dy, dsum, eps):
    """(dx, dw) and the sums of magnitudes that bound their rounding."""
    h, dy = np.asarray(h, np.float64), np.asarray(dy, np.float64)
    g = dy if w is None else dy * np.asarray(w, np.float64)
    rstd = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    dx = rstd * g - h * rstd ** 3 * (g * h).mean(-1, keepdims=True)
    mag = rstd * np.abs(g) + np.abs(h) * rstd ** 3 * np.abs(g * h).mean(-1, keepdims=True)
    if dsum is not None:
        dx, mag = dx + dsum, mag + np.abs(dsum)
    return dx, (dy * h * rstd).sum(0), mag, np.abs(dy * h * rstd).sum(0)


def block_scales(x, block_rows):
    """The scale of every block of x [R, C] in 64 bits, and the same spread over x's elements."""
    R, C = x.shape
    full = np.zeros((-(-R // block_rows) * block_rows, padded(C)))
    full[:R, :C] = np.abs(x)
    t = full.reshape(full.shape[0] // block_rows, block_rows, -1, BLOCK)
    s = np.maximum(t.max((1, 3)) / 448.0, TINY)
    return s, np.repeat(np.repeat(s, block_rows, 0)[:R], BLOCK, 1)[:, :C]


def half_step(v):
    """Half the distance between the e4m3 values around |v| <= 448: the largest error of a nearest rounding."""
    a = np.maximum(np.abs(v), 2.0 ** -6)
    return 2.0 ** (np.floor(np.log2(a)) - 4)


def spread(s, rows, block_rows):
    return np.repeat(np.repeat(np.asarray(s, np.float64), block_rows, 0)[:rows], BLOCK, 1)


def matmul(a, sa, b, sb, b_block_rows):
    """(C, sum of the products' magnitudes) of e4m3 codes (uint8) and scales."""
    x = E4M3[a] * spread(sa, a.shape[0], 1)
    y = E4M3[b] * spread(sb, b.shape[0], b_block_rows)
    return x @ y.T, np.abs(x) @ np.abs(y).T
