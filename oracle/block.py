"""Layer norm, SwiGLU with 8-bit checkpoints and ragged expert products in float64 (oracle; test
infrastructure). Plain definitions on numpy arrays; rounding to BF16 or MXFP8 happens only where an
operator's definition has it."""
import numpy as np

from .formats import bf16_bits_to_f64, e4m3_to_f64, e8m0_to_f64, f64_to_bf16_bits
from .mx import quantize_blocks


def bf16(v):
    """float64 -> the nearest BF16 value, as float64."""
    return bf16_bits_to_f64(f64_to_bf16_bits(np.asarray(v, dtype=np.float64)))


def mx_rows(v):
    """Row-wise MXFP8 of v [rows, cols] with a short last group: (codes [rows, cols], bytes [rows, G]). The
    missing elements of a short group are zeros, which change neither its maximum nor the other codes."""
    v = np.asarray(v, dtype=np.float64)
    rows, cols = v.shape
    G = -(-cols // 32)
    p = np.zeros((rows, G * 32))
    p[:, :cols] = v
    q, s = quantize_blocks(p.reshape(rows, G, 32))
    return q.reshape(rows, G * 32)[:, :cols], s


def mx_values(q, s):
    """The float64 values of codes [rows, cols] and bytes [rows, G]."""
    return e4m3_to_f64(q) * np.repeat(e8m0_to_f64(s), 32, axis=1)[:, :q.shape[1]]


def layer_norm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd, xh)."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    xh = (x - mean[:, None]) * rstd[:, None]
    return xh * (1.0 if w is None else w) + (0.0 if b is None else b), mean, rstd, xh


def layer_norm_grads(dy, xh, rstd, w=None):
    """(dx, dw, db)."""
    g = dy * (1.0 if w is None else w)
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def sigmoid(g):
    return 1.0 / (1.0 + np.exp(-g))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_grads(dh, g, u):
    """(dg, du)."""
    s = sigmoid(g)
    return dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s


def grouped_fwd(x, w, offs):
    y = np.zeros((x.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        y[offs[e]:offs[e + 1]] = x[offs[e]:offs[e + 1]] @ w[e].T
    return y


def grouped_dgrad(dy, w, offs):
    dx = np.zeros((dy.shape[0], w.shape[2]))
    for e in range(w.shape[0]):
        dx[offs[e]:offs[e + 1]] = dy[offs[e]:offs[e + 1]] @ w[e]
    return dx


def grouped_wgrad(dy, x, offs):
    return np.stack([dy[a:b].T @ x[a:b] for a, b in zip(offs[:-1], offs[1:])])
