"""The routed experts of examples/expert_mlp_mxfp4.py (every 4-bit operator together) against a float64 MLP that quantises at the
same places.

Tolerance, normwise. The chains differ by BF16 roundings (2^-8 of a value at most each), and a rounding in front of a
quantiser can move a value over the border between two codes: at a border v the codes are at least 0.285 v apart (3 and 4), so
at most a share 2 x 2^-8 / 0.285 = 0.027 of the values moves, each by at most half of itself (4 and 6 around 5 less, below 1 more
but of small values): sqrt(0.027) / 2 = 0.083 for each quantiser that is fed a rounded tensor, which the product behind it passes
on; moved scales and the 8-bit checkpoint's codes (steps of 2^-4) are an order below. Together with the roundings 0.1 a quantiser on
the way; E4M3 operands move by 2^-4: sqrt(2 x 2^-8 x 16) / 16 = 0.022."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from gpu_util import require_gpu
from oracle import block as ob
from oracle import mxfp4 as o4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def f64(t):
    return t.detach().double().cpu().numpy()


def load():
    spec = importlib.util.spec_from_file_location("expert_mlp_mxfp4", os.path.join(ROOT, "examples", "expert_mlp_mxfp4.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def q(v, e4m3=False):
    """Quantised along the last axis and read back."""
    return o4.values(*o4.operand(v, e4m3))[:, :v.shape[1]]


def qt(v):
    """Quantised along the first axis."""
    return q(np.ascontiguousarray(v.T)).T


def near(got, ref, tol, what):
    d = np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)
    assert d <= tol, (what, d)


def reference(w13, w2, x, choice, weight, dy, e4m3=False):
    w13, w2, x, dy, p, choice = f64(w13), f64(w2), f64(x), f64(dy), f64(weight), choice.cpu().numpy()
    E, F, k = w13.shape[0], w2.shape[2], choice.shape[1]
    flat = choice.reshape(-1)
    order = np.argsort(flat, kind="stable")
    counts = np.bincount(flat, minlength=E)
    tok, pr = order // k, p.reshape(-1)[order][:, None]
    seg = np.concatenate([[0], counts.cumsum()])
    y, dx = x.copy(), dy.copy()
    dw13, dw2, dweight = np.zeros_like(w13), np.zeros_like(w2), np.zeros(flat.size)
    for e in range(E):
        a, b = seg[e], seg[e + 1]
        if a == b:
            continue
        t = tok[a:b]
        xe = x[t]
        gu = ob.bf16(q(xe, e4m3) @ q(w13[e]).T)
        h = ob.bf16(ob.swiglu(gu[:, :F], gu[:, F:]))
        yp = ob.bf16(q(h, e4m3) @ q(w2[e]).T)
        np.add.at(y, t, yp * pr[a:b])
        dweight[order[a:b]] = (dy[t] * yp).sum(1)
        dyp = ob.bf16(dy[t] * pr[a:b])
        dh = ob.bf16(q(dyp) @ qt(w2[e]))
        pad = np.zeros((-(b - a) % 128, 1))  # column groups start at the segment's first row
        cols = lambda v: qt(np.concatenate([v, np.zeros((pad.shape[0], v.shape[1]))]))[:b - a]  # noqa: E731
        dw2[e] = cols(dyp).T @ cols(h)
        keep = lambda v: ob.mx_values(*ob.mx_rows(v))  # noqa: E731
        dgu = ob.bf16(np.concatenate(ob.swiglu_grads(dh, keep(gu[:, :F]), keep(gu[:, F:])), 1))
        np.add.at(dx, t, q(dgu) @ qt(w13[e]))
        dw13[e] = cols(dgu).T @ cols(xe)
    return y, dx, dweight.reshape(choice.shape), dw13, dw2


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,F,E,k", [(96, 128, 64, 8, 3), (33, 96, 160, 5, 2), (1, 256, 128, 16, 4), (300, 320, 200, 4, 2)])
def test_mlp_against_float64(T, D, F, E, k):
    require_gpu()
    ex = load()
    w13, w2 = ex.make(D, F, E)
    w13, w2 = w13 * 4, w2 * 4  # (so that y is not x alone)
    mlp = ex.ExpertMlp4(w13, w2)
    x, choice, weight, dy = ex.tokens(T, D, E, k)
    y, kept = mlp.forward(x, choice, weight)
    dx, dweight, dw13, dw2 = mlp.backward(dy, kept)
    ry, rdx, rdweight, rdw13, rdw2 = reference(w13, w2, x, choice, weight, dy)
    near(y.float() - x.float(), ry - f64(x), 0.1, "y")            # h
    near(dweight, rdweight, 0.1, "dweight")
    near(dx.float() - dy.float(), rdx - f64(dy), 0.2, "dx")       # dyp, dgu
    near(dw2, rdw2, 0.2, "dw2")                                   # dyp, h
    near(dw13, rdw13, 0.2, "dw13")                                # dyp, dgu
    served = reference(w13, w2, x, choice, weight, dy, e4m3=True)[0]
    near(mlp.serve(x, choice, weight).float() - x.float(), served - f64(x), 0.04, "served")


@pytest.mark.gpu
def test_step_captured_and_replayed():
    """Forward and backward in one graph, replayed on new inputs beside eager steps."""
    require_gpu()
    ex = load()
    mlp = ex.ExpertMlp4(*ex.make(256, 128, 8))
    x, choice, weight, dy = ex.tokens(64, 256, 8, 2)

    def step():
        y, kept = mlp.forward(x, choice, weight)
        return (y, *mlp.backward(dy, kept))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in range(3):
        for a, b in zip((x, choice, weight, dy), ex.tokens(64, 256, 8, 2, seed=seed + 5)):
            a.copy_(b)
        want = step()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
