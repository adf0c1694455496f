"""The expert block of examples/expert_block.py (every operator together) against a float64 block that rounds to
MXFP8 where the block keeps 8 bits, and nowhere else.

Tolerance, normwise: the block rounds to BF16 (2^-9 of a value in the mean square at most 2^-9, worst 2^-8) at
n, gu, h, yp and y forward, and at dyp, dh, dgu, h', dxp, dn and dx backward; errors of different elements are
independent, each stage passes them on with a factor of order one: at most 7 x 2^-8 = 0.027."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from gpu_util import require_gpu
from oracle import block as ob

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOL = 7 * 2.0 ** -8


def f64(t):
    return t.detach().double().cpu().numpy()


def load():
    spec = importlib.util.spec_from_file_location("expert_block", os.path.join(ROOT, "examples", "expert_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def near(got, ref, what):
    d = np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)
    assert d <= TOL, (what, d)


def reference(block, x, choice, weight, dy):
    nw, nb, w13, w2 = (f64(t) for t in (block.norm_w, block.norm_b, block.w13, block.w2))
    x, dy, p, choice = f64(x), f64(dy), f64(weight), choice.cpu().numpy()
    T, k = choice.shape
    F = w2.shape[2]
    n, _, rstd, xh = ob.layer_norm(x, nw, nb)
    order = np.argsort(choice.reshape(-1), kind="stable")  # rows: by expert, then by assignment
    offs = np.concatenate([[0], np.bincount(choice.reshape(-1), minlength=w13.shape[0]).cumsum()])
    tok = order // k
    xp = n[tok]
    gu = ob.grouped_fwd(xp, w13, offs)
    yp = ob.grouped_fwd(ob.swiglu(gu[:, :F], gu[:, F:]), w2, offs)
    pr = p.reshape(-1)[order][:, None]
    y = x.copy()
    np.add.at(y, tok, yp * pr)
    # backward from the 8-bit copies
    keep = lambda v: ob.mx_values(*ob.mx_rows(ob.bf16(v)))  # noqa: E731
    dyp = dy[tok] * pr
    dh = ob.grouped_dgrad(dyp, w2, offs)
    g, u = keep(gu[:, :F]), keep(gu[:, F:])
    dgu = np.concatenate(ob.swiglu_grads(dh, g, u), 1)
    dw2 = ob.grouped_wgrad(dyp, ob.swiglu(g, u), offs)
    dw13 = ob.grouped_wgrad(dgu, keep(xp), offs)
    dn = np.zeros_like(x)
    np.add.at(dn, tok, ob.grouped_dgrad(dgu, w13, offs))
    dx, dnw, dnb = ob.layer_norm_grads(dn, keep(xh), rstd, nw)
    return y, (dx + dy, dnw, dnb, dw13, dw2)


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,F,E,k", [(96, 128, 64, 8, 3), (33, 64, 96, 5, 2), (1, 256, 160, 16, 4)])
def test_block_against_float64(T, D, F, E, k):
    require_gpu()
    ex = load()
    block = ex.make(D, F, E)
    x, choice, weight, dy = ex.tokens(T, D, E, k)
    y, kept = block.forward(x, choice, weight)
    grads = block.backward(dy, kept)
    ry, rg = reference(block, x, choice, weight, dy)
    near(y, ry, "y")
    for name, a, b in zip(("dx", "dnorm_w", "dnorm_b", "dw13", "dw2"), grads, rg):
        near(a, b, name)
    near(block.forward(x, choice, weight, keep=False), ry, "y without keeping")

