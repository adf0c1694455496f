"""The float64 oracle of layer norm, SwiGLU and the ragged expert products: its gradients against torch's
float64 autograd and against differences, its MXFP8 rows against the whole-block quantizer."""
import numpy as np
import pytest
import torch

from oracle import block as ob
from oracle.mx import quantize_rowwise

D = torch.float64


def _rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("rows,cols,affine", [(1, 1, True), (3, 5, True), (4, 33, False), (7, 64, True)])
def test_layer_norm_against_autograd_and_differences(rows, cols, affine):
    r = _rng(rows * 100 + cols)
    x, dy = r.normal(size=(rows, cols)), r.normal(size=(rows, cols))
    w, b = (r.normal(size=cols), r.normal(size=cols)) if affine else (None, None)
    y, mean, rstd, xh = ob.layer_norm(x, w, b)
    dx, dw, db = ob.layer_norm_grads(dy, xh, rstd, w)
    tx = torch.tensor(x, requires_grad=True)
    tw = torch.tensor(np.ones(cols) if w is None else w, requires_grad=True)
    tb = torch.tensor(np.zeros(cols) if b is None else b, requires_grad=True)
    ty = torch.nn.functional.layer_norm(tx, (cols,), tw, tb, 1e-5)
    ty.backward(torch.tensor(dy))
    for a, t in ((y, ty.detach()), (dx, tx.grad), (dw, tw.grad), (db, tb.grad)):
        # float64 sums of at most 64 terms of order one, scaled by rstd (at most 1/sqrt(eps) = 316)
        np.testing.assert_allclose(a, t.numpy(), rtol=1e-9, atol=1e-10)
    v, h = r.normal(size=x.shape), 1e-5
    diff = ((ob.layer_norm(x + h * v, w, b)[0] - ob.layer_norm(x - h * v, w, b)[0]) * dy).sum() / (2 * h)
    # central difference: truncation h^2 |y'''| / 6 with derivatives up to rstd^3 (cols = 1: y is constant)
    assert abs(diff - (dx * v).sum()) <= 1e-4 * max(1.0, np.abs(dx).max()) * rows * cols


def test_swiglu_against_autograd_and_differences():
    r = _rng(1)
    g, u, dh = r.normal(size=(5, 9)), r.normal(size=(5, 9)), r.normal(size=(5, 9))
    tg, tu = torch.tensor(g, requires_grad=True), torch.tensor(u, requires_grad=True)
    th = torch.nn.functional.silu(tg) * tu
    th.backward(torch.tensor(dh))
    dg, du = ob.swiglu_grads(dh, g, u)
    np.testing.assert_allclose(ob.swiglu(g, u), th.detach().numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(dg, tg.grad.numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(du, tu.grad.numpy(), rtol=1e-12, atol=1e-13)
    h = 1e-5
    diff = ((ob.swiglu(g + h, u) - ob.swiglu(g - h, u)) / (2 * h)) * dh
    np.testing.assert_allclose(dg, diff, rtol=0, atol=1e-8 * 20)


def test_grouped_products_are_each_others_gradients():
    """The products are bilinear, so a difference over any step equals the gradient."""
    r = _rng(2)
    offs = [0, 3, 3, 8, 9]
    x, w, dy = r.normal(size=(9, 6)), r.normal(size=(4, 5, 6)), r.normal(size=(9, 5))
    vx, vw = r.normal(size=x.shape), r.normal(size=w.shape)
    base = (ob.grouped_fwd(x, w, offs) * dy).sum()
    np.testing.assert_allclose((ob.grouped_fwd(x + vx, w, offs) * dy).sum() - base,
                               (ob.grouped_dgrad(dy, w, offs) * vx).sum(), rtol=1e-11, atol=1e-11)
    np.testing.assert_allclose((ob.grouped_fwd(x, w + vw, offs) * dy).sum() - base,
                               (ob.grouped_wgrad(dy, x, offs) * vw).sum(), rtol=1e-11, atol=1e-11)
    assert np.all(ob.grouped_wgrad(dy, x, offs)[1] == 0)


def test_mx_rows_matches_the_block_quantizer_and_its_short_group():
    r = _rng(3)
    v = ob.bf16(r.normal(size=(6, 96)) * np.exp2(r.integers(-30, 30, size=(6, 1)).astype(float)))
    v[2, 32:64] = 0
    q, s = ob.mx_rows(v)
    rq, rs = quantize_rowwise(v)
    assert np.array_equal(q, rq) and np.array_equal(s, rs)
    q2, s2 = ob.mx_rows(v[:, :70])  # groups 0 and 1 are whole, the third has six elements
    assert np.array_equal(q2[:, :64], rq[:, :64]) and np.array_equal(s2[:, :2], rs[:, :2]) and s2.shape == (6, 3)
    err = np.abs(ob.mx_values(q2, s2) - v[:, :70])
    top = np.abs(v[:, 64:70]).max(1)
    # a code is within half a step (2^-4 of its value) or half the smallest step, 2^-10 of 2^e with
    # 2^e <= amax / 2^8, except above 448 x 2^e (up to amax = 512 x 2^e: an eighth)
    assert np.all(err[:, 64:70] <= np.maximum(np.abs(v[:, 64:70]) / 8, top[:, None] * 2.0 ** -18))
