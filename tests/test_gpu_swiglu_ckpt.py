"""SwiGLU with 8-bit checkpoints on the GPU against the float64 oracle.

Tolerances: the sigmoid comes from the hardware exponential and reciprocal (1 ulp each of FP32, and the
argument g log2(e) rounded, so 2^-23 |g| more in the exponent), a few FP32 products and one rounding to
BF16 (2^-8). (3 + |g|) 2^-22 bounds the FP32 part relative to the result's magnitude; the checkpoint's
bytes are those of the oracle."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu
from oracle import block as ob

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, mag, what):
    bad = ~(np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + mag * 2.0 ** -22 + 2.0 ** -126)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist())


def inputs(rows, F, seed, scale=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    gu = (torch.randn((rows, 2 * F), generator=g, device="cuda") * scale).bfloat16()
    return gu, torch.randn((rows, F), generator=g, device="cuda").bfloat16()


def check(mx, gu, dh, F):
    v, d = f64(gu), f64(dh)
    rows = v.shape[0]
    h, q, s = mx.swiglu_ckpt_fwd(gu)
    g, u = v[:, :F], v[:, F:]
    close(h, ob.swiglu(g, u), (3 + np.abs(g)) * np.abs(ob.swiglu(g, u)), "h")
    rq, rs = ob.mx_rows(v.reshape(2 * rows, F))
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    # the library's own decoder reads the checkpoint
    assert np.array_equal(f64(mx.dequantize(q, s, torch.float32)), ob.mx_values(rq, rs))
    dec = ob.mx_values(rq, rs).reshape(rows, 2 * F)
    g, u = dec[:, :F], dec[:, F:]
    dgu, h2 = mx.swiglu_ckpt_bwd(dh, q, s)
    dg, du = ob.swiglu_grads(d, g, u)
    sg = ob.sigmoid(g)
    # dg's two terms, sg and g sg (1 - sg), may cancel: the bound is on their magnitudes
    mg = np.abs(d * u) * (sg + np.abs(g) * sg * (1 - sg) + np.abs(g) * sg * 2.0 ** -2)
    close(dgu[:, :F], dg, (4 + np.abs(g)) * mg, "dg")
    close(dgu[:, F:], du, (3 + np.abs(g)) * np.abs(du), "du")
    close(h2, ob.swiglu(g, u), (3 + np.abs(g)) * np.abs(ob.swiglu(g, u)), "h again")
    only, none = mx.swiglu_ckpt_bwd(dh, q, s, recompute=False)
    assert none is None and torch.equal(only, dgu)


@pytest.mark.parametrize("rows,F", [(1, 1), (3, 2), (5, 8), (1, 31), (2, 32), (7, 33), (9, 40), (4, 77), (130, 96),
                                    (3, 1408), (2, 1411), (1, 8200), (5000, 16)])
def test_forward_and_backward(rows, F):
    mx = require_gpu()
    gu, dh = inputs(rows, F, rows * 31 + F)
    check(mx, gu, dh, F)


def test_wide_range_of_values():
    mx = require_gpu()
    gu, dh = inputs(64, 160, 3)
    e = torch.arange(64, device="cuda").float().sub(32).mul(0.5)[:, None]
    check(mx, (gu.float() * torch.exp2(e)).clamp(-80, 80).bfloat16(), dh, 160)
    z = torch.zeros_like(gu)
    check(mx, z, dh, 160)


def test_strided_rows_and_untouched_gaps():
    mx = require_gpu()
    for rows, F, pad in ((6, 64, 16), (6, 64, 5), (4, 37, 3)):
        gu, dh = inputs(rows, F, 8)
        wide = torch.full((rows, 2 * F + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :2 * F] = gu
        dwide = torch.full((rows, F + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        dwide[:, :F] = dh
        a, b = mx.swiglu_ckpt_fwd(gu), mx.swiglu_ckpt_fwd(wide[:, :2 * F])
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        p, r = mx.swiglu_ckpt_bwd(dh, a[1], a[2]), mx.swiglu_ckpt_bwd(dwide[:, :F], a[1], a[2])
        assert all(torch.equal(x, y) for x, y in zip(p, r))
        out = torch.full((rows, 2 * F + pad), 5.0, dtype=torch.bfloat16, device="cuda")
        ho = torch.full((rows, F + pad), 5.0, dtype=torch.bfloat16, device="cuda")
        mx.mxf_swiglu_ckpt_bwd(dh, F, a[1], a[2], rows, F, out, 2 * F + pad, ho, F + pad)
        assert torch.equal(out[:, :2 * F], p[0]) and torch.equal(ho[:, :F], p[1])
        assert bool((out[:, 2 * F:] == 5).all()) and bool((ho[:, F:] == 5).all())


def test_non_finite_groups_stay_in_their_groups():
    mx = require_gpu()
    F = 96
    gu, dh = inputs(4, F, 11)
    h0, q0, s0 = mx.swiglu_ckpt_fwd(gu)
    bad = gu.clone()
    bad[1, 40] = float("nan")    # gate, group 1
    bad[2, F + 5] = float("inf")  # up, group 0
    h, q, s = mx.swiglu_ckpt_fwd(bad)
    q, s, q0, s0 = (t.view(4, 2, -1) for t in (q, s, q0, s0))
    assert int((s == 255).sum()) == 2 and int(s[1, 0, 1]) == 255 and int(s[2, 1, 0]) == 255
    same = torch.ones_like(q, dtype=torch.bool)
    same[1, 0, 32:64] = False
    same[2, 1, :32] = False
    assert torch.equal(q[same], q0[same]) and bool(((q[~same] & 0x7F) == 0x7F).all())
    hs = torch.ones_like(h, dtype=torch.bool)
    hs[1, 40] = hs[2, 5] = False
    assert torch.equal(h[hs], h0[hs]) and bool(h[1, 40].isnan()) and bool(h[2, 5].isinf())


def test_no_rows_and_gradient_against_differences():
    mx = require_gpu()
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    h, q, s = mx.swiglu_ckpt_fwd(e)
    assert h.shape == (0, 32) and mx.swiglu_ckpt_bwd(h, q, s)[0].shape == (0, 64)
    # differences of the float64 forward at the decoded point: truncation 1e-10 x |h'''|, BF16 outputs
    gu, dh = inputs(3, 64, 5)
    _, q, s = mx.swiglu_ckpt_fwd(gu)
    dec = ob.mx_values(q.cpu().numpy(), s.cpu().numpy()).reshape(3, 128)
    g, u, d, t = dec[:, :64], dec[:, 64:], f64(dh), 1e-5
    dgu = f64(mx.swiglu_ckpt_bwd(dh, q, s)[0])
    dg = (ob.swiglu(g + t, u) - ob.swiglu(g - t, u)) / (2 * t) * d
    du = (ob.swiglu(g, u + t) - ob.swiglu(g, u - t)) / (2 * t) * d
    np.testing.assert_allclose(dgu[:, :64], dg, rtol=2.0 ** -8, atol=1e-6)
    np.testing.assert_allclose(dgu[:, 64:], du, rtol=2.0 ** -8, atol=1e-6)


def last_rows(mx, rows, F, bwd_rows=None):
    """The last rows of a large call are those of a call with them alone."""
    n = 4
    gu, dh = inputs(n, F, 17)
    one = mx.swiglu_ckpt_fwd(gu)
    big = torch.zeros((rows, 2 * F), dtype=torch.bfloat16, device="cuda")
    big[-n:] = gu
    h, q, s = mx.swiglu_ckpt_fwd(big)
    assert torch.equal(h[-n:], one[0]) and torch.equal(q[-2 * n:], one[1]) and torch.equal(s[-2 * n:], one[2])
    del big, h, q, s
    torch.cuda.empty_cache()
    rows = bwd_rows or rows
    q = torch.zeros((2 * rows, F), dtype=torch.uint8, device="cuda")
    s = torch.zeros((2 * rows, -(-F // 32)), dtype=torch.uint8, device="cuda")
    d = torch.zeros((rows, F), dtype=torch.bfloat16, device="cuda")
    q[-2 * n:], s[-2 * n:], d[-n:] = one[1], one[2], dh
    dgu, h = mx.swiglu_ckpt_bwd(d, q, s)
    dgu1, h1 = mx.swiglu_ckpt_bwd(dh, one[1], one[2])
    assert torch.equal(dgu[-n:], dgu1) and torch.equal(h[-n:], h1)
    assert not bool(dgu[:n].any()) and not bool(h[:n].any())
    del q, s, d, dgu, h
    torch.cuda.empty_cache()


@pytest.mark.parametrize("F", [7200, 7203])
def test_offsets_past_32_bits(F):
    mx = require_gpu()
    last_rows(mx, (1 << 31) // F + 100, F)


def test_more_chunks_than_a_launch_takes():
    mx = require_gpu()
    last_rows(mx, (1 << 29) + 1000, 1, (1 << 31) + 1000)


def test_same_bits_again_on_a_stream_and_in_a_graph():
    mx = require_gpu()
    gu, dh = inputs(300, 1411, 7)

    def step():
        h, q, s = mx.swiglu_ckpt_fwd(gu)
        return (h, q, s, *mx.swiglu_ckpt_bwd(dh, q, s))
    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mx.swiglu_ckpt_fwd(gu, stream=side)
    other = (*other, *mx.swiglu_ckpt_bwd(dh, *other[1:], stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        gu.copy_(inputs(300, 1411, 60 + k)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step())), k
