"""Layer norm on the GPU against the float64 oracle: widths from one column to rows that do not fit
registers, unaligned and strided rows, both element types, absent weights, checkpoints, rows with NaN.

Tolerances. With n = 128 bounding the roundings a register-path sum goes through (at most 32 in a thread,
6 in a wavefront, 16 across it; rows past 16384 columns: cols / 1024 + 22), a sum's error is at most
n 2^-24 times the sum of magnitudes. So xh is off by at most T (rstd mean|x| + |xh| + 1) with
T = 2 n 2^-24, y by |w| times that plus a rounding, and a BF16 result by 2^-8 of itself more."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu
from oracle import block as ob

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def slack(cols):
    return 2 * max(128, cols / 1024 + 22) * 2.0 ** -24


def close(got, ref, tol, what):
    """got within tol of ref, and one rounding to got's type more."""
    g = f64(got)
    extra = np.abs(ref) * (2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -23)
    bad = ~(np.abs(g - ref) <= tol + extra)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.abs(g - ref)[bad].max()))


def strided(t, pad, shift):
    """A copy of t whose rows have `pad` columns between them and start `shift` elements into a buffer."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + shift + 8,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] if rows else t
    v.copy_(t)
    return v


def problem(rows, cols, kind, wkind, seed):
    g = gen(seed)
    x = (randn(g, rows, cols) * torch.exp(0.5 * randn(g, rows, 1)) + 2.0 * randn(g, rows, 1)).to(TYPES[kind])
    dy = randn(g, rows, cols).to(TYPES[kind])
    w = b = None
    if wkind:
        w, b = (1 + 0.5 * randn(g, cols)).to(TYPES[wkind]), randn(g, cols).to(TYPES[wkind])
    return x, dy, w, b


SHAPES = [(1, 1), (3, 2), (5, 7), (4, 8), (9, 31), (2, 33), (130, 64), (6, 511), (7, 513), (3, 1024), (5, 1411),
          (11, 2048), (3, 2056), (2, 4100), (3, 8192), (2, 9000), (2, 16385), (2, 32768), (2, 33000), (5000, 40)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind,wkind", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", None)])
def test_forward_and_backward(rows, cols, kind, wkind):
    mx = require_gpu()
    x, dy, w, b = problem(rows, cols, kind, wkind, rows * 7 + cols)
    fw, fb = (None, None) if w is None else (f64(w), f64(b))
    y, mean, rstd = mx.layer_norm_fwd(x, w, b, eps=1e-5)
    ry, rmean, rrstd, rxh = ob.layer_norm(f64(x), fw, fb, 1e-5)
    T = slack(cols)
    ax = np.abs(f64(x)).mean(1)
    close(mean, rmean, T * ax, "mean")
    close(rstd, rrstd, T * rrstd * (1 + rrstd * ax), "rstd")
    txh = T * (rrstd * ax + 1)[:, None] + T * np.abs(rxh)
    close(y, ry, txh * (1.0 if w is None else np.abs(fw)) + 2.0 ** -22 * (np.abs(ry) + (0 if b is None else np.abs(fb))), "y")
    # the gradients, from the statistics that the kernel itself returned
    xh = (f64(x) - f64(mean)[:, None]) * f64(rstd)[:, None]
    check_grads(mx.layer_norm_bwd(dy, x, mean, rstd, w), f64(dy), xh, f64(rstd), fw, rows, cols,
                T * (f64(rstd) * ax + 1)[:, None] + T * np.abs(xh))


def check_grads(got, dy, xh, rstd, w, rows, cols, txh):
    dx, dw, db = got
    rdx, rdw, rdb = ob.layer_norm_grads(dy, xh, rstd, w)
    g = np.abs(dy * (1.0 if w is None else w))
    T = slack(cols)
    # |dx| <= rstd (|g| + mean|g| + |xh| mean|g xh|); each of the sums carries T, xh carries txh
    mg, mgx = g.mean(1, keepdims=True), (g * np.abs(xh)).mean(1, keepdims=True)
    tdx = rstd[:, None] * (T * (g + mg + np.abs(xh) * mgx) + txh * mgx + np.abs(xh) * (g * txh).mean(1, keepdims=True))
    close(dx, rdx, tdx, "dx")
    # column sums: at most rows / 4 + 44 additions in a chain (one block's rows, its wavefronts, the partial rows)
    C = (rows / 4 + 44) * 2.0 ** -24
    close(dw, rdw, C * np.abs(dy * xh).sum(0) + (np.abs(dy) * txh).sum(0), "dweight")
    close(db, rdb, C * np.abs(dy).sum(0), "dbias")


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_checkpoint(rows, cols, kind):
    mx = require_gpu()
    x, dy, w, b = problem(rows, cols, kind, kind, rows + 13 * cols)
    y, rstd, q, s = mx.layer_norm_ckpt_fwd(x, w, b)
    y2, _, rstd2 = mx.layer_norm_fwd(x, w, b)
    assert torch.equal(y, y2) and torch.equal(rstd, rstd2)  # the checkpoint changes nothing else
    # without weights y is xh: its BF16 rounding quantized by the oracle gives the same bytes
    rq, rs = ob.mx_rows(f64(mx.layer_norm_fwd(x, stats=False).bfloat16()))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    xh = ob.mx_values(rq, rs)
    T = slack(cols)
    check_grads(mx.layer_norm_ckpt_bwd(dy, q, s, rstd, w), f64(dy), xh, f64(rstd), f64(w), rows, cols, T * np.abs(xh))


@pytest.mark.parametrize("rows,cols", [(70, 1030), (1400, 1411), (7, 1536), (41, 2049), (600, 2304), (9, 2560), (13, 2561),
                                       (520, 2816), (3, 3000)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_widths_between_powers_of_two(rows, cols, kind):
    test_forward_and_backward(rows, cols, kind, kind)
    test_checkpoint(rows, cols, kind)


@pytest.mark.parametrize("rows,cols", [(700, 8200), (129, 9003), (260, 16392)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_many_long_rows(rows, cols, kind):
    test_forward_and_backward(rows, cols, kind, kind)
    test_checkpoint(rows, cols, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,shift", [(5, 64, 8, 0), (5, 64, 3, 0), (4, 96, 0, 1), (6, 2048, 24, 8), (3, 33000, 5, 3)])
def test_strides_and_offsets_give_the_same_bits(rows, cols, pad, shift, kind):
    mx = require_gpu()
    x, dy, w, b = problem(rows, cols, kind, kind, 5)
    xs, dys = strided(x, pad, shift), strided(dy, pad, shift)
    a, c = mx.layer_norm_fwd(x, w, b), mx.layer_norm_fwd(xs, w, b)
    for p, r in zip(a, c):
        # sums run in another order where the rows' alignment decides the elements a thread owns
        close(p, f64(r), 2.0 ** -18 * (1 + np.abs(f64(r))), "strided forward")
    ga, gc = mx.layer_norm_bwd(dy, x, a[1], a[2], w), mx.layer_norm_bwd(dys, xs, a[1], a[2], w)
    for p, r in zip(ga, gc):
        close(p, f64(r), 2.0 ** -17 * (1 + np.abs(f64(r))), "strided backward")


def test_outputs_stay_inside_their_rows_and_in_place_is_allowed():
    mx = require_gpu()
    rows, cols, pad = 7, 72, 24
    x, dy, w, b = problem(rows, cols, "bf16", "bf16", 9)
    y, mean, rstd = mx.layer_norm_fwd(x, w, b)
    dx, dw, db = mx.layer_norm_bwd(dy, x, mean, rstd, w)
    big = torch.full((rows, cols + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    d = mx.NormDesc(rows, cols, cols, cols + pad, cols + pad, 1e-5, 0)
    mx.mxf_layer_norm_fwd(d, x, w, b, big, None, None, None, None)
    assert torch.equal(big[:, :cols], y) and bool((big[:, cols:] == 7.0).all())
    inplace = x.clone()
    mx.mxf_layer_norm_fwd(mx.NormDesc(rows, cols, cols, cols, cols, 1e-5, 0), inplace, w, b, inplace, None, None, None, None)
    assert torch.equal(inplace, y)
    g = dy.clone()
    mx.mxf_layer_norm_bwd(mx.NormDesc(rows, cols, cols, cols, cols, 0.0, 0), g, x, None, None, mean, rstd, w, g, None,
                          None, None)
    assert torch.equal(g, dx)


@pytest.mark.parametrize("cols", [40, 2048, 2051, 33000])
def test_a_bad_row_touches_no_other(cols):
    mx = require_gpu()
    x, dy, w, b = problem(6, cols, "bf16", "bf16", 3)
    good = mx.layer_norm_ckpt_fwd(x, w, b)
    bad = x.clone()
    bad[1, cols // 2] = float("nan")
    bad[4, 0] = float("inf")
    y, rstd, q, s = mx.layer_norm_ckpt_fwd(bad, w, b)
    keep = [0, 2, 3, 5]
    for a, c in zip((y, rstd, q, s), good):
        assert torch.equal(a[keep], c[keep])
    assert bool(y[[1, 4]].isnan().all()) and bool((s[[1, 4]] == 255).all())
    assert bool(((q[[1, 4]] & 0x7F) == 0x7F).all())
    dx, _, _ = mx.layer_norm_ckpt_bwd(dy, q, s, rstd, w)
    dx0, _, _ = mx.layer_norm_ckpt_bwd(dy, good[2], good[3], good[1], w)
    assert torch.equal(dx[keep], dx0[keep]) and bool(dx[[1, 4]].isnan().all())


def test_constant_and_large_mean_rows():
    mx = require_gpu()
    x = torch.full((3, 1000), 250.0, device="cuda")
    y, mean, rstd = mx.layer_norm_fwd(x, eps=1e-5)
    assert bool((y == 0).all()) and bool((mean == 250.0).all())
    close(rstd, np.full(3, 1e-5 ** -0.5), 1e-4, "rstd")
    g = gen(1)
    x = 1000.0 + randn(g, 4, 2048)  # the centred second pass keeps the variance
    y, mean, rstd = mx.layer_norm_fwd(x)
    ry = ob.layer_norm(f64(x))[0]
    close(y, ry, slack(2048) * 1001 * 1.1, "y")


def test_no_rows():
    mx = require_gpu()
    x = torch.empty((0, 48), dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = mx.layer_norm_fwd(x)
    dx, dw, db = mx.layer_norm_bwd(x, x, mean, rstd)
    assert y.shape == (0, 48) and dx.shape == (0, 48)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_gradient_against_differences():
    """(L(x + h v) - L(x - h v)) / 2h of the float64 forward, L = sum y dy, against <dx, v>: truncation is
    h^2 / 6 of third derivatives of order sum |dy| rstd^3 < 1e4 here, and dx carries 1e-4 of its norm."""
    mx = require_gpu()
    x, dy, w, b = problem(9, 300, "f32", "f32", 21)
    _, mean, rstd = mx.layer_norm_fwd(x, w, b)
    dx, dw, db = (f64(t) for t in mx.layer_norm_bwd(dy, x, mean, rstd, w))
    r, h = np.random.default_rng(0), 1e-5
    v, vw = r.normal(size=(9, 300)), r.normal(size=300)
    L = lambda a, c: (ob.layer_norm(a, c, f64(b))[0] * f64(dy)).sum()  # noqa: E731
    num = (L(f64(x) + h * v, f64(w)) - L(f64(x) - h * v, f64(w))) / (2 * h)
    assert abs(num - (dx * v).sum()) <= 1e-4 * np.linalg.norm(dx) * np.linalg.norm(v) / 50 + 1e-5
    num = (L(f64(x), f64(w) + h * vw) - L(f64(x), f64(w) - h * vw)) / (2 * h)
    assert abs(num - (dw * vw).sum()) <= 1e-5 * np.linalg.norm(dw) * np.linalg.norm(vw)
    np.testing.assert_allclose(db, f64(dy).sum(0), atol=1e-5)


def test_same_bits_again_and_on_another_stream():
    mx = require_gpu()
    x, dy, w, b = problem(3000, 1024, "bf16", "bf16", 2)
    _, mean, rstd = mx.layer_norm_fwd(x, w, b)
    first = mx.layer_norm_bwd(dy, x, mean, rstd, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mx.layer_norm_bwd(dy, x, mean, rstd, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    again = mx.layer_norm_bwd(dy, x, mean, rstd, w)
    for a, c, d in zip(first, other, again):
        assert torch.equal(a, c) and torch.equal(a, d)


def test_graph_replays():
    mx = require_gpu()
    x, dy, w, b = problem(200, 1024, "bf16", "bf16", 4)

    def step():
        y, rstd, q, s = mx.layer_norm_ckpt_fwd(x, w, b)
        return (y, *mx.layer_norm_ckpt_bwd(dy, q, s, rstd, w))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(problem(200, 1024, "bf16", None, 50 + k)[0])
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(out, step()):
            assert torch.equal(a, c), k


@pytest.mark.parametrize("base", [0, 480, 1376, 2976, 5120, 9984])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_last_group_of_every_length(base, kind):
    """Checkpoints byte for byte where the last group of 32 is short: ends on whole 16-byte chunks and inside one,
    for each number of threads that a row takes. The group's largest value visits every place in it."""
    mx = require_gpu()
    for rem in [r for r in range(4, 32, 4)] + [3, 13, 27, 31]:
        rows, cols = 8 * rem, base + rem
        x = problem(rows, cols, kind, None, base + rem)[0]
        r = torch.arange(rows, device="cuda")
        x[r, base + r % rem] = 12.0 * (1 + x[r, base + r % rem].abs())
        _, rstd, q, s = mx.layer_norm_ckpt_fwd(x)
        y, _, rstd2 = mx.layer_norm_fwd(x)
        rq, rs = ob.mx_rows(f64(y.bfloat16()))
        bad = [int(v) for v in ((s.cpu().numpy() != rs).any(1).sum(), (q.cpu().numpy() != rq).any(1).sum())]
        assert bad == [0, 0] and torch.equal(rstd, rstd2), (cols, "rows with wrong scales, codes", bad)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,shift", [(5, 64, 3, 1), (9, 24, 8, 0), (40, 1411, 5, 3), (33, 1536, 1, 0), (33, 2560, 7, 1),
                                                 (33, 3064, 0, 3), (33, 3071, 2, 0), (300, 8200, 3, 1), (30, 16400, 1, 5)])
def test_strides_and_alignment_change_no_bit(rows, cols, pad, shift, kind):
    """The columns a thread owns and the order of its sums are the width's alone."""
    mx = require_gpu()
    x, dy, w, b = problem(rows, cols, kind, kind, cols)
    xs, dys = strided(x, pad, shift), strided(dy, pad, shift)
    y, mean, rstd = mx.layer_norm_fwd(x, w, b)
    _, _, q, s = a = mx.layer_norm_ckpt_fwd(x, w, b)
    pairs = [((y, mean, rstd), mx.layer_norm_fwd(xs, w, b)), (a, mx.layer_norm_ckpt_fwd(xs, w, b)),
             (mx.layer_norm_bwd(dy, x, mean, rstd, w), mx.layer_norm_bwd(dys, xs, mean, rstd, w)),
             (mx.layer_norm_ckpt_bwd(dy, q, s, rstd, w), mx.layer_norm_ckpt_bwd(dys, q, s, rstd, w))]
    for i, (p, r) in enumerate(pairs):
        assert all(torch.equal(u, v) for u, v in zip(p, r)), i


@pytest.mark.parametrize("rows,cols", [(1536000, 2816), (300000, 14400), (131100, 32800)])
def test_offsets_past_32_bits(rows, cols):
    """Codes past 2^32 bytes, rows of x, y, dy and dx past 2^33: the last rows are those of a call with them alone."""
    mx = require_gpu()
    n = 8
    x, dy, w, b = problem(n, cols, "bf16", "bf16", 6)
    assert (rows - n) * cols > 1 << 32
    big = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    big[-n:] = x
    y, rstd, q, s = mx.layer_norm_ckpt_fwd(big, w, b)
    y1, rstd1, q1, s1 = mx.layer_norm_ckpt_fwd(x, w, b)
    assert all(torch.equal(u[-n:], v) for u, v in ((y, y1), (rstd, rstd1), (q, q1), (s, s1)))
    mean1 = mx.layer_norm_fwd(x, w, b)[1]
    mean = torch.zeros(rows, device="cuda")
    mean[-n:] = mean1
    del y
    g = torch.zeros_like(big)
    g[-n:] = dy
    assert torch.equal(mx.layer_norm_ckpt_bwd(g, q, s, rstd, w)[0][-n:], mx.layer_norm_ckpt_bwd(dy, q1, s1, rstd1, w)[0])
    assert torch.equal(mx.layer_norm_bwd(g, big, mean, rstd, w)[0][-n:], mx.layer_norm_bwd(dy, x, mean1, rstd1, w)[0])
    del big, g, q, s
    torch.cuda.empty_cache()
