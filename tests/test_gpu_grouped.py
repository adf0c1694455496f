"""Ragged expert products on the GPU against float64 products of the same BF16 numbers.

Tolerance per element: FP32 accumulation over n terms is off by at most n 2^-23 of the sum of magnitudes
(2^-23: the matrix cores' additions need not round to nearest), and BF16 outputs by 2^-8 of themselves."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu
from oracle import block as ob

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, mag, n, what):
    g = f64(got)
    tol = n * 2.0 ** -23 * mag + np.abs(ref) * (2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -23)
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(np.abs(g - ref))))


def problem(counts, N, K, seed, tail=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    offs = [0] + np.cumsum(counts).tolist()
    M = offs[-1] + tail
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return offs, torch.tensor(offs, dtype=torch.int32, device="cuda"), r(M, K), r(len(counts), N, K), r(M, N)


def reference(x, w, dy, offs):
    """The three products and the same of magnitudes, in float64 on the GPU's float64 units."""
    X, W, G = x.double(), w.double(), dy.double()

    def three(X, W, G):
        seg = list(zip(offs[:-1], offs[1:]))
        y = torch.zeros((X.shape[0], W.shape[1]), dtype=torch.float64, device="cuda")
        dx = torch.zeros_like(X)
        dw = torch.zeros_like(W)
        for e, (a, b) in enumerate(seg):
            y[a:b] = X[a:b] @ W[e].t()
            dx[a:b] = G[a:b] @ W[e]
            dw[e] = G[a:b].t() @ X[a:b]
        return [t.cpu().numpy() for t in (y, dx, dw)]
    return three(X, W, G), three(X.abs(), W.abs(), G.abs())


def check_all(counts, N, K, seed, out=torch.bfloat16):
    mx = require_gpu()
    offs, toffs, x, w, dy = problem(counts, N, K, seed)
    (y, dx, dw), (my, mdx, mdw) = reference(x, w, dy, offs)
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    close(mx.grouped_gemm_fwd(x, w, toffs, out_dtype=out, status=st), y, my, K, "fwd")
    assert int(st) == mx.DEV_OK
    close(mx.grouped_gemm_dgrad(dy, w, toffs, out_dtype=out, status=st), dx, mdx, N, "dgrad")
    assert int(st) == mx.DEV_OK
    close(mx.grouped_gemm_wgrad(dy, x, toffs, out_dtype=out, status=st), dw, mdw, max(counts), "wgrad")
    assert int(st) == mx.DEV_OK
    # from the 8-bit checkpoint of x, decoded exactly
    xf = ob.mx_rows(f64(x))
    q, s = (torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in xf)
    xd = torch.from_numpy(ob.mx_values(*xf)).cuda()
    rd = np.stack([(dy[a:b].double().t() @ xd[a:b]).cpu().numpy() for a, b in zip(offs[:-1], offs[1:])])
    md = np.stack([(dy[a:b].double().abs().t() @ xd[a:b].abs()).cpu().numpy() for a, b in zip(offs[:-1], offs[1:])])
    close(mx.grouped_gemm_wgrad(dy, (q, s), toffs, out_dtype=out), rd, md, max(counts), "wgrad of codes")


CASES = [
    ([1], 1, 1), ([1], 8, 8), ([3, 0, 2], 16, 24), ([0, 0, 5], 7, 13), ([1, 1, 1, 1], 64, 64),
    ([17, 0, 130, 1], 96, 160), ([64, 65, 63], 128, 64), ([200], 264, 72), ([129, 127], 130, 128),
    ([5, 9, 0, 31, 1, 2, 8, 7], 256, 512), ([300, 1, 0, 513], 320, 96), ([33, 300], 77, 101),
    ([256, 512], 512, 256), ([1000], 520, 1032), ([2] * 70, 40, 48), ([0] * 66 + [9, 0, 100], 48, 40),
]


@pytest.mark.parametrize("counts,N,K", CASES)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_products(counts, N, K, out):
    check_all(counts, N, K, sum(counts) + N + K, out)


@pytest.mark.parametrize("counts,N,K", [([0, 3, 1, 0] * 256, 40, 48), ([0] * 1023 + [150], 40, 48), ([20, 0, 13, 30] * 256, 24, 40),
                                        ([1] * 1024, 33, 17)])
def test_a_thousand_experts(counts, N, K):
    check_all(counts, N, K, 1024)


@pytest.mark.parametrize("counts,N,K", [([700, 0, 1400, 260, 1, 2000], 1408, 768), ([1900, 333], 1000, 2056),
                                        ([40, 11, 0, 90], 2816, 2048)])
def test_larger_products(counts, N, K):
    check_all(counts, N, K, 77)


@pytest.mark.parametrize("counts,N,K", [
    ([5000, 0, 3000, 130, 3900, 1], 2816, 192),  # 550 tiles of 256 x 256: the last 38 run as quarters
    ([9000], 2560, 136),                         # 360: the last 104 as halves
    ([4000, 100, 257, 4643], 2560, 64),          # 370: no split; an expert that ends in a tile's first half
    ([5000, 0, 3000, 130, 3900, 1], 2811, 197),  # the same, rows of any alignment
    ([9000], 2555, 131)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_large_tiles(counts, N, K, out):
    """Row counts that fill the chip with the largest tiles, in the forward and (N, K exchanged) the input
    gradient."""
    mx = require_gpu()
    offs, toffs, x, w, dy = problem(counts, N, K, N)
    (y, _, _), (my, _, _) = reference(x, w, dy, offs)
    close(mx.grouped_gemm_fwd(x, w, toffs, out_dtype=out), y, my, K, "fwd")
    del y, my
    offs, toffs, x, w, dy = problem(counts, K, N, N + 1)
    (_, dx, _), (_, mdx, _) = reference(x, w, dy, offs)
    close(mx.grouped_gemm_dgrad(dy, w, toffs, out_dtype=out), dx, mdx, K, "dgrad")


@pytest.mark.parametrize("counts,tail", [([1000, 0, 900, 300], 0), ([2304], 0), ([130, 0, 100, 7], 1963), ([0, 0, 600, 3], 1600)])
@pytest.mark.parametrize("N,K", [(4600, 72), (4599, 71)])
def test_less_than_a_round_of_large_tiles(counts, tail, N, K):
    """Fewer large tiles than compute units, and a capacity of rows that is mostly not used: what is there runs
    whole, as halves or as quarters."""
    mx = require_gpu()
    for n, k, op in ((N, K, mx.grouped_gemm_fwd), (K, N, mx.grouped_gemm_dgrad)):
        offs, toffs, x, w, dy = problem(counts, n, k, n, tail)
        (y, dx, _), (my, mdx, _) = reference(x, w, dy, offs)
        fwd = op is mx.grouped_gemm_fwd
        got = op(x if fwd else dy, w, toffs)
        end = offs[-1]
        close(got[:end], (y if fwd else dx)[:end], (my if fwd else mdx)[:end], K, "product")


@pytest.mark.parametrize("counts,N,K", [([100, 0, 333, 64, 1, 70], 1500, 2000), ([100, 0, 333, 64, 1, 70], 1501, 1999),
                                        ([65] * 5 + [0] * 63, 400, 504)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_large_weight_gradients(counts, N, K, out):
    """More output tiles than compute units, from BF16 rows and from codes; and more than 64 experts."""
    mx = require_gpu()
    offs, toffs, x, w, dy = problem(counts, N, K, 5)
    (_, _, dw), (_, _, mdw) = reference(x, w, dy, offs)
    close(mx.grouped_gemm_wgrad(dy, x, toffs, out_dtype=out), dw, mdw, max(counts), "wgrad")
    q, s = ob.mx_rows(f64(x))
    xd = torch.from_numpy(ob.mx_values(q, s)).cuda()
    (_, _, dw), (_, _, mdw) = reference(xd, w, dy, offs)
    q, s = torch.from_numpy(np.ascontiguousarray(q)).cuda(), torch.from_numpy(s).cuda()
    close(mx.grouped_gemm_wgrad(dy, (q, s), toffs, out_dtype=out), dw, mdw, max(counts), "wgrad of codes")


@pytest.mark.parametrize("counts,N,K", [
    ([0, 1, 15, 16, 17, 31, 33, 48, 63, 64, 65, 127, 128, 129, 200, 7] * 4, 768, 784),  # 64 experts of 42 tiles of 128
    ([3, 0, 70, 16, 1, 0, 130] * 30, 264, 520)])                                      # 210 of 15, by index
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_weight_gradients_of_many_tiles_and_few_rows_each(counts, N, K, out):
    """Thousands of output tiles, from BF16 rows and from codes; a non-finite row stays in its expert; sums join
    those that are there; bad offsets."""
    mx = require_gpu()
    offs, toffs, x, w, dy = problem(counts, N, K, 6)
    (_, _, dw), (_, _, mdw) = reference(x, w, dy, offs)
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    got = mx.grouped_gemm_wgrad(dy, x, toffs, out_dtype=out, status=st)
    assert int(st) == mx.DEV_OK
    close(got, dw, mdw, max(counts), "wgrad")
    if out == torch.float32:
        acc = torch.randn(got.shape, device="cuda")
        start = f64(acc)
        mx.grouped_gemm_wgrad(dy, x, toffs, accumulate=acc)
        close(acc, start + dw, mdw + np.abs(start), max(counts), "accumulate")
    e = 13  # an expert with rows, between others
    dy2 = dy.clone()
    dy2[offs[e]] = float("inf")
    bad = mx.grouped_gemm_wgrad(dy2, x, toffs, out_dtype=out)
    keep = [i for i in range(len(counts)) if i != e]
    assert not bool(bad[e].isfinite().any()) and torch.equal(bad[keep], got[keep])
    q, s = ob.mx_rows(f64(x))
    xd = torch.from_numpy(ob.mx_values(q, s)).cuda()
    (_, _, dw), (_, _, mdw) = reference(xd, w, dy, offs)
    q, s = torch.from_numpy(np.ascontiguousarray(q)).cuda(), torch.from_numpy(s).cuda()
    close(mx.grouped_gemm_wgrad(dy, (q, s), toffs, out_dtype=out), dw, mdw, max(counts), "wgrad of codes")
    toffs[5] = offs[-1] + 1
    kept = torch.full(got.shape, 3.0, dtype=out, device="cuda")
    d = mx.GroupedDesc(len(counts), mx.GROUPED_OUT_F32 if out == torch.float32 else 0, offs[-1], N, K, K, N)
    mx.mxf_grouped_gemm_wgrad(d, toffs, dy, x, None, None, kept, st)
    assert int(st) == mx.DEV_BAD_OFFSETS and bool((kept == 3).all())


@pytest.mark.parametrize("N,K", [(64, 512), (63, 257)])
def test_every_code_and_scale_enters_the_product_unrounded(N, K):
    """dy = the identity: dw[n, k] is the decoded x[n, k] itself. Scales that keep a code's value a normal BF16
    number (from 2^-117: the smallest code is 2^-9)."""
    mx = require_gpu()
    r = np.random.default_rng(1)
    q = r.integers(0, 256, size=(N, K)).astype(np.uint8)
    q[(q & 0x7F) == 0x7F] = 0  # NaN codes: below
    s = r.integers(10, 246, size=(N, -(-K // 32))).astype(np.uint8)
    dy = torch.eye(N, dtype=torch.bfloat16, device="cuda")
    offs = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    tq, ts = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    got = mx.grouped_gemm_wgrad(dy, (tq, ts), offs, out_dtype=torch.float32)
    assert np.array_equal(f64(got)[0], ob.mx_values(q, s))
    # a NaN scale and a NaN code: NaN in the columns of its group (0 x NaN), in its column, in no other
    ts[5, 2] = 255
    tq[9, 40] = 0x7F
    tq[5, 64:96] = 0x12
    bad = mx.grouped_gemm_wgrad(dy, (tq, ts), offs, out_dtype=torch.float32)[0].isnan()
    want = torch.zeros_like(bad)
    want[:, 64:96] = True
    want[:, 40] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 64, 65, 100])
def test_few_rows_in_one_expert_of_many(rows):
    """Serving: a handful of rows, all in one expert or one each."""
    mx = require_gpu()
    for counts in ([0, rows, 0, 0], [1] * min(rows, 8) + [rows - min(rows, 8)]):
        offs, toffs, x, w, dy = problem(counts, 200, 328, rows)
        (y, _, _), (my, _, _) = reference(x, w, dy, offs)
        for out in (torch.bfloat16, torch.float32):
            close(mx.grouped_gemm_fwd(x, w, toffs, out_dtype=out), y, my, 328, "fwd")


@pytest.mark.parametrize("K,pad,shift", [(8, 0, 0), (10, 2, 0), (330, 0, 0), (1788, 4, 2), (334, 1, 0), (328, 0, 2), (326, 0, 1)])
def test_few_rows_at_any_alignment(K, pad, shift):
    """Rows of any even or odd alignment, NaN around them."""
    mx = require_gpu()
    offs, toffs, x, w, dy = problem([0, 3, 0, 17, 1, 9], 72, K, K)
    (y, _, _), (my, _, _) = reference(x, w, dy, offs)
    buf = torch.full((30 * (K + pad) + 16,), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = buf[shift:shift + 30 * (K + pad)].view(30, K + pad)[:, :K]
    v.copy_(x)
    wb = torch.full((w.numel() + 16,), float("nan"), dtype=torch.bfloat16, device="cuda")
    wv = wb[shift:shift + w.numel()].view(w.shape)
    wv.copy_(w)
    for out in (torch.bfloat16, torch.float32):
        close(mx.grouped_gemm_fwd(v, wv, toffs, out_dtype=out), y, my, K, "fwd")
    v[5] = float("inf")  # a row of its expert alone
    bad = ~mx.grouped_gemm_fwd(v, wv, toffs).isfinite()
    assert bool(bad[5].all()) and not bool(bad[:5].any()) and not bool(bad[6:].any())


def test_rows_past_the_segments_are_neither_read_nor_written():
    mx = require_gpu()
    for N, K in ((96, 160), (77, 101)):
        offs, toffs, x, w, dy = problem([40, 0, 131], N, K, 5, tail=70)
        (y, dx, dw), (my, mdx, mdw) = reference(x, w, dy, offs)
        end = offs[-1]
        x[end:] = float("nan")
        dy[end:] = float("nan")
        d = mx.GroupedDesc(3, 0, x.shape[0], N, K, K, N)
        out = torch.full((x.shape[0], N), 3.0, dtype=torch.bfloat16, device="cuda")
        mx.mxf_grouped_gemm_fwd(d, toffs, x, w, out)
        close(out[:end], y[:end], my[:end], K, "fwd")
        assert bool((out[end:] == 3.0).all())
        out = torch.full((x.shape[0], K), 3.0, dtype=torch.bfloat16, device="cuda")
        mx.mxf_grouped_gemm_dgrad(d, toffs, dy, w, out)
        close(out[:end], dx[:end], mdx[:end], N, "dgrad")
        assert bool((out[end:] == 3.0).all())
        close(mx.grouped_gemm_wgrad(dy, x, toffs), dw, mdw, 131, "wgrad")


@pytest.mark.parametrize("N,K", [(96, 160), (77, 101), (264, 320)])
def test_non_finite_rows_stay_in_their_experts(N, K):
    """A NaN in one expert's rows or weight reaches only what the formulas let it reach."""
    mx = require_gpu()
    offs, toffs, x, w, dy = problem([37, 91, 20], N, K, 6)
    base = [mx.grouped_gemm_fwd(x, w, toffs), mx.grouped_gemm_dgrad(dy, w, toffs), mx.grouped_gemm_wgrad(dy, x, toffs)]
    x2, dy2, w2 = x.clone(), dy.clone(), w.clone()
    x2[50], dy2[60], w2[0, 3] = float("nan"), float("inf"), float("nan")
    y, dx, dw = (mx.grouped_gemm_fwd(x2, w2, toffs), mx.grouped_gemm_dgrad(dy2, w2, toffs),
                 mx.grouped_gemm_wgrad(dy2, x2, toffs))
    bad = y.isnan()
    want = torch.zeros_like(bad)
    want[50] = True
    want[:37, 3] = True
    assert torch.equal(bad, want) and torch.equal(y[~want], base[0][~want])
    keep = [i for i in range(37, 148) if i != 60]
    assert bool(dx[:37].isnan().all()) and torch.equal(dx[keep], base[1][keep]) and not bool(dx[60].isfinite().any())
    assert not bool(dw[1].isfinite().any()) and torch.equal(dw[[0, 2]], base[2][[0, 2]])


def test_strided_rows():
    mx = require_gpu()
    for N, K, pad in ((96, 160, 16), (96, 160, 3), (130, 72, 8)):
        offs, toffs, x, w, dy = problem([30, 0, 150], N, K, 8)
        xs = torch.full((180, K + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        ds = torch.full((180, N + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        xs[:, :K], ds[:, :N] = x, dy
        (y, dx, dw), (my, mdx, mdw) = reference(x, w, dy, offs)
        close(mx.grouped_gemm_fwd(xs[:, :K], w, toffs), y, my, K, "fwd")
        close(mx.grouped_gemm_dgrad(ds[:, :N], w, toffs), dx, mdx, N, "dgrad")
        close(mx.grouped_gemm_wgrad(ds[:, :N], xs[:, :K], toffs), dw, mdw, 150, "wgrad")
        out = torch.full((180, N + pad), 2.0, dtype=torch.bfloat16, device="cuda")
        mx.mxf_grouped_gemm_fwd(mx.GroupedDesc(3, 0, 180, N, K, K, N + pad), toffs, x, w, out)
        close(out[:, :N], y, my, K, "strided output")
        assert bool((out[:, N:] == 2.0).all())


@pytest.mark.parametrize("N,K", [(96, 160), (51, 33)])
def test_accumulation_and_empty_experts(N, K):
    mx = require_gpu()
    offs, toffs, x, w, dy = problem([12, 0, 70], N, K, 9)
    (_, _, dw), (_, _, mdw) = reference(x, w, dy, offs)
    acc = torch.randn((3, N, K), device="cuda")
    start = f64(acc)
    got = mx.grouped_gemm_wgrad(dy, x, toffs, accumulate=acc)
    assert got is acc
    close(acc, start + dw, mdw + np.abs(start), 70, "accumulate")
    assert np.array_equal(f64(acc)[1], start[1])
    fresh = mx.grouped_gemm_wgrad(dy, x, toffs)
    assert bool((fresh[1] == 0).all())
    # no rows at all
    e = torch.empty((0, N), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert bool((mx.grouped_gemm_wgrad(e, e.new_empty((0, K)), z) == 0).all())
    assert mx.grouped_gemm_fwd(e.new_empty((0, K)), w, z).shape == (0, N)


@pytest.mark.parametrize("N,K", [(96, 160), (77, 101)])
@pytest.mark.parametrize("offs", [[1, 5, 10, 20], [0, 12, 10, 20], [0, 5, 10, 21], [0, -3, 10, 20], [0, 5, 10, -1],
                                  [-2147483648, 2147483647, 5, 20]])
def test_bad_offsets_write_nothing_and_say_so(offs, N, K):
    mx = require_gpu()
    _, _, x, w, dy = problem([20], N, K, 4)
    w = w.expand(3, N, K).contiguous()
    t = torch.tensor(offs, dtype=torch.int32, device="cuda")
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    d = mx.GroupedDesc(3, 0, 20, N, K, K, N)
    y = torch.full((20, N), 3.0, dtype=torch.bfloat16, device="cuda")
    mx.mxf_grouped_gemm_fwd(d, t, x, w, y, st)
    assert int(st) == mx.DEV_BAD_OFFSETS and bool((y == 3).all())
    st.fill_(-1)
    dx = torch.full((20, K), 3.0, dtype=torch.bfloat16, device="cuda")
    mx.mxf_grouped_gemm_dgrad(d, t, dy, w, dx, st)
    assert int(st) == mx.DEV_BAD_OFFSETS and bool((dx == 3).all())
    st.fill_(-1)
    dw = torch.full((3, N, K), 3.0, dtype=torch.bfloat16, device="cuda")
    mx.mxf_grouped_gemm_wgrad(d, t, dy, x, None, None, dw, st)
    assert int(st) == mx.DEV_BAD_OFFSETS and bool((dw == 3).all())


def test_offsets_past_32_bits():
    """Rows whose byte offset passes 2^32: only the last rows are used, through a view of a wide buffer."""
    mx = require_gpu()
    K, N, ld = 64, 64, 1 << 20
    rows = 2100  # 2100 x 2^20 elements: 4.4 GB
    buf = torch.zeros(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(rows, ld)[:, :K]
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x.copy_(torch.randn((rows, K), generator=g, device="cuda"))
    offs = [0, 1500, 2100]
    toffs = torch.tensor(offs, dtype=torch.int32, device="cuda")
    w = torch.randn((2, N, K), generator=g, device="cuda").bfloat16()
    dy = torch.randn((rows, N), generator=g, device="cuda").bfloat16()
    xc = x.contiguous()
    (y, _, dw), (my, _, mdw) = reference(xc, w, dy, offs)
    close(mx.grouped_gemm_fwd(x, w, toffs), y, my, K, "fwd")
    close(mx.grouped_gemm_wgrad(dy, x, toffs), dw, mdw, 1500, "wgrad")


def test_same_bits_again_on_a_stream_and_in_a_graph():
    mx = require_gpu()
    offs, toffs, x, w, dy = problem([100, 0, 300, 57], 264, 320, 12)

    def step():
        return mx.grouped_gemm_fwd(x, w, toffs), mx.grouped_gemm_dgrad(dy, w, toffs), mx.grouped_gemm_wgrad(dy, x, toffs)
    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mx.grouped_gemm_wgrad(dy, x, toffs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, first[2])
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(problem([100, 0, 300, 57], 264, 320, 90 + k)[2])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step())), k


@pytest.mark.parametrize("N,K", [(96, 160), (77, 101)])
def test_the_stride_of_x_is_not_used_with_codes(N, K):
    mx = require_gpu()
    offs, toffs, x, _, dy = problem([30, 0, 150], N, K, 3)
    q, s = (torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in ob.mx_rows(f64(x)))
    want = mx.grouped_gemm_wgrad(dy, (q, s), toffs)
    for ldx in (0, -1, 1 << 40):
        dw = torch.full_like(want, 3.0)
        mx.mxf_grouped_gemm_wgrad(mx.GroupedDesc(3, 0, offs[-1], N, K, ldx, N), toffs, dy, None, q, s, dw)
        assert torch.equal(dw, want), ldx


@pytest.mark.parametrize("E,e,rows,N,K", [(256, 200, 2000, 264, 520), (32, 20, 4000, 1032, 1024), (32, 31, 4001, 1025, 1023)])
def test_all_rows_in_one_expert(E, e, rows, N, K):
    """A collapsed router, where few rows per expert on average choose the kernel."""
    check_all([0] * e + [rows] + [0] * (E - 1 - e), N, K, E)


def test_few_rows_among_many_experts():
    """The forward where every block looks for its expert past the first 64, and counts, widths and lengths on either
    side of the choice between blocks of few rows and tiles."""
    mx = require_gpu()
    for E, M, N, K, out in [(1024, 8, 200, 1024, torch.bfloat16), (300, 7, 128, 40, torch.float32), (128, 32, 264, 1022, torch.bfloat16),
                            (65, 200, 96, 2048, torch.bfloat16), (65, 200, 520, 512, torch.bfloat16),
                            (256, 256, 264, 520, torch.float32), (256, 256, 264, 522, torch.bfloat16),
                            (16, 64, 2048, 1024, torch.bfloat16), (32, 64, 2048, 1024, torch.bfloat16),
                            (48, 144, 2040, 2000, torch.bfloat16), (48, 144, 2040, 1998, torch.bfloat16)]:
        r = np.random.default_rng(E + M)
        counts = np.bincount(np.concatenate([r.integers(0, E, M - 1), [E - 1]]), minlength=E).tolist()
        offs, toffs, x, w, dy = problem(counts, N, K, E)
        (y, _, _), (my, _, _) = reference(x, w, dy, offs)
        st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        close(mx.grouped_gemm_fwd(x, w, toffs, out_dtype=out, status=st), y, my, K, (E, M, N, K))
        assert int(st) == mx.DEV_OK
