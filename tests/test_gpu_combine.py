"""Dispatch, combine and their gradients on the GPU against float64.

Tolerances per element: a sum of n FP32 terms is off by at most n 2^-24 of the sum of magnitudes (products are fused or add
one more 2^-24 each: n + 1), an output by half a step of its type (BF16 2^-8 of itself, FP32 2^-24)."""
import pytest
import torch

import mxfp8_mixed_precision_amd as mx
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def half_step(t):
    return torch.finfo(t).eps / 2


def make_plan(T, topk, E, pad, seed, drop=0.0, slack=0):
    """A plan of route_plan; `drop`: share of ids that no expert has; slack: rows past the layout."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ids = torch.randint(0, E, (T, topk), generator=g, device="cuda", dtype=torch.int32)
    ids = torch.where(torch.rand((T, topk), generator=g, device="cuda") < drop, torch.full_like(ids, -1), ids)
    cap = T * topk + E * (pad - 1) + slack
    plan = mx.route_plan(ids, E, pad, cap)
    return plan, int(plan["offs"][-1])


def rnd(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def strided(t, ld, off):
    """t in a wider matrix whose storage starts `off` elements later (other alignments and strides)."""
    if ld == 0:
        return t
    buf = torch.full((t.shape[0] * (t.shape[1] + ld) + off + 8,), float("nan"), device="cuda").to(t.dtype)
    v = buf[off:off + t.shape[0] * (t.shape[1] + ld)].view(t.shape[0], -1)[:, :t.shape[1]]
    v.copy_(t)
    return v


def close(got, ref, mag, n, what):
    tol = (n + 1) * 2.0 ** -24 * mag + ref.abs() * half_step(got.dtype) * (1 + 1e-9)
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist())


def gathered(h, idx):
    z = torch.zeros((idx.numel(), h.shape[1]), dtype=torch.float64, device="cuda")
    ok = idx >= 0
    z[ok] = h[idx[ok].long()].double()
    return z


CASES = [  # T, topk, E, D, pad, drop, stride, offset
    (1, 1, 1, 1, 1, 0.0, 0, 0), (3, 2, 4, 7, 1, 0.3, 3, 1), (8, 6, 64, 2048, 1, 0.0, 0, 0), (5, 64, 8, 40, 1, 0.2, 0, 0),
    (17, 8, 16, 129, 16, 0.1, 1, 1), (64, 4, 8, 64, 128, 0.0, 8, 0), (33, 9, 5, 256, 1, 0.5, 0, 0), (100, 1, 3, 8, 4, 0.0, 0, 0),
    (40, 3, 1024, 513, 1, 0.0, 5, 3), (2, 7, 2, 7168, 128, 0.0, 0, 0), (300, 2, 7, 1411, 1, 0.06, 0, 0), (6, 2, 4, 96, 1, 1.0, 0, 0),
    (513, 17, 9, 33, 3, 0.02, 0, 0), (70, 5, 6, 4099, 2, 0.1, 2, 1), (9, 2, 3, 15, 1, 0.0, 0, 1), (9, 2, 3, 16, 1, 0.0, 0, 0)]


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("T,topk,E,D,pad,drop,ld,off", CASES)
def test_against_float64(T, topk, E, D, pad, drop, ld, off, t):
    require_gpu()
    plan, end = make_plan(T, topk, E, pad, T * 7 + D, drop, slack=5)
    rows, a = plan["row_assign"].numel(), plan["row_assign"][:end].long()
    tok = torch.where((a >= 0) & (a < T * topk), a // topk, -1)
    x, h, dy = (strided(rnd(s, n, D).to(t), ld, off) for s, n in ((1, T), (2, rows), (3, T)))
    res = rnd(4, T, D).to(t)
    # pad rows of h, and those past the layout, hold nothing that counts
    h[:end][a < 0] = float("nan")
    h[end:] = float("inf")
    xe = mx.dispatch_fwd(x, plan)
    assert torch.equal(xe[:end].double(), gathered(x, tok))
    assert torch.equal(mx.dispatch_fwd(x, plan)[:end], xe[:end])
    H = gathered(h, plan["assign_row"]).view(T, topk, D)
    close(mx.dispatch_bwd(h, plan, T), H.sum(1), H.abs().sum(1), topk, "dispatch_bwd")
    for wt in (BF, F32):
        w = rnd(5, T, topk).to(wt)
        W = w.double()[:, :, None]
        close(mx.combine_fwd(h, w, plan), (H * W).sum(1), (H * W).abs().sum(1), topk, "combine_fwd")
        R = res.double()
        close(mx.combine_fwd(h, w, plan, res), R + (H * W).sum(1), R.abs() + (H * W).abs().sum(1), topk + 1, "residual")
        dh, dw = mx.combine_bwd(dy, h, w, plan)
        want = gathered(dy, tok) * gathered(w.reshape(-1, 1), torch.where((a >= 0) & (a < T * topk), a, -1))
        close(dh[:end], want, want.abs(), 0, "dh")
        G = (H * dy.double()[:, None])
        ok = plan["assign_row"].view(T, topk) >= 0
        close(dw, G.sum(2), G.abs().sum(2), D, "dweights")
        assert (dw[~ok] == 0).all()
        alone, none = mx.combine_bwd(dy, None, w, plan)
        assert none is None and torch.equal(alone[:end], dh[:end])
        again = mx.combine_bwd(dy, h, w, plan)
        assert torch.equal(again[0][:end], dh[:end]) and torch.equal(again[1], dw)


# h, or h and dh, larger than the last-level cache
@pytest.mark.parametrize("T,topk,D,t", [(4096, 8, 4096, BF), (4096, 6, 2048, F32), (8192, 4, 2048, BF)])
def test_rows_past_the_cache(T, topk, D, t):
    test_against_float64(T, topk, 16, D, 128, 0.01, 0, 0, t)


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int8, torch.float16, torch.int32, torch.int64, torch.float64])
@pytest.mark.parametrize("D", [1, 3, 16, 65, 1000])
def test_dispatch_moves_any_type(dtype, D):
    require_gpu()
    plan, end = make_plan(50, 3, 8, 4, D, 0.1)
    x = (rnd(D, 50, D + 3) * 50).to(dtype)[:, 1:D + 1]
    a = plan["row_assign"][:end].long()
    want = torch.where((a >= 0)[:, None], x[(a.clamp_min(0) // 3)], torch.zeros((), dtype=dtype, device="cuda"))
    assert torch.equal(mx.dispatch_fwd(x, plan)[:end], want)


@pytest.mark.parametrize("t", [BF, F32])
def test_rows_and_columns_outside_are_left(t):
    """Rows past the layout and the gaps of strided outputs stay as they were (raw calls)."""
    require_gpu()
    T, topk, E, D, pad = 21, 3, 4, 77, 8
    plan, end = make_plan(T, topk, E, pad, 3, 0.1, slack=40)
    rows, ld = plan["row_assign"].numel(), D + 6
    flags = (mx.ROUTE_F32 if t == F32 else 0) | mx.ROUTE_WEIGHT_F32
    x, h, dy, w = rnd(1, T, D).to(t), rnd(2, rows, D).to(t), rnd(3, T, D).to(t), rnd(4, T, topk)
    big = [torch.full((n, ld), 7.0, dtype=t, device="cuda") for n in (rows, T, rows)]
    dw = torch.empty((T, topk), device="cuda")
    sz = x.element_size()
    mx.mxf_dispatch_fwd(mx.RouteDesc(T, rows, D, D, ld, D, topk, E, sz, 0), plan["offs"], plan["row_assign"], plan["assign_row"],
                        x, big[0])
    mx.mxf_combine_fwd(mx.RouteDesc(T, rows, D, ld, D, D, topk, E, 0, flags), plan["assign_row"], h, w, None, big[1])
    mx.mxf_combine_bwd(mx.RouteDesc(T, rows, D, D, D, ld, topk, E, 0, flags), plan["offs"], plan["row_assign"], plan["assign_row"],
                       dy, h, w, big[2], dw)
    assert torch.equal(big[0][:end, :D], mx.dispatch_fwd(x, plan)[:end])
    assert torch.equal(big[1][:, :D], mx.combine_fwd(h, w, plan))
    assert torch.equal(big[2][:end, :D], mx.combine_bwd(dy, h, w, plan)[0][:end])
    for b, n in zip(big, (end, T, end)):
        assert (b[:, D:] == 7).all() and (b[n:] == 7).all()


def test_a_plan_over_its_capacity():
    """Assignments whose row is past m_capacity have none: they are dropped."""
    require_gpu()
    ids = torch.randint(0, 4, (64, 2), device="cuda", dtype=torch.int32)
    plan = mx.route_plan(ids, 4, 1, 100)
    assert int(plan["status"]) == mx.DEV_OVERFLOW and (plan["assign_row"] < 0).sum() == 28
    x, w = rnd(1, 64, 48), rnd(2, 64, 2)
    xe = mx.dispatch_fwd(x, plan)
    assert torch.equal(xe, x[plan["row_assign"].long() // 2])
    H = gathered(xe, plan["assign_row"]).view(64, 2, 48)
    close(mx.combine_fwd(xe, w, plan), (H * w.double()[:, :, None]).sum(1), (H * w.double()[:, :, None]).abs().sum(1), 2, "y")
    dh, dw = mx.combine_bwd(x, xe, w, plan)
    G = H * x.double()[:, None]
    close(dw, G.sum(2), G.abs().sum(2), 48, "dw")
    assert torch.isfinite(dh).all()


def test_maps_out_of_range_are_dropped():
    """Entries of the maps outside their ranges count as dropped (assign_row) and as pad rows (row_assign)."""
    require_gpu()
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = {"offs": torch.tensor([0, 4], **i32), "row_assign": torch.tensor([0, 1, 2 ** 31 - 1, -5], **i32),
            "assign_row": torch.tensor([0, 1, 4, 2 ** 31 - 1, -7, -2 ** 31], **i32)}
    x, w = rnd(1, 3, 24), torch.ones((3, 2), device="cuda")
    h = rnd(2, 4, 24)
    xe = mx.dispatch_fwd(x, plan)
    assert torch.equal(xe, torch.stack([x[0], x[0], torch.zeros_like(x[0]), torch.zeros_like(x[0])]))
    y = mx.combine_fwd(h, w, plan)
    assert torch.equal(y[0], h[0] + h[1]) and (y[1:] == 0).all()
    dh, dw = mx.combine_bwd(x, h, w, plan)
    assert torch.equal(dh, xe) and (dw[1:] == 0).all()


def test_nothing_to_do():
    require_gpu()
    i32 = dict(dtype=torch.int32, device="cuda")
    e = {"offs": torch.zeros(3, **i32), "row_assign": torch.zeros(0, **i32), "assign_row": torch.zeros(0, **i32)}
    x, w = torch.zeros((0, 16), device="cuda"), torch.zeros((0, 2), device="cuda")
    assert mx.dispatch_fwd(x, e).shape == (0, 16) and mx.combine_fwd(x, w, e).shape == (0, 16)
    dh, dw = mx.combine_bwd(x, x, w, e)
    assert dh.shape == (0, 16) and dw.shape == (0, 2)
    # no tokens, pad rows alone; all assignments dropped, no rows
    pads = {"offs": torch.tensor([0, 8], **i32), "row_assign": torch.full((8,), -1, **i32), "assign_row": torch.zeros(0, **i32)}
    assert (mx.dispatch_fwd(x, pads) == 0).all() and (mx.combine_bwd(x, None, w, pads)[0] == 0).all()
    gone = {**e, "assign_row": torch.full((6,), -1, **i32)}
    assert (mx.combine_fwd(x, torch.ones((3, 2), device="cuda"), gone) == 0).all()
    assert (mx.combine_bwd(torch.ones((3, 16), device="cuda"), x, torch.ones((3, 2), device="cuda"), gone)[1] == 0).all()


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31 (and bytes past 2^32)."""
    require_gpu()
    D, rows, T = 8192, 300000, 8
    i32 = dict(dtype=torch.int32, device="cuda")
    row = torch.tensor([299999, 3, 262144, 131073, 280001, 0, 262145, 150000], **i32)
    ra = torch.full((rows,), -1, **i32)
    ra[row.long()] = torch.arange(8, **i32)
    plan = {"offs": torch.tensor([0, rows], **i32), "row_assign": ra, "assign_row": row}
    x, w = rnd(1, T, D).bfloat16(), rnd(2, T, 1)
    xe = mx.dispatch_fwd(x, plan)
    assert torch.equal(xe[row.long()], x)
    assert int((xe != 0).any(1).sum()) == 8
    assert torch.equal(mx.dispatch_bwd(xe, plan, T), x)
    dh, dw = mx.combine_bwd(x, xe, w, plan)
    assert torch.equal(dh[row.long()], (x.float() * w).bfloat16())
    S = x.double().square().sum(1, keepdim=True)
    close(dw, S, S, D, "dw")


def test_streams_and_graphs():
    require_gpu()
    T, topk, E, D = 96, 4, 8, 640
    plan, _ = make_plan(T, topk, E, 16, 5, 0.1)
    rows = plan["row_assign"].numel()
    x, h, w, dy = rnd(1, T, D).bfloat16(), rnd(2, rows, D).bfloat16(), rnd(3, T, topk), rnd(4, T, D).bfloat16()
    end = int(plan["offs"][-1])

    def step():
        xe = mx.dispatch_fwd(x, plan)
        y = mx.combine_fwd(h, w, plan, x)
        dh, dw = mx.combine_bwd(dy, h, w, plan)
        return xe, y, dh, dw, mx.dispatch_bwd(h, plan, T)

    def same(a, b):
        return all(torch.equal(u[:end] if u.shape[0] == rows else u, v[:end] if v.shape[0] == rows else v) for u, v in zip(a, b))

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert same(got, want)
    y = mx.combine_fwd(h, w, plan, x, stream=s)
    s.synchronize()
    assert torch.equal(y, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in range(3):
        for t in (x, h, dy):
            t.copy_(rnd(seed * 10 + t.shape[0], *t.shape))
        want = step()
        g.replay()
        torch.cuda.synchronize()
        assert same(out, want)
