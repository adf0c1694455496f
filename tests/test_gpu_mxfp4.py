"""MXFP4 operands on the GPU against the float64 oracle, byte for byte."""
import numpy as np
import pytest
import torch

import mxfp8_mixed_precision_amd as mx
from gpu_util import require_gpu
from oracle import mxfp4 as o4

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def np_(t):
    return t.cpu().numpy()


def matrix(rows, cols, t, seed):
    """Values over many binades, with zero groups, zeros of both signs and ties."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    v = r(rows, cols) * torch.exp2((10 * r(rows, 1)).round()) * torch.exp2((6 * r(1, cols)).round())
    v = torch.where(torch.rand((rows, cols), generator=g, device="cuda") < 0.1, -0.0 * v, v)
    v = torch.where(torch.rand((rows, cols), generator=g, device="cuda") < 0.2, (v / 0.25).round() * 0.25, v)
    if cols > 40:
        v[::3, 32:64] = 0
    return v.to(t)


def check(got, v, e4m3, what):
    q, s = o4.operand(v, e4m3)
    assert np.array_equal(np_(got[1]), s), (what, "scales", np.argwhere(np_(got[1]) != s)[:4].tolist())
    assert np.array_equal(np_(got[0]), q), (what, "codes", np.argwhere(np_(got[0]) != q)[:4].tolist())


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 31), (32, 32), (33, 65), (128, 128), (127, 129), (130, 256), (257, 1000), (4, 1411), (200, 3),
          (48, 2048), (1, 4097)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_operands_equal_the_oracle(rows, cols, t, e4m3):
    require_gpu()
    x = matrix(rows, cols, t, rows * 31 + cols)
    v = np_(x.double())
    q, s, qt, st = mx.mxfp4_quantize(x, mx.ROW | mx.COL, e4m3=e4m3)
    check((q, s), v, e4m3, "rows")
    check((qt, st), v.T, e4m3, "columns")
    r = mx.mxfp4_quantize(x, e4m3=e4m3)
    assert torch.equal(r[0], q) and torch.equal(r[1], s) and r[2] is None and r[3] is None
    c = mx.mxfp4_quantize(x, mx.COL, e4m3=e4m3)
    assert torch.equal(c[2], qt) and torch.equal(c[3], st) and c[0] is None and c[1] is None
    want = o4.values(*o4.operand(v, e4m3))[:, :cols]
    f = mx.mxfp4_dequantize(q, s, cols, F32)
    assert np.array_equal(np_(f.double()), want.astype(np.float32).astype(np.float64))
    b = mx.mxfp4_dequantize(q, s, cols)
    assert torch.equal(b, f.bfloat16())
    assert np.array_equal(np_(mx.mxfp4_dequantize(qt, st, rows, F32).double()),
                          o4.values(*o4.operand(v.T, e4m3))[:, :rows].astype(np.float32).astype(np.float64))


def test_every_bf16_in_a_group():
    """All finite BF16 patterns, each beside an element that sets the scale, against the oracle."""
    require_gpu()
    bits = torch.arange(65536, dtype=torch.int32, device="cuda")
    bits = bits[(bits & 0x7F80) != 0x7F80]
    for top in (1.0, 2.0 ** -126, 2.0 ** -133, 1.75 * 2.0 ** 127, 6.0):
        x = torch.zeros((bits.numel(), 32), dtype=BF, device="cuda")
        x[:, 5] = bits.to(torch.int16).view(BF)
        x[:, 6] = top
        q, s, _, _ = mx.mxfp4_quantize(x)
        check((q, s), np_(x.double()), False, top)


def test_ties_and_borders_in_float32():
    """Values one step of FP32 from the rounding borders and from a change of the scale."""
    require_gpu()
    edge = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], dtype=np.float32)
    near = np.concatenate([edge, np.nextafter(edge, np.float32(0)), np.nextafter(edge, np.float32(9))])
    amax = np.array([4.0, np.nextafter(np.float32(4), np.float32(0)), np.nextafter(np.float32(8), np.float32(0)), 8.0], dtype=np.float32)
    rows = []
    for a in amax:
        for e in (-130, -100, 0, 60):
            g = np.zeros(32, dtype=np.float32)
            g[:near.size] = np.ldexp(near * np.where(np.arange(near.size) % 2, -1, 1), e).astype(np.float32)
            g[-1] = np.ldexp(a, e)
            rows.append(np.where(np.abs(g) > np.abs(g[-1]), 0, g))
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).cuda()
    q, s, qt, st = mx.mxfp4_quantize(x, mx.ROW | mx.COL)
    check((q, s), np_(x.double()), False, "rows")
    check((qt, st), np_(x.double()).T, False, "columns")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("t", [BF, F32])
def test_groups_that_are_not_finite(t, e4m3):
    require_gpu()
    x = matrix(70, 96, t, 5)
    x[3, 40], x[20, 7], x[66, 95] = float("nan"), float("inf"), float("-inf")
    q, s, qt, st = mx.mxfp4_quantize(x, mx.ROW | mx.COL, e4m3=e4m3)
    y, yt = mx.mxfp4_dequantize(q, s, 96), mx.mxfp4_dequantize(qt, st, 70)
    bad = torch.zeros((70, 96), dtype=torch.bool, device="cuda")
    bad[3, 32:64] = bad[20, :32] = bad[66, 64:] = True
    badt = torch.zeros((96, 70), dtype=torch.bool, device="cuda")
    badt[40, :32] = badt[7, :32] = badt[95, 64:] = True
    assert torch.equal(y.isnan(), bad) and torch.equal(yt.isnan(), badt)
    clean = np_(torch.where(x.isfinite(), x, torch.zeros_like(x)).double())
    w = torch.from_numpy(o4.values(*o4.operand(clean, e4m3))[:, :96]).cuda()
    assert torch.equal(y.double()[~bad], w[~bad].bfloat16().double())
    assert (s[0, 3, 1] == 255) and int((s == 255).sum()) == 3 and int((st == 255).sum()) == 3


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("cols,ld,off", [(96, 8, 0), (65, 3, 1), (200, 1, 5), (7, 2, 1)])
def test_strides_and_alignment(cols, ld, off, t):
    require_gpu()
    x = matrix(50, cols, t, cols)
    buf = torch.full((50 * (cols + ld) + off,), float("nan"), device="cuda").to(t)
    v = buf[off:].view(50, cols + ld)[:, :cols]
    v.copy_(x)
    for a, b in zip(mx.mxfp4_quantize(v, mx.ROW | mx.COL), mx.mxfp4_quantize(x, mx.ROW | mx.COL)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,rows,cols", [(3, 40, 72), (5, 128, 256), (2, 130, 33), (0, 4, 32), (2, 0, 32)])
def test_batches(n, rows, cols, e4m3):
    require_gpu()
    x = torch.stack([matrix(rows, cols, BF, i) for i in range(n)]) if n else torch.zeros((0, rows, cols), dtype=BF, device="cuda")
    got = mx.mxfp4_quantize(x, mx.ROW | mx.COL, e4m3=e4m3)
    for i in range(n):
        for a, b in zip(got, mx.mxfp4_quantize(x[i], mx.ROW | mx.COL, e4m3=e4m3)):
            assert torch.equal(a[i], b)
    back = mx.mxfp4_dequantize(got[0], got[1], cols)
    for i in range(n):
        assert torch.equal(back[i], mx.mxfp4_dequantize(got[0][i].contiguous(), got[1][i].contiguous(), cols))


@pytest.mark.parametrize("T,topk,E,D,pad,slack", [(8, 6, 16, 2048, 1, 3), (50, 3, 4, 100, 128, 300), (33, 2, 5, 257, 16, 0), (1, 1, 1, 8, 1, 7),
                                                  (200, 2, 70, 64, 1, 0)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("t", [BF, F32])
def test_gathered_by_a_plan(T, topk, E, D, pad, slack, e4m3, t):
    require_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    ids = torch.randint(-1, E, (T, topk), generator=g, device="cuda", dtype=torch.int32)
    plan = mx.route_plan(ids, E, pad, T * topk + E * (pad - 1) + slack)
    end, rows = int(plan["offs"][-1]), plan["row_assign"].numel()
    x = matrix(T, D, t, D)
    if pad > 1:
        x[0, 0] = float("nan")  # (a token without rows may hold anything: pad rows read none)
        ids[0] = -1
        plan = mx.route_plan(ids, E, pad, rows)
        end = int(plan["offs"][-1])
    xe = mx.dispatch_fwd(x, plan)
    xe[end:] = 0
    ref = mx.mxfp4_quantize(xe, mx.ROW | mx.COL, e4m3=e4m3)
    # outputs whose former contents show: rows past the layout along rows, planes past it along columns
    P, Pr = (D + 127) // 128, (rows + 127) // 128
    m = 2 if e4m3 else 1
    out = [torch.full(s, 0xAA, dtype=torch.uint8, device="cuda") for s in ((m * P, rows, 64), (P, rows, 4), (m * Pr, D, 64), (Pr, D, 4))]
    flags = (mx.OPERAND_F32 if t == F32 else 0) | (mx.OPERAND_E4M3 if e4m3 else 0)
    mx.mxf_mxfp4_quantize(mx.OperandDesc(1, rows, D, D, T, topk, E, flags), x, plan["offs"], plan["row_assign"], *out)
    for i in (0, 1):
        assert torch.equal(out[i][:, :end], ref[i][:, :end]) and (out[i][:, end:] == 0xAA).all()
    last = (end + 127) // 128
    for i, k in ((2, m), (3, 1)):
        assert torch.equal(out[i][:k * last], ref[i][:k * last]) and (out[i][k * last:] == 0xAA).all()
    got = mx.mxfp4_quantize(x, mx.ROW | mx.COL, e4m3=e4m3, plan=plan)
    assert torch.equal(got[0][:, :end], ref[0][:, :end]) and torch.equal(got[2][:m * last], ref[2][:m * last])


def test_no_tokens_pad_rows_alone():
    require_gpu()
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = {"offs": torch.tensor([0, 40], **i32), "row_assign": torch.full((40,), -1, **i32), "assign_row": torch.zeros(0, **i32)}
    for t in mx.mxfp4_quantize(torch.zeros((0, 100), device="cuda"), mx.ROW | mx.COL, plan=plan):
        assert (t == 0).all()


def test_bytes_past_32_bits():
    """A matrix and an operand of more than 2^32 bytes: the last rows."""
    require_gpu()
    rows, cols = 1050000, 4096
    x = torch.zeros((rows, cols), dtype=BF, device="cuda")
    x[-5:] = matrix(5, cols, BF, 1)
    q, s, _, _ = mx.mxfp4_quantize(x, e4m3=True)
    r = mx.mxfp4_quantize(x[-5:].contiguous(), e4m3=True)
    assert torch.equal(q[:, -5:], r[0]) and torch.equal(s[:, -5:], r[1]) and not q[:, :-5].any()
    y = mx.mxfp4_dequantize(q, s, cols)
    assert torch.equal(y[-5:], mx.mxfp4_dequantize(r[0], r[1], cols))


def test_streams_and_graphs():
    require_gpu()
    x = matrix(300, 520, BF, 3)
    f = lambda: [*mx.mxfp4_quantize(x, mx.ROW | mx.COL), *(lambda q: [mx.mxfp4_dequantize(q[0], q[1], 520)])(mx.mxfp4_quantize(x))]  # noqa: E731
    want = f()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = f()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    for seed in range(3):
        x.copy_(matrix(300, 520, BF, seed + 10))
        want = f()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
