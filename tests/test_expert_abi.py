"""What dispatch, combine, the MXFP4 operands and their products refuse before anything is launched (CPU), and their
kernels' resources."""
import pytest
import torch

import mxfp8_mixed_precision_amd as mx
from mxfp8_mixed_precision_amd import _abi
from test_kernel_resources import LDS_LIMIT, _kernel_metadata

P = 1 << 20  # an aligned address that no call reaches
F32 = mx.ROUTE_F32


def refused(fn, *a, **kw):
    with pytest.raises(mx.MxfError) as ei:
        fn(*a, stream=0, **kw)
    assert mx.last_error()
    return ei.value.status


def route(tokens=8, rows=32, D=64, ldx=64, ldh=64, lddh=64, topk=2, E=4, element=2, flags=0):
    return mx.RouteDesc(tokens, rows, D, ldx, ldh, lddh, topk, E, element, flags)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), _abi.E_SHAPE), (dict(rows=-1), _abi.E_SHAPE), (dict(rows=(1 << 30) + 1), _abi.E_SHAPE),
    (dict(D=0), _abi.E_SHAPE), (dict(D=(1 << 20) + 1, ldx=1 << 21, ldh=1 << 21, lddh=1 << 21), _abi.E_SHAPE),
    (dict(ldx=63), _abi.E_SHAPE), (dict(ldh=63), _abi.E_SHAPE), (dict(topk=0), _abi.E_SHAPE), (dict(topk=65), _abi.E_SHAPE),
    (dict(E=0), _abi.E_SHAPE), (dict(E=1025), _abi.E_SHAPE), (dict(tokens=(1 << 29) + 1), _abi.E_SHAPE),
    (dict(tokens=1 << 28, D=8192, ldx=8192, ldh=8192, lddh=8192), _abi.E_SHAPE), (dict(flags=4), _abi.E_ARG)])
def test_route_descriptor(kw, code):
    d = route(**kw)
    assert refused(mx.mxf_dispatch_fwd, d, P, P, P, P, P) == code
    assert refused(mx.mxf_combine_fwd, d, P, P, P, None, P) == code
    assert refused(mx.mxf_combine_bwd, d, P, P, P, P, P, P, P, P) == code


def test_route_pointers():
    f, c, b = mx.mxf_dispatch_fwd, mx.mxf_combine_fwd, mx.mxf_combine_bwd
    for k in range(5):
        a = [P] * 5
        a[k] = None
        assert refused(f, route(), *a) == _abi.E_NULL
    for n in (0, 3, 16, -1):
        assert refused(f, route(element=n), P, P, P, P, P) == _abi.E_ARG
    assert refused(f, route(flags=F32), P, P, P, P, P) == _abi.E_ARG
    assert refused(f, route(element=8), P, P, P, P + 4, P) == _abi.E_ALIGN
    assert refused(f, route(), P, P + 2, P, P, P) == _abi.E_ALIGN
    for k in (0, 1, 4):
        a = [P, P, P, None, P]
        a[k] = None
        assert refused(c, route(), *a) == _abi.E_NULL
    assert refused(c, route(), P + 2, P, P, None, P) == _abi.E_ALIGN
    assert refused(c, route(), P, P + 1, P, None, P) == _abi.E_ALIGN
    assert refused(c, route(flags=F32), P, P, P, None, P + 2) == _abi.E_ALIGN
    assert refused(c, route(flags=F32), P, P, P, P + 2, P) == _abi.E_ALIGN
    assert refused(c, route(flags=mx.ROUTE_WEIGHT_F32), P, P, P + 2, None, P) == _abi.E_ALIGN
    assert refused(c, route(lddh=63), P, P, P, P, P) == _abi.E_SHAPE       # the residual's stride
    assert refused(b, route(lddh=63), P, P, P, P, P, P, P, P) == _abi.E_SHAPE
    for k in (0, 1, 2, 3, 4, 5, 6):
        a = [P] * 8
        a[k] = None
        assert refused(b, route(), *a) == _abi.E_NULL
    assert refused(b, route(), P, P, P, P, P, P, P, P + 2) == _abi.E_ALIGN
    assert refused(b, route(flags=F32), P, P, P, P, P, P, P + 2, P) == _abi.E_ALIGN
    # nothing to do
    f(route(rows=0), None, None, P, P, None, stream=0)
    c(route(tokens=0), None, None, None, None, None, stream=0)
    b(route(tokens=0, rows=0), None, None, None, None, None, None, None, None, stream=0)


def operand(batch=1, rows=64, cols=96, ldx=96, tokens=8, topk=2, E=4, flags=0):
    return mx.OperandDesc(batch, rows, cols, ldx, tokens, topk, E, flags)


def test_operands():
    q, d = mx.mxf_mxfp4_quantize, mx.mxf_mxfp4_dequantize
    for kw, code in [(dict(batch=-1), _abi.E_SHAPE), (dict(rows=-1), _abi.E_SHAPE), (dict(cols=0), _abi.E_SHAPE),
                     (dict(cols=(1 << 20) + 1, ldx=1 << 21), _abi.E_SHAPE), (dict(flags=4), _abi.E_ARG),
                     (dict(rows=1 << 30, cols=1 << 12, ldx=1 << 12), _abi.E_SHAPE), (dict(batch=1 << 25), _abi.E_SHAPE)]:
        assert refused(q, operand(**kw), P, None, None, P, P, P, P) == code
        assert refused(d, operand(**kw), P, P, P) == code
    assert refused(q, operand(ldx=95), P, None, None, P, P, P, P) == _abi.E_SHAPE
    assert refused(q, operand(ldx=1 << 33), P, None, None, P, P, P, P) == _abi.E_SHAPE
    assert refused(q, operand(), None, None, None, P, P, P, P) == _abi.E_NULL
    assert refused(q, operand(), P, None, None, None, None, None, None) == _abi.E_NULL
    assert refused(q, operand(), P, None, None, P, None, P, P) == _abi.E_NULL
    assert refused(q, operand(), P, None, None, P, P, None, P) == _abi.E_NULL
    assert refused(q, operand(), P, None, P, P, P, P, P) == _abi.E_NULL                 # row_assign without offs
    assert refused(q, operand(batch=2), P, P, P, P, P, P, P) == _abi.E_SHAPE
    assert refused(q, operand(topk=0), P, P, P, P, P, P, P) == _abi.E_SHAPE
    assert refused(q, operand(), P + 1, None, None, P, P, P, P) == _abi.E_ALIGN
    assert refused(q, operand(flags=mx.OPERAND_F32), P + 2, None, None, P, P, P, P) == _abi.E_ALIGN
    assert refused(q, operand(), P, None, None, P + 8, P, P, P) == _abi.E_ALIGN
    assert refused(q, operand(), P, None, None, P, P + 2, P, P) == _abi.E_ALIGN
    assert refused(q, operand(), P, None, None, P, P, P + 8, P) == _abi.E_ALIGN
    for k in range(3):
        a = [P] * 3
        a[k] = None
        assert refused(d, operand(), *a) == _abi.E_NULL
        a[k] = P + 1
        assert refused(d, operand(), *a) == _abi.E_ALIGN
    q(operand(rows=0), None, None, None, None, None, None, None, stream=0)
    d(operand(batch=0), None, None, None, stream=0)


def grouped(E=4, flags=0, M=128, N=64, K=96, ldx=0, ldy=64):
    return mx.GroupedDesc(E, flags, M, N, K, ldx, ldy)


def test_products():
    f, w = mx.mxf_grouped_gemm_mxfp4_fwd, mx.mxf_grouped_gemm_mxfp4_wgrad
    acc = mx.GROUPED_ACCUM | mx.GROUPED_OUT_F32
    for fn in (f, w):
        for kw, code in [(dict(E=0), _abi.E_SHAPE), (dict(E=1025), _abi.E_SHAPE), (dict(M=-1), _abi.E_SHAPE),
                         (dict(N=0), _abi.E_SHAPE), (dict(K=(1 << 20) + 1), _abi.E_SHAPE), (dict(flags=8), _abi.E_ARG),
                         (dict(flags=mx.GROUPED_ACCUM), _abi.E_ARG)]:
            assert refused(fn, grouped(**kw), P, P, P, P, P, P) == code
        for k in range(6):
            a = [P] * 6
            a[k] = None
            assert refused(fn, grouped(), *a) == _abi.E_NULL
        for k, off in ((0, 2), (1, 8), (2, 2), (3, 8), (4, 2), (5, 1)):
            a = [P] * 6
            a[k] = P + off
            assert refused(fn, grouped(), *a) == _abi.E_ALIGN
        assert refused(fn, grouped(), P, P, P, P, P, P, P + 2) == _abi.E_ALIGN  # status
        assert refused(fn, grouped(flags=mx.GROUPED_OUT_F32), P, P, P, P, P, P + 2) == _abi.E_ALIGN
        assert refused(fn, grouped(E=1024, M=1 << 30, N=1 << 20, K=1 << 20, ldy=1 << 20), P, P, P, P, P, P) == _abi.E_SHAPE
    assert refused(f, grouped(flags=acc), P, P, P, P, P, P) == _abi.E_ARG
    assert refused(f, grouped(ldy=63), P, P, P, P, P, P) == _abi.E_SHAPE


def test_tensor_calls_refuse_what_does_not_fit():
    bf, u8, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.uint8), dict(dtype=torch.int32)
    x, h, w, dy = torch.zeros((4, 8), **bf), torch.zeros((10, 8), **bf), torch.zeros(4, 2), torch.zeros((4, 8), **bf)
    plan = {"offs": torch.zeros(4, **i32), "row_assign": torch.zeros(10, **i32), "assign_row": torch.zeros(8, **i32)}
    q, s = torch.zeros((2, 10, 64), **u8), torch.zeros((2, 10, 4), **u8)
    wq, ws = torch.zeros((3, 2, 6, 64), **u8), torch.zeros((3, 2, 6, 4), **u8)
    gq, gs = torch.zeros((2, 6, 64), **u8), torch.zeros((2, 6, 4), **u8)
    offs = torch.zeros(4, **i32)

    def but(**kw):
        return {**plan, **kw}

    bad = [
        (mx.dispatch_fwd, (x[0], plan)), (mx.dispatch_fwd, (x.t(), plan)), (mx.dispatch_fwd, (x[:3], plan)),
        (mx.dispatch_fwd, (x, but(offs=None))), (mx.dispatch_fwd, (x, but(offs=plan["offs"][:1]))),
        (mx.dispatch_fwd, (x, but(row_assign=plan["row_assign"].long()))), (mx.dispatch_fwd, (x, but(assign_row=plan["assign_row"][::2]))),
        (mx.dispatch_fwd, (x[:0], plan)), (mx.dispatch_fwd, (x, but(assign_row=plan["assign_row"][:3]))),
        (mx.dispatch_bwd, (h, plan, 3)), (mx.dispatch_bwd, (h[:9], plan, 4)), (mx.dispatch_bwd, (h.half(), plan, 4)),
        (mx.dispatch_bwd, (h, plan, 16)), (mx.dispatch_bwd, (h, plan, -4)),
        (mx.combine_fwd, (h, None, plan)), (mx.combine_fwd, (h, w[:3], plan)), (mx.combine_fwd, (h, w.half(), plan)),
        (mx.combine_fwd, (h, w[:, :1], plan)), (mx.combine_fwd, (h, w, plan, x.float())), (mx.combine_fwd, (h, w, plan, x[:3])),
        (mx.combine_bwd, (dy, h[:9], w, plan)), (mx.combine_bwd, (dy, h.float(), w, plan)), (mx.combine_bwd, (dy, h, None, plan)),
        (mx.combine_bwd, (dy, h, w[:, :1], plan)), (mx.combine_bwd, (dy[:3], h, w, plan)),
        (mx.mxfp4_quantize, (x.half(),)), (mx.mxfp4_quantize, (x, 4)), (mx.mxfp4_quantize, (x, 0)), (mx.mxfp4_quantize, (x[0],)),
        (mx.mxfp4_quantize, (x.view(2, 2, 8), mx.ROW, False, plan)), (mx.mxfp4_quantize, (x.view(2, 2, 8)[:, :, :4],)),
        (mx.mxfp4_dequantize, (q, None, 200)), (mx.mxfp4_dequantize, (q, s, 128)), (mx.mxfp4_dequantize, (q, s, 257)),
        (mx.mxfp4_dequantize, (q[:, :9], s, 200)), (mx.mxfp4_dequantize, (q[:1], s, 200)), (mx.mxfp4_dequantize, (q, s, 200, torch.half)),
        (mx.grouped_gemm_mxfp4_fwd, ((q, s), (wq[:, :1], ws[:, :1]), offs)), (mx.grouped_gemm_mxfp4_fwd, ((q, s), (wq, ws), offs[:3])),
        (mx.grouped_gemm_mxfp4_fwd, ((q, s), (wq, ws), offs.long())), (mx.grouped_gemm_mxfp4_fwd, ((q, s), (wq, ws), None)),
        (mx.grouped_gemm_mxfp4_fwd, ((q, s), (torch.zeros((3, 4, 6, 64), **u8), ws), offs)),  # 8-bit weights
        (mx.grouped_gemm_mxfp4_fwd, ((q, s), (wq, ws), offs, torch.half)), (mx.grouped_gemm_mxfp4_fwd, ((q, s), (gq, gs), offs)),
        (mx.grouped_gemm_mxfp4_wgrad, ((gq, gs), (q[:1], s[:1]), offs)), (mx.grouped_gemm_mxfp4_wgrad, ((gq, None), (q, s), offs)),
        (mx.grouped_gemm_mxfp4_wgrad, ((gq, gs), (q, s), offs[0])),
        (mx.grouped_gemm_mxfp4_wgrad, ((gq, gs), (q, s), offs, None, torch.zeros((3, 6, 9)))),
        (mx.grouped_gemm_mxfp4_wgrad, ((gq, gs), (q, s), offs, torch.bfloat16, torch.zeros((3, 6, 10)))),
        # not on a GPU
        (mx.dispatch_fwd, (x, plan)), (mx.combine_fwd, (h, w, plan)), (mx.combine_bwd, (dy, h, w, plan)),
        (mx.mxfp4_quantize, (x,)), (mx.mxfp4_dequantize, (q, s, 200)), (mx.grouped_gemm_mxfp4_fwd, ((q, s), (wq, ws), offs)),
        (mx.grouped_gemm_mxfp4_wgrad, ((gq, gs), (q, s), offs)),
    ]
    wrong = []
    for i, (fn, args) in enumerate(bad):
        try:
            fn(*args)
        except ValueError:
            continue
        except Exception as e:  # noqa: BLE001
            wrong.append((i, fn.__name__, type(e).__name__, str(e)))
            continue
        wrong.append((i, fn.__name__, "accepted"))
    assert not wrong


@pytest.mark.parametrize("src", ["combine.hip", "mxfp4.hip", "grouped_mx.hip"])
def test_no_scratch_and_lds_fits(src):
    for k in _kernel_metadata(src):
        assert int(k.get("private_segment_fixed_size", 0)) == 0, (k["name"], "uses scratch")
        assert int(k.get("vgpr_spill_count", 0)) == 0, (k["name"], "spills VGPRs")
        assert int(k.get("group_segment_fixed_size", 0)) <= LDS_LIMIT, (k["name"], "LDS over 160 KB")
