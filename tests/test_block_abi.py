"""What the training-block operators refuse before anything is launched (CPU), and their kernels' resources."""
import pytest
import torch

import mxfp8_mixed_precision_amd as mx
from mxfp8_mixed_precision_amd import _abi
from test_kernel_resources import LDS_LIMIT, _kernel_metadata

P = 1 << 20  # an aligned address that no call reaches


def refused(fn, *a, **kw):
    with pytest.raises(mx.MxfError) as ei:
        fn(*a, stream=0, **kw)
    assert mx.last_error()
    return ei.value.status


def norm(rows=4, cols=64, ldx=64, ldy=64, lddx=64, eps=1e-5, flags=0):
    return mx.NormDesc(rows, cols, ldx, ldy, lddx, eps, flags)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), _abi.E_SHAPE), (dict(cols=0), _abi.E_SHAPE), (dict(cols=(1 << 20) + 1), _abi.E_SHAPE),
    (dict(ldx=63), _abi.E_SHAPE), (dict(ldy=63), _abi.E_SHAPE), (dict(eps=-1.0), _abi.E_ARG),
    (dict(eps=float("nan")), _abi.E_ARG), (dict(flags=4), _abi.E_ARG)])
def test_norm_descriptor(kw, code):
    assert refused(mx.mxf_layer_norm_fwd, norm(**kw), P, P, P, P, P, P, None, None) == code
    assert refused(mx.mxf_layer_norm_bwd, norm(**kw), P, P, None, None, P, P, P, P, P, P, P) == code
    assert mx.layer_norm_workspace_bytes(norm(**kw)) == 0


def test_norm_pointers():
    f, b = mx.mxf_layer_norm_fwd, mx.mxf_layer_norm_bwd
    assert refused(f, norm(), None, P, P, P, P, P, None, None) == _abi.E_NULL
    assert refused(f, norm(), P, P, P, None, P, P, None, None) == _abi.E_NULL
    assert refused(f, norm(), P, P, P, P, P, P, P, None) == _abi.E_NULL             # half a checkpoint
    assert refused(f, norm(), P + 1, P, P, P, P, P, None, None) == _abi.E_ALIGN
    assert refused(f, norm(flags=mx.NORM_F32), P + 2, P, P, P, P, P, None, None) == _abi.E_ALIGN
    assert refused(f, norm(flags=mx.NORM_WEIGHT_F32), P, P + 2, P, P, P, P, None, None) == _abi.E_ALIGN
    assert refused(f, norm(), P, P, P, P, P + 2, P, None, None) == _abi.E_ALIGN
    assert refused(b, norm(lddx=63), P, P, None, None, P, P, P, P, P, P, P) == _abi.E_SHAPE
    assert refused(b, norm(), None, P, None, None, P, P, P, P, P, P, P) == _abi.E_NULL
    assert refused(b, norm(), P, None, None, None, P, P, P, P, P, P, P) == _abi.E_NULL   # neither x nor checkpoint
    assert refused(b, norm(), P, P, None, None, None, P, P, P, P, P, P) == _abi.E_NULL   # x without mean
    assert refused(b, norm(), P, P, P, P, P, P, P, P, P, P, P) == _abi.E_ARG             # both
    assert refused(b, norm(), P, P, None, None, P, P, P, P, P, P, None) == _abi.E_NULL   # workspace
    mx.mxf_layer_norm_fwd(norm(rows=0), None, None, None, None, None, None, None, None, stream=0)
    mx.mxf_layer_norm_bwd(norm(rows=0), None, None, None, None, None, None, None, None, None, None, None, stream=0)
    assert mx.layer_norm_workspace_bytes(norm()) % (2 * 64 * 4) == 0


def test_swiglu():
    f, b = mx.mxf_swiglu_ckpt_fwd, mx.mxf_swiglu_ckpt_bwd
    assert refused(f, P, -1, 64, 128, P, 64, P, P) == _abi.E_SHAPE
    assert refused(f, P, 4, 0, 128, P, 64, P, P) == _abi.E_SHAPE
    assert refused(f, P, 4, 64, 127, P, 64, P, P) == _abi.E_SHAPE
    assert refused(f, P, 4, 64, 128, P, 63, P, P) == _abi.E_SHAPE
    assert refused(f, None, 4, 64, 128, P, 64, P, P) == _abi.E_NULL
    assert refused(f, P, 4, 64, 128, P, 64, P, None) == _abi.E_NULL
    assert refused(f, P + 1, 4, 64, 128, P, 64, P, P) == _abi.E_ALIGN
    assert refused(b, P, 63, P, P, 4, 64, P, 128, P, 64) == _abi.E_SHAPE
    assert refused(b, P, 64, P, P, 4, 64, P, 128, P, 63) == _abi.E_SHAPE
    assert refused(b, None, 64, P, P, 4, 64, P, 128, P, 64) == _abi.E_NULL
    assert refused(b, P, 64, P, P, 4, 64, P + 1, 128, P, 64) == _abi.E_ALIGN
    mx.mxf_swiglu_ckpt_fwd(None, 0, 64, 128, None, 64, None, None, stream=0)


def grouped(E=4, flags=0, M=128, N=64, K=96, ldx=96, ldy=64):
    return mx.GroupedDesc(E, flags, M, N, K, ldx, ldy)


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), _abi.E_SHAPE), (dict(E=1025), _abi.E_SHAPE), (dict(M=-1), _abi.E_SHAPE),
    (dict(M=(1 << 30) + 1), _abi.E_SHAPE), (dict(N=0, ldy=64), _abi.E_SHAPE), (dict(K=0), _abi.E_SHAPE),
    (dict(ldx=95), _abi.E_SHAPE), (dict(ldy=63), _abi.E_SHAPE), (dict(flags=4), _abi.E_ARG)])
def test_grouped_descriptor(kw, code):
    d = grouped(**kw)
    assert refused(mx.mxf_grouped_gemm_fwd, d, P, P, P, P) == code
    assert refused(mx.mxf_grouped_gemm_dgrad, d, P, P, P, P) == code
    assert refused(mx.mxf_grouped_gemm_wgrad, d, P, P, P, None, None, P) == code


def test_grouped_pointers_and_flags():
    f, g, w = mx.mxf_grouped_gemm_fwd, mx.mxf_grouped_gemm_dgrad, mx.mxf_grouped_gemm_wgrad
    acc = mx.GROUPED_ACCUM | mx.GROUPED_OUT_F32
    assert refused(f, grouped(flags=acc), P, P, P, P) == _abi.E_ARG                       # accumulation is wgrad's
    assert refused(w, grouped(flags=mx.GROUPED_ACCUM), P, P, P, None, None, P) == _abi.E_ARG  # and FP32's
    for fn in (f, g):
        for k in range(4):
            a = [P, P, P, P]
            a[k] = None
            assert refused(fn, grouped(), *a) == _abi.E_NULL
        assert refused(fn, grouped(), P + 2, P, P, P) == _abi.E_ALIGN
        assert refused(fn, grouped(), P, P + 1, P, P) == _abi.E_ALIGN
        assert refused(fn, grouped(), P, P, P, P, P + 2) == _abi.E_ALIGN                  # status
        assert refused(fn, grouped(flags=mx.GROUPED_OUT_F32), P, P, P, P + 2) == _abi.E_ALIGN
    assert refused(w, grouped(), P, P, None, None, None, P) == _abi.E_NULL
    assert refused(w, grouped(), P, P, None, P, None, P) == _abi.E_NULL
    assert refused(w, grouped(), P, P, P, P, P, P) == _abi.E_ARG
    assert refused(w, grouped(), P, None, P, None, None, P) == _abi.E_NULL
    assert refused(w, grouped(), P, P, P, None, None, None) == _abi.E_NULL
    assert refused(f, grouped(M=1 << 30, N=1 << 20, ldy=1 << 20), P, P, P, P) == _abi.E_SHAPE  # tiles


def test_the_stride_of_x_is_not_used_with_codes():
    w = mx.mxf_grouped_gemm_wgrad
    for ldx in (95, 0, -1, 1 << 40):
        assert refused(w, grouped(ldx=ldx), P, P, None, P, P, None) == _abi.E_NULL  # dw: past the descriptor's checks
    assert refused(w, grouped(ldx=95), P, P, P, None, None, None) == _abi.E_SHAPE
    assert refused(w, grouped(ldy=63), P, P, None, P, P, None) == _abi.E_SHAPE


def test_tensor_calls_refuse_what_does_not_fit():
    bf = dict(dtype=torch.bfloat16)
    x, w, offs = torch.zeros((4, 8), **bf), torch.zeros((2, 6, 8), **bf), torch.zeros(3, dtype=torch.int32)
    dy, u8 = torch.zeros((4, 6), **bf), dict(dtype=torch.uint8)
    bad = [
        (mx.layer_norm_fwd, (x.half(),)), (mx.layer_norm_fwd, (x[0],)), (mx.layer_norm_fwd, (x.t(),)),
        (mx.layer_norm_fwd, (x, torch.zeros(7, **bf))), (mx.layer_norm_fwd, (x, torch.zeros(8), torch.zeros(8, **bf))),
        (mx.layer_norm_fwd, (x[:1].expand(4, 8),)),
        (mx.layer_norm_bwd, (x, x[:3], torch.zeros(4), torch.zeros(4))),
        (mx.layer_norm_bwd, (x, x, torch.zeros(3), torch.zeros(4))),
        (mx.layer_norm_ckpt_bwd, (x, torch.zeros((4, 7), **u8), torch.zeros((4, 1), **u8), torch.zeros(4))),
        (mx.swiglu_ckpt_fwd, (x.float(),)), (mx.swiglu_ckpt_fwd, (torch.zeros((4, 7), **bf),)),
        (mx.swiglu_ckpt_bwd, (x, torch.zeros((4, 8), **u8), torch.zeros((8, 1), **u8))),
        (mx.grouped_gemm_fwd, (x.float(), w, offs)), (mx.grouped_gemm_fwd, (x, w[:, :, :7], offs)),
        (mx.grouped_gemm_fwd, (x, w, offs[:2])), (mx.grouped_gemm_fwd, (x, w, offs.long())),
        (mx.grouped_gemm_fwd, (x, w, offs, torch.float16)),
        (mx.grouped_gemm_dgrad, (x, w, offs)),
        (mx.grouped_gemm_wgrad, (dy, x[:3], offs)), (mx.grouped_gemm_wgrad, (dy, (torch.zeros((4, 8), **u8), torch.zeros((4, 2), **u8)), offs)),
        (mx.grouped_gemm_wgrad, (dy, x, offs, torch.bfloat16, torch.zeros((2, 6, 8)))),
        (mx.layer_norm_fwd, (x,)), (mx.swiglu_ckpt_fwd, (x,)), (mx.grouped_gemm_fwd, (x, w, offs)),  # not on a GPU
    ]
    for fn, args in bad:
        with pytest.raises(ValueError):
            fn(*args)


def test_tensor_calls_refuse_what_is_empty_or_absent():
    bf, u8 = dict(dtype=torch.bfloat16), dict(dtype=torch.uint8)
    x, w, offs = torch.zeros((4, 8), **bf), torch.zeros((2, 6, 8), **bf), torch.zeros(3, dtype=torch.int32)
    dy, f, q, s = torch.zeros((4, 6), **bf), torch.zeros(4), torch.zeros((4, 8), **u8), torch.zeros((4, 1), **u8)
    bad = [
        (mx.layer_norm_fwd, (x[0, 0],)), (mx.layer_norm_bwd, (x[0, 0], x, f, f)),
        (mx.layer_norm_bwd, (x, x, None, f)), (mx.layer_norm_bwd, (x, x, f, None)), (mx.layer_norm_bwd, (x, None, f, f)),
        (mx.layer_norm_ckpt_bwd, (x, None, s, f)), (mx.layer_norm_ckpt_bwd, (x, q, None, f)),
        (mx.layer_norm_ckpt_bwd, (x, q, s, None)),
        (mx.swiglu_ckpt_bwd, (x, None, s)), (mx.swiglu_ckpt_bwd, (x, torch.zeros((8, 8), **u8), None)),
        (mx.grouped_gemm_wgrad, (dy, None, offs)), (mx.grouped_gemm_wgrad, (dy, (None, s), offs)),
        (mx.grouped_gemm_wgrad, (dy, (q, None), offs)),
    ]
    for o in (None, offs[:0], offs[0], offs.view(1, 3)):
        bad += [(mx.grouped_gemm_fwd, (x, w, o)), (mx.grouped_gemm_dgrad, (dy, w, o)), (mx.grouped_gemm_wgrad, (dy, x, o)),
                (mx.grouped_gemm_wgrad, (dy, (q, s), o)),
                (mx.grouped_gemm_wgrad, (dy, x, o, None, torch.zeros((2, 6, 8))))]
    wrong = []
    for fn, args in bad:
        try:
            fn(*args)
        except ValueError:
            continue
        except Exception as e:  # noqa: BLE001
            wrong.append((fn.__name__, type(e).__name__))
            continue
        wrong.append((fn.__name__, "accepted"))
    assert not wrong


@pytest.mark.parametrize("src", ["norm.hip", "swiglu_ckpt.hip", "grouped.hip"])
def test_no_scratch_and_lds_fits(src):
    for k in _kernel_metadata(src):
        assert int(k.get("private_segment_fixed_size", 0)) == 0, (k["name"], "uses scratch")
        assert int(k.get("vgpr_spill_count", 0)) == 0, (k["name"], "spills VGPRs")
        assert int(k.get("group_segment_fixed_size", 0)) <= LDS_LIMIT, (k["name"], "LDS over 160 KB")
