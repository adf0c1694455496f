"""Sizes that the routed-expert calls' documented limits allow are not refused, and those past them are (CPU: a call inside the
limits gets as far as the missing device), and on the GPU one such call."""
import pytest
import torch

import mxfp8_mixed_precision_amd as mx
from gpu_util import require_gpu
from mxfp8_mixed_precision_amd import _abi
from test_expert_abi import P, grouped, refused, route
from test_gpu_grouped_mx import close, operand, values

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that a kernel must not reach")


@no_gpu
@pytest.mark.parametrize("kw,inside", [
    (dict(E=1, M=65536, N=262144), True), (dict(E=1, M=1 << 20, N=16384), True), (dict(E=1024, M=1024, N=1 << 20), True),
    (dict(E=2, M=(1 << 30) - 512, N=512), True), (dict(E=2, M=1 << 30, N=512), False), (dict(E=1024, M=1 << 24, N=1 << 20), False)])
def test_forward_products(kw, inside):
    d = grouped(**kw, ldy=kw["N"])
    assert (refused(mx.mxf_grouped_gemm_mxfp4_fwd, d, P, P, P, P, P, P) != _abi.E_SHAPE) == inside


@no_gpu
@pytest.mark.parametrize("kw,inside", [
    (dict(E=1024, N=8192, K=65280), True), (dict(E=1024, N=16384, K=32512), True), (dict(E=1024, N=8192, K=65536), False),
    (dict(E=512, N=32768, K=32768), False)])
def test_weight_gradients(kw, inside):
    assert (refused(mx.mxf_grouped_gemm_mxfp4_wgrad, grouped(**kw), P, P, P, P, P, P) != _abi.E_SHAPE) == inside


@no_gpu
@pytest.mark.parametrize("tokens,D,topk,inside", [(1 << 20, 8192, 1, True), (1 << 29, 1, 2, True), (1 << 30, 1024, 1, True), (1 << 24, 65536, 64, True),
                                                  (1 << 30, 1025, 1, False), (1 << 24, 65537, 64, False)])
def test_rows_of_tokens(tokens, D, topk, inside):
    d = route(tokens=tokens, D=D, ldx=D, ldh=D, lddh=D, topk=topk, rows=1 << 30)
    for fn, n in ((mx.mxf_dispatch_fwd, 5), (mx.mxf_combine_bwd, 8)):
        assert (refused(fn, d, *[P] * n) != _abi.E_SHAPE) == inside
    assert (refused(mx.mxf_combine_fwd, d, P, P, P, None, P) != _abi.E_SHAPE) == inside


@no_gpu
def test_a_residual_in_the_result_s_place():
    """The last two chunks of a row overlap: a row would be read where it is written."""
    assert refused(mx.mxf_combine_fwd, route(), P, P, P, P << 1, P << 1) == _abi.E_ARG
    assert refused(mx.mxf_combine_fwd, route(), P, P, None, P << 1, P << 1) == _abi.E_ARG
    assert refused(mx.mxf_combine_fwd, route(), P, P, P, P << 2, P << 1) not in (_abi.E_ARG, _abi.E_SHAPE, _abi.E_ALIGN, _abi.E_NULL)


@pytest.mark.gpu
def test_rows_in_more_blocks_than_a_row_of_the_grid():
    """2^29 - 2^20 tokens of one element, two rows each, and 2^21 pad rows."""
    require_gpu()
    T, R = (1 << 29) - (1 << 20), 1 << 30
    i32 = dict(dtype=torch.int32, device="cuda")
    row = torch.arange(2 * T, **i32) ^ 0x15555  # its own inverse
    plan = {"offs": torch.tensor([0, R], **i32), "row_assign": torch.cat([row, torch.full((R - 2 * T,), -1, **i32)]), "assign_row": row}
    x = torch.randint(1, 100, (T, 1), dtype=torch.uint8, device="cuda")
    xe = mx.dispatch_fwd(x, plan)
    assert torch.equal(xe[:2 * T], x[row.long() // 2]) and not xe[2 * T:].any()
    h, dy, w = xe.bfloat16(), x.bfloat16(), torch.full((T, 2), 0.5, dtype=torch.bfloat16, device="cuda")
    w[:, 1] = 2
    del xe
    assert torch.equal(mx.combine_fwd(h, w, plan), (2.5 * x.float()).bfloat16())
    assert torch.equal(mx.dispatch_bwd(h, plan, T), 2 * dy)
    dh, dw = mx.combine_bwd(dy, h, w, plan)
    assert torch.equal(dh[:2 * T], (dy[row.long() // 2] * w.view(-1)[row.long()][:, None])) and not dh[2 * T:].any()
    assert torch.equal(dw, x.float().square().expand(T, 2))


@pytest.mark.gpu
def test_many_wide_rows():
    """2^20 tokens of 8192."""
    require_gpu()
    T, D = 1 << 20, 8192
    i32 = dict(dtype=torch.int32, device="cuda")
    row = torch.arange(T, **i32) ^ 0x5555
    plan = {"offs": torch.tensor([0, T], **i32), "row_assign": row, "assign_row": row}
    x = torch.randint(0, 100, (T, D), dtype=torch.int16, device="cuda").bfloat16()
    w = torch.full((T, 1), 0.5, device="cuda")
    xe = mx.dispatch_fwd(x, plan)
    assert torch.equal(xe, x[row.long()])
    assert torch.equal(mx.combine_fwd(xe, w, plan), 0.5 * x)
    dh, dw = mx.combine_bwd(x, xe, w, plan)
    assert torch.equal(dh, 0.5 * xe)
    assert (dw[:, 0].double() - torch.stack([v.double().square().sum(1) for v in x.split(1 << 16)]).view(-1)).abs().max() <= D * 2.0 ** -24 * D * 1e4


@pytest.mark.gpu
def test_forward_product_of_many_tiles():
    """2^20 rows and 16392 columns: zeros but for the first and last rows."""
    require_gpu()
    M, N, K = 1 << 20, 16392, 128
    small, w = operand(600, K, 1), operand(N, K, 2, lead=(1,))
    q = torch.zeros((1, M, 64), dtype=torch.uint8, device="cuda")
    s = torch.zeros((1, M, 4), dtype=torch.uint8, device="cuda")
    for t, v in ((q, small[0]), (s, small[1])):
        t[:, :300], t[:, -300:] = v[:, :300], v[:, 300:]
    y = mx.grouped_gemm_mxfp4_fwd((q, s), w, torch.tensor([0, M], dtype=torch.int32, device="cuda"))
    X, W = values(*small), values(*w)[0]
    close(torch.cat([y[:300], y[-300:]]), X @ W.t(), X.abs() @ W.abs().t(), K, None, "rows")
    assert not y[300:-300].any()
