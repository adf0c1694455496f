"""Sizes that the routed-expert calls' documented limits allow are not refused, and those past them are (CPU: a call inside the
limits gets as far as the missing device), and on the GPU one such call."""
import pytest
import torch

import mxfp8_mixed_precision_amd as mx
from gpu_util import require_gpu
from mxfp8_mixed_precision_amd import _abi
from test_expert_abi import P, grouped, refused
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
