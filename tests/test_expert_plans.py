"""A plan knows the number of its experts per token: calls with another number of tokens that divides the assignments are refused."""
import pytest
import torch

import mxfp8_mixed_precision_amd as mx
from gpu_util import require_gpu


def calls(plan, dev="cpu"):
    """Calls with 16 tokens on a plan of 8 tokens and 6 experts each, and with 8 tokens and weights for 6 and for 3."""
    rows = plan["row_assign"].numel()
    x, h, w = torch.zeros((16, 32), device=dev), torch.zeros((rows, 32), device=dev), torch.zeros((16, 3), device=dev)
    return [lambda: mx.dispatch_fwd(x, plan), lambda: mx.dispatch_bwd(h, plan, 16), lambda: mx.combine_fwd(h, w, plan),
            lambda: mx.combine_bwd(x, h, w, plan), lambda: mx.mxfp4_quantize(x, plan=plan), lambda: mx.dispatch_bwd(h, plan, 0)]


def test_another_number_of_tokens_is_refused():
    i32 = dict(dtype=torch.int32)
    plan = {"offs": torch.zeros(5, **i32), "row_assign": torch.zeros(48, **i32), "assign_row": torch.zeros(48, **i32), "topk": 6}
    for i, fn in enumerate(calls(plan)):
        with pytest.raises(ValueError, match="tokens"):
            fn()
    with pytest.raises(ValueError, match="GPU"):  # (the right number gets further)
        mx.dispatch_bwd(torch.zeros((48, 32)), plan, 8)
    with pytest.raises(ValueError, match="topk"):
        mx.dispatch_bwd(torch.zeros((48, 32)), {**plan, "topk": 0}, 8)


@pytest.mark.gpu
def test_plans_of_route_plan():
    require_gpu()
    for T, k in ((8, 6), (0, 6), (5, 1)):
        plan = mx.route_plan(torch.zeros((T, k), dtype=torch.int32, device="cuda"), 4, 1, T * k)
        assert plan["topk"] == k
        x = torch.randn((T, 32), device="cuda")
        xe = mx.dispatch_fwd(x, plan)
        assert torch.equal(mx.combine_fwd(xe, torch.full((T, k), 0.0, device="cuda"), plan, x), x)
    plan = mx.route_plan(torch.zeros((8, 6), dtype=torch.int32, device="cuda"), 4, 1, 48)
    for fn in calls(plan, "cuda"):
        with pytest.raises(ValueError, match="tokens"):
            fn()
