"""Routed experts with 4-bit products: a training step, and serving of a few tokens with 8-bit rows.

    python examples/expert_mlp_mxfp4.py [--tokens 4096 --model 2048 --hidden 1408 --experts 16 --topk 6]

y = x + sum_k p[t, k] W2[e] swiglu(W13[e] x[t]),  e = choice[t, k]

Routing plan (segments of whole 128-row panels) -> tokens gathered and quantised along both directions in one pass ->
product -> SwiGLU -> quantised -> product -> combine onto x. Every product, forward and backward, has both operands in
MXFP4: the forward along rows, the input gradients with the weights' operands along columns, the weight gradients with all
operands along columns. Quantisation counts as the identity in the chain rule. Between forward and backward the block keeps
operands along columns (4.25 bits an element), the gate and up rows in MXFP8 and the second product's BF16 rows, which the
gradient of the router's weights takes.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_mixed_precision_amd as mx  # noqa: E402

BOTH = mx.ROW | mx.COL


class ExpertMlp4:
    """w13 [E, 2F, D] (gate rows, then up rows), w2 [E, D, F], BF16 or FP32: quantised once per set of weights."""

    def __init__(self, w13, w2):
        self.E = w13.shape[0]
        q, s, qt, st = mx.mxfp4_quantize(w13, BOTH)
        self.w13, self.w13_t = (q, s), (qt, st)
        q, s, qt, st = mx.mxfp4_quantize(w2, BOTH)
        self.w2, self.w2_t = (q, s), (qt, st)

    def forward(self, x, choice, weight):
        """x [T, D] BF16, choice [T, k] int32 experts, weight [T, k]. Returns y and what backward takes."""
        T, k = choice.shape
        plan = mx.route_plan(choice, self.E, 128, (T * k + self.E * 127) // 128 * 128)
        offs = plan["offs"]
        xq, xs, xqt, xst = mx.mxfp4_quantize(x, BOTH, plan=plan)
        gu = mx.grouped_gemm_mxfp4_fwd((xq, xs), self.w13, offs)
        h, qg, sg = mx.swiglu_ckpt_fwd(gu)
        hq, hs, hqt, hst = mx.mxfp4_quantize(h, BOTH)
        yp = mx.grouped_gemm_mxfp4_fwd((hq, hs), self.w2, offs)
        return mx.combine_fwd(yp, weight, plan, x), dict(x=(xqt, xst), gu=(qg, sg), h=(hqt, hst), yp=yp, plan=plan, weight=weight)

    def backward(self, dy, kept):
        """dy [T, D] BF16. Returns dx (BF16), and FP32 gradients of the router's weights, w13 and w2."""
        plan = kept["plan"]
        offs = plan["offs"]
        dyp, dweight = mx.combine_bwd(dy, kept["yp"], kept["weight"], plan)
        q, s, qt, st = mx.mxfp4_quantize(dyp, BOTH)
        dh = mx.grouped_gemm_mxfp4_fwd((q, s), self.w2_t, offs)
        dw2 = mx.grouped_gemm_mxfp4_wgrad((qt, st), kept["h"], offs, out_dtype=torch.float32)
        dgu, _ = mx.swiglu_ckpt_bwd(dh, *kept["gu"], recompute=False)
        q, s, qt, st = mx.mxfp4_quantize(dgu, BOTH)
        dxe = mx.grouped_gemm_mxfp4_fwd((q, s), self.w13_t, offs)
        dw13 = mx.grouped_gemm_mxfp4_wgrad((qt, st), kept["x"], offs, out_dtype=torch.float32)
        return mx.dispatch_bwd(dxe, plan, dy.shape[0]) + dy, dweight, dw13, dw2

    def serve(self, x, choice, weight):
        """The forward alone for a few tokens: rows in MXFP8, weights in MXFP4, no padding."""
        T, k = choice.shape
        plan = mx.route_plan(choice, self.E, 1, T * k)
        offs = plan["offs"]
        gu = mx.grouped_gemm_mxfp4_fwd(mx.mxfp4_quantize(x, e4m3=True, plan=plan)[:2], self.w13, offs)
        h, _, _ = mx.swiglu_ckpt_fwd(gu)
        yp = mx.grouped_gemm_mxfp4_fwd(mx.mxfp4_quantize(h, e4m3=True)[:2], self.w2, offs)
        return mx.combine_fwd(yp, weight, plan, x)


def make(D, F, E, seed=0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s: 0.02 * torch.randn(s, generator=g, device=device)  # noqa: E731
    return r(E, 2 * F, D).bfloat16(), r(E, D, F).bfloat16()


def tokens(T, D, E, k, seed=1, device="cuda"):
    """Inputs, k distinct experts per token with uneven popularity, weights that sum to one, output gradients."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    x = torch.randn((T, D), generator=g, device=device).bfloat16()
    logits = torch.randn((T, E), generator=g, device=device) + torch.randn((1, E), generator=g, device=device)
    top, choice = logits.topk(k, 1)
    return x, choice.int(), top.softmax(1), torch.randn((T, D), generator=g, device=device).bfloat16()


def _ms(fn, n=10):
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(n):
        fn()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / n * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, v in (("tokens", 4096), ("model", 2048), ("hidden", 1408), ("experts", 16), ("topk", 6)):
        ap.add_argument("--" + name, type=int, default=v)
    a = ap.parse_args()
    w13, w2 = make(a.model, a.hidden, a.experts)
    mlp = ExpertMlp4(w13, w2)
    x, choice, weight, dy = tokens(a.tokens, a.model, a.experts, a.topk)
    y, kept = mlp.forward(x, choice, weight)
    grads = mlp.backward(dy, kept)
    print(f"{a.tokens} tokens: |y| {y.float().norm():.1f}, |dweight| {grads[1].norm():.3g}, |dw13| {grads[2].norm():.3g}, "
          f"|dw2| {grads[3].norm():.3g}")
    print(f"weights quantised {_ms(lambda: ExpertMlp4(w13, w2)):.3f} ms, forward {_ms(lambda: mlp.forward(x, choice, weight)):.3f} ms, "
          f"backward {_ms(lambda: mlp.backward(dy, kept)):.3f} ms")
    x1, c1, p1 = x[:8], choice[:8].contiguous(), weight[:8]
    print(f"8 tokens served: {_ms(lambda: mlp.serve(x1, c1, p1)):.3f} ms")


if __name__ == "__main__":
    main()
