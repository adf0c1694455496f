"""A pre-norm expert block in BF16 on unpadded rows, its activations kept in 8 bits until the backward.

    python examples/expert_block.py [--tokens 4096 --model 2048 --hidden 1408 --experts 16 --topk 6]

y = x + sum_k p[t, k] W2[e] swiglu(W13[e] norm(x)[t]),  e = choice[t, k]

Layer norm -> routing plan and dispatch (segments not padded) -> ragged product -> SwiGLU -> ragged product ->
combine. What the backward needs is kept as MXFP8: the normalised rows, the first product's input and
the gate and up rows (1.03 bytes per element instead of 2); the second product's input is computed again.
The router is an input here: its choices and weights are given.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_mixed_precision_amd as mx  # noqa: E402


class ExpertBlock:
    """norm_w, norm_b [D]; w13 [E, 2F, D] (gate rows, then up rows); w2 [E, D, F]; all BF16."""

    def __init__(self, norm_w, norm_b, w13, w2):
        self.norm_w, self.norm_b, self.w13, self.w2 = norm_w, norm_b, w13, w2

    def forward(self, x, choice, weight, keep=True):
        """x [T, D] BF16, choice [T, k] int32 experts, weight [T, k] FP32. Returns y and, with keep, what
        backward takes."""
        (T, D), k, E = x.shape, choice.shape[1], self.w13.shape[0]
        if keep:
            n, rstd, qn, sn = mx.layer_norm_ckpt_fwd(x, self.norm_w, self.norm_b)
        else:
            n = mx.layer_norm_fwd(x, self.norm_w, self.norm_b, stats=False)
        plan = mx.route_plan(choice, E, 1, T * k)  # pad_multiple 1: every row is a token's
        offs = plan["offs"]
        xp = mx.dispatch_fwd(n, plan)
        gu = mx.grouped_gemm_fwd(xp, self.w13, offs)
        h, qh, sh = mx.swiglu_ckpt_fwd(gu)
        yp = mx.grouped_gemm_fwd(h, self.w2, offs)
        y = mx.combine_fwd(yp, weight, plan, x)
        if not keep:
            return y
        qx, sx, _, _ = mx.quantize(xp, mx.ROW)
        return y, dict(norm=(qn, sn, rstd), x=(qx, sx), h=(qh, sh), plan=plan, weight=weight)

    def backward(self, dy, kept):
        """dy [T, D] BF16. Returns dx (BF16) and the FP32 gradients of norm_w, norm_b, w13 and w2."""
        plan = kept["plan"]
        offs = plan["offs"]
        dyp, _ = mx.combine_bwd(dy, None, kept["weight"], plan)  # (the weights are given: no gradient of theirs)
        dh = mx.grouped_gemm_dgrad(dyp, self.w2, offs)
        dgu, h = mx.swiglu_ckpt_bwd(dh, *kept["h"])
        dw2 = mx.grouped_gemm_wgrad(dyp, h, offs, out_dtype=torch.float32)
        dxp = mx.grouped_gemm_dgrad(dgu, self.w13, offs)
        dw13 = mx.grouped_gemm_wgrad(dgu, kept["x"], offs, out_dtype=torch.float32)
        dn = mx.dispatch_bwd(dxp, plan, dy.shape[0])
        dx, dnw, dnb = mx.layer_norm_ckpt_bwd(dn, *kept["norm"], self.norm_w)
        return (dx.float() + dy.float()).bfloat16(), dnw, dnb, dw13, dw2


def make(D, F, E, seed=0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    return ExpertBlock((1 + 0.1 * r(D)).bfloat16(), (0.1 * r(D)).bfloat16(), (0.02 * r(E, 2 * F, D)).bfloat16(),
                       (0.02 * r(E, D, F)).bfloat16())


def tokens(T, D, E, k, seed=1, device="cuda"):
    """Inputs, k distinct experts per token with uneven popularity, weights that sum to one, output gradients."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    x = torch.randn((T, D), generator=g, device=device).bfloat16()
    logits = torch.randn((T, E), generator=g, device=device) + torch.randn((1, E), generator=g, device=device)
    top, choice = logits.topk(k, 1)
    dy = torch.randn((T, D), generator=g, device=device).bfloat16()
    return x, choice.int(), top.softmax(1), dy


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
    block = make(a.model, a.hidden, a.experts)
    x, choice, weight, dy = tokens(a.tokens, a.model, a.experts, a.topk)
    y, kept = block.forward(x, choice, weight)
    grads = block.backward(dy, kept)
    size = sum(t.numel() * t.element_size() for v in (kept["norm"], kept["x"], kept["h"]) for t in v)
    print(f"{a.tokens} tokens, kept for the backward: {size / 2**20:.1f} MiB; |y| {y.float().norm():.1f}, "
          f"|dw13| {grads[3].norm():.3g}, |dw2| {grads[4].norm():.3g}")
    print(f"forward {_ms(lambda: block.forward(x, choice, weight)):.3f} ms, "
          f"backward {_ms(lambda: block.backward(dy, kept)):.3f} ms")
    x1, c1, w1 = x[:8], choice[:8].contiguous(), weight[:8]
    print(f"8 tokens, forward alone: {_ms(lambda: block.forward(x1, c1, w1, keep=False)):.3f} ms")


if __name__ == "__main__":
    main()
