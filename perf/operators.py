"""Workloads of the training-block operators: layer norm, ragged expert products, SwiGLU with 8-bit checkpoints.

``run`` computes an operator either in its plain form (elementary torch operations in float32, rounded once at the
end) or, with ``own`` set, through the package's entry points. ``exact`` is the definition in float64.

Checkpoints are row-wise MXFP8: groups of 32 along a row (the last may be short), E4M3 codes and one E8M0 scale byte
per group. They are returned as torch's float8 types, i.e. as the numbers the bytes stand for.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the norm in front of a block while eight sequences are decoded: one row each, latency counts
        {"name": "norm_fwd_decode", "op": "norm_fwd", "rows": 8, "cols": 2048, "type": "bf16", "ckpt": False},
        # the same norm in training at the wide model size, its normalised rows kept in 8 bits for the backward pass
        {"name": "norm_fwd_train_ckpt", "op": "norm_fwd", "rows": 8192, "cols": 7168, "type": "bf16", "ckpt": True},
        # backward of an odd-sized float32 norm (small models, a float32 residual stream)
        {"name": "norm_bwd_f32_odd", "op": "norm_bwd", "rows": 4093, "cols": 1411, "type": "f32", "ckpt": False},
        # backward at the narrow model size from the 8-bit checkpoint
        {"name": "norm_bwd_train_ckpt", "op": "norm_bwd", "rows": 16384, "cols": 2048, "type": "bf16", "ckpt": True},
        # one expert-parallel rank of a 16-expert block: first product forward
        {"name": "gemm_fwd_rank", "op": "gemm_fwd", "E": 16, "M": 24576, "N": 2816, "K": 2048, "out": "bf16"},
        # the same product while eight tokens with six experts each are decoded: the weights' bytes count
        {"name": "gemm_fwd_decode", "op": "gemm_fwd", "E": 16, "M": 48, "N": 2816, "K": 2048, "out": "bf16"},
        # input gradient of the second product at the wide model size
        {"name": "gemm_dgrad_wide", "op": "gemm_dgrad", "E": 8, "M": 16384, "N": 7168, "K": 2048, "out": "bf16"},
        # weight gradient of the rank's first product into float32 gradients
        {"name": "gemm_wgrad_rank", "op": "gemm_wgrad", "E": 16, "M": 24576, "N": 2816, "K": 2048, "out": "f32",
         "ckpt": False},
        # weight gradient from an input kept in 8 bits, many small experts and odd sizes
        {"name": "gemm_wgrad_ckpt_odd", "op": "gemm_wgrad", "E": 40, "M": 6001, "N": 1400, "K": 1056, "out": "bf16",
         "ckpt": True},
        # activation of a short prompt
        {"name": "swiglu_fwd_prompt", "op": "swiglu_fwd", "rows": 192, "F": 1408},
        # activation of one rank's training step, forward and backward
        {"name": "swiglu_fwd_rank", "op": "swiglu_fwd", "rows": 24576, "F": 1408},
        {"name": "swiglu_bwd_rank", "op": "swiglu_bwd", "rows": 24576, "F": 1408},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if v != 3072:
            return min(max(v, lo), hi)


def _width(rng, lo, hi):
    """A width: one in four as drawn (odd ones among them), the others multiples of 32, as models have."""
    v = _log(rng, lo, hi)
    if rng.random() < 0.25:
        return v
    v = max(32, v // 32 * 32)
    return v if v != 3072 else 3104


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "gemm_fwd", "gemm_dgrad", "gemm_wgrad", "swiglu_fwd", "swiglu_bwd"])
    if op.startswith("norm"):
        cols = _width(rng, 64, 14336)
        rows = _log(rng, 1, min(32768, (1 << 26) // cols))
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["bf16", "bf16", "f32"]),
                "ckpt": rng.random() < 0.5}
    if op.startswith("swiglu"):
        F = _width(rng, 64, 14336)
        return {"op": op, "rows": _log(rng, 1, min(32768, (1 << 25) // F)), "F": F}
    while True:
        E, M = _log(rng, 1, 64), _log(rng, 1, 32768)
        N, K = _width(rng, 64, 8192), _width(rng, 64, 8192)
        if M * N * K <= 1.4e11 and E * N * K <= 3e8:
            break
    case = {"op": op, "E": E, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "f32"])}
    if op == "gemm_wgrad":
        case["ckpt"] = rng.random() < 0.4
    return case


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        R, C, b = case["rows"], case["cols"], BYTES[case["type"]]
        ck = R * C + R * -(-C // 32)
        if op == "norm_fwd":  # x, w, b -> y, and mean and rstd or rstd and the checkpoint
            return {"bytes": 2 * b * R * C + 2 * b * C + (ck + 4 * R if case["ckpt"] else 8 * R), "flops": 8 * R * C}
        # dy, x or its checkpoint, w -> dx, dw, db
        seen = ck + 4 * R if case["ckpt"] else b * R * C + 8 * R
        return {"bytes": 2 * b * R * C + seen + b * C + 8 * C, "flops": 12 * R * C}
    if op.startswith("swiglu"):
        R, F = case["rows"], case["F"]
        ck = 2 * R * F + 2 * R * -(-F // 32)
        return {"bytes": (6 * R * F if op == "swiglu_fwd" else 8 * R * F) + ck, "flops": (6 if op == "swiglu_fwd" else 14) * R * F}
    E, M, N, K, o = case["E"], case["M"], case["N"], case["K"], BYTES[case["out"]]
    met = min(E, M)  # experts that can have a row
    if op == "gemm_fwd":
        moved = 2 * M * K + 2 * met * N * K + o * M * N
    elif op == "gemm_dgrad":
        moved = 2 * M * N + 2 * met * N * K + o * M * K
    else:
        moved = 2 * M * N + (M * K + M * -(-K // 32) if case["ckpt"] else 2 * M * K) + o * E * N * K
    return {"bytes": moved, "flops": 2 * M * N * K}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


def _residual(g, rows, cols):
    """A residual stream: rows of differing scale and mean, a few columns much larger than the others."""
    x = _normal(g, rows, cols) * torch.exp(0.5 * _normal(g, rows, 1)) + 0.3 * _normal(g, rows, 1)
    return x * (1.0 + 15.0 * (torch.rand((1, cols), generator=g, device=DEV) < 0.005))


def _counts(g, E, M):
    """Rows per expert, uneven as a router leaves them; from eight experts on some get none."""
    share = torch.rand(E, generator=g, device=DEV).cpu() ** 2 + 1e-3
    if E >= 8:
        share[torch.randperm(E, generator=g, device=DEV).cpu()[: E // 8]] = 0.0
    edge = torch.cumsum(share.double() / share.double().sum(), 0) * M
    edge = edge.round().to(torch.int64).clamp(0, M)
    edge[-1] = M
    return [0] + edge.tolist()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op.startswith("norm"):
        t = TYPES[case["type"]]
        x = _residual(g, case["rows"], case["cols"]).to(t)
        s["w"] = (1.0 + _normal(g, case["cols"], std=0.1)).to(t)
        if op == "norm_fwd":
            s["x"], s["b"] = x, _normal(g, case["cols"], std=0.1).to(t)
            return s
        s["dy"] = _normal(g, case["rows"], case["cols"]).to(t)
        xf = x.float()
        mean = xf.mean(1)
        s["rstd"] = ((xf - mean[:, None]).square().mean(1) + EPS).rsqrt()
        if case["ckpt"]:
            s["q"], s["s"] = _mx((xf - mean[:, None]) * s["rstd"][:, None])
        else:
            s["x"], s["mean"] = x, mean
        return s
    if op.startswith("swiglu"):
        gu = _normal(g, case["rows"], 2 * case["F"], std=1.5).bfloat16()
        if op == "swiglu_fwd":
            s["gu"] = gu
            return s
        q, sc = _mx(gu.float().view(2 * case["rows"], case["F"]))
        s["q"], s["s"] = q, sc
        s["dh"] = _normal(g, case["rows"], case["F"]).bfloat16()
        return s
    E, M, N, K = case["E"], case["M"], case["N"], case["K"]
    s["bounds"] = _counts(g, E, M)
    s["offs"] = torch.tensor(s["bounds"], dtype=torch.int32, device=DEV)
    if op != "gemm_wgrad":
        s["w"] = (torch.randn((E, N, K), generator=g, device=DEV, dtype=torch.bfloat16) * 0.02)
    if op != "gemm_dgrad":
        s["x"] = _normal(g, M, K).bfloat16()
    if op != "gemm_fwd":
        s["dy"] = _normal(g, M, N).bfloat16()
    if case.get("ckpt"):
        s["q"], s["s"] = _mx(s.pop("x").float())
    return s


# ------------------------------------------------------------------ plain forms

def _pow2(byte):
    """2^(byte - 127) as float32 for bytes 0..254, from its bits."""
    return torch.where(byte == 0, 0x00400000, byte.to(torch.int32) << 23).to(torch.int32).view(torch.float32)


def _mx(v):
    """Row-wise MXFP8 of float32 v [rows, cols], rounded to BF16 first: codes [rows, cols] and scale bytes, uint8."""
    rows, cols = v.shape
    n = -(-cols // 32)
    p = torch.nn.functional.pad(v.bfloat16().float(), (0, n * 32 - cols)).view(rows, n, 32)
    amax = p.abs().amax(2)
    byte = torch.where(amax == 0, 0, (torch.frexp(amax).exponent - 1 - 8).clamp(-127, 127) + 127)
    q = (p * _pow2(254 - byte)[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(rows, n * 32)[:, :cols].contiguous().view(torch.uint8), byte.to(torch.uint8)


def _unmx(q, s):
    """The float32 values of codes and scale bytes."""
    scale = _pow2(s.to(torch.int32)).repeat_interleave(32, 1)[:, : q.shape[1]]
    return q.view(torch.float8_e4m3fn).float() * scale


def _numbers(q, s):
    """Codes and scale bytes as the numbers that they stand for."""
    return q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)


def _plain(s):
    op = s["op"]
    if op == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = (xc.square().mean(1, keepdim=True) + EPS).rsqrt()
        xh = xc * rstd
        y = (xh * s["w"].float() + s["b"].float()).to(s["x"].dtype)
        return (y, rstd[:, 0], *_numbers(*_mx(xh))) if s["ckpt"] else (y, mean[:, 0], rstd[:, 0])
    if op == "norm_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = _unmx(s["q"], s["s"]) if s["ckpt"] else (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["w"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        return dx.to(s["dy"].dtype), (dy * xh).sum(0), dy.sum(0)
    if op == "swiglu_fwd":
        g, u = s["gu"].float().chunk(2, 1)
        h = (g * torch.sigmoid(g) * u).bfloat16()
        return (h, *_numbers(*_mx(s["gu"].float().view(-1, s["F"]))))
    if op == "swiglu_bwd":
        g, u = _unmx(s["q"], s["s"]).view(-1, 2 * s["F"]).chunk(2, 1)
        dh, sg = s["dh"].float(), torch.sigmoid(g)
        dgu = torch.cat([dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg], 1)
        return dgu.bfloat16(), (g * sg * u).bfloat16()
    at, out = s["bounds"], TYPES[s["out"]]
    # one library product per expert that has rows: the fewest operations that elementary torch needs here
    segments = [(e, a, b) for e, (a, b) in enumerate(zip(at, at[1:])) if b > a]
    if op == "gemm_fwd":
        return torch.cat([s["x"][a:b].float() @ s["w"][e].float().t() for e, a, b in segments]).to(out)
    if op == "gemm_dgrad":
        return torch.cat([s["dy"][a:b].float() @ s["w"][e].float() for e, a, b in segments]).to(out)
    x = _unmx(s["q"], s["s"]) if s["ckpt"] else s["x"].float()
    dy = s["dy"].float()
    dw = torch.zeros((s["E"], s["N"], s["K"]), dtype=torch.float32, device=dy.device)
    for e, a, b in segments:
        torch.mm(dy[a:b].t(), x[a:b], out=dw[e])
    return dw.to(out)


# ------------------------------------------------------------------ one pass

def _own(s):
    import mxfp8_mixed_precision_amd as mx
    op = s["op"]
    if op == "norm_fwd":
        if s["ckpt"]:
            y, rstd, q, sc = mx.layer_norm_ckpt_fwd(s["x"], s["w"], s["b"], eps=EPS)
            return (y, rstd, *_numbers(q, sc))
        return mx.layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS)
    if op == "norm_bwd":
        if s["ckpt"]:
            return mx.layer_norm_ckpt_bwd(s["dy"], s["q"], s["s"], s["rstd"], s["w"])
        return mx.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    if op == "swiglu_fwd":
        h, q, sc = mx.swiglu_ckpt_fwd(s["gu"])
        return (h, *_numbers(q, sc))
    if op == "swiglu_bwd":
        return mx.swiglu_ckpt_bwd(s["dh"], s["q"], s["s"])
    out = TYPES[s["out"]]
    if op == "gemm_fwd":
        return mx.grouped_gemm_fwd(s["x"], s["w"], s["offs"], out_dtype=out)
    if op == "gemm_dgrad":
        return mx.grouped_gemm_dgrad(s["dy"], s["w"], s["offs"], out_dtype=out)
    if s["ckpt"]:
        return mx.grouped_gemm_wgrad(s["dy"], (s["q"], s["s"]), s["offs"], out_dtype=out)
    return mx.grouped_gemm_wgrad(s["dy"], s["x"], s["offs"], out_dtype=out)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ float64

def _two64(e):
    """2^e for whole e, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _codes64(v):
    """MXFP8 of v, whose definition rounds it to BF16 first: codes and scales as numbers, from the logarithm's floor."""
    rows, cols = v.shape
    n = -(-cols // 32)
    p = torch.zeros((rows, n * 32), dtype=torch.float64, device=v.device)
    p[:, :cols] = v.to(torch.bfloat16).double()
    p = p.view(rows, n, 32)
    top = p.abs().amax(2)
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    e = torch.where(_two64(e) > top, e - 1, e)
    e = torch.where(_two64(e + 1) <= top, e + 1, e)
    e = torch.where(top > 0, (e - 8).clamp(-127, 127), torch.full_like(e, -127))
    r = p / _two64(e)[:, :, None]
    step = _two64(torch.floor(torch.log2(r.abs().clamp_min(2.0 ** -6))) - 3)
    codes = (torch.round(r / step) * step).clamp(-448.0, 448.0)
    return codes.view(rows, n * 32)[:, :cols], _two64(e)


def _decode64(q, s):
    """E4M3 and E8M0 bytes as numbers, from their bit fields."""
    i = q.to(torch.int64)
    field, frac = (i >> 3) & 15, (i & 7).double()
    v = torch.where(field == 0, frac * 2.0 ** -9, (8 + frac) * _two64(field - 10))
    v = torch.where(i >= 128, -v, v)
    return v * _two64(s.to(torch.int64) - 127).repeat_interleave(32, 1)[:, : q.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        x = s["x"].double()
        mean = x.sum(1) / case["cols"]
        var = (x - mean[:, None]).square().sum(1) / case["cols"]
        rstd = 1.0 / torch.sqrt(var + EPS)
        xh = (x - mean[:, None]) * rstd[:, None]
        y = xh * s["w"].double() + s["b"].double()
        # the checkpoint is taken of rows rounded to BF16: where that rounding is nearly a tie, float32 and float64 may
        # fall on either side and a code (a sixteenth of its value) or a scale follows, so it has no one value here
        return (y, rstd, None, None) if case["ckpt"] else (y, mean, rstd)
    if op == "norm_bwd":
        dy, rstd, C = s["dy"].double(), s["rstd"].double()[:, None], case["cols"]
        xh = _decode64(s["q"], s["s"]) if case["ckpt"] else (s["x"].double() - s["mean"].double()[:, None]) * rstd
        g = dy * s["w"].double()
        dx = (g - g.sum(1, keepdim=True) / C - xh * ((g * xh).sum(1, keepdim=True) / C)) * rstd
        return dx, (dy * xh).sum(0), dy.sum(0)
    if op == "swiglu_fwd":
        v, F = s["gu"].double(), case["F"]
        return (v[:, :F] / (1.0 + torch.exp(-v[:, :F])) * v[:, F:], *_codes64(v.view(-1, F)))
    if op == "swiglu_bwd":
        F = case["F"]
        v = _decode64(s["q"], s["s"]).view(-1, 2 * F)
        g, u, dh = v[:, :F], v[:, F:], s["dh"].double()
        sg = 1.0 / (1.0 + torch.exp(-g))
        return torch.cat([dh * u * (sg + g * sg * (1.0 - sg)), dh * g * sg], 1), g * sg * u
    at = s["bounds"]
    if op == "gemm_wgrad":
        x = _decode64(s["q"], s["s"]) if case["ckpt"] else s["x"].double()
        dw = torch.zeros((case["E"], case["N"], case["K"]), dtype=torch.float64, device=x.device)
        for e in range(case["E"]):
            dw[e] = s["dy"][at[e]:at[e + 1]].double().t() @ x[at[e]:at[e + 1]]
        return dw
    a, w = (s["x"], s["w"].transpose(1, 2)) if op == "gemm_fwd" else (s["dy"], s["w"])
    y = torch.zeros((case["M"], w.shape[2]), dtype=torch.float64, device=a.device)
    for e in range(case["E"]):
        y[at[e]:at[e + 1]] = a[at[e]:at[e + 1]].double() @ w[e].double()
    return y
