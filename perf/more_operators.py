"""Workloads of the routed-expert operators around the products: token rows sorted by expert and back with the
router's weights, their gradients, microscaled 4-bit operands, and the expert products on them.

``run`` computes an operator either in its plain form (elementary torch operations in float32, rounded once at the
end) or, with ``own`` set, through the package's entry points. ``exact`` is the definition in float64.

A microscaled operand holds a matrix [rows, K] for products along K: per 128 of K a plane of scale bytes
[rows, 4] (E8M0, one per group of 32) and panels of codes, 64 bytes a row: one panel of E2M1 codes, two to a byte, the
lower K in the lower four bits, or two panels of E4M3 codes. K is padded to 128 with zeros. Codes are returned
as the values that they stand for, scale bytes as torch's float8_e8m0fnu.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the experts' rows of eight decoded tokens weighted and added up: latency counts
        {"name": "combine_fwd_decode", "op": "combine_fwd", "T": 8, "topk": 6, "E": 64, "D": 2048, "pad": 1,
         "type": "bf16", "weights": "f32", "drop": 0.0},
        # the same for one rank's training step: 24576 rows before padding
        {"name": "combine_fwd_rank", "op": "combine_fwd", "T": 4096, "topk": 6, "E": 16, "D": 2048, "pad": 128,
         "type": "bf16", "weights": "bf16", "drop": 0.0},
        # its gradient at the wide model size: every row's gradient, and each weight's from two long rows
        {"name": "combine_bwd_wide", "op": "combine_bwd", "T": 4096, "topk": 8, "E": 32, "D": 7168, "pad": 128,
         "type": "bf16", "weights": "f32", "drop": 0.0},
        # tokens copied to their experts' rows
        {"name": "dispatch_fwd_rank", "op": "dispatch_fwd", "T": 4096, "topk": 6, "E": 16, "D": 2048, "pad": 128,
         "type": "bf16", "drop": 0.0},
        # its gradient in float32 at odd sizes, where a capacity has dropped some of the assignments
        {"name": "dispatch_bwd_odd_f32", "op": "dispatch_bwd", "T": 1531, "topk": 2, "E": 7, "D": 1411, "pad": 1,
         "type": "f32", "drop": 0.06},
        # eight decoded tokens gathered by expert and quantised to 8-bit operands
        {"name": "quant_decode_e4m3", "op": "quant", "T": 8, "topk": 6, "E": 16, "cols": 2048, "pad": 1, "type": "bf16",
         "e4m3": True, "col": False},
        # the rank's tokens gathered by expert and quantised to 4 bits, as they lie for the forward product and
        # transposed for the weight gradient
        {"name": "quant_rank_dual", "op": "quant", "T": 4096, "topk": 6, "E": 16, "cols": 2048, "pad": 128,
         "type": "bf16", "e4m3": False, "col": True},
        # expert weights quantised from their float32 masters
        {"name": "quant_weights_f32", "op": "quant", "T": 0, "topk": 0, "E": 16, "rows": 2816, "cols": 2048, "pad": 1,
         "type": "f32", "e4m3": False, "col": False},
        # first product of the rank with both operands in 4 bits
        {"name": "gemm_fwd_rank", "op": "gemm_fwd", "E": 16, "M": 24576, "N": 2816, "K": 2048, "e4m3": False,
         "out": "bf16"},
        # the same product for eight decoded tokens with 8-bit rows: the weights' bytes count
        {"name": "gemm_fwd_decode_e4m3", "op": "gemm_fwd", "E": 16, "M": 48, "N": 2816, "K": 2048, "e4m3": True,
         "out": "bf16"},
        # a product of the wide model size (as the input gradient is: the gradient's rows times transposed weights)
        {"name": "gemm_fwd_wide", "op": "gemm_fwd", "E": 8, "M": 16384, "N": 4096, "K": 7168, "e4m3": False,
         "out": "bf16"},
        # weight gradient of the rank's first product into float32 gradients
        {"name": "gemm_wgrad_rank", "op": "gemm_wgrad", "E": 16, "M": 24576, "N": 2816, "K": 2048, "e4m3": False,
         "out": "f32"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def _width(rng, lo, hi):
    """A width: one in four as drawn (odd ones among them), the others multiples of 32, as models have."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.25 else max(32, v // 32 * 32)


def draw(rng):
    op = rng.choice(["combine_fwd", "combine_bwd", "dispatch_fwd", "dispatch_bwd", "quant", "quant", "gemm_fwd",
                     "gemm_fwd", "gemm_wgrad"])
    if op.startswith("gemm"):
        while True:
            E, M = _log(rng, 1, 64), _log(rng, 1, 32768)
            N, K = _width(rng, 64, 8192), _width(rng, 64, 8192)
            if M * N * K <= 4.8e11 and E * N * K <= 3e8:
                break
        e4m3 = rng.random() < 0.35
        # (a product with 8-bit rows is added up in the matrix cores to 4e-5, so it has no float32 result to speak of)
        return {"op": op, "E": E, "M": M, "N": N, "K": K, "e4m3": e4m3, "out": "bf16" if e4m3 else rng.choice(["bf16", "f32"])}
    topk = rng.choice([1, 2, 4, 6, 8])
    E = max(topk, _log(rng, 1, 256))
    D = _width(rng, 64, 8192)
    T = _log(rng, 1, min(16384, max(1, (1 << 26) // (topk * D))))
    pad = rng.choice([1, 1, 16, 128])
    case = {"op": op, "T": T, "topk": topk, "E": E, "pad": pad if T * topk >= 4 * E * pad else 1,
            "type": rng.choice(["bf16", "bf16", "f32"])}
    if op == "quant":
        case |= {"cols": D, "e4m3": rng.random() < 0.35, "col": rng.random() < 0.5}
        if rng.random() < 0.3:
            rows = _width(rng, 32, 8192)
            while case["E"] * rows * D > 1e8:
                case["E"] = (case["E"] + 1) // 2
                if case["E"] == 1:
                    rows = min(rows, int(1e8 // D))
            case |= {"T": 0, "topk": 0, "rows": rows, "pad": 1}
        return case
    case |= {"D": D, "drop": rng.choice([0.0, 0.0, 0.05, 0.4]) if T >= 16 else 0.0}
    if op.startswith("combine"):
        case["weights"] = rng.choice(["f32", "bf16"])
    return case


def work(case):
    op = case["op"]
    if op.startswith("gemm"):
        E, M, N, K, o = case["E"], case["M"], case["N"], case["K"], BYTES[case["out"]]
        left = 1.0 if case["e4m3"] else 0.5
        if op == "gemm_fwd":
            moved = M * K * (left + 1 / 32) + min(E, M) * N * K * (0.5 + 1 / 32) + o * M * N
        else:
            moved = M * N * (left + 1 / 32) + M * K * (0.5 + 1 / 32) + o * E * N * K
        return {"bytes": moved, "flops": 2 * M * N * K}
    b = BYTES[case["type"]]
    if op == "quant":  # quantised, and read back into bf16 for each direction
        C = case["cols"]
        n = (case["E"] * case["rows"] if case["T"] == 0 else _rows(case["T"], case["topk"], case["E"], case["pad"])) * C
        seen = n if case["T"] == 0 else case["T"] * C
        codes = (1.0 if case["e4m3"] else 0.5) + 1 / 32
        return {"bytes": b * seen + (2 if case["col"] else 1) * n * (2 * codes + 2), "flops": 4 * n}
    T, k, D = case["T"], case["topk"], case["D"]
    n, rows = T * k * (1.0 - case["drop"]), _rows(T, k, case["E"], case["pad"])
    if op == "combine_bwd":  # dy and h read, dh written
        return {"bytes": b * D * (T + n + rows) + 12 * T * k, "flops": 3 * n * D}
    # rows to tokens, or tokens to rows: each side once
    return {"bytes": b * D * (T + (rows if op == "dispatch_fwd" else n)) + 8 * T * k, "flops": 2 * n * D}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


def _residual(g, rows, cols):
    """Hidden states: rows of differing scale, a few columns much larger than the others."""
    x = _normal(g, rows, cols) * torch.exp(0.5 * _normal(g, rows, 1))
    return x * (1.0 + 15.0 * (torch.rand((1, cols), generator=g, device=DEV) < 0.005))


def _rows(T, topk, E, pad):
    """Rows of the padded layout: the most that the segments' pad rows can come to."""
    return (T * topk + E * (pad - 1)) // pad * pad


def _plan(g, T, topk, E, pad, drop):
    """A routing plan as ``route_plan`` gives it: topk different experts per token, some preferred, a share of the
    assignments dropped. The last segment's pad rows reach to a capacity that any routing fits in, as in a program whose
    buffers keep their size."""
    liking = _normal(g, T, E) + _normal(g, 1, E)
    ids = liking.topk(topk, 1).indices.reshape(-1)
    ids = torch.where(torch.rand(T * topk, generator=g, device=DEV) < drop, E, ids)
    counts = torch.bincount(ids, minlength=E + 1)[:E]
    seg = (counts + pad - 1) // pad * pad
    offs = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), seg.cumsum(0)])
    offs[E] = _rows(T, topk, E, pad)
    order = torch.argsort(ids, stable=True)[: int(counts.sum())]
    e = ids[order]
    rank = torch.arange(order.numel(), device=DEV) - (counts.cumsum(0) - counts)[e]
    row = offs[e] + rank
    row_assign = torch.full((_rows(T, topk, E, pad),), -1, dtype=torch.int32, device=DEV)
    row_assign[row] = order.int()
    assign_row = torch.full((T * topk,), -1, dtype=torch.int32, device=DEV)
    assign_row[order] = row.int()
    return {"offs": offs.int(), "counts": counts.int(), "row_assign": row_assign, "assign_row": assign_row,
            "status": torch.zeros(1, dtype=torch.int32, device=DEV)}


def _counts(g, E, M):
    """Rows per expert, uneven as a router leaves them; from eight experts on some get none."""
    share = torch.rand(E, generator=g, device=DEV).cpu() ** 2 + 1e-3
    if E >= 8:
        share[torch.randperm(E, generator=g, device=DEV).cpu()[: E // 8]] = 0.0
    edge = torch.cumsum(share.double() / share.double().sum(), 0) * M
    edge = edge.round().to(torch.int64).clamp(0, M)
    edge[-1] = M
    return [0] + edge.tolist()


def _codes_of(x, e4m3):
    """A microscaled operand (codes, scales) of float32 x [..., rows, K]."""
    v, byte = _mx(x, e4m3)
    *lead, rows, K = v.shape
    n = len(lead)
    if e4m3:
        c = v.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        mag = v.abs().contiguous()
        c = torch.bucketize(mag, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)).to(torch.uint8)
        c = c + 8 * torch.signbit(v).to(torch.uint8)
        c = c[..., 0::2] | c[..., 1::2] << 4
    back = (*range(n), n + 1, n, n + 2)
    return (c.view(*lead, rows, -1, 64).permute(back).contiguous(), byte.view(*lead, rows, -1, 4).permute(back).contiguous())


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op.startswith("gemm"):
        E, M, N, K = case["E"], case["M"], case["N"], case["K"]
        if op == "gemm_fwd":
            s["bounds"] = _counts(g, E, M)
            s["a"] = _codes_of(_residual(g, M, K), case["e4m3"])
            w = [_codes_of(_normal(g, N, K, std=0.02), False) for _ in range(E)]
            s["b"] = tuple(torch.stack(t) for t in zip(*w))
        else:  # segments are whole panels of 128 rows; rows that an expert lacks are zero
            part = _counts(g, E, -(-M // 128))
            s["bounds"] = [128 * v for v in part]
            real = (torch.arange(s["bounds"][-1], device=DEV) < M).float()
            s["a"] = _codes_of(_normal(g, N, s["bounds"][-1]) * real, case["e4m3"])
            s["b"] = _codes_of(_residual(g, s["bounds"][-1], K).t() * real, False)
        s["offs"] = torch.tensor(s["bounds"], dtype=torch.int32, device=DEV)
        return s
    t = TYPES[case["type"]]
    if op == "quant":
        if case["T"] == 0:
            s["x"] = _normal(g, case["E"], case["rows"], case["cols"], std=0.02).to(t)
            s["plan"] = None
        else:
            s["x"] = _residual(g, case["T"], case["cols"]).to(t)
            s["plan"] = _plan(g, case["T"], case["topk"], case["E"], case["pad"], 0.0)
        return s
    T, k, D = case["T"], case["topk"], case["D"]
    s["plan"] = _plan(g, T, k, case["E"], case["pad"], case["drop"])
    rows = s["plan"]["row_assign"].numel()
    if op == "dispatch_fwd":
        s["x"] = _residual(g, T, D).to(t)
    else:
        s["h"] = _normal(g, rows, D).to(t)
    if op.startswith("combine"):
        s["w"] = torch.softmax(_normal(g, T, k), 1).to(TYPES[case["weights"]])
    if op == "combine_bwd":
        s["dy"] = _normal(g, T, D).to(t)
    return s


# ------------------------------------------------------------------ plain forms

def _pow2(byte):
    """2^(byte - 127) as float32 for bytes 0..254, from its bits."""
    return torch.where(byte == 0, 0x00400000, byte.to(torch.int32) << 23).to(torch.int32).view(torch.float32)


def _mx(x, e4m3):
    """float32 x [..., K]: the codes' values, padded to 128, and the scale bytes of the groups of 32."""
    K = x.shape[-1]
    p = torch.nn.functional.pad(x, (0, -K % 128)).unflatten(-1, (-1, 32))
    amax = p.abs().amax(-1)
    top = 8 if e4m3 else 2
    byte = torch.where(amax == 0, 0, (torch.frexp(amax).exponent - 1 - top).clamp(-127, 127) + 127)
    # (2^127 - byte has no float32 of its own at 0: two steps, both exact)
    half = (254 - byte) // 2
    r = p * _pow2(half + 63)[..., None] * _pow2(254 - byte - half + 64)[..., None]
    if e4m3:
        v = r.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    else:  # steps of 1/2 below 2, of 1 below 4, of 2 up to 6; halves go to the even code
        m = r.abs()
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
        v = torch.copysign((torch.round(m / step) * step).clamp(max=6.0), r)
    return v.flatten(-2), byte.to(torch.uint8)


def _planes(byte):
    """Scale bytes [..., rows, groups] as they lie in an operand, as numbers."""
    b = byte.unflatten(-1, (-1, 4)).transpose(-3, -2)
    return b.contiguous().view(torch.float8_e8m0fnu)


def _values(q, s):
    """The float32 matrix [..., rows, K padded] of an operand."""
    rows = s.shape[-2]
    if q.shape[-3] != s.shape[-3]:
        c = q.view(torch.float8_e4m3fn).float()
    else:
        mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
        mag = torch.cat([mag, -mag])
        c = mag[torch.stack([q & 15, q >> 4], -1).int()]
        c = c.flatten(-2)
    c = c.transpose(-3, -2).flatten(-2)
    sc = _pow2(s.transpose(-3, -2).flatten(-2).to(torch.int32))
    return (c.unflatten(-1, (-1, 32)) * sc[..., None]).flatten(-2).view(*s.shape[:-3], rows, -1)


def _gather(x, index):
    """Rows of x, zeros where the index is negative."""
    return torch.where(index[:, None] >= 0, x[index.clamp_min(0).long()], torch.zeros((), dtype=x.dtype, device=x.device))


def _tokens(s):
    """Token of each row, -1 for a pad row."""
    a = s["plan"]["row_assign"]
    return torch.where(a >= 0, a // s["topk"], -1)


def _plain(s):
    op = s["op"]
    if op == "dispatch_fwd":
        return _gather(s["x"], _tokens(s))
    if op == "dispatch_bwd":
        return _gather(s["h"], s["plan"]["assign_row"]).float().view(s["T"], s["topk"], -1).sum(1).to(s["h"].dtype)
    if op == "combine_fwd":
        h = _gather(s["h"], s["plan"]["assign_row"]).float().view(s["T"], s["topk"], -1)
        return (h * s["w"].float()[:, :, None]).sum(1).to(s["h"].dtype)
    if op == "combine_bwd":
        a, r = s["plan"]["row_assign"], s["plan"]["assign_row"]
        dy = s["dy"].float()
        dh = _gather(dy, _tokens(s)) * _gather(s["w"].float().view(-1, 1), a)
        h = _gather(s["h"], r).float().view(s["T"], s["topk"], -1)
        return dh.to(s["h"].dtype), (h * dy[:, None]).sum(2)
    if op == "quant":
        x = s["x"].float()
        if s["plan"] is not None:
            x = _gather(x, _tokens(s))
        out = []
        for m in ([x, x.transpose(-2, -1)] if s["col"] else [x]):
            v, byte = _mx(m, s["e4m3"])
            v = (v.unflatten(-1, (-1, 32)) * _pow2(byte.to(torch.int32))[..., None]).flatten(-2)
            out += [v[..., : m.shape[-1]].bfloat16(), _planes(byte)]
        return out
    at, out = s["bounds"], TYPES[s["out"]]
    a, b = _values(*s["a"]), _values(*s["b"])
    # one library product per expert that has rows: the fewest operations that elementary torch needs here
    segments = [(e, lo, hi) for e, (lo, hi) in enumerate(zip(at, at[1:])) if hi > lo]
    if op == "gemm_fwd":
        return torch.cat([a[lo:hi] @ b[e].t() for e, lo, hi in segments]).to(out)
    dw = torch.zeros((s["E"], s["N"], s["K"]), dtype=torch.float32, device=a.device)
    for e, lo, hi in segments:
        torch.mm(a[:, lo:hi], b[:, lo:hi].t(), out=dw[e])
    return dw.to(out)


# ------------------------------------------------------------------ one pass

def _own(s):
    import mxfp8_mixed_precision_amd as mx
    op = s["op"]
    if op == "dispatch_fwd":
        return mx.dispatch_fwd(s["x"], s["plan"])
    if op == "dispatch_bwd":
        return mx.dispatch_bwd(s["h"], s["plan"], s["T"])
    if op == "combine_fwd":
        return mx.combine_fwd(s["h"], s["w"], s["plan"])
    if op == "combine_bwd":
        return mx.combine_bwd(s["dy"], s["h"], s["w"], s["plan"])
    if op == "quant":
        mode = mx.ROW | mx.COL if s["col"] else mx.ROW
        q, sc, qt, sct = mx.mxfp4_quantize(s["x"], mode, e4m3=s["e4m3"], plan=s["plan"])
        out = [mx.mxfp4_dequantize(q, sc, s["cols"]), sc.view(torch.float8_e8m0fnu)]
        if s["col"]:
            rows = s["x"].shape[-2] if s["plan"] is None else s["plan"]["row_assign"].numel()
            out += [mx.mxfp4_dequantize(qt, sct, rows), sct.view(torch.float8_e8m0fnu)]
        return out
    if op == "gemm_fwd":
        return mx.grouped_gemm_mxfp4_fwd(s["a"], s["b"], s["offs"], out_dtype=TYPES[s["out"]])
    return mx.grouped_gemm_mxfp4_wgrad(s["a"], s["b"], s["offs"], out_dtype=TYPES[s["out"]])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ float64

def _two64(e):
    """2^e for whole e, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _quantised64(x, e4m3):
    """x [rows, K] in float64 as its definition quantises it: values [rows, K] and scales [planes, rows, 4]."""
    rows, K = x.shape
    n = -(-K // 128) * 4
    p = torch.zeros((rows, n * 32), dtype=torch.float64, device=x.device)
    p[:, :K] = x
    p = p.view(rows, n, 32)
    top = p.abs().amax(2)
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    e = torch.where(_two64(e) > top, e - 1, e)
    e = torch.where(_two64(e + 1) <= top, e + 1, e)
    e = torch.where(top > 0, (e - (8 if e4m3 else 2)).clamp(-127, 127), torch.full_like(e, -127))
    scale = _two64(e)
    low, bits, most = (-6.0, 3, 448.0) if e4m3 else (0.0, 1, 6.0)
    r = p / scale[:, :, None]
    step = _two64(torch.floor(torch.log2(r.abs().clamp_min(2.0 ** low))) - bits)
    v = (torch.round(r / step) * step).clamp(-most, most) * scale[:, :, None]
    return v.view(rows, n * 32)[:, :K], scale.view(rows, n // 4, 4).permute(1, 0, 2).contiguous()


def _operand64(q, s):
    """An operand [planes, rows, ...] as its numbers [rows, K], from the codes' bit fields."""
    planes, rows, _ = s.shape
    i = q.to(torch.int64)
    if q.shape[0] == planes:  # E2M1
        i = torch.stack([i % 16, i // 16], 3).view(planes, rows, 128)
        field, frac, sign = (i >> 1) & 3, (i & 1).double(), i >= 8
        v = torch.where(field == 0, frac * 0.5, (1 + frac * 0.5) * _two64(field - 1))
    else:
        field, frac, sign = (i >> 3) & 15, (i & 7).double(), i >= 128
        v = torch.where(field == 0, frac * 2.0 ** -9, (8 + frac) * _two64(field - 10))
    v = torch.where(sign, -v, v)
    v = v.permute(1, 0, 2).reshape(rows, planes * 4, 32)
    return (v * _two64(s.permute(1, 0, 2).reshape(rows, planes * 4).to(torch.int64) - 127)[:, :, None]).view(rows, planes * 128)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("gemm"):
        at, E = s["bounds"], case["E"]
        a = _operand64(*s["a"])
        if op == "gemm_fwd":
            y = torch.zeros((case["M"], case["N"]), dtype=torch.float64, device=a.device)
            for e in range(E):
                y[at[e]:at[e + 1]] = a[at[e]:at[e + 1]] @ _operand64(s["b"][0][e], s["b"][1][e]).t()
            return y
        b = _operand64(*s["b"])
        dw = torch.zeros((E, case["N"], case["K"]), dtype=torch.float64, device=a.device)
        for e in range(E):
            dw[e] = a[:, at[e]:at[e + 1]] @ b[:, at[e]:at[e + 1]].t()
        return dw
    plan = s["plan"]
    if op == "quant":
        x = s["x"].double()
        if plan is None:
            every = [[_quantised64(m, case["e4m3"]) for m in ([x[e], x[e].t()] if case["col"] else [x[e]])]
                     for e in range(case["E"])]
            return [torch.stack([every[e][d][i] for e in range(case["E"])]) for d in range(len(every[0])) for i in range(2)]
        rows = torch.zeros((plan["row_assign"].numel(), case["cols"]), dtype=torch.float64, device=x.device)
        at = torch.nonzero(plan["row_assign"] >= 0)[:, 0]
        rows[at] = x[plan["row_assign"][at].long() // case["topk"]]
        return [t for m in ([rows, rows.t()] if case["col"] else [rows]) for t in _quantised64(m, case["e4m3"])]
    T, k, D = case["T"], case["topk"], case["D"]
    at = torch.nonzero(plan["assign_row"] >= 0)[:, 0]  # assignments that have a row
    row, tok = plan["assign_row"][at].long(), at // k
    if op == "dispatch_fwd":
        out = torch.zeros((plan["row_assign"].numel(), D), dtype=torch.float64, device=at.device)
        out[row] = s["x"].double()[tok]
        return out
    w = s["w"].double().view(-1)[at] if "w" in s else torch.ones(at.numel(), dtype=torch.float64, device=at.device)
    if op == "combine_bwd":
        dh = torch.zeros(s["h"].shape, dtype=torch.float64, device=at.device)
        dw = torch.zeros(T * k, dtype=torch.float64, device=at.device)
        for part in torch.arange(at.numel(), device=at.device).split(4096):
            g = s["dy"][tok[part]].double()
            dh[row[part]] = g * w[part, None]
            dw[at[part]] = (g * s["h"][row[part]].double()).sum(1)
        return dh, dw.view(T, k)
    y = torch.zeros((T, D), dtype=torch.float64, device=at.device)
    for part in torch.arange(at.numel(), device=at.device).split(4096):
        y.index_add_(0, tok[part], s["h"][row[part]].double() * w[part, None])
    return y
