"""Tensor-level calls around the routed experts' products: token rows to their experts' rows and back, MXFP4 operands and
the products on them (include/mxfp8.h).

As in block_ops.py each call checks its tensors (ValueError), allocates its outputs with torch and makes one library call
(MxfError) on the current stream of the tensors' device, or on ``stream=``.

``plan`` is what ``route_plan`` returns: a dict with int32 tensors offs [E + 1], row_assign [rows] and assign_row [tokens *
topk], and topk, which a call's number of tokens has to match (a plan made elsewhere may lack it: then it is assignments over
tokens). Rows at or past offs[E] of an output with expert rows are left as allocated.

An MXFP4 operand of a matrix [rows, K] is a pair (q, s): uint8 codes [P, rows, 64] and scale bytes [P, rows, 4], P = ceil(K /
128); with E4M3 elements q is [2 P, rows, 64]. K is padded with zeros, so only P is left of it. A batch of matrices has
one more dimension in front.
"""
from . import _abi
from ._abi import GroupedDesc, OperandDesc, RouteDesc
from .block_ops import _bad, _dense, _on, _on_stream, _ptr, _rows, _run, _stream_of, _t


def _plan(plan, device, rows=None):
    """offs, row_assign, assign_row of a plan on `device`, each a dense vector."""
    torch = _t()
    for name in ("offs", "row_assign", "assign_row"):
        t = plan.get(name)
        if t is None or not (t.dim() == 1 and t.dtype == torch.int32 and t.is_contiguous()):
            _bad(f"plan: {name} has to be a dense int32 vector")
        if t.device != device:
            _on(t, device, name)
    if plan["offs"].numel() < 2:
        _bad("plan: offs [E + 1] is needed")
    if rows is not None and plan["row_assign"].numel() != rows:
        _bad(f"plan: row_assign has {plan['row_assign'].numel()} rows, the matrix {rows}")
    return plan["offs"], plan["row_assign"], plan["assign_row"]


def _topk(plan, tokens):
    """Experts per token: the plan's own where it has them, else assignments over tokens."""
    n, topk = plan["assign_row"].numel(), plan.get("topk")
    if tokens < 0:
        _bad(f"{tokens} tokens")
    if topk is not None:
        if topk < 1:
            _bad(f"plan: topk = {topk}")
        if tokens * topk != n:
            _bad(f"plan: {n} assignments, {topk} per token, are not of {tokens} tokens")
        return topk
    if tokens == 0:
        if n:
            _bad(f"plan: {n} assignments of no tokens")
        return 1
    if n % tokens or n < tokens:
        _bad(f"plan: {n} assignments are not a multiple of {tokens} tokens")
    return n // tokens


def _float_flag(t, name):
    torch = _t()
    if t.dtype not in (torch.bfloat16, torch.float32):
        _bad(f"{name}: bfloat16 or float32 is needed, not {t.dtype}")
    return 1 if t.dtype == torch.float32 else 0


# ------------------------------------------------------------------ token rows to experts and back

@_on_stream
def dispatch_fwd(x, plan):
    """xe [rows, D]: row r is token row_assign[r] // topk of x [tokens, D], zeros for a pad row. Any type with
    elements of 1, 2, 4 or 8 bytes."""
    torch = _t()
    tokens, D, ld = _rows(x, "x")
    dev = x.device
    offs, row_assign, assign_row = _plan(plan, dev)
    topk, rows = _topk(plan, tokens), row_assign.numel()
    xe = torch.empty((rows, D), dtype=x.dtype, device=dev)
    _run("mxf_dispatch_fwd", RouteDesc(tokens, rows, D, ld, D, D, topk, offs.numel() - 1, x.element_size(), 0),
         offs.data_ptr(), row_assign.data_ptr(), assign_row.data_ptr(), x.data_ptr(), xe.data_ptr(), _stream_of(dev))
    return xe


def _combine(h, weights, plan, tokens, residual=None):
    torch = _t()
    rows, D, ld = _rows(h, "h")
    dev = h.device
    offs, _, assign_row = _plan(plan, dev, rows)
    topk = _topk(plan, tokens)
    flags = _float_flag(h, "h")
    if weights is not None:
        flags |= 2 * _float_flag(weights, "weights")
        _dense(weights, (tokens, topk if tokens else weights.shape[1]), weights.dtype, dev, "weights")
    ldr = D
    if residual is not None:
        if residual.dtype != h.dtype or tuple(residual.shape) != (tokens, D):
            _bad(f"residual: a {h.dtype} tensor [{tokens}, {D}] is needed")
        _on(residual, dev, "residual")
        ldr = _rows(residual, "residual")[2]
    y = torch.empty((tokens, D), dtype=h.dtype, device=dev)
    _run("mxf_combine_fwd", RouteDesc(tokens, rows, D, D, ld, ldr, topk, offs.numel() - 1, 0, flags), assign_row.data_ptr(),
         h.data_ptr(), _ptr(weights), _ptr(residual), y.data_ptr(), _stream_of(dev))
    return y


@_on_stream
def dispatch_bwd(dxe, plan, tokens):
    """dx [tokens, D] of dispatch_fwd: each token's rows of dxe [rows, D] (BF16 or FP32) added up."""
    return _combine(dxe, None, plan, tokens)


@_on_stream
def combine_fwd(h, weights, plan, residual=None):
    """y [tokens, D]: each token's rows of h [rows, D] (BF16 or FP32) times weights [tokens, topk] (BF16 or FP32), added up,
    and onto residual [tokens, D] if there is one (of h's type; y is rounded once)."""
    if weights is None or weights.dim() != 2:
        _bad("weights [tokens, topk] are needed")
    return _combine(h, weights, plan, weights.shape[0], residual)


@_on_stream
def combine_bwd(dy, h, weights, plan):
    """(dh, dweights) of combine_fwd: dh [rows, D] like dy, zeros in pad rows, and dweights [tokens, topk] FP32 (None where h
    is None: h is only needed for it)."""
    torch = _t()
    tokens, D, ldy = _rows(dy, "dy")
    dev = dy.device
    rows, ldh = None, D
    if h is not None:
        rows, Dh, ldh = _rows(h, "h")
        if Dh != D or h.dtype != dy.dtype:
            _bad("h and dy differ in type or width")
        _on(h, dev, "h")
    offs, row_assign, assign_row = _plan(plan, dev, rows)
    rows, topk = row_assign.numel(), _topk(plan, tokens)
    if weights is None or weights.dim() != 2:
        _bad("weights [tokens, topk] are needed")
    flags = _float_flag(dy, "dy") | 2 * _float_flag(weights, "weights")
    _dense(weights, (tokens, topk if tokens else weights.shape[1]), weights.dtype, dev, "weights")
    dh = torch.empty((rows, D), dtype=dy.dtype, device=dev)
    dw = torch.empty(tuple(weights.shape), dtype=torch.float32, device=dev) if h is not None else None
    _run("mxf_combine_bwd", RouteDesc(tokens, rows, D, ldy, ldh, D, topk, offs.numel() - 1, 0, flags), offs.data_ptr(),
         row_assign.data_ptr(), assign_row.data_ptr(), dy.data_ptr(), _ptr(h), weights.data_ptr(), dh.data_ptr(), _ptr(dw),
         _stream_of(dev))
    return dh, dw


# ------------------------------------------------------------------ MXFP4 operands

def _new_operand(lead, rows, K, e4m3, device):
    torch = _t()
    P = (K + 127) // 128
    return (torch.empty((*lead, 2 * P if e4m3 else P, rows, 64), dtype=torch.uint8, device=device),
            torch.empty((*lead, P, rows, 4), dtype=torch.uint8, device=device))


@_on_stream
def mxfp4_quantize(x, mode=_abi.ROW, e4m3=False, plan=None):
    """Operands of x [rows, cols] (BF16 or FP32, any row stride) or of a dense batch [n, rows, cols]: (q_row, s_row, q_col,
    s_col), as ``quantize`` returns them; with mode ROW along the rows, with COL along the columns (the operand of the
    transposed matrix), None for what mode leaves out. e4m3: 8-bit elements. plan: the rows are those that dispatch_fwd
    would lay out of the tokens x."""
    flags = _float_flag(x, "x") | (_abi.OPERAND_E4M3 if e4m3 else 0)
    if mode not in (_abi.ROW, _abi.COL, _abi.ROW | _abi.COL):
        _bad(f"mode {mode}: ROW, COL or both")
    dev = x.device
    lead, offs, row_assign, tokens, topk, E = (), None, None, 0, 1, 1
    if x.dim() == 3:
        if plan is not None or not x.is_contiguous():
            _bad("x: a batch has to be dense, and without a plan")
        lead, (rows, cols) = (x.shape[0],), x.shape[1:]
        ld = cols
    else:
        rows, cols, ld = _rows(x, "x")
        if plan is not None:
            offs, row_assign, _ = _plan(plan, dev)
            tokens, topk, E = rows, _topk(plan, rows), offs.numel() - 1
            rows = row_assign.numel()
    q = s = qt = st = None
    if mode & _abi.ROW:
        q, s = _new_operand(lead, rows, cols, e4m3, dev)
    if mode & _abi.COL:
        qt, st = _new_operand(lead, cols, rows, e4m3, dev)
    _run("mxfp4_quantize", OperandDesc(lead[0] if lead else 1, rows, cols, ld, tokens, topk, E, flags), x.data_ptr(), _ptr(offs),
         _ptr(row_assign), _ptr(q), _ptr(s), _ptr(qt), _ptr(st), _stream_of(dev))
    return q, s, qt, st


def _operand(q, s, lead, device, name):
    """(planes, rows, whether E4M3) of an operand with `lead` leading dimensions."""
    torch = _t()
    for t in (q, s):
        if t is None or not (t.dtype == torch.uint8 and t.dim() == lead + 3 and t.is_contiguous()):
            _bad(f"{name}: dense uint8 codes [.., P, rows, 64] and scales [.., P, rows, 4] are needed")
        if t.device != device:
            _on(t, device, name)
    P, rows, n = s.shape[lead:]
    panels = q.shape[lead]
    if n != 4 or q.shape[-1] != 64 or q.shape[-2] != rows or q.shape[:lead] != s.shape[:lead] or panels not in (P, 2 * P):
        _bad(f"{name}: codes {tuple(q.shape)} and scales {tuple(s.shape)} are no operand")
    return P, rows, panels != P


@_on_stream
def mxfp4_dequantize(q, s, cols, out_dtype=None):
    """The matrix [rows, cols] (or batch) of an operand along its rows, BF16 (default) or FP32."""
    torch = _t()
    out_dtype = out_dtype or torch.bfloat16
    if s is None or s.dim() not in (3, 4):
        _bad("s: scales [P, rows, 4], or a batch of them, are needed")
    lead, dev = s.dim() - 3, s.device
    P, rows, e4m3 = _operand(q, s, lead, dev, "operand")
    if not (P > 0 and 128 * (P - 1) < cols <= 128 * P):
        _bad(f"cols = {cols} does not fit {P} planes of 128")
    out = torch.empty((*s.shape[:lead], rows, cols), dtype=out_dtype, device=dev)
    flags = _float_flag(out, "out_dtype") | (_abi.OPERAND_E4M3 if e4m3 else 0)
    _run("mxfp4_dequantize", OperandDesc(s.shape[0] if lead else 1, rows, cols, cols, 0, 1, 1, flags), q.data_ptr(), s.data_ptr(),
         out.data_ptr(), _stream_of(dev))
    return out


# ------------------------------------------------------------------ expert products on operands

def _grouped(offs, device, out_dtype, status, e4m3):
    torch = _t()
    if offs is None or not (offs.dim() == 1 and offs.numel() >= 2 and offs.dtype == torch.int32 and offs.is_contiguous()):
        _bad("offs: a dense int32 tensor [E + 1] is needed")
    _on(offs, device, "offs")
    if status is not None:
        if not (status.dtype == torch.int32 and status.numel() >= 1):
            _bad("status: an int32 tensor is needed")
        _on(status, device, "status")
    if out_dtype not in (torch.bfloat16, torch.float32):
        _bad(f"out_dtype {out_dtype}: bfloat16 or float32 is needed")
    return (_abi.GROUPED_OUT_F32 if out_dtype == torch.float32 else 0) | (_abi.GROUPED_LEFT_E4M3 if e4m3 else 0)


@_on_stream
def grouped_gemm_mxfp4_fwd(x, w, offs, out_dtype=None, status=None):
    """y [M, N]: rows [offs[e], offs[e+1]) of x times w[e] transposed, from the operands x = (q, s) of [M, K] (4 or 8 bits) and
    w = (q, s) of E matrices [N, K] (4 bits). With dy and the weights' operands along columns it is the input gradient."""
    torch = _t()
    out_dtype = out_dtype or torch.bfloat16
    (xq, xs), (wq, ws) = x, w
    if xs is None:
        _bad("x: a pair of codes and scales is needed")
    dev = xs.device
    P, M, e4m3 = _operand(xq, xs, 0, dev, "x")
    Pw, N, w8 = _operand(wq, ws, 1, dev, "w")
    if Pw != P or w8:
        _bad(f"w: 4-bit codes over {P} planes are needed")
    flags = _grouped(offs, dev, out_dtype, status, e4m3)
    E = ws.shape[0]
    if offs.numel() != E + 1:
        _bad(f"offs has {offs.numel()} entries for {E} experts")
    y = torch.empty((M, N), dtype=out_dtype, device=dev)
    _run("grouped_gemm_mxfp4_fwd", GroupedDesc(E, flags, M, N, 128 * P, 0, N), offs.data_ptr(), xq.data_ptr(), xs.data_ptr(),
         wq.data_ptr(), ws.data_ptr(), y.data_ptr(), _ptr(status), _stream_of(dev))
    return y


@_on_stream
def grouped_gemm_mxfp4_wgrad(dy, x, offs, out_dtype=None, accumulate=None, status=None):
    """dw [E, N, K]: for each expert the product of its rows of dy (4 or 8 bits) and x (4 bits), from their operands along
    columns: dy = (q, s) of [N, M], x = (q, s) of [K, M]. offs are multiples of 128. accumulate: an FP32 [E, N, K] tensor
    that the gradient is added to and that is returned."""
    torch = _t()
    (gq, gs), (xq, xs) = dy, x
    if gs is None:
        _bad("dy: a pair of codes and scales is needed")
    dev = gs.device
    P, N, e4m3 = _operand(gq, gs, 0, dev, "dy")
    Px, K, x8 = _operand(xq, xs, 0, dev, "x")
    if Px != P or x8:
        _bad(f"x: 4-bit codes over {P} planes are needed")
    if accumulate is not None:
        if out_dtype not in (None, torch.float32):
            _bad("accumulate: the output is float32")
        out_dtype = torch.float32
    out_dtype = out_dtype or torch.bfloat16
    flags = _grouped(offs, dev, out_dtype, status, e4m3)
    E = offs.numel() - 1
    if accumulate is not None:
        _dense(accumulate, (E, N, K), torch.float32, dev, "accumulate")
        flags, dw = flags | _abi.GROUPED_ACCUM, accumulate
    else:
        dw = torch.empty((E, N, K), dtype=out_dtype, device=dev)
    _run("grouped_gemm_mxfp4_wgrad", GroupedDesc(E, flags, 128 * P, N, K, 0, 0), offs.data_ptr(), gq.data_ptr(), gs.data_ptr(),
         xq.data_ptr(), xs.data_ptr(), dw.data_ptr(), _ptr(status), _stream_of(dev))
    return dw
