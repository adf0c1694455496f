"""Tensor-level calls of the training-block operators: layer norm, SwiGLU with 8-bit checkpoints and
ragged expert products (include/mxfp8.h).

Each call checks its tensors, allocates its outputs with torch and makes one library call on the current
stream of the tensors' device, or on ``stream=`` (a torch stream, or a hipStream_t as an int), which the outputs
and the workspace then belong to; inputs that another stream made are the caller's to order.
Checkpoints are row-wise MXFP8: uint8 codes and E8M0 scale bytes, which ``dequantize`` reads back. A violated check raises ValueError before anything is launched;
what the library itself refuses raises MxfError.
"""
import functools

from . import _abi
from ._abi import GroupedDesc, NormDesc

_torch = None


def _t():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _bad(what):
    raise ValueError(what)


def _rows(t, name):
    """A matrix with adjacent columns as (rows, cols, row stride)."""
    if not (t.dim() == 2 and (t.shape[1] <= 1 or t.stride(1) == 1)):
        _bad(f"{name}: a 2-D tensor with adjacent columns is needed")
    rows, cols = t.shape
    ld = t.stride(0) if rows > 1 else cols
    if not (ld >= cols):
        _bad(f"{name}: rows overlap (stride {ld} < {cols})")
    return rows, cols, ld


def _on(t, device, name):
    if not (t.device == device):
        _bad(f"{name} is on {t.device}, not on {device}")


def _dense(t, shape, dtype, device, name):
    if t is None or not (t.dtype == dtype and tuple(t.shape) == shape and t.is_contiguous()):
        _bad(f"{name}: a dense {dtype} tensor of shape {shape} is needed")
    _on(t, device, name)


def _stream_of(device):
    """The current stream of the tensors' device, which has to be the current device."""
    if device.type != "cuda":
        _bad(f"tensors on {device}: a GPU is needed")
    torch = _t()
    if device.index != torch.cuda.current_device():
        _bad(f"tensors are on {device}, not on the current device")
    return torch._C._cuda_getCurrentRawStream(device.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _run(name, *args):
    """One library call (looked up once), its status checked."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(_abi.lib(), name)
    status = fn(*args)
    if status:
        _abi._check(status)


_entry = {}


def _on_stream(fn):
    """Adds ``stream=``: the call runs, and allocates, with that stream as the current one."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        cuda = _t().cuda
        with cuda.stream(stream if isinstance(stream, cuda.Stream) else cuda.ExternalStream(stream)):
            return fn(*args, **kw)
    return call


# ------------------------------------------------------------------ layer norm

def _norm_args(x, weight, bias):
    torch = _t()
    if not (x.dtype in (torch.bfloat16, torch.float32)):
        _bad(f"element type {x.dtype}: bfloat16 or float32 is needed")
    flags = _abi.NORM_F32 if x.dtype == torch.float32 else 0
    cols = x.shape[-1]
    for name, v in (("weight", weight), ("bias", bias)):
        if v is not None:
            if not (v.dtype in (torch.bfloat16, torch.float32)):
                _bad(f"{name}: bfloat16 or float32 is needed")
            _dense(v, (cols,), v.dtype, x.device, name)
            if v.dtype == torch.float32:
                flags |= _abi.NORM_WEIGHT_F32
    if not (weight is None or bias is None or weight.dtype == bias.dtype):
        _bad("weight and bias differ in type")
    return flags


def _norm_fwd(x, weight, bias, eps, stats, ckpt):
    torch = _t()
    rows, cols, ld = _rows(x, "x")
    flags = _norm_args(x, weight, bias)
    dev = x.device
    y = torch.empty((rows, cols), dtype=x.dtype, device=dev)
    mean = torch.empty(rows, dtype=torch.float32, device=dev) if stats and not ckpt else None
    rstd = torch.empty(rows, dtype=torch.float32, device=dev) if stats or ckpt else None
    q = torch.empty((rows, cols), dtype=torch.uint8, device=dev) if ckpt else None
    s = torch.empty((rows, (cols + 31) // 32), dtype=torch.uint8, device=dev) if ckpt else None
    _run("mxf_layer_norm_fwd", NormDesc(rows, cols, ld, cols, cols, eps, flags), x.data_ptr(), _ptr(weight),
         _ptr(bias), y.data_ptr(), _ptr(mean), _ptr(rstd), _ptr(q), _ptr(s), _stream_of(dev))
    return y, mean, rstd, q, s


@_on_stream
def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, stats=True):
    """Layer norm of x [rows, cols] (BF16 or FP32, any row stride): (y, mean, rstd), or y alone with
    stats=False."""
    y, mean, rstd, _, _ = _norm_fwd(x, weight, bias, eps, stats, False)
    return (y, mean, rstd) if stats else y


@_on_stream
def layer_norm_ckpt_fwd(x, weight=None, bias=None, eps=1e-5):
    """Layer norm that keeps its normalised rows in 8 bits: (y, rstd, q, s). x is not needed for the
    backward."""
    y, _, rstd, q, s = _norm_fwd(x, weight, bias, eps, True, True)
    return y, rstd, q, s


def _norm_bwd(dy, x, q, s, mean, rstd, weight):
    torch = _t()
    rows, cols, ldy = _rows(dy, "dy")
    flags = _norm_args(dy, weight, None)
    dev = dy.device
    ldx = cols
    if x is not None:
        if not (x.dtype == dy.dtype and tuple(x.shape) == (rows, cols)):
            _bad("x and dy differ in type or shape")
        _on(x, dev, "x")
        ldx = _rows(x, "x")[2]
        _dense(mean, (rows,), torch.float32, dev, "mean")
    else:
        _dense(q, (rows, cols), torch.uint8, dev, "q")
        _dense(s, (rows, (cols + 31) // 32), torch.uint8, dev, "s")
    _dense(rstd, (rows,), torch.float32, dev, "rstd")
    desc = NormDesc(rows, cols, ldx, ldy, cols, 0.0, flags)
    dx = torch.empty((rows, cols), dtype=dy.dtype, device=dev)
    dw = torch.empty((2, cols), dtype=torch.float32, device=dev)
    ws = torch.empty(_abi.layer_norm_workspace_bytes(desc), dtype=torch.uint8, device=dev)
    dw, db = dw.unbind(0)
    _run("mxf_layer_norm_bwd", desc, dy.data_ptr(), _ptr(x), _ptr(q), _ptr(s), _ptr(mean), rstd.data_ptr(),
         _ptr(weight), dx.data_ptr(), dw.data_ptr(), db.data_ptr(), ws.data_ptr(), _stream_of(dev))
    return dx, dw, db


@_on_stream
def layer_norm_bwd(dy, x, mean, rstd, weight=None):
    """(dx, dweight, dbias) of layer_norm_fwd; dweight and dbias are FP32."""
    if x is None:
        _bad("x is needed")
    return _norm_bwd(dy, x, None, None, mean, rstd, weight)


@_on_stream
def layer_norm_ckpt_bwd(dy, q, s, rstd, weight=None):
    """(dx, dweight, dbias) of layer_norm_ckpt_fwd, from its 8-bit checkpoint."""
    return _norm_bwd(dy, None, q, s, None, rstd, weight)


# ------------------------------------------------------------------ SwiGLU

@_on_stream
def swiglu_ckpt_fwd(gu):
    """h = BF16(g sigmoid(g) u) of gu [rows, 2F] BF16 (gate | up), and gu in 8 bits: (h, q, s) with q
    [2 rows, F] and s [2 rows, ceil(F / 32)]."""
    torch = _t()
    if not (gu.dtype == torch.bfloat16):
        _bad("gu: bfloat16 is needed")
    rows, cols, ld = _rows(gu, "gu")
    if not (cols % 2 == 0):
        _bad(f"gu: an even number of columns is needed, not {cols}")
    F, dev = cols // 2, gu.device
    h = torch.empty((rows, F), dtype=torch.bfloat16, device=dev)
    q = torch.empty((2 * rows, F), dtype=torch.uint8, device=dev)
    s = torch.empty((2 * rows, (F + 31) // 32), dtype=torch.uint8, device=dev)
    _run("mxf_swiglu_ckpt_fwd", gu.data_ptr(), rows, F, ld, h.data_ptr(), F, q.data_ptr(), s.data_ptr(),
         _stream_of(dev))
    return h, q, s


@_on_stream
def swiglu_ckpt_bwd(dh, q, s, recompute=True):
    """(dgu, h) of swiglu_ckpt_fwd from its checkpoint: dgu [rows, 2F], and the activation h again (None
    with recompute=False)."""
    torch = _t()
    if not (dh.dtype == torch.bfloat16):
        _bad("dh: bfloat16 is needed")
    rows, F, ld = _rows(dh, "dh")
    dev = dh.device
    _dense(q, (2 * rows, F), torch.uint8, dev, "q")
    _dense(s, (2 * rows, (F + 31) // 32), torch.uint8, dev, "s")
    dgu = torch.empty((rows, 2 * F), dtype=torch.bfloat16, device=dev)
    h = torch.empty((rows, F), dtype=torch.bfloat16, device=dev) if recompute else None
    _run("mxf_swiglu_ckpt_bwd", dh.data_ptr(), ld, q.data_ptr(), s.data_ptr(), rows, F, dgu.data_ptr(), 2 * F,
         _ptr(h), F, _stream_of(dev))
    return dgu, h


# ------------------------------------------------------------------ ragged expert products

def _grouped_args(w_shape, offs, device, out_dtype, status):
    torch = _t()
    E = w_shape[0]
    _dense(offs, (E + 1,), torch.int32, device, "offs")
    if status is not None:
        if not (status.dtype == torch.int32 and status.numel() >= 1):
            _bad("status: an int32 tensor is needed")
        _on(status, device, "status")
    if not (out_dtype in (torch.bfloat16, torch.float32)):
        _bad(f"out_dtype {out_dtype}: bfloat16 or float32 is needed")
    return _abi.GROUPED_OUT_F32 if out_dtype == torch.float32 else 0


@_on_stream
def grouped_gemm_fwd(x, w, offs, out_dtype=None, status=None):
    """y [M, N]: rows [offs[e], offs[e+1]) of x [M, K] times w[e] [N, K] transposed. Rows at or past
    offs[E] are left as allocated."""
    torch = _t()
    out_dtype = out_dtype or torch.bfloat16
    if not (x.dtype == torch.bfloat16 and w.dtype == torch.bfloat16 and w.dim() == 3):
        _bad("x and w [E, N, K]: bfloat16 is needed")
    M, K, ld = _rows(x, "x")
    if not (w.shape[2] == K and w.is_contiguous()):
        _bad(f"w: a dense [E, N, {K}] tensor is needed")
    _on(w, x.device, "w")
    flags = _grouped_args(w.shape, offs, x.device, out_dtype, status)
    E, N, _ = w.shape
    y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _run("grouped_gemm_fwd", GroupedDesc(E, flags, M, N, K, ld, N), offs.data_ptr(), x.data_ptr(), w.data_ptr(),
         y.data_ptr(), _ptr(status), _stream_of(x.device))
    return y


@_on_stream
def grouped_gemm_dgrad(dy, w, offs, out_dtype=None, status=None):
    """dx [M, K]: rows [offs[e], offs[e+1]) of dy [M, N] times w[e] [N, K]."""
    torch = _t()
    out_dtype = out_dtype or torch.bfloat16
    if not (dy.dtype == torch.bfloat16 and w.dtype == torch.bfloat16 and w.dim() == 3):
        _bad("dy and w [E, N, K]: bfloat16 is needed")
    M, N, ld = _rows(dy, "dy")
    if not (w.shape[1] == N and w.is_contiguous()):
        _bad(f"w: a dense [E, {N}, K] tensor is needed")
    _on(w, dy.device, "w")
    flags = _grouped_args(w.shape, offs, dy.device, out_dtype, status)
    E, _, K = w.shape
    dx = torch.empty((M, K), dtype=out_dtype, device=dy.device)
    _run("grouped_gemm_dgrad", GroupedDesc(E, flags, M, N, K, K, ld), offs.data_ptr(), dy.data_ptr(), w.data_ptr(),
         dx.data_ptr(), _ptr(status), _stream_of(dy.device))
    return dx


@_on_stream
def grouped_gemm_wgrad(dy, x, offs, out_dtype=None, accumulate=None, status=None):
    """dw [E, N, K]: for each expert the product of its rows of dy [M, N], transposed, and of x [M, K].
    x is BF16, or a pair (q, s): its row-wise MXFP8 codes [M, K] and scales [M, ceil(K / 32)].
    accumulate: an FP32 [E, N, K] tensor that the gradient is added to and that is returned."""
    torch = _t()
    if not (dy.dtype == torch.bfloat16):
        _bad("dy: bfloat16 is needed")
    M, N, ldy = _rows(dy, "dy")
    q = s = None
    if isinstance(x, (tuple, list)):
        q, s = x
        x = None
        if q is None or q.dim() != 2:
            _bad("q: a 2-D tensor is needed")
        K = ldx = q.shape[1]
        _dense(q, (M, K), torch.uint8, dy.device, "q")
        _dense(s, (M, (K + 31) // 32), torch.uint8, dy.device, "s")
    else:
        if x is None or x.dtype != torch.bfloat16:
            _bad("x: bfloat16 is needed")
        rows, K, ldx = _rows(x, "x")
        if not (rows == M):
            _bad(f"x has {rows} rows, dy {M}")
        _on(x, dy.device, "x")
    if offs is None or offs.dim() != 1 or offs.numel() == 0:
        _bad("offs: a 1-D int32 tensor [E + 1] is needed")
    E = offs.numel() - 1
    if accumulate is not None:
        if not (out_dtype in (None, torch.float32)):
            _bad("accumulate: the output is float32")
        _dense(accumulate, (E, N, K), torch.float32, dy.device, "accumulate")
        out_dtype, dw = torch.float32, accumulate
    else:
        out_dtype = out_dtype or torch.bfloat16
        dw = torch.empty((E, N, K), dtype=out_dtype, device=dy.device)
    flags = _grouped_args((E,), offs, dy.device, out_dtype, status)
    if accumulate is not None:
        flags |= _abi.GROUPED_ACCUM
    _run("grouped_gemm_wgrad", GroupedDesc(E, flags, M, N, K, ldx, ldy), offs.data_ptr(), dy.data_ptr(), _ptr(x),
         _ptr(q), _ptr(s), dw.data_ptr(), _ptr(status), _stream_of(dy.device))
    return dw

