"""Operators around the joint attention: layer norm, the projection with low-rank adapters, and
cross attention to an encoder's states.  Argument marshalling only, as in ``_ffi``: every step
runs in the library's kernels, on the tensors' device and on ``stream`` (default: the current
stream of that device).  Outputs are tensors of the caller, which overlap no other operand except
where a call says that they may be one; scratch memory comes from PyTorch's allocator on that
stream, so calls of these functions on different streams, and graphs captured from them, never
share it.  (A `ProjectedLayer` keeps buffers of its own: see there.)
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _ffi
from ._ffi import BF16, F16, F32, AdapterSizes, CrossSizes, NormSizes, _check, lib

_CODE = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}
_INT32_MAX = 2 ** 31 - 1


def _tensor(t, name, dtypes, shape=None, device=None):
    """Checks one tensor argument."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _contiguous(t, name, dtypes, shape, device):
    # (one look at everything first: the messages cost only a call that is refused)
    if isinstance(t, torch.Tensor) and t.device == device and t.dtype in dtypes and t.shape == shape and t.is_contiguous():
        return
    _tensor(t, name, dtypes, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows_apart(t, name, out=False):
    """Checks that the last dimension is contiguous and (for an output) that no two elements
    share memory."""
    if t.is_contiguous():
        return
    if t.numel() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if out and t.numel():
        need = 1
        for st, n in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n > 1):
            if st < need:
                raise ValueError(f"{name} overlaps itself (strides {t.stride()})")
            need = st * (n - 1) + need


def _ptr(t):
    return None if t is None else t.data_ptr()


@contextlib.contextmanager
def _other(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):     # scratch memory then belongs to `stream`
                yield


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """Makes `device`, and `stream` if given, current for the call."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    if stream is None and torch.cuda.current_device() == device.index:
        return _HERE
    return _other(device, stream)


def _workspace(what, device, query, *args):
    need = ctypes.c_size_t()
    _check(what, query(*args, ctypes.byref(need)))
    return torch.empty(need.value, dtype=torch.uint8, device=device) if need.value else None


def _stream(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def operator_status(stream=None) -> int:
    """Waits for `stream` (default: the current one), then returns and clears the device-side
    status of this module's operators on the stream's device (0: no kernel's wait ran out)."""
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        return lib().ultragen_operator_status(s.cuda_stream)


# ------------------------------------------------------------------------------- layer norm
def _batched(t):
    return t if t.dim() == 3 else t.unsqueeze(0)


def _norm_sizes(x, weight, bias, plus_one, eps):
    _tensor(x, "x", tuple(_CODE))
    if x.dim() not in (2, 3):
        raise ValueError("x must be [rows, cols] or [batch, rows, cols]")
    _rows_apart(x, "x")
    x3 = _batched(x)
    B, R, C = x3.shape
    if C < 1 or B * R > _INT32_MAX:
        raise ValueError(f"x has shape {tuple(x.shape)}")
    n = NormSizes(batch=B, rows=R, cols=C, dtype=_CODE[x.dtype], wdtype=_CODE[x.dtype],
                  plus_one=1 if plus_one else 0, eps=float(eps), x_row=x3.stride(1), x_batch=x3.stride(0))
    t = bias if weight is None else weight
    if t is not None:
        if not isinstance(t, torch.Tensor) or t.dtype not in (x.dtype, torch.float32):
            raise ValueError("weight and bias must have x's dtype or float32")
        per_sample = t.dim() == 2
        if per_sample and x.dim() != 3:
            raise ValueError("a weight per sample needs x [batch, rows, cols]")
        n.per_sample = 1 if per_sample else 0
        n.wdtype = _CODE[t.dtype]
        shape = (B, C) if per_sample else (C,)
        if weight is not None:
            _contiguous(weight, "weight", (t.dtype,), shape, x.device)
        if bias is not None:
            _contiguous(bias, "bias", (t.dtype,), shape, x.device)
    return n, x3


def layer_norm(x, y, weight=None, bias=None, eps: float = 1e-6, plus_one: bool = False, mean=None,
               rstd=None, stream=None):
    """y = (x - mean) * rstd * w' + bias over the last dimension of x [rows, cols] or
    [batch, rows, cols] (bf16, fp16 or fp32; any row and batch strides; y may be x), with
    w' = weight, or 1 + weight (plus_one).  weight and bias are [cols], or [batch, cols] for one
    modulation per sample, in x's dtype or fp32.  mean and rstd, fp32 of x.shape[:-1], receive
    the statistics the backward pass needs."""
    n, x3 = _norm_sizes(x, weight, bias, plus_one, eps)
    _tensor(y, "y", (x.dtype,), x.shape, x.device)
    _rows_apart(y, "y", out=True)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t is not None:
            _contiguous(t, name, (torch.float32,), x.shape[:-1], x.device)
    y3 = _batched(y)
    n.y_row, n.y_batch = y3.stride(1), y3.stride(0)
    with _on(x.device, stream):
        _check("ultragen_layer_norm", lib().ultragen_layer_norm(
            n, x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), _ptr(mean), _ptr(rstd),
            _stream(x.device)))
    return y


def layer_norm_backward(dy, x, mean, rstd, dx, weight=None, plus_one: bool = False, dweight=None,
                        dbias=None, stream=None):
    """Gradients of layer_norm: dx (may be dy or x), and dweight, dbias (bf16, fp16 or fp32)
    shaped [cols] or [batch, cols] as the forward pass's weight and bias; each may be None.
    mean and rstd as layer_norm wrote them."""
    shaped = [t for t in (weight, dweight, dbias) if t is not None]
    if len({tuple(t.shape) for t in shaped}) > 1:
        raise ValueError("weight, dweight and dbias must share a shape")
    n, x3 = _norm_sizes(x, weight, None, plus_one, 0.0)
    B, R, C = x3.shape
    for t, name in ((dy, "dy"), (dx, "dx")):
        _tensor(t, name, (x.dtype,), x.shape, x.device)
        _rows_apart(t, name, out=name == "dx")
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _contiguous(t, name, (torch.float32,), x.shape[:-1], x.device)
    grads = [t for t in (dweight, dbias) if t is not None]
    if weight is None and grads:
        if grads[0].dim() == 2 and x.dim() != 3:
            raise ValueError("a gradient per sample needs x [batch, rows, cols]")
        n.per_sample = 1 if grads[0].dim() == 2 else 0
    for t in grads:
        _contiguous(t, "dweight and dbias", tuple(_CODE), (B, C) if n.per_sample else (C,), x.device)
    if len({t.dtype for t in grads}) > 1:
        raise ValueError("dweight and dbias must share a dtype")
    dy3, dx3 = _batched(dy), _batched(dx)
    n.dy_row, n.dy_batch = dy3.stride(1), dy3.stride(0)
    n.y_row, n.y_batch = dx3.stride(1), dx3.stride(0)
    with _on(x.device, stream):
        ws = None
        if grads:
            ws = _workspace("ultragen_layer_norm_backward_workspace", x.device,
                            lib().ultragen_layer_norm_backward_workspace, n)
        _check("ultragen_layer_norm_backward", lib().ultragen_layer_norm_backward(
            n, dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(),
            _ptr(dweight), _ptr(dbias), _CODE[grads[0].dtype] if grads else F32, _ptr(ws),
            ws.numel() if ws is not None else 0, _stream(x.device)))
    return dx


# ------------------------------------------------------------------------------- adapters
def adapter_project(x, w, y, a, b, ids, scales=None, bias=None, stream=None):
    """y[m] = w x[m] + bias + scales[id] b[id] (a[id] x[m]), id = ids[m]: a projection shared by
    all rows with each row's own low-rank adapter beside it; an id outside [0, adapters) means
    none.  x [rows, k] and y [rows, n] (bf16, fp16 or fp32, any row stride), w [n, k], bias [n],
    a [adapters, rank, k], b [adapters, n, rank] in x's dtype, scales [adapters] fp32 (None: 1),
    ids [rows] int32."""
    _tensor(x, "x", tuple(_CODE))
    if x.dim() != 2 or not isinstance(w, torch.Tensor) or w.dim() != 2 or \
            not isinstance(a, torch.Tensor) or a.dim() != 3:
        raise ValueError("x must be [rows, k], w [n, k] and a [adapters, rank, k]")
    M, K = x.shape
    N = w.shape[0]
    A, R = a.shape[:2]
    if max(M, N, K) > _INT32_MAX:
        raise ValueError("sizes past int32")
    dev, dt = x.device, (x.dtype,)
    _rows_apart(x, "x")
    _contiguous(w, "w", dt, (N, K), dev)
    _tensor(y, "y", dt, (M, N), dev)
    _rows_apart(y, "y", out=True)
    _contiguous(a, "a", dt, (A, R, K), dev)
    _contiguous(b, "b", dt, (A, N, R), dev)
    _contiguous(ids, "ids", (torch.int32,), (M,), dev)
    if bias is not None:
        _contiguous(bias, "bias", dt, (N,), dev)
    if scales is not None:
        _contiguous(scales, "scales", (torch.float32,), (A,), dev)
    c = AdapterSizes(rows=M, k=K, n=N, rank=R, adapters=A, dtype=_CODE[x.dtype], x_row=x.stride(0),
                     y_row=y.stride(0))
    with _on(dev, stream):
        ws = _workspace("ultragen_adapter_project_workspace", dev, lib().ultragen_adapter_project_workspace, c)
        _check("ultragen_adapter_project", lib().ultragen_adapter_project(
            c, x.data_ptr(), w.data_ptr(), _ptr(bias), a.data_ptr(), b.data_ptr(), _ptr(scales),
            ids.data_ptr(), y.data_ptr(), _ptr(ws), ws.numel() if ws is not None else 0, _stream(dev)))
    return y


# ------------------------------------------------------------------------------- cross attention
_HALF = (torch.bfloat16, torch.float16)


def _cross_sizes(q, k, v, kv_lens, key_mask, scale):
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _tensor(t, name, _HALF)
        if t.dim() != 4:
            raise ValueError(f"{name} must be [batch, length, heads, head_dim]")
    B, Nq, H, D = q.shape
    S, G = k.shape[1:3]
    for t, name in ((k, "k"), (v, "v")):
        _tensor(t, name, (q.dtype,), (B, S, G, D), q.device)
    if G < 1 or H % G:
        raise ValueError(f"{H} query heads cannot share {G} key/value heads")
    if kv_lens is not None:
        _contiguous(kv_lens, "kv_lens", (torch.int32,), (B,), q.device)
    if key_mask is not None:
        _contiguous(key_mask, "key_mask", (torch.bool, torch.uint8), (B, S), q.device)
    return CrossSizes(batch=B, nq=Nq, ns=S, heads=H, kv_heads=G, head_dim=D, dtype=_CODE[q.dtype],
                      masked=0 if key_mask is None else 1,
                      scale=float(D ** -0.5 if scale is None else scale))


def _cross_strides(c, tensors):
    for i, (t, name, out) in enumerate(tensors):
        if t is None:
            continue
        _rows_apart(t, name, out)
        if t.numel() == 0:
            continue
        # a dimension of one element is never stepped over: its stride may be anything
        st = [s if n > 1 else 8 for s, n in zip(t.stride(), t.shape)][:3]
        if t.data_ptr() % 16 or any(s % 8 for s in st):
            raise ValueError(f"{name}: address and strides must be multiples of 16 bytes")
        c.stride[i][:] = st


def cross_attention(q, k, v, o, kv_lens=None, key_mask=None, scale=None, lse=None, stream=None):
    """o = softmax(scale q k^T) v over the visible keys: q, o [batch, nq, heads, D] attend to
    k, v [batch, ns, kv_heads, D] (bf16 or fp16, D 64 or 128, heads a multiple of kv_heads; any
    strides that are multiples of 16 bytes).  kv_lens [batch] int32 leaves keys [0, kv_lens[b])
    visible, key_mask [batch, ns] (bool) those that are true; hidden keys and values may hold
    anything.  A query without a visible key gets zeros.  o may be q.  scale defaults to D^-1/2; lse
    [batch, heads, nq] fp32 receives the log-sum-exp the backward pass needs."""
    c = _cross_sizes(q, k, v, kv_lens, key_mask, scale)
    _tensor(o, "o", (q.dtype,), q.shape, q.device)
    B, Nq, H, _ = q.shape
    if lse is not None:
        _contiguous(lse, "lse", (torch.float32,), (B, H, Nq), q.device)
    _cross_strides(c, ((q, "q", False), (k, "k", False), (v, "v", False), (o, "o", True)))
    with _on(q.device, stream):
        ws = _workspace("ultragen_cross_attention_workspace", q.device,
                        lib().ultragen_cross_attention_workspace, c, 0)
        _check("ultragen_cross_attention", lib().ultragen_cross_attention(
            c, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(kv_lens), _ptr(key_mask), o.data_ptr(), _ptr(lse),
            _ptr(ws), ws.numel() if ws is not None else 0, _stream(q.device)))
    return o


def cross_attention_backward(do, q, k, v, o, lse, dq, dk, dv, kv_lens=None, key_mask=None, scale=None,
                             stream=None):
    """Gradients of cross_attention for do = dLoss/do: dq [batch, nq, heads, D], dk and dv
    [batch, ns, kv_heads, D], all written in full (zeros for hidden keys and values, and for a
    query without a visible key).  o and lse as cross_attention wrote them; the other arguments
    as there."""
    c = _cross_sizes(q, k, v, kv_lens, key_mask, scale)
    B, Nq, H, _ = q.shape
    for t, name in ((do, "do"), (o, "o"), (dq, "dq")):
        _tensor(t, name, (q.dtype,), q.shape, q.device)
    for t, name in ((dk, "dk"), (dv, "dv")):
        _tensor(t, name, (q.dtype,), k.shape, q.device)
    _contiguous(lse, "lse", (torch.float32,), (B, H, Nq), q.device)
    _cross_strides(c, ((q, "q", False), (k, "k", False), (v, "v", False), (o, "o", False), (do, "do", False),
                       (dq, "dq", True), (dk, "dk", True), (dv, "dv", True)))
    with _on(q.device, stream):
        ws = _workspace("ultragen_cross_attention_workspace", q.device,
                        lib().ultragen_cross_attention_workspace, c, 1)
        _check("ultragen_cross_attention_backward", lib().ultragen_cross_attention_backward(
            c, do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
            _ptr(kv_lens), _ptr(key_mask), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(ws),
            ws.numel() if ws is not None else 0, _stream(q.device)))
    return dq, dk, dv


# ------------------------------------------------------------------------------- layers
class ProjectedLayer:
    """One attention layer from hidden states: layer norm (modulated per sample), the Q, K and V
    projections with each token's adapter beside them, the joint attention of `Layer`, and, where
    states are given, cross attention of the normed tokens' queries to an encoder's states.  Every
    step runs on `stream`.  The buffers between the steps belong to the instance and stay resident, as
    `Layer`'s and its plan's do, so calls of one instance, and replays of graphs captured from it, must
    follow one another: on one stream, or with an event between streams.  cross() reads what the last
    call normed, so it runs behind that call.  Layers that run at once need an instance and a plan each."""

    def __init__(self, plan, batch: int, channels: int, device="cuda"):
        i = plan.info
        self.layer = _ffi.Layer(plan, batch, device)
        self.shape = (batch, i["N_raster"], i["heads"], i["head_dim"])
        self.norm = torch.empty((batch, i["N_raster"], channels), dtype=torch.bfloat16, device=device)
        self.q, self.k, self.v, self.xq = (torch.empty(self.shape, dtype=torch.bfloat16, device=device)
                                           for _ in range(4))

    def project(self, w, out, a, b, ids, scales=None, bias=None, stream=None):
        """out [batch, N_raster, heads, head_dim] = the projection of the normed tokens."""
        B, N, H, D = self.shape
        adapter_project(self.norm.view(B * N, -1), w, out.view(B * N, H * D), a, b, ids, scales=scales,
                        bias=bias, stream=stream)
        return out

    def __call__(self, x, o, w, a, b, ids, scales=None, bias=None, weight=None, shift=None, eps: float = 1e-6,
                 plus_one: bool = True, stream=None):
        """x [batch, N_raster, channels] bf16, o [batch, N_raster, heads, head_dim]; w, a, b (and bias)
        are triples for Q, K and V as adapter_project takes them; ids [batch * N_raster]; weight and
        shift are the norm's weight and bias."""
        if not isinstance(o, torch.Tensor) or o.device != self.norm.device:
            raise ValueError(f"o must be on {self.norm.device}")
        with _on(self.norm.device, stream):     # `Layer` runs on the current device
            layer_norm(x, self.norm, weight, shift, eps=eps, plus_one=plus_one, stream=stream)
            for i, out in enumerate((self.q, self.k, self.v)):
                self.project(w[i], out, a[i], b[i], ids, scales, None if bias is None else bias[i], stream)
            return self.layer(self.q, self.k, self.v, o, stream)

    def cross(self, o, w, a, b, ids, k, v, scales=None, bias=None, kv_lens=None, key_mask=None, lse=None,
              stream=None):
        """o = cross attention of the tokens normed by the last call, projected by w, to the states'
        keys and values k, v [batch, ns, kv_heads, head_dim]."""
        self.project(w, self.xq, a, b, ids, scales, bias, stream)
        return cross_attention(self.xq, k, v, o, kv_lens=kv_lens, key_mask=key_mask, lse=lse, stream=stream)
