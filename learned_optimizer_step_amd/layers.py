"""Norms, embedding and distillation loss over liblopt, for PyTorch tensors.

They produce the gradients that ``lopt.LearnedOptimizer`` steps with:

* ``layer_norm``, ``rms_norm``  a transformer's norms
* ``embedding``                 a token lookup with scaling, its gradient by sorted tokens
* ``distill_loss``              a loss from a teacher's top logits, where a backward pass begins

These are differentiable (``torch.autograd``; gradients of gradients are not
supported).  The ``*_forward`` and ``*_backward`` functions below them make
one call of the library each (include/lopt.h has the formulas); they take
buffers for the parameters' gradients and can add to what is there, so a
training step captured into a HIP graph keeps the gradients where the
optimizer's step reads them.

Everything runs on the GPU, on the tensors' device and its current stream;
nothing waits.  Tensors may be fp32, bf16 or fp16, of any leading shape; a
tensor whose last dimension is not contiguous, or whose rows are not equally
spaced, is copied first.  Bad arguments raise ``ValueError``, errors of the
library ``lopt.LoptError``.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import lopt as L

_DTYPES = {torch.float32: L.LOPT_F32, torch.bfloat16: L.LOPT_BF16, torch.float16: L.LOPT_F16}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, not {t.dtype}")
    return code


def _on(device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _gpu(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU: there is no CPU path")
    return t.device


def _matrix(t: torch.Tensor, name: str) -> torch.Tensor:
    """t as rows of its last dimension, with unit stride in a row and rows that do not overlap."""
    if t.dim() == 0:
        raise ValueError(f"{name} needs at least one dimension")
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1]) if t.shape[-1] else t.reshape(0, 0)
    if t.shape[1] < 1:
        raise ValueError(f"{name}: the last dimension is empty")
    if (t.stride(1) != 1 and t.shape[1] > 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        t = t.contiguous()
    return t


def _vector(t: Optional[torch.Tensor], n: int, name: str):
    """A vector of n elements, contiguous."""
    if t is None:
        return None
    if t.shape != (n,):
        raise ValueError(f"{name} must have shape ({n},), not {tuple(t.shape)}")
    return t.contiguous()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _call(fn, device, *args) -> None:
    if torch.cuda.current_device() == device.index:
        fn(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            fn(*args, _stream(device))


def _out(t: Optional[torch.Tensor], shape, device, name: str, make_dtype) -> torch.Tensor:
    """A caller's contiguous output buffer, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=make_dtype, device=device)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} on {device}")
    _dtype(t, name)
    return t


# ---------------------------------------------------------------------------
# norms

def norm_forward(x, weight=None, bias=None, eps: float = 1e-5, rms: bool = False):
    """(y, mean, rstd) of a layer norm, or of an RMS norm (mean: None) over x's last dimension.

    y is like x; mean and rstd are float32, one value a row (x's leading shape
    flattened), for ``norm_backward``.  weight and bias: vectors of one type,
    or None."""
    dev = _gpu(x, "x")
    _on(dev, weight=weight, bias=bias)
    code = _dtype(x, "x")
    m = _matrix(x, "x")
    rows, cols = m.shape
    weight, bias = _vector(weight, cols, "weight"), _vector(bias, cols, "bias")
    if rms and bias is not None:
        raise ValueError("an RMS norm has no bias")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have the same type")
    w = weight if weight is not None else bias
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    stats = torch.empty((1 if rms else 2, rows), dtype=torch.float32, device=dev)
    mean, rstd = (None, stats[0]) if rms else (stats[0], stats[1])
    _call(L.lopt_norm_forward, dev, L.LOPT_NORM_RMS if rms else L.LOPT_NORM_LAYER, rows, cols, code, m.data_ptr(),
          m.stride(0), _ptr(weight), _ptr(bias), 0 if w is None else _dtype(w, "weight"), eps, y.data_ptr(), cols,
          _ptr(mean), rstd.data_ptr())
    return y, mean, rstd


def norm_backward(grad_y, x, weight, mean, rstd, *, rms: bool = False, grad_weight=None, grad_bias=None,
                  accumulate: bool = False, need_x: bool = True, need_weight: bool = True,
                  need_bias: Optional[bool] = None, grad_dtype: Optional[torch.dtype] = None):
    """(grad_x, grad_weight, grad_bias) of ``norm_forward``; None where not needed.

    grad_weight, grad_bias: buffers to write, or, with accumulate, to add to;
    made anew where None (of grad_dtype, else of the weight's type, else
    float32).  An RMS norm has no grad_bias."""
    dev = _gpu(x, "x")
    _on(dev, grad_y=grad_y, weight=weight, mean=mean, rstd=rstd)
    code = _dtype(x, "x")
    if grad_y.shape != x.shape or grad_y.dtype != x.dtype:
        raise ValueError("grad_y must have the shape and type of x")
    m, g = _matrix(x, "x"), _matrix(grad_y, "grad_y")
    rows, cols = m.shape
    weight = _vector(weight, cols, "weight")
    need_bias = (not rms) if need_bias is None else need_bias
    if rms and (need_bias or grad_bias is not None):
        raise ValueError("an RMS norm has no bias")
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is None:
            if name == "mean" and rms:
                continue
            raise ValueError(f"{name} is missing")
        if t.dtype != torch.float32 or t.shape != (rows,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 vector of {rows} values")
    if accumulate and ((need_weight and grad_weight is None) or (need_bias and grad_bias is None)):
        raise ValueError("accumulate needs the buffers to add to")
    make = grad_dtype if grad_dtype is not None else torch.float32 if weight is None else weight.dtype
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if need_x else None
    dw = _out(grad_weight, (cols,), dev, "grad_weight", make) if need_weight else None
    db = _out(grad_bias, (cols,), dev, "grad_bias", make if dw is None else dw.dtype) if need_bias else None
    if dw is not None and db is not None and dw.dtype != db.dtype:
        raise ValueError("grad_weight and grad_bias must have the same type")
    gw = dw if dw is not None else db
    ws, ws_bytes = None, 0
    if gw is not None:
        ws_bytes = L.lopt_norm_backward_workspace(rows, cols)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _call(L.lopt_norm_backward, dev, L.LOPT_NORM_RMS if rms else L.LOPT_NORM_LAYER, rows, cols, code, g.data_ptr(),
          g.stride(0), m.data_ptr(), m.stride(0), _ptr(weight), 0 if weight is None else _dtype(weight, "weight"),
          None if rms else mean.data_ptr(), rstd.data_ptr(), _ptr(dx), cols, _ptr(dw), _ptr(db),
          0 if gw is None else _dtype(gw, "grad_weight"), int(accumulate), _ptr(ws), ws_bytes)
    return dx, dw, db


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, rms):
        y, mean, rstd = norm_forward(x, weight, bias, eps, rms)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.rms = rms
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        x, weight, mean, rstd = ctx.saved_tensors
        nx, nw, nb = ctx.needs_input_grad[:3]
        dx, dw, db = norm_backward(grad_y, x, weight, mean, rstd, rms=ctx.rms, need_x=nx, need_weight=nw, need_bias=nb,
                                   grad_dtype=ctx.bias_dtype if weight is None else None)
        return dx, dw, db, None, None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm over x's last dimension: (x - mean) / sqrt(var + eps) * weight + bias."""
    return _Norm.apply(x, weight, bias, eps, False)


def rms_norm(x, weight=None, eps: float = 1e-6):
    """RMS norm over x's last dimension: x / sqrt(mean(x^2) + eps) * weight."""
    return _Norm.apply(x, weight, None, eps, True)


# ---------------------------------------------------------------------------
# embedding

def _ids(ids, name: str) -> int:
    n = _ID_BYTES.get(ids.dtype)
    if n is None:
        raise ValueError(f"{name} must be int32 or int64, not {ids.dtype}")
    return n


def embedding_forward(ids, weight, scale: float = 1.0, row0: int = 0, dtype: Optional[torch.dtype] = None):
    """scale * weight[ids - row0], of shape ids.shape + (weight.shape[1],) and type dtype (default: the weight's).

    An id that names no row of weight (padding, or a row of another shard of
    the table whose first row here is row0) gives zeros."""
    dev = _gpu(weight, "weight")
    _on(dev, ids=ids)
    code = _dtype(weight, "weight")
    if weight.dim() != 2:
        raise ValueError("weight must have two dimensions")
    nb = _ids(ids, "ids")
    w = _matrix(weight, "weight")
    rows, cols = w.shape
    ids = ids.contiguous()
    out = torch.empty((*ids.shape, cols), dtype=weight.dtype if dtype is None else dtype, device=dev)
    _call(L.lopt_embedding_forward, dev, ids.numel(), ids.data_ptr(), nb, rows, cols, row0, w.data_ptr(), w.stride(0), code,
          scale, out.data_ptr(), cols, _dtype(out, "dtype"))
    return out


def embedding_backward(grad_out, ids, rows: int, scale: float = 1.0, row0: int = 0, *, out=None, accumulate: bool = False,
                       dtype: torch.dtype = torch.float32):
    """The gradient of ``embedding_forward`` for a weight of `rows` rows.

    out: a buffer (rows, grad_out.shape[-1]) to write or, with accumulate, to
    add to (only the rows that ids name are touched then); made anew, of type
    dtype, where None."""
    dev = _gpu(grad_out, "grad_out")
    _on(dev, ids=ids)
    code = _dtype(grad_out, "grad_out")
    nb = _ids(ids, "ids")
    if grad_out.shape[:-1] != ids.shape:
        raise ValueError("grad_out must have the shape of ids and one dimension more")
    g = _matrix(grad_out, "grad_out")
    n, cols = g.shape
    if accumulate and out is None:
        raise ValueError("accumulate needs a buffer to add to")
    dw = _out(out, (rows, cols), dev, "out", dtype)
    ids = ids.contiguous()
    ws_bytes = L.lopt_embedding_backward_workspace(n, rows, cols)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _call(L.lopt_embedding_backward, dev, n, ids.data_ptr(), nb, g.data_ptr(), g.stride(0), code, rows, cols, row0, scale,
          dw.data_ptr(), cols, _dtype(dw, "out"), int(accumulate), ws.data_ptr(), ws_bytes)
    return dw


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, scale, row0, dtype):
        ctx.save_for_backward(ids)
        ctx.args = (weight.shape[0], scale, row0, weight.dtype)
        return embedding_forward(ids, weight, scale, row0, dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        rows, scale, row0, dtype = ctx.args
        dw = None
        if ctx.needs_input_grad[1]:
            dw = embedding_backward(grad_out, ctx.saved_tensors[0], rows, scale, row0, dtype=dtype)
        return None, dw, None, None, None


def embedding(ids, weight, scale: float = 1.0, row0: int = 0, dtype: Optional[torch.dtype] = None):
    """scale * weight[ids - row0]; see ``embedding_forward``.  The gradient is dense, like weight."""
    return _Embedding.apply(ids, weight, scale, row0, dtype)


# ---------------------------------------------------------------------------
# distillation from a teacher's top logits

def _lists(logits, ids, teacher):
    dev = _gpu(logits, "logits")
    _on(dev, teacher_ids=ids, teacher_logits=teacher)
    if ids.shape != teacher.shape or ids.dim() == 0 or ids.shape[:-1] != logits.shape[:-1]:
        raise ValueError("teacher_ids and teacher_logits must have one shape, the logits' but for the last dimension")
    return (dev, _dtype(logits, "logits"), _ids(ids, "teacher_ids"), _dtype(teacher, "teacher_logits"),
            _matrix(logits, "logits"), _matrix(ids, "teacher_ids"), _matrix(teacher, "teacher_logits"))


def distill_forward(logits, teacher_ids, teacher_logits, temperature: float = 1.0):
    """(loss, lse), float32 and one value a row of logits: temperature^2 times the divergence KL(teacher || student),
    the teacher renormalised over its list, and log sum exp(logits / temperature) for ``distill_backward``.

    Entries with an id outside the vocabulary (say -1) or a logit of -inf are
    absent; a row without entries has loss 0."""
    dev, code, nb, ucode, z, i, u = _lists(logits, teacher_ids, teacher_logits)
    rows, cols = z.shape
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=dev)
    lse = torch.empty(logits.shape[:-1], dtype=torch.float32, device=dev)
    _call(L.lopt_distill_forward, dev, rows, cols, code, z.data_ptr(), z.stride(0), i.shape[1], i.data_ptr(), i.stride(0), nb,
          u.data_ptr(), u.stride(0), ucode, temperature, loss.data_ptr(), lse.data_ptr())
    return loss, lse


def distill_backward(grad_loss, logits, teacher_ids, teacher_logits, lse, temperature: float = 1.0, *, out=None):
    """The gradient of ``distill_forward``'s loss for the logits, of their type.

    grad_loss: one float32 value a row.  out: a contiguous buffer like logits;
    it may be logits itself, which the gradient then replaces."""
    dev, code, nb, ucode, z, i, u = _lists(logits, teacher_ids, teacher_logits)
    _on(dev, grad_loss=grad_loss, lse=lse)
    rows, cols = z.shape
    for name, t in (("grad_loss", grad_loss), ("lse", lse)):
        if t.dtype != torch.float32 or t.shape != logits.shape[:-1]:
            raise ValueError(f"{name} must be float32, one value a row of logits")
    dz = _out(out, logits.shape, dev, "out", logits.dtype)
    if dz.dtype != logits.dtype:
        raise ValueError("out must have the type of logits")
    g, lse = grad_loss.reshape(-1), lse.contiguous()
    _call(L.lopt_distill_backward, dev, rows, cols, code, g.data_ptr(), g.stride(0), z.data_ptr(), z.stride(0), i.shape[1],
          i.data_ptr(), i.stride(0), nb, u.data_ptr(), u.stride(0), ucode, temperature, lse.data_ptr(), dz.data_ptr(), cols)
    return dz


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, teacher, temperature):
        loss, lse = distill_forward(logits, ids, teacher, temperature)
        ctx.save_for_backward(logits, ids, teacher, lse)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss):
        logits, ids, teacher, lse = ctx.saved_tensors
        return distill_backward(grad_loss, logits, ids, teacher, lse, ctx.temperature), None, None, None


def distill_loss(logits, teacher_ids, teacher_logits, temperature: float = 1.0):
    """The distillation loss of every row of logits (float32); see ``distill_forward``.

    Differentiable in the logits; the teacher is a constant."""
    if teacher_logits.requires_grad:
        raise ValueError("the loss has no gradient for teacher_logits: detach them")
    return _Distill.apply(logits, teacher_ids, teacher_logits, temperature)
