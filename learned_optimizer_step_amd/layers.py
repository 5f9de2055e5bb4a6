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
optimizer's step reads them.  The differentiable functions can be captured
with ``torch.autograd.grad`` too; before a ``backward()`` is captured, let go of
every eager graph of the same leaves: torch accumulates into a leaf on the
stream where its first live graph was made, which cannot join a capture when
it is the default stream.

Everything runs on the GPU, on the tensors' device and its current stream;
nothing waits.  Tensors may be fp32, bf16 or fp16, of any leading shape; a
tensor whose last dimension is not contiguous, or whose rows are not equally
spaced, is copied first.  Bad arguments raise ``ValueError``, errors of the
library ``lopt.LoptError``.

The calls are compiled (csrc/layers.cpp, built into _layers.so by
``python -m learned_optimizer_step_amd.build``); importing this module fails
when they are not built.  They run from the library that ``lopt`` has loaded.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _layers as _C


# ---------------------------------------------------------------------------
# norms

def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm over x's last dimension: (x - mean) / sqrt(var + eps) * weight + bias."""
    return _C.norm(x, weight, bias, eps, False)


def rms_norm(x, weight=None, eps: float = 1e-6):
    """RMS norm over x's last dimension: x / sqrt(mean(x^2) + eps) * weight."""
    return _C.norm(x, weight, None, eps, True)


def norm_forward(x, weight=None, bias=None, eps: float = 1e-5, rms: bool = False):
    """(y, mean, rstd) of a layer norm, or of an RMS norm (mean: None) over x's last dimension.

    y is like x; mean and rstd are float32, one value a row (x's leading shape
    flattened), for ``norm_backward``.  weight and bias: vectors of one type,
    or None."""
    return _C.norm_forward(x, weight, bias, eps, rms)


def norm_backward(grad_y, x, weight, mean, rstd, *, rms: bool = False, grad_weight=None, grad_bias=None,
                  accumulate: bool = False, need_x: bool = True, need_weight: bool = True,
                  need_bias: Optional[bool] = None, grad_dtype: Optional[torch.dtype] = None):
    """(grad_x, grad_weight, grad_bias) of ``norm_forward``; None where not needed.

    grad_weight, grad_bias: buffers to write, or, with accumulate, to add to;
    made anew where None (of grad_dtype, else of the weight's type, else
    float32).  An RMS norm has no grad_bias."""
    return _C.norm_backward(grad_y, x, weight, mean, rstd, rms, grad_weight, grad_bias, accumulate, need_x, need_weight,
                            not rms if need_bias is None else need_bias, grad_dtype)


# ---------------------------------------------------------------------------
# embedding

def embedding(ids, weight, scale: float = 1.0, row0: int = 0, dtype: Optional[torch.dtype] = None):
    """scale * weight[ids - row0]; see ``embedding_forward``.  The gradient is dense, like weight."""
    return _C.embedding(ids, weight, scale, row0, dtype)


def embedding_forward(ids, weight, scale: float = 1.0, row0: int = 0, dtype: Optional[torch.dtype] = None):
    """scale * weight[ids - row0], of shape ids.shape + (weight.shape[1],) and type dtype (default: the weight's).

    An id that names no row of weight (padding, or a row of another shard of
    the table whose first row here is row0) gives zeros."""
    return _C.embedding_forward(ids, weight, scale, row0, dtype)


def embedding_backward(grad_out, ids, rows: int, scale: float = 1.0, row0: int = 0, *, out=None, accumulate: bool = False,
                       dtype: torch.dtype = torch.float32):
    """The gradient of ``embedding_forward`` for a weight of `rows` rows.

    out: a buffer (rows, grad_out.shape[-1]) to write or, with accumulate, to
    add to (only the rows that ids name are touched then); made anew, of type
    dtype, where None."""
    return _C.embedding_backward(grad_out, ids, rows, scale, row0, out, accumulate, dtype)


# ---------------------------------------------------------------------------
# distillation from a teacher's top logits

def distill_loss(logits, teacher_ids, teacher_logits, temperature: float = 1.0):
    """The distillation loss of every row of logits (float32); see ``distill_forward``.

    Differentiable in the logits; the teacher is a constant.  A list of one entry
    of any finite logit is a target: at temperature 1 the loss is the
    cross-entropy of that token, 0 for an id outside the vocabulary."""
    return _C.distill(logits, teacher_ids, teacher_logits, temperature)


def distill_forward(logits, teacher_ids, teacher_logits, temperature: float = 1.0):
    """(loss, lse), float32 and one value a row of logits: temperature^2 times the divergence KL(teacher || student),
    the teacher renormalised over its list, and log sum exp(logits / temperature) for ``distill_backward``.

    Entries with an id outside the vocabulary (say -1) or a logit of -inf are
    absent; a row without entries has loss 0."""
    return _C.distill_forward(logits, teacher_ids, teacher_logits, temperature)


def distill_backward(grad_loss, logits, teacher_ids, teacher_logits, lse, temperature: float = 1.0, *, out=None):
    """The gradient of ``distill_forward``'s loss for the logits, of their type.

    grad_loss: one float32 value a row.  out: a contiguous buffer like logits;
    it may be logits itself, which the gradient then replaces."""
    return _C.distill_backward(grad_loss, logits, teacher_ids, teacher_logits, lse, temperature, out)
